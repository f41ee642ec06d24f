"""How far an output row of tq_paged_attend may lie from the oracle's, with the roundings taken as independent.

Every rounding to fp16 or to the 16-bit integers of a decode step is off by at most u = 2^-11 of what it rounds, with
either sign, and is made anew for every token (and coordinate). A row is sum_t p_t v_t:
* p_t enters the products in fp16, and v_t has its levels, the rotation, the opened tile (and its residual norm) in
  fp16: four parts of u each, 2 u together (root sum square), per token. They are independent between tokens, so the
  row is off by sqrt(sum_t p_t^2 |v_t|^2 (4 u^2 + e_t^2)) with the scores' e_t, not by their plain sum.
* the score of a token takes the levels, the rotation and the opened tile in fp16, per coordinate: off by
  u scale sqrt(sum_i q'_i^2 k'_i^2) in the rotated basis, u scale |q| |k| / sqrt(d) by the rotation's entries (which
  spread a rounding over all coordinates), and u scale sqrt(sum_j q_j^2 k_j^2). Together it is off by e_t, which moves
  p_t by as much, relatively. (A decode step's integers are finer: 2^-16 of the largest coordinate or level, which is
  seldom above 3 times the usual one.)
* the levels' roundings are the same for all tokens; what they share is a factor within 2 u of the whole row.
* the output is rounded to bf16 (2^-8), and fp32 sums add 2^-20 of sum_t p_t |v_t|.
The parts above are largest values of what is spread evenly below them (1 / sqrt(3) of it on average), so four times
their root sum square is seven standard deviations: no row of the tests' 10^5 reaches it by chance.
"""
from __future__ import annotations

import numpy as np

from oracle import paged as OP

U = 2.0**-11
TIMES = 4.0


def bounds(q, k, v, Pi, kv_len, scale, **kw):
    """(exact rows [Qn, Hq, d], bound per row [Qn, Hq], whether a row sees anything) of one sequence; as OP.attend."""
    Qn, Hq, d = q.shape
    g = Hq // k.shape[0]
    p = OP.softmax_weights(q, k, kv_len, scale, **kw)
    out, tol, sees = np.zeros((Qn, Hq, d)), np.zeros((Qn, Hq)), np.zeros((Qn, Hq), bool)
    turn = Pi.T.astype(np.float64)
    for h in range(Hq):
        w, qh, kh, vh = p[:, h], q[:, h], k[h // g], v[h // g]
        out[:, h] = w @ vh
        sees[:, h] = w.sum(-1) > 0
        e2 = (qh**2 @ (kh**2).T + (qh @ turn) ** 2 @ ((kh @ turn) ** 2).T +
              (qh**2).sum(-1)[:, None] * (kh**2).sum(-1)[None] / d) * (scale * U) ** 2
        size = np.linalg.norm(vh, axis=1)
        each = np.sqrt(((w * size) ** 2 * (4 * U**2 + e2)).sum(-1))
        tol[:, h] = (2.0**-8 + 2 * U) * np.linalg.norm(out[:, h], axis=-1) + TIMES * each + 2.0**-20 * (w @ size)
    return out, tol, sees


def random_records(rng, n, Hkv, d, k_levels, v_levels, Pi, S=None):
    """Decoded keys and values [Hkv, n, d] of random codes, with the norms of the GPU tests' pools."""
    def norms(size):
        return size * np.exp(0.4 * rng.standard_normal((Hkv, n, 1)))
    k = norms(6.0) * (rng.choice(k_levels, (Hkv, n, d)) @ Pi)
    v = rng.choice(v_levels, (Hkv, n, d)) @ Pi
    if S is not None:
        v = v + np.sqrt(np.pi / 2) / d * norms(0.35) * (rng.choice([-1.0, 1.0], (Hkv, n, d)) @ S)
    return k, norms(6.0) * v
