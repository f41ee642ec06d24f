"""The bound of tests/paged_bound.py rejects outputs that are wrong by little: a row of zeros, sixteen tokens left out, a
single token at a mask's edge left out or let in."""
import numpy as np
import pytest

import kv_cache_vector_encode_b200 as tq
import paged_bound as PB
import workloads as W
from oracle import paged as OP

# length, queries, heads, KV heads, d, key bits, value codebook bits, Algorithm 2, options
CASES = [
    (150, 1, 8, 2, 128, 3, 2, True, {}),
    (150, 70, 8, 2, 64, 4, 4, False, {}),
    (700, 1, 8, 2, 128, 3, 3, False, {}),
    (900, 40, 4, 4, 64, 1, 1, False, dict(window=64)),
    (640, 128, 14, 2, 128, 3, 3, True, dict(prefix=200, slopes=True)),
    (1300, 1, 7, 1, 128, 2, 1, False, dict(window=100, softcap=20.0)),
    (2000, 1, 4, 4, 128, 4, 3, True, {}),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_bound_rejects_small_mistakes(case):
    n, qn, Hq, Hkv, d, kb, vb, alg2, opt = CASES[case]
    rng = np.random.default_rng(case)
    Pi, S = W.rotation(d), W.jl_matrix(d)
    kl, vl = (np.array(tq.tq_codebook_init(d, b).c[: 1 << b]) for b in (kb, vb))
    k, v = PB.random_records(rng, n, Hkv, d, kl, vl, Pi, S if alg2 else None)
    q = rng.standard_normal((qn, Hq, d))
    opt = dict(opt)
    if opt.get("slopes"):
        opt["slopes"] = 2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)
    scale = d**-0.5
    want, tol, sees = PB.bounds(q, k, v, Pi, n, scale, **opt)
    assert sees.all()
    same, _, _ = OP.attend(q, k, v, n, scale, **opt)
    assert np.allclose(same, want, rtol=0, atol=1e-12)
    assert np.mean(np.linalg.norm(want, axis=-1) > tol) == 1.0   # zeros

    weight = OP.softmax_weights(q, k, n, scale, **opt)

    def caught(wrong, rows):
        return np.mean((np.linalg.norm(wrong - want, axis=-1) > tol)[rows])

    def without(out):                                            # some tokens not seen
        return OP.attend(q, k, v, n, scale, present=~out, **opt)[0]

    t = np.arange(n)
    first = n - qn - 32                                          # a block that every query sees
    block = (t >= first) & (t < first + 16)
    hit = weight[..., block].sum(-1) > 8.0 / n                   # rows of a steep bias give it no weight
    assert hit.mean() > 0.4 and caught(without(block), hit) > 0.99
    seen = min(n, opt.get("window", n))
    if seen <= 1000:                                             # beyond, one token is less than the roundings allow
        hit = np.zeros((qn, Hq), bool)
        hit[-1] = weight[-1, :, -1] > 0.5 / seen
        assert hit.any() and caught(without(t == n - 1), hit) >= 0.75
    if "window" in opt:
        for more in (-1, 1):
            other = OP.attend(q, k, v, n, scale, **{**opt, "window": opt["window"] + more})[0]
            assert caught(other, slice(None)) > 0.95
