"""Oracle (numpy, fp64) of the paged packed cache: rotary positions, append, attention of new tokens.

Not part of the TurboQuant write-ups: the operators around the cache that a decoder with paged memory
needs. Records are those of oracle.quant.
"""
from __future__ import annotations

import math

import numpy as np

from . import quant as Q


def rope_freqs(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, low_turns: float = 1.0,
               high_turns: float = 32.0, original_len: float = 0.0) -> np.ndarray:
    """Angle per position of each pair [rot/2]."""
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "blend":
        turns = original_len * f / (2.0 * math.pi)
        keep = np.clip((turns - low_turns) / (high_turns - low_turns), 0.0, 1.0)
        return keep * f + (1.0 - keep) * f / factor
    return f


def rope_table(n_pos: int, freqs: np.ndarray, magnitude: float = 1.0) -> np.ndarray:
    """(cos, sin) [n_pos, rot/2, 2]."""
    a = np.arange(n_pos)[:, None] * freqs
    return magnitude * np.stack([np.cos(a), np.sin(a)], -1)


def rope(x: np.ndarray, positions: np.ndarray, table: np.ndarray, pairs: bool, inverse: bool = False) -> np.ndarray:
    """x [tokens, heads, d]; rows with a negative position come back as they are."""
    h = table.shape[1]
    out = x.astype(np.float64).copy()
    on = positions >= 0
    c, s = (table[positions[on]][:, None, :, k].astype(np.float64) for k in (0, 1))
    if inverse:
        s = -s
    first, second = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if pairs else (slice(0, h), slice(h, 2 * h))
    a, b = out[on][..., first], out[on][..., second]
    turned = out[on]
    turned[..., first], turned[..., second] = a * c - b * s, b * c + a * s
    out[on] = turned
    return out


def dequant(codes: np.ndarray, norms: np.ndarray, levels: np.ndarray, Pi: np.ndarray, S: np.ndarray | None = None,
            signs: np.ndarray | None = None, gammas: np.ndarray | None = None) -> np.ndarray:
    """Vectors [n, d] of records [n]; levels fp32 of the codebook."""
    d = Pi.shape[0]
    bits = codes.shape[-1]
    x = levels.astype(np.float64)[Q.unpack_planes(codes, bits)] @ Pi.astype(np.float64)
    if signs is not None:
        z = 2.0 * Q.unpack_signs(signs) - 1.0
        x = x + Q.qjl_alpha(d) * gammas.astype(np.float64)[:, None] * (z @ S.astype(np.float64))
    return norms.astype(np.float64)[:, None] * x


def visible(Qn: int, kv_len: int, window: int = 0, prefix: int = 0, present: np.ndarray | None = None):
    """Positions [Qn] of the newest Qn of kv_len tokens, and which tokens each sees [Qn, kv_len]."""
    t = np.arange(kv_len)
    pos = kv_len - Qn + np.arange(Qn)
    seen = t[None] <= pos[:, None]
    if window:
        seen &= t[None] > pos[:, None] - window
    seen |= t[None] < prefix
    if present is not None:
        seen &= present[None]
    return pos, seen


def softmax_weights(q: np.ndarray, k: np.ndarray, kv_len: int, scale: float, softcap: float = 0.0, window: int = 0,
                    prefix: int = 0, slopes: np.ndarray | None = None, present: np.ndarray | None = None) -> np.ndarray:
    """Weights [Qn, Hq, kv_len] of one sequence: q [Qn, Hq, d], k [Hkv, kv_len, d]; 0 for what a query does not see."""
    Qn, Hq, d = q.shape
    g = Hq // k.shape[0]
    pos, seen = visible(Qn, kv_len, window, prefix, present)
    t = np.arange(kv_len)
    out = np.zeros((Qn, Hq, kv_len))
    for h in range(Hq):
        x = scale * (q[:, h].astype(np.float64) @ k[h // g].T)
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x + float(slopes[h]) * (t[None] - pos[:, None])
        x = np.where(seen, x, -np.inf)
        top = x.max(-1, keepdims=True, initial=-np.inf)
        p = np.where(seen, np.exp(x - np.where(np.isfinite(top), top, 0.0)), 0.0)
        total = p.sum(-1, keepdims=True)
        out[:, h] = np.where(total > 0, p / np.where(total > 0, total, 1.0), 0.0)
    return out


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, kv_len: int, scale: float, softcap: float = 0.0, window: int = 0,
           prefix: int = 0, slopes: np.ndarray | None = None, present: np.ndarray | None = None):
    """One sequence: q [Qn, Hq, d], k / v [Hkv, kv_len, d] -> out [Qn, Hq, d] and, for error bounds, the weighted
    length of the values sum_t p_t |v_t| and the largest scale |q| |k_t| of the seen tokens, both [Qn, Hq]."""
    Qn, Hq, d = q.shape
    g = Hq // k.shape[0]
    w = softmax_weights(q, k, kv_len, scale, softcap, window, prefix, slopes, present)
    out, size, reach = np.zeros((Qn, Hq, d)), np.zeros((Qn, Hq)), np.zeros((Qn, Hq))
    _, seen = visible(Qn, kv_len, window, prefix, present)
    for h in range(Hq):
        kh, vh, p = k[h // g], v[h // g], w[:, h]
        out[:, h] = p @ vh
        size[:, h] = p @ np.linalg.norm(vh, axis=1)
        if kv_len:
            reach[:, h] = (np.where(seen, np.linalg.norm(kh, axis=1)[None], 0.0).max(-1, initial=0.0) * scale *
                           np.linalg.norm(q[:, h], axis=1))
    return out, size, reach
