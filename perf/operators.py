"""Measured cases of the paged-cache operators: rotary positions (tq_rope), the append of new keys
and values to a paged packed cache (tq_paged_append) and attention of new tokens over it
(tq_paged_attend).

Each operator is given here in its plain form (elementary torch operations) and, where `own` is
true, as the call that a user makes. Shapes: 32 query heads over 8 KV heads of 128 coordinates, or
32 heads of 64; keys by Algorithm 1, values by Algorithm 1 or 2 of the packed format.
"""
import functools
import math
import types

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- the packed format: codebook, rotation, planes -----------------------------------------------

@functools.lru_cache(maxsize=None)
def codebook(d, bits):
    """(levels, boundaries) in float32 of the Lloyd-Max quantiser for the density (1 - x^2)^((d-3)/2)."""
    half = 1 << (bits - 1)
    theta = np.linspace(0.0, math.pi / 2, 400001)
    w = np.cos(theta) ** (d - 2)
    x = np.sin(theta)
    mass = np.concatenate([[0.0], np.cumsum((w[1:] + w[:-1]) * 0.5)])
    wx = w * x
    moment = np.concatenate([[0.0], np.cumsum((wx[1:] + wx[:-1]) * 0.5)])
    c = (np.arange(half) + 0.5) / half * 3.0 / math.sqrt(d)
    for _ in range(2000):
        edge = np.concatenate([[0.0], (c[1:] + c[:-1]) / 2, [1.0]])
        m, f = np.interp(edge, x, mass), np.interp(edge, x, moment)
        new = np.diff(f) / np.diff(m)
        moved = np.abs(new - c).max()
        c = new
        if moved < 1e-13:
            break
    levels = np.concatenate([-c[::-1], c])
    bounds = (levels[1:] + levels[:-1]) / 2
    bounds[half - 1] = 0.0
    return levels.astype(np.float32), bounds.astype(np.float32)


def matrices(d, gen):
    """A random rotation Pi and a Gaussian S, float32."""
    a = torch.randn(d, d, generator=gen, device="cuda", dtype=torch.float64)
    q, r = torch.linalg.qr(a)
    Pi = (q * torch.sign(torch.diagonal(r))).float().contiguous()
    return Pi, torch.randn(d, d, generator=gen, device="cuda")


def planes(bits_of):
    """int32 words of truth values [..., 32]: value l in bit l."""
    shift = torch.arange(32, device=bits_of.device, dtype=torch.int32)
    return (bits_of.to(torch.int32) << shift).sum(-1, dtype=torch.int32)


def pack(idx, bits):
    """idx [n, d] -> codes [n, d/32, bits]."""
    groups = idx.reshape(idx.shape[0], -1, 1, 32)
    p = torch.arange(bits, device=idx.device).reshape(1, 1, bits, 1)
    return planes((groups >> p) & 1)


def unpack(codes):
    """codes [..., G, bits] -> indices [..., 32 G]."""
    shift = torch.arange(32, device=codes.device, dtype=torch.int32)
    p = torch.arange(codes.shape[-1], device=codes.device, dtype=torch.int32)
    idx = (((codes[..., None] >> shift) & 1) << p[:, None]).sum(-2, dtype=torch.int32)
    return idx.reshape(*codes.shape[:-2], -1)


def signs_of(words):
    """words [..., G] -> -1 / +1 [..., 32 G]."""
    shift = torch.arange(32, device=words.device, dtype=torch.int32)
    z = (words[..., None] >> shift) & 1
    return (2 * z - 1).reshape(*words.shape[:-1], -1).float()


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 64 running sequences: queries and keys of a fused projection
        {"name": "rope_step", "op": "rope", "tokens": 64, "heads": 40, "d": 128, "rot": 128, "layout": "half",
         "inverse": False, "type": "bf16", "far": 131072},
        # a prefill chunk, queries and keys together
        {"name": "rope_chunk", "op": "rope", "tokens": 8192, "heads": 40, "d": 128, "rot": 128, "layout": "half",
         "inverse": False, "type": "bf16", "far": 32768},
        # the gradient's way back through interleaved pairs of a part of the head, odd token count
        {"name": "rope_back_part", "op": "rope", "tokens": 4099, "heads": 32, "d": 64, "rot": 48,
         "layout": "pairs", "inverse": True, "type": "f32", "far": 4200},
        # the new token of 64 running sequences
        {"name": "append_step", "op": "append", "tokens": 64, "hkv": 8, "d": 128, "rot": 128, "layout": "half",
         "type": "bf16", "k_bits": 3, "v_bits": 2, "v_alg": 2, "page": 16, "far": 131072, "skip": 0.0},
        # a prefill chunk entering the cache
        {"name": "append_chunk", "op": "append", "tokens": 8192, "hkv": 8, "d": 128, "rot": 128, "layout": "half",
         "type": "bf16", "k_bits": 3, "v_bits": 3, "v_alg": 2, "page": 64, "far": 32768, "skip": 0.0},
        # heads of 64, interleaved partial rotation, a padded batch, values by Algorithm 1
        {"name": "append_part", "op": "append", "tokens": 1027, "hkv": 32, "d": 64, "rot": 32, "layout": "pairs",
         "type": "bf16", "k_bits": 4, "v_bits": 4, "v_alg": 1, "page": 32, "far": 4096, "skip": 0.1},
        # one decode step of a few short sequences
        {"name": "attend_step_short", "op": "attend", "batch": 4, "hq": 32, "hkv": 8, "d": 128, "q_len": 1,
         "kv_len": 1000, "ragged": True, "k_bits": 3, "v_bits": 2, "v_alg": 2, "page": 16, "cap": 0.0,
         "window": 0, "slopes": False, "prefix": False},
        # one decode step over long contexts
        {"name": "attend_step_long", "op": "attend", "batch": 16, "hq": 32, "hkv": 8, "d": 128, "q_len": 1,
         "kv_len": 32768, "ragged": True, "k_bits": 3, "v_bits": 2, "v_alg": 2, "page": 64, "cap": 0.0,
         "window": 0, "slopes": False, "prefix": False},
        # a decode step without shared heads, capped scores and a sliding window
        {"name": "attend_step_window", "op": "attend", "batch": 32, "hq": 32, "hkv": 32, "d": 64, "q_len": 1,
         "kv_len": 4096, "ragged": True, "k_bits": 4, "v_bits": 4, "v_alg": 1, "page": 32, "cap": 30.0,
         "window": 1024, "slopes": False, "prefix": False},
        # a batch of chunks of many lengths, single tokens among them; distance bias and prefix mask
        {"name": "attend_mixed", "op": "attend", "batch": 7, "hq": 32, "hkv": 8, "d": 128, "q_len": 300,
         "kv_len": 2500, "ragged": True, "k_bits": 3, "v_bits": 3, "v_alg": 1, "page": 16, "cap": 0.0,
         "window": 0, "slopes": True, "prefix": True},
        # a chunk of a long prompt, values by Algorithm 2
        {"name": "attend_chunk", "op": "attend", "batch": 1, "hq": 32, "hkv": 8, "d": 128, "q_len": 2048,
         "kv_len": 8192, "ragged": False, "k_bits": 3, "v_bits": 2, "v_alg": 2, "page": 64, "cap": 0.0,
         "window": 0, "slopes": False, "prefix": False},
        # the largest: a chunk at the end of a long prompt, values by Algorithm 1, capped scores
        {"name": "attend_chunk_long", "op": "attend", "batch": 2, "hq": 32, "hkv": 8, "d": 128, "q_len": 2048,
         "kv_len": 16384, "ragged": False, "k_bits": 3, "v_bits": 3, "v_alg": 1, "page": 128, "cap": 50.0,
         "window": 0, "slopes": False, "prefix": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    d = rng.choice([64, 128])
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 8192), "heads": rng.randint(1, 40), "d": d,
                "rot": 2 * rng.randint(1, d // 2), "layout": rng.choice(["half", "pairs"]),
                "inverse": rng.random() < 0.5, "type": rng.choice(["bf16", "f16", "f32"]),
                "far": _log(rng, 16, 131072)}
    v_alg = rng.choice([1, 2])
    pool = {"k_bits": rng.randint(1, 4), "v_bits": rng.randint(2, 4), "v_alg": v_alg, "page": rng.choice([16, 32, 64, 128])}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 8192), "hkv": rng.randint(1, 8), "d": d,
                "rot": rng.choice([0, 2 * rng.randint(1, d // 2), d]), "layout": rng.choice(["half", "pairs"]),
                "type": rng.choice(["bf16", "f32"]), "far": _log(rng, 16, 131072), "skip": rng.choice([0.0, 0.2]), **pool}
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 7, 8, 16])
    q_len = rng.choice([1, 1, _log(rng, 2, 600)])
    return {"op": op, "batch": rng.randint(1, 16 if q_len == 1 else 4), "hq": hq, "hkv": hkv, "d": d, "q_len": q_len,
            "kv_len": max(q_len, _log(rng, 1, 16000 if q_len == 1 else 4000)), "ragged": rng.random() < 0.7,
            "cap": rng.choice([0.0, 0.0, 20.0]), "window": rng.choice([0, 0, _log(rng, 1, 4000)]),
            "slopes": rng.random() < 0.25, "prefix": rng.random() < 0.25, **pool}


# ---- inputs --------------------------------------------------------------------------------------

def vectors(n, d, gen):
    """Rows as KV heads give them: unit Gaussian coordinates, a few strong channels, a spread of lengths."""
    x = torch.randn(n, d, generator=gen, device="cuda")
    strong = torch.randperm(d, generator=gen, device="cuda")[: max(1, d // 40)]
    x[:, strong] *= 8.0
    return x * torch.exp(0.5 * torch.randn(n, 1, generator=gen, device="cuda"))


def angles(rot, far, positions):
    """The rows of the (cos, sin) table that `positions` may name: float32 [far][rot/2][2]."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = positions.double()[:, None] * freq
    table = torch.zeros(far, rot // 2, 2, device="cuda")
    table[positions] = torch.stack([a.cos(), a.sin()], -1).float()
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = types.SimpleNamespace(**case)
    if s.op == "rope":
        prepare_rope(s, gen)
    elif s.op == "append":
        prepare_append(s, gen)
    else:
        prepare_attend(s, gen)
    if own:
        prepare_handles(s)
    return s


def positions_of(tokens, far, gen):
    """Where the tokens stand: a run of positions where it fits, else anywhere."""
    if tokens > far or tokens < 100:
        return torch.randint(0, far, (tokens,), generator=gen, device="cuda")
    first = torch.randint(0, far - tokens + 1, (1,), generator=gen, device="cuda")
    return first + torch.arange(tokens, device="cuda")


def prepare_rope(s, gen):
    pos = positions_of(s.tokens, s.far, gen)
    s.x = torch.randn(s.tokens, s.heads, s.d, generator=gen, device="cuda").to(TYPES[s.type])
    s.out = torch.zeros_like(s.x)
    s.positions, s.table = pos.int(), angles(s.rot, s.far, pos)


def empty_pool(s, pages):
    """The cache's arrays, with what an allocator leaves in them: anything (here zeros, norms NaN)."""
    g, kb = s.d // 32, s.k_bits
    vb = s.v_bits - (s.v_alg == 2)
    word = functools.partial(torch.zeros, dtype=torch.int32, device="cuda")
    half = functools.partial(torch.full, fill_value=float("nan"), dtype=torch.float16, device="cuda")
    at = (pages, s.hkv, s.page)
    s.k_codes, s.k_norms, s.v_codes, s.v_norms = word((*at, g, kb)), half(at), word((*at, g, vb)), half(at)
    s.v_signs, s.v_gammas = (word((*at, g)), half(at)) if s.v_alg == 2 else (None, None)
    s.cb_k, s.cb_v = codebook(s.d, kb), codebook(s.d, vb)


def prepare_append(s, gen):
    n = s.tokens * s.hkv
    s.k = vectors(n, s.d, gen).reshape(s.tokens, s.hkv, s.d).to(TYPES[s.type])
    s.v = vectors(n, s.d, gen).reshape(s.tokens, s.hkv, s.d).to(TYPES[s.type])
    s.k[s.tokens // 2, 0] = 0  # a dead head
    s.v[s.tokens // 3, -1] = 0
    pages = -(-s.tokens // s.page) + 2
    empty_pool(s, pages)
    s.k_norms.zero_(), s.v_norms.zero_()
    if s.v_gammas is not None:
        s.v_gammas.zero_()
    slots = torch.randperm(pages, generator=gen, device="cuda")[:, None] * s.page + torch.arange(s.page, device="cuda")
    s.slots = slots.reshape(-1)[: s.tokens].clone()
    if s.tokens < 100:  # single tokens of many sequences lie anywhere
        s.slots = torch.randperm(pages * s.page, generator=gen, device="cuda")[: s.tokens]
    s.slots[torch.rand(s.tokens, generator=gen, device="cuda") < s.skip] = -1  # rows that only pad the batch
    pos = positions_of(s.tokens, s.far, gen)
    s.positions, s.table = (pos.int(), angles(s.rot, s.far, pos)) if s.rot else (None, None)
    s.Pi, s.S = matrices(s.d, gen)


def prepare_attend(s, gen):
    host = np.random.RandomState(100003 * s.batch + 1009 * s.kv_len + s.q_len)  # the lengths belong to the case
    if s.ragged:
        kv = np.maximum(1, (s.kv_len * (1 - 0.7 * host.rand(s.batch) ** 2)).astype(np.int64))
        kv[0] = s.kv_len
        ql = np.minimum(kv, np.maximum(1, (s.q_len * host.rand(s.batch) ** 2).astype(np.int64)))
        ql[-1] = min(kv[-1], s.q_len)
    else:
        kv, ql = np.full(s.batch, s.kv_len), np.full(s.batch, s.q_len)
    start = np.concatenate([[0], np.cumsum(ql)])
    total = int(start[-1])
    s.max_q, s.max_kv, s.total = int(ql.max()), int(kv.max()), total
    s.q = torch.randn(total, s.hq, s.d, generator=gen, device="cuda").bfloat16()
    s.out = torch.zeros_like(s.q)
    as_int = lambda a: torch.from_numpy(np.ascontiguousarray(a)).int().cuda()  # noqa: E731
    s.q_start, s.kv_lens = as_int(start), as_int(kv)
    need = -(-kv // s.page)
    pages = int(need.sum())
    table = np.full((s.batch, int(need.max())), -1)
    order = torch.randperm(pages, generator=gen, device="cuda").cpu().numpy()
    at = 0
    for b in range(s.batch):
        table[b, : need[b]] = order[at : at + need[b]]
        at += need[b]
    s.pages = as_int(table)
    s.prefix_lens = as_int(np.minimum(kv, (host.rand(s.batch) * kv).astype(np.int64))) if s.prefix else None
    s.alibi = (2.0 ** (-8.0 * torch.arange(1, s.hq + 1, device="cuda") / s.hq)).float() if s.slopes else None
    s.scale = 1.0 / math.sqrt(s.d)
    s.Pi, s.S = matrices(s.d, gen)
    empty_pool(s, pages)
    fill_pool(s, table, kv, gen)
    rows = np.repeat(np.arange(s.batch), ql)
    s.row_b = torch.from_numpy(rows).cuda()
    s.row_j = torch.from_numpy(np.arange(total) - start[rows]).cuda()


def fill_pool(s, table, kv, gen):
    """Encodes random vectors into every slot that a sequence has filled; the others stay as they are."""
    t = np.arange(table.shape[1] * s.page)
    slots = (table.repeat(s.page, axis=1) * s.page + t % s.page)[t[None] < kv[:, None]]
    slots = torch.from_numpy(slots).cuda()
    for part in slots.split(1 << 16):
        at = (part // s.page, slice(None), part % s.page)
        n = part.numel() * s.hkv
        for codes, norms, cb, alg2 in ((s.k_codes, s.k_norms, s.cb_k, False), (s.v_codes, s.v_norms, s.cb_v, s.v_alg == 2)):
            x = vectors(n, s.d, gen)
            norm = x.norm(dim=1, keepdim=True)
            levels, bounds = (torch.from_numpy(a).cuda() for a in cb)
            y = (x / norm) @ s.Pi.T
            idx = torch.bucketize(y, bounds)
            codes[at] = pack(idx, codes.shape[-1]).reshape(part.numel(), s.hkv, *codes.shape[3:])
            norms[at] = norm.half().reshape(part.numel(), s.hkv)
            if alg2:
                r = x / norm - levels[idx] @ s.Pi
                s.v_signs[at] = planes(((r @ s.S.T) >= 0).reshape(n, -1, 32)).reshape(part.numel(), s.hkv, -1)
                s.v_gammas[at] = r.norm(dim=1).half().reshape(part.numel(), s.hkv)


def prepare_handles(s):
    """What a user's program keeps between calls: the prepared rotation, the cache's handle, a workspace."""
    import kv_cache_vector_encode_b200 as tq
    s.tq = tq
    if s.op == "rope":
        s.style = tq.TQ_ROPE_HALF if s.layout == "half" else tq.TQ_ROPE_PAIRS
        return

    def book(cb):
        c = tq.Codebook(d=s.d, bits=int(cb[0].size).bit_length() - 1, levels=cb[0].size)
        c.c[: c.levels], c.t[: c.levels - 1] = cb[0].tolist(), cb[1].tolist()
        c.c64[: c.levels], c.t64[: c.levels - 1] = cb[0].tolist(), cb[1].tolist()
        return c

    s.rotation = tq.tq_rotation_prepare(s.Pi, s.S)
    s.kv = tq.PagedKV(book(s.cb_k), book(s.cb_v), s.k_codes, s.k_norms, s.v_codes, s.v_norms, s.v_signs, s.v_gammas)
    if s.op == "append":
        s.style = tq.TQ_ROPE_HALF if s.layout == "half" else tq.TQ_ROPE_PAIRS
    else:
        need = tq.tq_paged_attend_workspace_bytes(s.kv, s.batch, s.hq, s.total, s.max_q, s.max_kv)
        s.ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


# ---- the operators -------------------------------------------------------------------------------

def run(s):
    if s.op == "rope":
        if own:
            s.tq.tq_rope(s.x, s.positions, s.table, out=s.out, layout=s.style, inverse=s.inverse)
            return s.out
        return rope(s.x.float(), s.positions, s.table, s.layout, s.inverse).to(s.x.dtype)
    if s.op == "append":
        if own:
            s.tq.tq_paged_append(s.kv, s.k, s.v, s.slots, s.rotation, positions=s.positions, table=s.table, layout=s.style)
        else:
            append(s)
        pools = {"k_codes": s.k_codes, "k_norms": s.k_norms, "v_codes": s.v_codes, "v_norms": s.v_norms}
        return pools | ({"v_signs": s.v_signs, "v_gammas": s.v_gammas} if s.v_alg == 2 else {})
    if own:
        s.tq.tq_paged_attend(s.kv, s.q, s.q_start, s.kv_lens, s.pages, s.rotation, s.out, max_q_len=s.max_q,
                             max_kv_len=s.max_kv, scale=s.scale, softcap=s.cap, window=s.window, slopes=s.alibi,
                             prefix_len=s.prefix_lens, ws=s.ws)
        return s.out
    return attend(s)


def rope(x, positions, table, layout, inverse):
    """Rotates pair i of the first 2 * table.shape[1] coordinates by the angle of (position, i)."""
    h = table.shape[1]
    c, sn = (table[positions.long()].to(x.dtype)[:, None, :, k] for k in (0, 1))
    sn = -sn if inverse else sn
    part, rest = x[..., : 2 * h], x[..., 2 * h :]
    if layout == "half":
        a, b = part[..., :h], part[..., h:]
        return torch.cat([a * c - b * sn, b * c + a * sn, rest], -1)
    a, b = part[..., 0::2], part[..., 1::2]
    return torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), rest], -1)


def encode(x, Pi, S, cb, alg2):
    """Codes, norms (and signs, residual norms) of the rows of x, in 64 bits: values next to a border count."""
    levels, bounds = (torch.from_numpy(a).to(x.device).double() for a in cb)
    Pi = Pi.double()
    norm = x.square().sum(-1, keepdim=True).sqrt()
    u = x / torch.where(norm > 0, norm, 1.0)
    idx = ((u @ Pi.T)[..., None, :] > bounds[:, None]).sum(-2)
    codes = pack(idx, levels.numel().bit_length() - 1)
    if not alg2:
        return codes, norm[:, 0].half(), None, None
    r = torch.where(norm > 0, u - levels[idx] @ Pi, 0.0)
    z = (r @ S.double().T) >= 0
    return codes, norm[:, 0].half(), planes(z.reshape(z.shape[0], -1, 32)), r.square().sum(-1).sqrt().half()


def append(s):
    k = s.k.double()
    if s.rot:
        k = rope(k, s.positions, s.table, s.layout, False)
    kc, kn, _, _ = encode(k.reshape(-1, s.d), s.Pi, s.S, s.cb_k, False)
    vc, vn, vz, vg = encode(s.v.double().reshape(-1, s.d), s.Pi, s.S, s.cb_v, s.v_alg == 2)
    live = s.slots >= 0
    slots = s.slots[live]
    at = (slots // s.page, slice(None), slots % s.page)
    new = lambda a: a.reshape(s.tokens, s.hkv, *a.shape[1:])[live]  # noqa: E731
    s.k_codes[at], s.k_norms[at], s.v_codes[at], s.v_norms[at] = new(kc), new(kn), new(vc), new(vn)
    if s.v_alg == 2:
        s.v_signs[at], s.v_gammas[at] = new(vz), new(vg)


def attend(s):
    d, g = s.d, s.hq // s.hkv
    alpha = math.sqrt(math.pi / 2) / d
    lev_k, lev_v = (torch.from_numpy(cb[0]).cuda() for cb in (s.cb_k, s.cb_v))
    pages = s.pages.long().clamp(min=0)
    t = torch.arange(pages.shape[1] * s.page, device="cuda")
    filled = t[None] < s.kv_lens[:, None]

    def seen(a):  # [pages][Hkv][page]... -> [B][Hkv][T]...
        return a[pages].transpose(1, 2).flatten(2, 3)

    k = seen(s.k_norms).float()[..., None] * (lev_k[unpack(seen(s.k_codes)).long()] @ s.Pi)
    v = lev_v[unpack(seen(s.v_codes)).long()] @ s.Pi
    if s.v_alg == 2:
        v = v + alpha * seen(s.v_gammas).float()[..., None] * (signs_of(seen(s.v_signs)) @ s.S)
    v = seen(s.v_norms).float()[..., None] * v
    v = torch.where(filled[:, None, :, None], v, 0.0)
    q_len = s.q_start[1:] - s.q_start[:-1]
    j = torch.arange(s.max_q, device="cuda")
    rows = (s.q_start[:-1, None] + j).clamp(max=s.total - 1).long()
    q = s.q.float()[rows].reshape(s.batch, s.max_q, s.hkv, g, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = (s.scale * (q @ k.transpose(-1, -2))).reshape(s.batch, s.hkv, g, s.max_q, -1)
    if s.cap:
        scores = s.cap * torch.tanh(scores / s.cap)
    pos = s.kv_lens[:, None] - q_len[:, None] + j
    ahead = t[None, None] - pos[..., None]  # how far token t lies behind query j
    if s.slopes:
        scores = scores + s.alibi.reshape(1, s.hkv, g, 1, 1) * ahead[:, None, None]
    ok = ahead <= 0
    if s.window:
        ok = ok & (ahead > -s.window)
    if s.prefix:
        ok = ok | (t[None, None] < s.prefix_lens[:, None, None])
    ok = (ok & filled[:, None])[:, None, None]
    scores = torch.where(ok, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).reshape(s.batch, s.hkv, g, s.max_q, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).flatten(2, 3)
    s.out.copy_(o[s.row_b, s.row_j].to(s.out.dtype))
    return s.out


# ---- what one pass cannot do without -------------------------------------------------------------

def work(case):
    s = types.SimpleNamespace(**case)
    if s.op == "rope":
        size = {"bf16": 2, "f16": 2, "f32": 4}[s.type]
        n = s.tokens * s.heads
        return {"bytes": 2 * n * s.d * size + 4 * s.tokens * (s.rot + 1), "flops": 3 * n * s.rot}
    g = s.d // 32
    k_rec, v_rec = 4 * g * s.k_bits + 2, 4 * g * s.v_bits + (4 if s.v_alg == 2 else 2)
    if s.op == "append":
        n = s.tokens * s.hkv
        size = 2 if s.type == "bf16" else 4
        products = 4 if s.v_alg == 2 else 2
        return {"bytes": n * (2 * s.d * size + k_rec + v_rec) + s.tokens * (8 + 4 * (s.rot + 1)),
                "flops": n * (2.0 * s.d * s.d * products + 3 * s.rot)}
    # ragged batches: their mean length
    kv = s.kv_len * (1 - 0.7 / 3) if s.ragged else s.kv_len
    ql = max(1.0, s.q_len / 3) if s.ragged else s.q_len
    ql = min(ql, kv)
    seen = kv - (ql - 1) / 2
    if s.window:
        seen = min(seen, s.window) if not s.prefix else seen
    read = min(kv, s.window + ql) if s.window and not s.prefix else kv
    return {"bytes": s.batch * (s.hkv * read * (k_rec + v_rec) + 4 * ql * s.hq * s.d),
            "flops": 4.0 * s.batch * s.hq * ql * seen * s.d}


# ---- in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if s.op == "rope":
        return exact_rope(s.x, s)
    return exact_append(s) if s.op == "append" else exact_attend(s)


def exact_rope(x, s):
    """As a product of complex numbers: (a + ib) (cos + i sin)."""
    x = x.double()
    turn = torch.view_as_complex(s.table[s.positions.long()].double())[:, None]
    if getattr(s, "inverse", False):
        turn = turn.conj()
    h = s.rot // 2
    if s.layout == "half":
        z = torch.complex(x[..., :h], x[..., h : 2 * h]) * turn
        return torch.cat([z.real, z.imag, x[..., 2 * h :]], -1)
    z = torch.view_as_complex(x[..., : 2 * h].reshape(*x.shape[:-1], h, 2)) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), x[..., 2 * h :]], -1)


def exact_append(s):
    """On the host, vector by vector in numpy."""
    Pi, S = s.Pi.double().cpu().numpy(), s.S.double().cpu().numpy()
    k = (exact_rope(s.k, s) if s.rot else s.k.double()).cpu().numpy()
    v, slots = s.v.double().cpu().numpy(), s.slots.cpu().numpy()
    live = np.flatnonzero(slots >= 0)
    page, off = slots[live] // s.page, slots[live] % s.page

    def words(b):
        return np.packbits(b.reshape(*b.shape[:-1], -1, 32).astype(np.uint8), axis=-1, bitorder="little").view(np.int32)[..., 0]

    def stored(pool, fill):
        a = pool.cpu().numpy().astype(np.float64 if pool.is_floating_point() else np.int32)
        a[page, :, off] = fill
        return torch.from_numpy(a)

    out = {}
    for name, x, cb, alg2 in (("k", k[live], s.cb_k, False), ("v", v[live], s.cb_v, s.v_alg == 2)):
        levels, bounds = cb[0].astype(np.float64), cb[1].astype(np.float64)
        n = np.sqrt(np.einsum("thi,thi->th", x, x))[..., None]
        y = np.einsum("ij,thj->thi", Pi, x, optimize=True)
        idx = np.searchsorted(bounds, y / np.where(n > 0, n, 1.0), side="left")
        codes = np.stack([words(idx >> p & 1) for p in range(len(levels).bit_length() - 1)], -1)
        out[name + "_codes"] = stored(getattr(s, name + "_codes"), codes)
        out[name + "_norms"] = stored(getattr(s, name + "_norms"), n[..., 0])
        if alg2:
            r = (x / np.where(n > 0, n, 1.0) - np.einsum("thi,ij->thj", levels[idx], Pi, optimize=True)) * (n > 0)
            out["v_signs"] = stored(s.v_signs, words(np.einsum("ij,thj->thi", S, r, optimize=True) >= 0))
            out["v_gammas"] = stored(s.v_gammas, np.sqrt(np.einsum("thi,thi->th", r, r)))
    return out


def exact_attend(s):
    """Sequence by sequence, KV head by KV head, query rows in parts; the scores in the rotated domain."""
    Pi, S, d, g = s.Pi.double(), s.S.double(), s.d, s.hq // s.hkv
    alpha = math.sqrt(math.pi / 2) / d
    lev_k, lev_v = (torch.from_numpy(cb[0]).cuda().double() for cb in (s.cb_k, s.cb_v))
    out = torch.zeros(s.total, s.hq, d, dtype=torch.float64, device="cuda")
    start, lens = s.q_start.tolist(), s.kv_lens.tolist()
    for b in range(s.batch):
        n, m = lens[b], start[b + 1] - start[b]
        if not m or not n:
            continue
        t = torch.arange(n, device="cuda")
        page, off = s.pages[b].long()[t // s.page], t % s.page
        q = s.q[start[b] : start[b + 1]].double() @ Pi.T
        for h in range(s.hkv):
            k = lev_k[unpack(s.k_codes[page, h, off]).long()] * s.k_norms[page, h, off].double()[:, None]
            v = lev_v[unpack(s.v_codes[page, h, off]).long()] @ Pi
            if s.v_alg == 2:
                v = v + alpha * s.v_gammas[page, h, off].double()[:, None] * (signs_of(s.v_signs[page, h, off]).double() @ S)
            v = v * s.v_norms[page, h, off].double()[:, None]
            for first in range(0, m, 256):
                rows = torch.arange(first, min(m, first + 256), device="cuda")
                x = torch.einsum("jgd,td->gjt", q[rows][:, h * g : (h + 1) * g], k) * s.scale
                if s.cap:
                    x = s.cap * torch.tanh(x / s.cap)
                pos = (n - m + rows)[:, None]
                if s.slopes:
                    x = x + s.alibi[h * g : (h + 1) * g].double()[:, None, None] * (t[None] - pos)
                ok = t[None] <= pos
                if s.window:
                    ok &= t[None] > pos - s.window
                if s.prefix:
                    ok |= t[None] < s.prefix_lens[b]
                x = x.masked_fill(~ok, float("-inf"))
                w = torch.softmax(x, -1).nan_to_num(0.0)
                out[start[b] + rows, h * g : (h + 1) * g] = torch.einsum("gjt,td->jgd", w, v)
    return out
