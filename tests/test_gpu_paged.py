"""GPU parity of the rotary and paged-cache operators against the oracle (B200).

Tolerances, from the roundings made on the way (a rounding is off by at most half a step, eps / 2 relative):
* tq_rope: products and sums in fp32, rounded once: eps/2 |out| + 2^-22 (|a c| + |b s|).
* tq_paged_append: indices and signs as in fp64 (both sides are sums of d fp64 products: 1e-12 of the scale), norms one
  rounding to fp16. The residual is a unit vector minus a product of split fp16 operands: three 2^-22 for the splits
  and 16 2^-23 for the accumulation make 2^-18.4 per coordinate at most, so its length is off by sqrt(d) 2^-18.4 at
  most before it is rounded to fp16.
* tq_paged_attend: scores take the queries (2^-11), the levels or opened keys (2^-11 each step, two at most) in fp16,
  so |x - x_exact| <= E = 3 2^-11 scale |q| max|k_t| (Cauchy); weights then are off by a factor within e^(+-2E), and
  weights, levels and opened values by 2^-11 each (four at most):
  |out - exact| <= (e^(2E) - 1 + 4 2^-11) sum_t p_t |v_t| per row (normwise), plus the bf16 rounding 2^-8 |out|.
"""
import math

import numpy as np
import pytest

import workloads as W
from oracle import paged as OP
from oracle import quant as Q
from parity import np_f16, np_u32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("kv_cache_vector_encode_b200")


@pytest.fixture(scope="module")
def dev(gpu_required):
    tq.lib()
    return torch.device("cuda")


_rot = {}


def rotation(d, dev):
    if d not in _rot:
        Pi, S = W.rotation(d), W.jl_matrix(d)
        _rot[d] = (Pi, S, tq.tq_rotation_prepare(torch.from_numpy(Pi).to(dev), torch.from_numpy(S).to(dev)))
    return _rot[d]


def i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).to(dev)


DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---- rotary positions ----------------------------------------------------------------------------

@pytest.mark.parametrize("kw", [dict(), dict(scaling=1, factor=4.0),
                                dict(scaling=2, factor=8.0, low_turns=1.0, high_turns=16.0, original_len=4096.0, magnitude=1.2)])
@pytest.mark.parametrize("rot", [2, 48, 128])
def test_rope_table(dev, rot, kw):
    n = 40001
    table = tq.tq_rope_table(n, rot, base=500000.0, **kw).cpu().numpy()
    args = {k: v for k, v in kw.items() if k not in ("scaling", "magnitude")}
    f = OP.rope_freqs(rot, 500000.0, ["plain", "linear", "blend"][kw.get("scaling", 0)], **args)
    want = OP.rope_table(n, f, kw.get("magnitude", 1.0))
    # fp64 angles up to 4e4, both sides with a relative error of a few 2^-53, then one rounding to fp32
    assert np.max(np.abs(table - want)) <= 2.0**-24 * kw.get("magnitude", 1.0) + 1e-10
    assert tq.tq_rope_table(0, rot).shape == (0, rot // 2, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("tokens,heads,d,rot,pad", [
    (1, 1, 2, 2, 0), (1, 32, 128, 128, 0), (3, 5, 64, 48, 0), (7, 3, 80, 20, 0), (5, 2, 33, 6, 0), (257, 40, 128, 128, 64),
    (64, 8, 96, 96, 3), (19, 3, 576, 512, 8),
])
def test_rope(dev, tokens, heads, d, rot, pad, pairs, dtype):
    rng = np.random.default_rng(tokens * 131 + d)
    n_pos = 5000
    table = tq.tq_rope_table(n_pos, rot)
    pos = rng.integers(0, n_pos, tokens)
    pos[0] = n_pos - 1
    if tokens > 2:
        pos[1], pos[2] = -1, 0
    buf = torch.from_numpy(rng.standard_normal((tokens, heads, d + pad))).to(dev).to(DTYPES[dtype])
    x = buf[:, :, :d]
    tab = table.cpu().numpy()
    xs = x.double().cpu().numpy()
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    for inverse in (False, True):
        want = OP.rope(xs, pos, tab, pairs, inverse)
        # |a c| + |b s| <= sqrt(2) times the pair's length, which the turn keeps
        partner = np.abs(OP.rope(xs, pos, tab, pairs, not inverse))
        tol = eps * np.abs(want) + 2.0**-22 * (np.abs(xs) + np.abs(want) + partner) * 1.5 + 2.0**-25
        out = torch.full((tokens, heads, d), 7.0, dtype=DTYPES[dtype], device=dev)
        assert tq.tq_rope(x, i32(pos, dev), table, out=out, layout=int(pairs), inverse=inverse) is out
        got = out.double().cpu().numpy()
        assert np.all(got[pos < 0] == 7.0)
        want[pos < 0] = 7.0
        assert np.all(np.abs(got - want) <= tol)
        before = buf.clone()
        y = buf.clone()
        tq.tq_rope(y[:, :, :d], i32(pos, dev), table, layout=int(pairs), inverse=inverse)      # in place
        assert torch.equal(y[:, :, :d][torch.from_numpy(pos >= 0).to(dev)], out[torch.from_numpy(pos >= 0).to(dev)])
        assert torch.equal(y[:, :, d:], before[:, :, d:])
        assert torch.equal(y[torch.from_numpy(pos < 0).to(dev)], before[torch.from_numpy(pos < 0).to(dev)])
    tq.tq_sync_check()


def test_rope_head_major_and_shared_input(dev):
    """Heads outside tokens, and one head's data broadcast over eight (stride 0) into an output of its own."""
    rng = np.random.default_rng(3)
    table = tq.tq_rope_table(300, 64)
    x = torch.from_numpy(rng.standard_normal((6, 11, 64))).to(dev).float()
    pos = rng.integers(0, 300, 11)
    want = OP.rope(x.transpose(0, 1).double().cpu().numpy(), pos, table.cpu().numpy(), False)
    y = x.clone()
    tq.tq_rope(y.transpose(0, 1), i32(pos, dev), table)
    assert np.max(np.abs(y.transpose(0, 1).double().cpu().numpy() - want)) <= 2.0**-19
    one = x[:1].transpose(0, 1).expand(11, 8, 64)
    out = torch.empty(11, 8, 64, device=dev)
    tq.tq_rope(one, i32(pos, dev), table, out=out)
    assert torch.equal(out[:, 3], y.transpose(0, 1)[:, 0])


def test_rope_inverse_is_the_gradient(dev):
    """The inverse turn of the output's gradient against the formula's gradient and central differences (fp32 input)."""
    rng = np.random.default_rng(5)
    table = tq.tq_rope_table(100, 24)
    tab = table.cpu().numpy()
    pos = rng.integers(0, 100, 4)
    x, go = rng.standard_normal((4, 2, 32)), rng.standard_normal((4, 2, 32)).astype(np.float32)
    gx = torch.from_numpy(go).to(dev)
    tq.tq_rope(gx, i32(pos, dev), table, layout=tq.TQ_ROPE_PAIRS, inverse=True)
    got = gx.double().cpu().numpy()
    for at in [(0, 0, 0), (1, 1, 7), (2, 0, 23), (3, 1, 30)]:
        h = 0.5                                                  # linear: differences are exact
        lo, hi = x.copy(), x.copy()
        lo[at] -= h
        hi[at] += h
        diff = ((OP.rope(hi, pos, tab, True) - OP.rope(lo, pos, tab, True)) / (2 * h) * go).sum()
        assert abs(diff - got[at]) <= 2.0**-21 * 4


def test_rope_reports_positions_out_of_range(dev):
    table = tq.tq_rope_table(10, 32)
    x = torch.ones(3, 1, 32, device=dev)
    tq.tq_rope(x, torch.tensor([1, 10, 2], dtype=torch.int32, device=dev), table)
    with pytest.raises(tq.TQError):
        tq.tq_sync_check()
    tq.tq_sync_check()
    assert torch.all(x[1] == 1) and not torch.all(x[2] == 1)


# ---- append --------------------------------------------------------------------------------------

def heads_data(rng, tokens, Hkv, d):
    x = rng.standard_normal((tokens, Hkv, d)) * np.exp(0.5 * rng.standard_normal((tokens, Hkv, 1)))
    x[..., rng.choice(d, 2, replace=False)] *= 8.0
    return x


def filled(dev, pages, Hkv, ps, d, kb, vb, alg, value=0x5A5A5A5A):
    """A cache whose arrays all hold a known pattern."""
    kv = tq.empty_paged(pages, Hkv, ps, d, kb, vb, alg, device=dev)
    for t in kv.tensors:
        if t is not None:
            t.view(torch.int32).fill_(value)
    return kv


def records(kv):
    """The arrays as numpy, vector by vector [pages, page_size, Hkv, ...]."""
    out = []
    for t in kv.tensors:
        out.append(None if t is None else (np_u32(t) if t.dtype is torch.int32 else np_f16(t)).swapaxes(1, 2))
    return out


def check_append(kv, before, k, v, slots, dev, alg):
    d, ps = kv.d, kv.page_size
    Pi, S, _ = rotation(d, dev)
    live = np.flatnonzero(slots >= 0)
    page, off = slots[live] // ps, slots[live] % ps
    after = records(kv)
    mask = np.ones((kv.num_pages, ps), bool)
    mask[page, off] = False
    for a, b in zip(after, before):
        if a is not None:                                        # every other slot as it was
            assert np.array_equal(a[mask].view(np.uint8), b[mask].view(np.uint8))
    kc, kn, vc, vn, vs, vg = [None if a is None else a[page, off].reshape(len(live) * kv.Hkv, *a.shape[3:]) for a in after]
    for x, codes, norms, signs, gammas in ((k, kc, kn, None, None), (v, vc, vn, vs, vg)):
        cb = Q_cb(d, codes.shape[-1])
        rows = x[live].reshape(-1, d)
        e = Q.encode_prod(rows, Pi, S, cb) if signs is not None else Q.encode_mse(rows, Pi, cb)
        idx = Q.unpack_planes(codes, codes.shape[-1])
        wrong = idx != e["idx"]
        near = np.min(np.abs(e["y"][..., None] - cb.t32.astype(np.float64)), -1) < 1e-12
        zero = ~(np.isfinite(e["n"]) & (e["n"] > 0))             # u = 0: y lies on a boundary, exactly
        assert not np.any(wrong & ~(near & ~zero[:, None]))
        same_norm = (norms == e["norms"]) | (np.isnan(norms) & np.isnan(e["norms"]))
        with np.errstate(invalid="ignore"):
            mid = np.abs(norms.astype(np.float64) - e["n"]) <= 2.0**-11 * (1 + 1e-9) * np.abs(e["n"]) + 2.0**-25
        assert np.all(same_norm | mid)
        if signs is not None:
            ok = ~wrong.any(1)
            z = Q.unpack_signs(signs)
            assert not np.any((z != e["z"])[ok] & ~(np.abs(e["s"]) < 1e-11)[ok])
            assert np.all((np.abs(gammas.astype(np.float64) - e["gamma"]) <= 2.0**-11 * e["gamma"] + math.sqrt(d) * 2.0**-18.4)[ok])


def Q_cb(d, bits):
    from oracle.codebook import lloyd_max
    return lloyd_max(d, bits)


@pytest.mark.parametrize("tokens,Hkv,d,kb,vb,alg,ps,rot,pairs,dtype", [
    (1, 1, 128, 3, 3, 2, 16, 128, False, "bf16"),
    (3, 2, 64, 4, 4, 1, 16, 64, True, "f32"),
    (17, 8, 128, 1, 2, 2, 32, 64, True, "bf16"),
    (33, 3, 64, 2, 1, 1, 64, 0, False, "bf16"),
    (50, 8, 128, 4, 4, 2, 128, 128, False, "f32"),
    (5, 2, 128, 2, 3, 1, 1024, 2, False, "bf16"),
    (700, 3, 128, 3, 3, 2, 64, 128, False, "bf16"),
    (1500, 2, 64, 4, 4, 1, 32, 32, True, "bf16"),
    (2111, 2, 64, 2, 2, 2, 16, 62, False, "f32"),
    (1025, 4, 128, 3, 2, 1, 16, 0, False, "f32"),
])
def test_append(dev, tokens, Hkv, d, kb, vb, alg, ps, rot, pairs, dtype):
    rng = np.random.default_rng(tokens + 7 * d + kb)
    pages = -(-tokens // ps) + 3
    kv = filled(dev, pages, Hkv, ps, d, kb, vb, alg)
    before = records(kv)
    buf = torch.from_numpy(np.stack([heads_data(rng, tokens, Hkv, d), heads_data(rng, tokens, Hkv, d)], 1)).to(dev).to(DTYPES[dtype])
    buf[tokens // 2, :, 0] = 0                                   # zero vectors
    k, v = buf[:, 0], buf[:, 1]                                  # token stride 2 Hkv d
    slots = rng.permutation(pages * ps)[:tokens]
    if tokens > 4:
        slots[[1, 4]] = -1, -7
    n_pos = 3000
    pos = rng.integers(0, n_pos, tokens)
    pos[-1] = n_pos - 1
    table = tq.tq_rope_table(n_pos, rot) if rot else None
    tq.tq_paged_append(kv, k, v, torch.from_numpy(slots).to(dev), rotation(d, dev)[2], positions=i32(pos, dev) if rot else None,
                       table=table, layout=int(pairs))
    tq.tq_sync_check()
    kt = k.double().cpu().numpy()
    if rot:
        kt = OP.rope(kt, pos, table.cpu().numpy(), pairs)
    check_append(kv, before, kt, v.double().cpu().numpy(), slots, dev, alg)


@pytest.mark.parametrize("tokens", [6, 900])
def test_append_values_at_the_edges(dev, tokens):
    """Rows with infinities, NaN, fp16-overflowing and vanishing lengths, next to ordinary ones; slots and positions
    out of range are reported and skipped."""
    rng = np.random.default_rng(9)
    d, Hkv, ps, pages = 128, 2, 16, tokens // 16 + 2
    kv = filled(dev, pages, Hkv, ps, d, 3, 3, 2)
    before = records(kv)
    k, v = heads_data(rng, tokens, Hkv, d).astype(np.float32), heads_data(rng, tokens, Hkv, d).astype(np.float32)
    for x in (k, v):
        x[0, 0, 5], x[0, 1, 6], x[1, 0, 3] = np.inf, np.nan, -np.inf
        x[2, 0] *= 1e6
        x[2, 1] *= 1e-30
        x[3, 0] = 0
        x[3, 1] = 1e38
        x[4, 0] = x[4, 0] * 1e-39                                # subnormal
        x[4, 1] = np.where(np.arange(d) == 7, 1e-45, 0)
        x[5, 0] = np.sign(x[5, 0]) * 3e38
    slots = rng.permutation(pages * ps)[:tokens]
    tq.tq_paged_append(kv, torch.from_numpy(k).to(dev), torch.from_numpy(v).to(dev), torch.from_numpy(slots).to(dev), rotation(d, dev)[2])
    tq.tq_sync_check()
    check_append(kv, before, k.astype(np.float64), v.astype(np.float64), slots, dev, 2)
    before = records(kv)
    bad = slots.copy()
    bad[0], bad[1] = pages * ps, 1 << 40
    table = tq.tq_rope_table(4, 8)
    pos = np.full(tokens, 2)
    pos[2], pos[3] = 4, -1
    tq.tq_paged_append(kv, torch.from_numpy(k[::-1].copy()).to(dev), torch.from_numpy(v[::-1].copy()).to(dev),
                       torch.from_numpy(bad).to(dev), rotation(d, dev)[2], positions=i32(pos, dev), table=table)
    with pytest.raises(tq.TQError):
        tq.tq_sync_check()
    bad[:4] = -1
    kt = OP.rope(k[::-1].astype(np.float64), np.minimum(pos, 3), table.cpu().numpy(), False)
    check_append(kv, before, kt, v[::-1].astype(np.float64), bad, dev, 2)


# ---- attention -----------------------------------------------------------------------------------

class Paged:
    """Sequences of random records in a shuffled pool; everything no sequence fills holds random codes and NaN norms."""

    def __init__(self, dev, lens, Hkv, d, kb, vb, alg, ps, seed=0, spare=2, first_page=0):
        rng = np.random.default_rng(seed)
        self.dev, self.lens, self.alg, self.d, self.Hkv, self.ps = dev, lens, alg, d, Hkv, ps
        need = [-(-n // ps) for n in lens]
        self.pages = sum(need) + spare
        self.kv = tq.empty_paged(first_page + self.pages, Hkv, ps, d, kb, vb, alg, device=dev)
        order = rng.permutation(self.pages)
        width = max(max(need), 1) + 1
        self.table = np.full((len(lens), width), -1)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.host = []
        used = np.zeros((self.pages, ps), bool)
        for b, n in enumerate(lens):
            t = np.arange(n)
            used[self.table[b, t // ps], t % ps] = True
        for i, t in enumerate(self.kv.tensors):
            if t is None:
                self.host.append(None)
                continue
            shape = (self.pages, *t.shape[1:])
            if t.dtype is torch.int32:
                a = rng.integers(-2**31, 2**31, shape, dtype=np.int64).astype(np.int32)
            else:
                a = (0.35 if i == 5 else 6.0) * np.exp(0.4 * rng.standard_normal(shape))
                a = np.where(used[:, None], a, np.nan).astype(np.float16)
            self.host.append(a)
        self.first_page = first_page
        self.upload()

    def upload(self):
        for a, t in zip(self.host, self.kv.tensors):
            if a is not None:
                t[self.first_page:] = torch.from_numpy(a).to(self.dev)

    def sequence(self, b):
        """Decoded keys and values [Hkv, n, d] of a sequence (fp64)."""
        Pi, S, _ = rotation(self.d, self.dev)
        t = np.arange(self.lens[b])
        page, off = self.table[b, t // self.ps], t % self.ps
        page = np.where((page >= 0) & (page < self.pages), page, 0)
        kc, kn, vc, vn, vs, vg = self.host
        lev = [np.array(tq.tq_codebook_init(self.d, c.shape[-1]).c[: 1 << c.shape[-1]], np.float32) for c in (kc, vc)]
        k = np.stack([OP.dequant(kc[page, h, off].view(np.uint32), kn[page, h, off], lev[0], Pi) for h in range(self.Hkv)])
        v = np.stack([OP.dequant(vc[page, h, off].view(np.uint32), vn[page, h, off], lev[1], Pi, *(() if vs is None else (
            S, vs[page, h, off].view(np.uint32), vg[page, h, off]))) for h in range(self.Hkv)])
        return k, v

    def call(self, q, q_lens, pad=0, max_q=None, max_kv=None, prefix=None, slopes=None, ws=None, stream=None, **kw):
        start = np.concatenate([[0], np.cumsum(q_lens)])
        rows = int(start[-1])
        out = torch.full((rows + pad, *q.shape[1:]), float("nan"), dtype=torch.bfloat16, device=self.dev)
        table = np.where(self.table >= 0, self.table + self.first_page, -1)
        tq.tq_paged_attend(self.kv, q, i32(start, self.dev), i32(self.lens, self.dev), i32(table, self.dev),
                           rotation(self.d, self.dev)[2], out, max_q_len=max(q_lens) if max_q is None else max_q,
                           max_kv_len=max(self.lens) if max_kv is None else max_kv,
                           prefix_len=None if prefix is None else i32(prefix, self.dev),
                           slopes=None if slopes is None else torch.from_numpy(slopes).to(self.dev), ws=ws, stream=stream, **kw)
        return out

    def check(self, out, q, q_lens, softcap=0.0, window=0, prefix=None, slopes=None, scale=None, present=None, skip=()):
        got = out.double().cpu().numpy()
        start = np.concatenate([[0], np.cumsum(q_lens)])
        assert np.all(np.isnan(got[start[-1]:]))                 # padding rows as they were
        sc = scale or 1.0 / math.sqrt(self.d)
        qs = q.double().cpu().numpy()
        for b, m in enumerate(q_lens):
            if not m or b in skip:
                continue
            k, v = self.sequence(b)
            if present is not None and present[b] is not None:
                k, v = (np.where(present[b][None, :, None], a, 0.0) for a in (k, v))
            rows = slice(start[b], start[b + 1])
            want, size, reach = OP.attend(qs[rows], k, v, self.lens[b], sc, softcap, window, 0 if prefix is None else prefix[b],
                                          slopes, None if present is None else present[b])
            E = 3 * 2.0**-11 * reach
            tol = (np.expm1(2 * E) + 4 * 2.0**-11) * size + 2.0**-8 * np.linalg.norm(want, axis=-1)
            err = np.linalg.norm(got[rows] - want, axis=-1)
            assert np.all(err <= tol), (b, float(np.max(err / np.maximum(tol, 1e-30))))
            empty = size == 0
            assert np.all(got[rows][empty] == 0)


def queries(rng, rows, Hq, d, dev):
    return torch.from_numpy(rng.standard_normal((rows, Hq, d))).to(dev).to(torch.bfloat16)


CASES = [
    # lens, q_lens, Hq, Hkv, d, kb, vb (codebook + sign), alg, page, options
    ([1], [1], 1, 1, 128, 3, 3, 2, 16, {}),
    ([5, 0, 33, 16, 17], [1, 1, 1, 1, 1], 8, 2, 128, 3, 3, 2, 16, {}),
    ([700, 1, 129], [1, 1, 1], 32, 8, 64, 4, 4, 1, 32, dict(softcap=20.0)),
    ([1300, 40], [1, 1], 7, 1, 128, 2, 2, 1, 64, dict(window=100)),
    ([515, 64], [1, 1], 16, 1, 64, 1, 2, 2, 128, dict(window=1)),
    ([2000], [1], 4, 4, 128, 4, 4, 2, 1024, dict(slopes=True)),
    ([90, 300], [5, 3], 4, 2, 128, 3, 2, 2, 16, dict(prefix=True)),
    ([300, 20, 7, 0, 450], [9, 0, 7, 2, 1], 8, 2, 64, 3, 1, 1, 16, dict(window=30, prefix=True, softcap=5.0)),
    # chunks
    ([200], [200], 4, 1, 128, 3, 3, 2, 16, {}),
    ([513, 700, 100], [257, 1, 100], 8, 2, 128, 3, 3, 1, 64, {}),
    ([1000, 130], [130, 129], 6, 2, 64, 2, 2, 2, 32, dict(softcap=15.0)),
    ([900], [300], 2, 2, 128, 4, 4, 1, 128, dict(window=150)),
    ([900, 300], [200, 300], 4, 4, 64, 1, 1, 1, 16, dict(window=64, prefix=True)),
    ([600, 640], [90, 128], 14, 2, 128, 3, 4, 2, 16, dict(slopes=True, prefix=True)),
    ([3000], [400], 32, 8, 128, 3, 3, 2, 64, dict(slopes=True, window=700, softcap=10.0)),
    ([20, 400], [64, 150], 8, 2, 128, 3, 3, 2, 16, {}),          # more queries than tokens: the first ones see nothing
    ([260], [140], 16, 1, 128, 3, 3, 1, 16, dict(window=1)),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend(dev, case):
    lens, q_lens, Hq, Hkv, d, kb, vb, alg, ps, opt = CASES[case]
    rng = np.random.default_rng(case)
    pool = Paged(dev, lens, Hkv, d, kb, vb, alg, ps, seed=case)
    rows = sum(q_lens)
    buf = queries(rng, rows + 3, Hq + 2, d, dev)
    q = buf[:, :Hq]                                              # token stride (Hq + 2) d
    opt = dict(opt)
    if opt.pop("prefix", False):
        opt["prefix"] = [min(n, int(rng.integers(0, n + 1))) if i else min(n, 40) for i, n in enumerate(lens)]
    if opt.pop("slopes", False):
        opt["slopes"] = (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)
    out = pool.call(q, q_lens, pad=3, **opt)
    tq.tq_sync_check()
    pool.check(out, q, q_lens, **opt)
    # larger limits and another scale: the launch's shape changes, the results' meaning does not
    out = pool.call(q, q_lens, pad=3, max_q=max(q_lens) + 70, max_kv=max(lens) + 900 if case % 2 else None, scale=0.05,
                    **opt) if pool.table.shape[1] * ps >= max(lens) + (900 if case % 2 else 0) else \
        pool.call(q, q_lens, pad=3, max_q=max(q_lens) + 70, scale=0.05, **opt)
    tq.tq_sync_check()
    pool.check(out, q, q_lens, scale=0.05, **opt)


@pytest.mark.parametrize("q_lens", [[1, 1], [180, 150]])
def test_attend_norms_far_apart(dev, q_lens):
    """Value norms over the whole fp16 range (a record's error is relative to the weights it meets), an outlier outside a
    window, and infinite and NaN norms that only some rows see: those rows are not finite, the others as without them."""
    lens, Hq, Hkv, d = [400, 333], 4, 2, 128
    rng = np.random.default_rng(2)
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 16, seed=4)
    q = queries(rng, sum(q_lens), Hq, d, dev)
    vn = pool.host[3]
    p, o = pool.table[0, 3], 5                                   # token 53 of sequence 0
    vn[p, :, o] = 60000.0
    page, off = pool.table[1, 100 // 16], 100 % 16
    vn[page, 0, off], vn[page, 1, off] = 6e-8, 1e-4
    pool.upload()
    pool.check(pool.call(q, q_lens), q, q_lens)
    pool.check(pool.call(q, q_lens, window=200), q, q_lens, window=200)
    small = vn.copy()
    pool.host[3] = (vn.astype(np.float32) * 2.0**-10).astype(np.float16)
    pool.upload()
    pool.check(pool.call(q, q_lens), q, q_lens)
    pool.host[3] = small
    pool.upload()
    good = pool.call(q, q_lens, window=60).double().cpu().numpy()
    start = np.concatenate([[0], np.cumsum(q_lens)])
    for which, what in ((3, np.inf), (1, np.nan), (5, np.nan)):
        keep = pool.host[which].copy()
        t = lens[0] - 70 if q_lens[0] > 1 else lens[0] - 60      # only some rows' window holds it
        pool.host[which][pool.table[0, t // 16], 1, t % 16] = what
        pool.upload()
        got = pool.call(q, q_lens, window=60).double().cpu().numpy()
        tq.tq_sync_check()
        pos = lens[0] - q_lens[0] + np.arange(q_lens[0])
        hit = np.zeros((got.shape[0], Hq), bool)
        hit[: start[1], 2:] = ((t <= pos) & (t > pos - 60))[:, None]
        if q_lens[0] == 1:
            assert hit.sum() == 2 or not hit.any()
        assert not np.any(np.isfinite(got).all(-1)[hit])
        assert np.array_equal(got[~hit], good[~hit])
        pool.host[which] = keep
    pool.upload()


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("q_lens", [[1, 1], [180, 150]])
def test_attend_not_finite(dev, q_lens, softcap):
    """Norms and queries that are not finite, with and without a cap (which would take an infinite score to a finite
    one): the rows that see or hold them are not finite whatever the sign of a score, and no others."""
    lens, Hq, Hkv, d = [400, 333], 4, 2, 128
    rng = np.random.default_rng(2)
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 16, seed=4)
    q = queries(rng, sum(q_lens), Hq, d, dev)
    good = pool.call(q, q_lens, window=60, softcap=softcap).double().cpu().numpy()
    assert np.all(np.isfinite(good))
    n0, pos = q_lens[0], lens[0] - q_lens[0] + np.arange(q_lens[0])
    for which, what in ((1, np.nan), (1, np.inf), (3, np.nan), (3, np.inf), (5, np.nan), (5, np.inf)):
        for t in (lens[0] - 60, lens[0] - 9):                    # both seen by the last query
            keep = pool.host[which].copy()
            pool.host[which][pool.table[0, t // 16], 1, t % 16] = what
            pool.upload()
            got = pool.call(q, q_lens, window=60, softcap=softcap).double().cpu().numpy()
            tq.tq_sync_check()
            hit = np.zeros((got.shape[0], Hq), bool)
            hit[:n0, 2:] = ((t <= pos) & (t > pos - 60))[:, None]
            assert hit.any()
            assert not np.any(np.isfinite(got).all(-1)[hit])
            assert np.array_equal(got[~hit], good[~hit])
            pool.host[which] = keep
    pool.upload()
    for what in (np.nan, np.inf, -np.inf):
        for window in (1, 60):                                   # one token seen, and many
            for row in range(0, n0, 7):
                bad = q.clone()
                bad[row, 1, 3] = what
                got = pool.call(bad, q_lens, window=window, softcap=softcap).double().cpu().numpy()
                ok = np.ones(got.shape[:2], bool)
                ok[row, 1] = False
                assert not np.isfinite(got[row, 1]).all()
                assert np.all(np.isfinite(got[ok]))


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [140, 70, 1]])
def test_attend_reports_bad_pages_and_lengths(dev, q_lens):
    """A page number out of range is reported and its tokens are not seen."""
    lens, Hq, Hkv, d, ps = [300, 200, 90], 4, 2, 64, 16
    rng = np.random.default_rng(3)
    pool = Paged(dev, lens, Hkv, d, 3, 3, 1, ps, seed=5)
    q = queries(rng, sum(q_lens), Hq, d, dev)
    true_table = pool.table.copy()
    for bad in (pool.pages, -1, 2**31 - 1):
        pool.table = true_table.copy()
        pool.table[0, 4] = bad
        start = np.concatenate([[0], np.cumsum(q_lens)])
        out = torch.full((sum(q_lens), Hq, d), float("nan"), dtype=torch.bfloat16, device=dev)
        tq.tq_paged_attend(pool.kv, q, i32(start, dev), i32(lens, dev), i32(pool.table, dev), rotation(d, dev)[2], out,
                           max_q_len=max(q_lens), max_kv_len=max(lens))
        with pytest.raises(tq.TQError):
            tq.tq_sync_check()
        present = np.ones(300, bool)
        present[64:80] = False
        pool.check(out, q, q_lens, present=[present, None, None])
    pool.table = true_table
    # longer than the launch was sized for: reported; the sequences within the limits are as ever
    out = pool.call(q, q_lens, max_kv=250)
    with pytest.raises(tq.TQError):
        tq.tq_sync_check()
    pool.check(out, q, q_lens, skip=[0])
    pool.check(pool.call(q, q_lens), q, q_lens)
    tq.tq_sync_check()


def test_attend_offsets_past_32_bits(dev):
    """Pages at the end of arrays beyond 2^33 bytes."""
    d, Hkv, ps = 128, 8, 128
    first = (1 << 33) // (Hkv * ps * 4 * 3 * 4) + 10
    rng = np.random.default_rng(6)
    for q_lens in ([1, 1], [130, 1]):
        pool = Paged(dev, [300, 77], Hkv, d, 3, 3, 2, ps, seed=6, first_page=first)
        assert pool.kv.tensors[0].numel() * 4 > 1 << 33
        q = queries(rng, sum(q_lens), 32, d, dev)
        out = pool.call(q, q_lens)
        tq.tq_sync_check()
        pool.check(out, q, q_lens)
        kv = pool.kv
        keep = kv.tensors[0][first - 9].clone()
        slots = torch.tensor([(first + pool.pages) * ps - 1, (first - 5) * ps], device=dev)
        x = queries(rng, 2, Hkv, d, dev)
        tq.tq_paged_append(kv, x, x, slots, rotation(d, dev)[2])
        tq.tq_sync_check()
        assert torch.equal(kv.tensors[0][first - 9], keep)
        cb = Q_cb(d, 3)
        e = Q.encode_mse(x.double().cpu().numpy().reshape(-1, d), rotation(d, dev)[0], cb)
        got = np_u32(kv.tensors[0][[first + pool.pages - 1, first - 5], :, [ps - 1, 0]])
        assert np.array_equal(got.reshape(-1, d // 32, 3), e["codes"])
        del pool, kv
        torch.cuda.empty_cache()


def test_attend_same_results_every_time(dev):
    """No atomics in the sums: repeated calls agree bit for bit, and so do calls on another stream and a captured
    graph, which follows its inputs when they change in place."""
    lens, Hq, Hkv, d = [5000, 1200, 64], 8, 2, 128
    rng = np.random.default_rng(8)
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 64, seed=8)
    for q_lens in ([1, 1, 1], [150, 80, 1]):
        q = queries(rng, sum(q_lens), Hq, d, dev)
        first = pool.call(q, q_lens)
        pool.check(first, q, q_lens)
        assert torch.equal(first, pool.call(q, q_lens))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert torch.equal(first, pool.call(q, q_lens))
        side.synchronize()
        start = i32(np.concatenate([[0], np.cumsum(q_lens)]), dev)
        kv_len, table, rot = i32(lens, dev), i32(pool.table, dev), rotation(d, dev)[2]
        out = torch.zeros_like(q)
        ws = torch.empty(tq.tq_paged_attend_workspace_bytes(pool.kv, 3, Hq, sum(q_lens), max(q_lens), max(lens)),
                         dtype=torch.uint8, device=dev)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tq.tq_paged_attend(pool.kv, q, start, kv_len, table, rot, out, max_q_len=max(q_lens), max_kv_len=max(lens), ws=ws)
        ws.fill_(255)                                            # nothing may be expected of the workspace
        graph.replay()
        assert torch.equal(first, out)
        kept, pool.lens = pool.lens, [4000, 1100, 2]
        kv_len.copy_(i32(pool.lens, dev))
        q.copy_(queries(rng, sum(q_lens), Hq, d, dev))
        graph.replay()
        tq.tq_sync_check()
        pool.check(out, q, q_lens)
        pool.lens = kept


def test_attend_opens_units_in_groups(dev):
    """Limits so large that the chunks' tiles are opened one (sequence, KV head) at a time."""
    pool = Paged(dev, [300, 190, 20], 2, 128, 3, 3, 2, 16, seed=2)
    q = queries(np.random.default_rng(2), 221, 4, 128, dev)
    pool.check(pool.call(q, [130, 90, 1], max_kv=1500000), q, [130, 90, 1])
    pool.check(pool.call(q, [130, 90, 1], max_kv=1500000, window=77), q, [130, 90, 1], window=77)
    tq.tq_sync_check()


@pytest.mark.parametrize("case", [8, 12, 14, 7])
def test_attend_many_times(dev, case):
    """The same call 40 times over, bit for bit: hand-offs between warps that a single call seldom shows."""
    lens, q_lens, Hq, Hkv, d, kb, vb, alg, ps, opt = CASES[case]
    rng = np.random.default_rng(case)
    pool = Paged(dev, lens, Hkv, d, kb, vb, alg, ps, seed=case)
    q = queries(rng, sum(q_lens), Hq, d, dev)
    opt = {k: v for k, v in opt.items() if k not in ("prefix", "slopes")}
    outs = [pool.call(q, q_lens, **opt) for _ in range(40)]
    tq.tq_sync_check()
    pool.check(outs[0], q, q_lens, **opt)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_attend_on_two_streams_at_once(dev):
    """Chunks and steps side by side, each with a workspace of its own, as they come and as a pair of captured graphs."""
    Hq, Hkv, d = 8, 2, 128
    rng = np.random.default_rng(12)
    pool = Paged(dev, [3000, 1200, 640], Hkv, d, 3, 3, 2, 64, seed=12)
    jobs = []
    for q_lens in ([1, 1, 1], [300, 150, 1]):
        q = queries(rng, sum(q_lens), Hq, d, dev)
        want = pool.call(q, q_lens)
        args = [i32(a, dev) for a in (np.concatenate([[0], np.cumsum(q_lens)]), pool.lens, pool.table)]
        ws = torch.empty(tq.tq_paged_attend_workspace_bytes(pool.kv, 3, Hq, sum(q_lens), max(q_lens), 3000), dtype=torch.uint8, device=dev)
        jobs.append((q, want, args, ws, torch.zeros_like(q), max(q_lens), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def go(job):
        q, want, args, ws, out, most, stream = job
        tq.tq_paged_attend(pool.kv, q, *args, rotation(d, dev)[2], out, max_q_len=most, max_kv_len=3000, ws=ws)

    for _ in range(20):
        for job in jobs:
            with torch.cuda.stream(job[6]):
                go(job)
    torch.cuda.synchronize()
    assert all(torch.equal(job[1], job[4]) for job in jobs)
    graphs = []
    for job in jobs:
        job[4].zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(job)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, job in zip(graphs, jobs):
            with torch.cuda.stream(job[6]):
                g.replay()
    torch.cuda.synchronize()
    tq.tq_sync_check()
    assert all(torch.equal(job[1], job[4]) for job in jobs)


def test_binding_refuses(dev):
    """What the C side cannot see: dtypes, shapes, layouts and devices of the tensors."""
    kv = tq.empty_paged(4, 2, 16, 64, 3, 3, device=dev)
    rot = rotation(64, dev)[2]
    bf = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=dev)
    pos, table = torch.zeros(3, dtype=torch.int32, device=dev), tq.tq_rope_table(8, 64)
    slots = torch.arange(3, device=dev)
    for bad in (dict(x=bf.double()), dict(positions=pos.long()), dict(positions=pos[:2]), dict(table=table.double()),
                dict(table=table[:, :, :1]), dict(out=bf.float()), dict(x=bf.transpose(1, 2)), dict(positions=pos.cpu())):
        with pytest.raises((ValueError, tq.TQError)):
            tq.tq_rope(**(dict(x=bf, positions=pos, table=table) | bad))
    for bad in (dict(k_new=bf.half()), dict(v_new=bf.float()), dict(slots=slots.int()), dict(slots=slots[:2]), dict(positions=None),
                dict(table=None), dict(k_new=torch.zeros(3, 64, 2, dtype=torch.bfloat16, device=dev).transpose(1, 2)),
                dict(k_new=bf[:, :, :32]), dict(rot=rot.cpu())):
        with pytest.raises(ValueError):
            tq.tq_paged_append(**(dict(kv=kv, k_new=bf, v_new=bf, slots=slots, rot=rot, positions=pos, table=table) | bad))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=dev)
    start, lens, pages = i32([0, 1, 3], dev), i32([5, 9], dev), i32([[0], [1]], dev)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(out=q[:2]), dict(q_start=start[:2]), dict(kv_len=lens.long()),
                dict(page_table=pages[0]), dict(prefix_len=lens[:1]), dict(slopes=torch.zeros(3, device=dev)),
                dict(ws=torch.zeros(1 << 20, dtype=torch.uint8)), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises((ValueError, IndexError)):
            tq.tq_paged_attend(**(dict(kv=kv, q=q, q_start=start, kv_len=lens, page_table=pages, rot=rot, out=torch.empty_like(q),
                                       max_q_len=2, max_kv_len=16) | bad))
    with pytest.raises(ValueError):
        tq.PagedKV(tq.tq_codebook_init(64, 3), tq.tq_codebook_init(64, 2), kv.tensors[0], kv.tensors[1].float(), *kv.tensors[2:])
    with pytest.raises(ValueError):
        tq.PagedKV(tq.tq_codebook_init(64, 3), tq.tq_codebook_init(64, 2), *kv.tensors[:5])
    tq.tq_sync_check()


def test_attend_dirty_workspace_and_single_rows(dev):
    """A workspace of NaN bytes, one token, one query of one head."""
    pool = Paged(dev, [1, 3], 1, 64, 1, 2, 2, 16, seed=1)
    q = queries(np.random.default_rng(1), 2, 1, 64, dev)
    ws = torch.full((tq.tq_paged_attend_workspace_bytes(pool.kv, 2, 1, 2, 1, 3),), 255, dtype=torch.uint8, device=dev)
    pool.check(pool.call(q, [1, 1], ws=ws), q, [1, 1])
    with pytest.raises(tq.TQError):
        pool.call(q, [1, 1], ws=ws[:16])


# ---- the operators together ----------------------------------------------------------------------

@pytest.mark.parametrize("alg", [1, 2])
def test_chunk_then_steps(dev, alg):
    """A prompt enters in two chunks, then single tokens follow, each step turning queries and keys, appending and
    attending; against the oracle on the records that the cache then holds."""
    Hq, Hkv, d, ps, B = 8, 2, 128, 16, 2
    rng = np.random.default_rng(alg)
    Pi, S, rot = rotation(d, dev)
    steps = [[70, 33], [150, 1], [1, 1], [1, 1]]
    pages_per = 20
    kv = filled(dev, B * pages_per, Hkv, ps, d, 3, 3, alg, value=0x7E007E00)       # NaN norms everywhere
    order = rng.permutation(B * pages_per).reshape(B, pages_per)
    table = tq.tq_rope_table(512, 64)
    lens = np.zeros(B, np.int64)
    for q_lens in steps:
        rows = sum(q_lens)
        pos = np.concatenate([n + np.arange(m) for n, m in zip(lens, q_lens)])
        seq = np.repeat(np.arange(B), q_lens)
        slots = order[seq, pos // ps] * ps + pos % ps
        qkv = torch.from_numpy(rng.standard_normal((rows, Hq + 2 * Hkv, d))).to(dev).to(torch.bfloat16)
        raw = qkv.clone()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        positions = i32(pos, dev)
        tq.tq_rope(q, positions, table)
        assert torch.equal(qkv[:, Hq:], raw[:, Hq:])
        tq.tq_paged_append(kv, k, v, torch.from_numpy(slots).to(dev), rot, positions=positions, table=table)
        lens = lens + q_lens
        out = torch.empty(rows, Hq, d, dtype=torch.bfloat16, device=dev)
        tq.tq_paged_attend(kv, q, i32(np.concatenate([[0], np.cumsum(q_lens)]), dev), i32(lens, dev), i32(order, dev), rot, out,
                           max_q_len=max(q_lens), max_kv_len=int(max(lens)))
        tq.tq_sync_check()
        view = object.__new__(Paged)
        view.dev, view.lens, view.alg, view.d, view.Hkv, view.ps, view.table = dev, [int(n) for n in lens], alg, d, Hkv, ps, order
        view.pages, view.kv = B * pages_per, kv
        view.host = [None if t is None else t.cpu().numpy() for t in kv.tensors]
        view.check(out, q, q_lens)
