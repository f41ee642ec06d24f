"""Refusals of the rotary and paged-cache entry points, and the fp16 levels of a cache handle (no GPU needed:
every check comes before a device is touched)."""
import ctypes

import numpy as np
import pytest

import kv_cache_vector_encode_b200 as tq
from oracle import paged as OP


@pytest.fixture(scope="module")
def L():
    from kv_cache_vector_encode_b200 import build
    build.build()
    return tq.lib()


P = 1 << 20          # a 16-byte aligned address that no call may touch
I64 = ctypes.c_int64


def handle(L, d=128, kb=3, vb=2, alg2=True, Hkv=8, page=16, pages=100, **kw):
    kv = tq._PagedKV()
    a = dict(kc=P, kn=P, vc=P, vs=P if alg2 else None, vn=P, vg=P if alg2 else None)
    a.update(kw)
    cbk, cbv = tq.tq_codebook_init(d if d in (64, 96, 128) else 128, kb), tq.tq_codebook_init(d if d in (64, 96, 128) else 128, vb)
    rc = L.tq_paged_kv_init(ctypes.byref(cbk), ctypes.byref(cbv), d, Hkv, page, pages, a["kc"], a["kn"], a["vc"], a["vs"],
                            a["vn"], a["vg"], ctypes.byref(kv))
    return rc, kv


def test_struct_mirrors_the_header(L):
    rc, kv = handle(L)
    assert rc == tq.TQ_OK
    assert (kv.d, kv.Hkv, kv.page_size, kv.v_alg, kv.num_pages, kv.k_bits, kv.v_bits) == (128, 8, 16, 2, 100, 3, 2)
    assert kv.k_codes == P and kv.v_gammas == P and kv.ready == 0x54515047


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [1, 2, 3, 4])
def test_fp16_levels_are_proportional(L, d, bits):
    """unit * level rounded to fp16 (half a step: 2^-11), the unit chosen so that the levels keep their ratios better
    than after scaling by a power of two."""
    rc, kv = handle(L, d=d, kb=bits, vb=min(bits, 3))
    assert rc == tq.TQ_OK
    c = np.array(tq.tq_codebook_init(d, bits).c[: 1 << bits], np.float32).astype(np.float64)
    h = np.array(kv.k_half[: 1 << bits], np.uint16).view(np.float16).astype(np.float64)
    err = np.max(np.abs(h / (kv.k_unit * c) - 1))
    unit = 2.0 ** np.floor(np.log2(1 / c[-1]) + 1)
    plain = np.max(np.abs((unit * c).astype(np.float16).astype(np.float64) / (unit * c) - 1))
    assert err <= min(2.0**-11, plain)
    assert np.all(np.sign(h) == np.sign(c)) and np.array_equal(h, -h[::-1])


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), tq.TQ_ERR_UNSUPPORTED), (dict(page=8), tq.TQ_ERR_UNSUPPORTED), (dict(page=48), tq.TQ_ERR_UNSUPPORTED),
    (dict(page=2048), tq.TQ_ERR_UNSUPPORTED), (dict(Hkv=0), tq.TQ_ERR_UNSUPPORTED), (dict(pages=0), tq.TQ_ERR_INVALID_ARG),
    (dict(kc=None), tq.TQ_ERR_INVALID_ARG), (dict(vg=None), tq.TQ_ERR_INVALID_ARG), (dict(kn=P + 2), tq.TQ_ERR_INVALID_ARG),
    (dict(vb=4), tq.TQ_ERR_UNSUPPORTED),
])
def test_handle_refusals(L, kw, code):
    rc, kv = handle(L, **kw)
    assert rc == code and L.tq_last_error()
    assert kv.ready == 0
    assert L.tq_paged_attend_workspace_bytes(ctypes.byref(kv), 1, 8, 1, 1, 1) == 0


def test_rope_table_refusals(L):
    def call(n=4, rot=8, base=1e4, sc=0, fac=1.0, lo=1.0, hi=32.0, orig=0.0, mag=1.0, table=P):
        return L.tq_rope_table(n, rot, base, sc, fac, lo, hi, orig, mag, table, None)
    bad, uns = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED
    assert call(n=-1) == bad and call(table=None) == bad and call(table=P + 4) == bad
    assert call(rot=7) == uns and call(rot=0) == uns and call(rot=514) == uns
    assert call(base=0.0) == bad and call(base=float("nan")) == bad and call(mag=float("inf")) == bad
    assert call(sc=3) == bad and call(sc=1, fac=0.0) == bad and call(sc=2, fac=2.0, orig=0.0) == bad
    assert call(sc=2, fac=2.0, orig=4096.0, lo=4.0, hi=4.0) == bad and call(n=1 << 31) == uns
    assert call(n=0, table=None) == tq.TQ_OK


def test_rope_refusals(L):
    def call(tokens=4, heads=2, d=64, rot=64, layout=0, inv=0, x=P, xt=128, xh=64, dt=tq.TQ_BF16, pos=P, table=P, n=9,
             out=P, ot=128, oh=64):
        return L.tq_rope(tokens, heads, d, rot, layout, inv, x, xt, xh, dt, pos, table, n, out, ot, oh, None)
    bad, uns = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED
    assert call(tokens=-1) == bad and call(heads=0) == bad and call(x=None) == bad and call(pos=None) == bad
    assert call(d=1, rot=2) == uns and call(rot=66) == uns and call(rot=3) == uns and call(d=4098) == uns
    assert call(layout=2) == bad and call(dt=5) == uns and call(x=P + 1, out=P + 1) == bad and call(table=P + 4) == bad
    assert call(ot=64) == bad and call(oh=32) == bad and call(xt=-1) == bad and call(out=P, xt=256) == bad
    assert call(ot=0) == bad and call(oh=0) == bad
    assert call(tokens=0, x=None, out=None, pos=None, table=None) == tq.TQ_OK


def test_append_refusals(L):
    rc, kv = handle(L)
    assert rc == tq.TQ_OK
    row = 8 * 128

    def call(h=kv, tokens=4, k=P, ks=row, v=P, vs=row, dt=tq.TQ_BF16, slots=P, pos=P, table=P, n=10, rot=128, layout=0, R=P):
        return L.tq_paged_append(ctypes.byref(h) if h is not None else None, tokens, k, ks, v, vs, dt, slots, pos, table, n,
                                 rot, layout, R, None)
    bad, uns = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED
    assert call(h=None) == bad and call(h=tq._PagedKV()) == bad and call(tokens=-1) == bad and call(n=-1) == bad
    assert call(dt=tq.TQ_F16) == uns and call(rot=130) == uns and call(rot=3) == uns and call(layout=7) == bad
    assert call(k=None) == bad and call(slots=None) == bad and call(R=None) == bad and call(pos=None) == bad
    assert call(ks=row - 8) == bad and call(ks=row + 4) == bad and call(k=P + 8) == bad and call(slots=P + 4) == bad
    assert call(tokens=1 << 30) == uns
    assert call(tokens=0, k=None, v=None, slots=None, R=None) == tq.TQ_OK


def test_attend_refusals(L):
    rc, kv = handle(L)
    assert rc == tq.TQ_OK

    def call(h=kv, B=2, Hq=32, total=4, mq=2, mkv=100, q=P, qs=32 * 128, dt=tq.TQ_BF16, start=P, lens=P, pages=P, mp=10,
             scale=0.0, cap=0.0, window=0, prefix=None, slopes=None, R=P, out=P, ws=P, wb=1 << 40):
        return L.tq_paged_attend(ctypes.byref(h), B, Hq, total, mq, mkv, q, qs, dt, start, lens, pages, mp, scale, cap, window,
                                 prefix, slopes, R, out, ws, wb, None)
    bad, uns = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED
    assert call(h=tq._PagedKV()) == bad and call(B=-1) == bad and call(total=-1) == bad and call(mkv=-1) == bad
    assert call(Hq=12) == uns and call(Hq=8 * 129) == uns and call(B=65535) == uns and call(mkv=1 << 31) == uns
    assert call(total=1 << 29, mq=2) == uns and call(mq=1 << 30) == uns
    assert call(q=None) == bad and call(lens=None) == bad and call(R=None) == bad and call(dt=tq.TQ_F32) == uns
    assert call(mp=-1) == bad and call(window=-1) == bad and call(cap=-1.0) == bad and call(cap=1e-38) == bad and call(cap=float("nan")) == bad
    assert call(scale=float("inf")) == bad and call(qs=32 * 128 - 8) == bad and call(qs=32 * 128 + 4) == bad
    assert call(q=P + 2) == bad and call(lens=P + 2) == bad and call(slopes=P + 1) == bad and call(out=P + 4) == bad
    need = L.tq_paged_attend_workspace_bytes(ctypes.byref(kv), 2, 32, 4, 2, 100)
    assert need > 0
    assert call(ws=None) == tq.TQ_ERR_WORKSPACE and call(wb=need - 1) == tq.TQ_ERR_WORKSPACE
    for none in (dict(B=0), dict(total=0), dict(mq=0)):
        assert call(q=None, start=None, lens=None, pages=None, R=None, out=None, ws=None, wb=0, **none) == tq.TQ_OK


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        tq.tq_rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(4, 32, 2))
    with pytest.raises(ValueError, match="CUDA"):
        tq.empty_paged(4, 2, 16, 64, 3, 3, device="cpu")


def test_oracle_rope_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 32))
    table = OP.rope_table(64, OP.rope_freqs(24))
    pos = np.array([0, 1, 63, 7, -1])
    for pairs in (False, True):
        y = OP.rope(x, pos, table, pairs)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.allclose(OP.rope(y, pos, table, pairs, inverse=True), x)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[4], x[4]) and np.array_equal(y[..., 24:], x[..., 24:])
    # a pair's product depends on the distance of the positions alone
    a, b = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32))
    dot = [float((OP.rope(a, np.array([p]), table, False) * OP.rope(b, np.array([p + 9]), table, False))[..., :24].sum())
           for p in (0, 20, 54)]
    assert np.allclose(dot, dot[0])
    blend = OP.rope_freqs(24, scaling="blend", factor=4.0, low_turns=1.0, high_turns=8.0, original_len=64.0)
    plain = OP.rope_freqs(24)
    assert blend[0] == plain[0] and np.isclose(blend[-1], plain[-1] / 4) and np.all(np.diff(blend) < 0)


def test_oracle_attend_masks():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((2, 9, 64)), rng.standard_normal((2, 9, 64))
    out, _, _ = OP.attend(q, k, v, 9, 0.1)
    w = np.exp(0.1 * k[1, :8] @ q[1, 3])
    assert np.allclose(out[1, 3], w @ v[1, :8] / w.sum())
    one, _, _ = OP.attend(q, k, v, 9, 0.1, window=1)
    assert np.allclose(one[:, 0], v[0, 6:9]) and np.allclose(one[:, 2], v[1, 6:9])
    full, _, _ = OP.attend(q, k, v, 9, 0.1, prefix=9, window=2)
    w = np.exp(0.1 * k[0] @ q[0, 1])
    assert np.allclose(full[0, 1], w @ v[0] / w.sum())
    none, _, _ = OP.attend(q, k[:, :2], v[:, :2], 2, 0.1)       # the first of three queries stands before every token
    assert np.all(none[0] == 0) and np.allclose(none[1, 0], v[0, 0])
