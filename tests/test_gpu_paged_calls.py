"""The paged operators' calls at the edges of what their documentation allows (B200)."""

import numpy as np
import pytest

import workloads as W
from oracle import quant as Q
from oracle.codebook import lloyd_max
from parity import np_u32
from test_gpu_paged import Paged, filled, i32, queries, rotation
from test_gpu_paged_formats import check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("kv_cache_vector_encode_b200")


@pytest.fixture(scope="module")
def dev(gpu_required):
    tq.lib()
    return torch.device("cuda")


# ---- reports ---------------------------------------------------------------------------------------

def status_of_check():
    try:
        tq.tq_sync_check()
    except tq.TQError as e:
        return e.status
    return tq.TQ_OK


@pytest.mark.parametrize("input_first", [True, False])
def test_bad_input_does_not_hide_a_timeout(dev, input_first):
    """Both between two checks: the timeout is reported first, the bad input by the next check, each once."""
    table = tq.tq_rope_table(10, 32)
    x = torch.ones(3, 1, 32, device=dev)
    pos = torch.tensor([1, 10, 2], dtype=torch.int32, device=dev)
    todo = [lambda: tq.tq_rope(x, pos, table), lambda: tq.tq_selftest_wait(1_000_000)]
    assert status_of_check() == tq.TQ_OK
    for call in todo if input_first else todo[::-1]:
        call()
    assert [status_of_check() for _ in range(3)] == [tq.TQ_ERR_DEVICE_TIMEOUT, tq.TQ_ERR_DEVICE_INPUT, tq.TQ_OK]


# ---- lengths past the limits ---------------------------------------------------------------------

@pytest.mark.parametrize("by_pages", [False, True])
@pytest.mark.parametrize("opt", [{}, dict(window=70), dict(window=240), dict(slopes=True), dict(prefix=[20, 9, 0])])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [9, 2, 1], [140, 70, 1]])
def test_attend_lengths_past_the_limits(dev, q_lens, opt, by_pages):
    """A length above max_kv_len, or above what max_pages hold, is reported; the tokens behind the limit are not seen,
    and the queries stand where the length says."""
    lens, Hq, Hkv, d, ps, most = [300, 200, 90], 4, 2, 64, 16, 240
    pool = Paged(dev, lens, Hkv, d, 3, 3, 1, ps, seed=5)
    q = queries(np.random.default_rng(3), sum(q_lens), Hq, d, dev)
    opt = dict(opt)
    if opt.pop("slopes", False):
        opt["slopes"] = (2.0 ** (-4.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)
    whole = pool.table
    if by_pages:
        pool.table = np.ascontiguousarray(whole[:, : most // ps])
    out = pool.call(q, q_lens, max_kv=max(lens) if by_pages else most, **opt)
    assert status_of_check() == tq.TQ_ERR_DEVICE_INPUT
    pool.table = whole
    check(pool, out, q, q_lens, present=[np.arange(300) < most, None, None], **opt)


# ---- rows that see nothing -----------------------------------------------------------------------

@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("lens,q_lens", [([20, 40], [150, 90]), ([3, 1], [9, 2])])
def test_attend_rows_that_see_nothing(dev, lens, q_lens, softcap):
    """More queries than tokens (a batch padded at its front): the first rows see nothing and are 0, whatever stands in
    their queries, in chunks as in steps."""
    Hq, Hkv, d = 4, 1, 128
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 16, seed=7)
    q = queries(np.random.default_rng(7), sum(q_lens), Hq, d, dev)
    start = np.concatenate([[0], np.cumsum(q_lens)])
    for what in (float("nan"), float("inf"), 3e38):
        bad = q.clone()
        for b, (n, m) in enumerate(zip(lens, q_lens)):
            bad[start[b]:start[b] + max(m - n, 0)] = what
        out = pool.call(bad, q_lens, softcap=softcap)
        tq.tq_sync_check()
        check(pool, out, q, q_lens, softcap=softcap)


@pytest.mark.parametrize("q_lens", [[1, 2], [150, 130]])
def test_attend_norms_of_tokens_that_nobody_sees(dev, q_lens):
    """Before the window of a sequence's first query records may hold anything: they change no bit, though some share a
    tile of opened tokens with those that are seen."""
    lens, Hq, Hkv, d, window = [500, 300], 4, 2, 128, 70
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 16, seed=21)
    for which in (1, 3):                                         # small norms, so that a large one's exponent shows
        pool.host[which] = (pool.host[which].astype(np.float32) * 2.0**-14).astype(np.float16)
    pool.upload()
    q = queries(np.random.default_rng(21), sum(q_lens), Hq, d, dev)
    want = pool.call(q, q_lens, window=window)
    tq.tq_sync_check()
    check(pool, want, q, q_lens, window=window)
    for what in (60000.0, np.inf, np.nan):
        for b, (n, m) in enumerate(zip(lens, q_lens)):
            t = np.arange(n - m + 1 - window)                    # before the first query's window
            for which in (1, 3):
                pool.host[which][pool.table[b, t // 16], :, t % 16] = what
        pool.upload()
        assert torch.equal(pool.call(q, q_lens, window=window), want)
    tq.tq_sync_check()


# ---- prefixes out of range -----------------------------------------------------------------------

@pytest.mark.parametrize("window", [0, 31])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [140, 130, 2]])
def test_attend_prefixes_out_of_range(dev, q_lens, window):
    """A negative prefix, down to the type's lowest value, is none; one past the sequence is all of it."""
    lens, Hq, Hkv, d = [300, 200, 90], 4, 2, 128
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 16, seed=15)
    q = queries(np.random.default_rng(15), sum(q_lens), Hq, d, dev)
    for prefix in ([-2**31, -1, 2**31 - 1], [2**31 - 1, -2**31, -2**31 + 100], [-2**31 + 5, 2**31 - 1, 0]):
        out = pool.call(q, q_lens, prefix=prefix, window=window)
        tq.tq_sync_check()
        check(pool, out, q, q_lens, prefix=prefix, window=window)


# ---- strides --------------------------------------------------------------------------

def test_rope_head_strides_past_32_bits(dev):
    """Heads outermost, further apart than 2^31 elements, in place and out of place."""
    far, tokens, d = (1 << 31) + 64, 3, 64
    rng = np.random.default_rng(1)
    buf = torch.empty(far + tokens * d, dtype=torch.bfloat16, device=dev)
    x = buf.as_strided((tokens, 2, d), (d, far, 1))
    x.copy_(torch.from_numpy(rng.standard_normal((tokens, 2, d))).to(dev))
    table, pos = tq.tq_rope_table(50, d), i32([7, 0, 49], dev)
    near = x.clone()
    tq.tq_rope(near, pos, table)
    out = torch.empty_like(near)
    tq.tq_rope(x, pos, table, out=out)
    assert torch.equal(out, near)
    tq.tq_rope(x, pos, table)
    assert torch.equal(x, near)


def test_rope_in_place_through_another_view(dev):
    """The stride of an axis of length one has no meaning."""
    table, pos = tq.tq_rope_table(50, 64), i32([7], dev)
    x = torch.randn(1, 4, 64, device=dev)
    want = tq.tq_rope(x.clone(), pos, table)
    tq.tq_rope(x, pos, table, out=x.as_strided((1, 4, 64), (64, 64, 1)))
    assert torch.equal(x, want)


# ---- ranges of the arguments ---------------------------------------------------------------------

def test_arguments_past_32_bits_are_refused(dev):
    """A window or a length that does not fit the C type is not cut to one that does."""
    pool = Paged(dev, [40], 1, 64, 3, 3, 1, 16, seed=1)
    q = queries(np.random.default_rng(1), 1, 1, 64, dev)
    for bad in (dict(window=(1 << 32) + 5), dict(window=-(1 << 32) + 5), dict(max_q=(1 << 32) + 1), dict(max_kv=(1 << 64) + 40)):
        with pytest.raises((ValueError, tq.TQError)):
            pool.call(q, [1], **bad)
    with pytest.raises((ValueError, tq.TQError)):
        tq.tq_paged_attend_workspace_bytes(pool.kv, 1, 1, 1, (1 << 32) + 1, 40)
    x = torch.ones(1, 1, 64, device=dev)
    with pytest.raises((ValueError, tq.TQError)):
        tq.tq_rope(x, i32([1], dev), tq.tq_rope_table(4, 64), layout=1 << 32)
    with pytest.raises((ValueError, tq.TQError)):
        tq.tq_paged_append(pool.kv, x, x, torch.zeros(1, dtype=torch.int64, device=dev), rotation(64, dev)[2], layout=1 << 32)
    tq.tq_sync_check()


# ---- large caps ----------------------------------------------------------------------------------

@pytest.mark.parametrize("softcap", [300.0, 1e3, 1e4, 1e6, 1e12, 1e30])
@pytest.mark.parametrize("q_lens", [[1, 1], [150, 3]])
def test_attend_large_caps(dev, q_lens, softcap):
    """A cap far above the scores changes nothing, and takes no precision from them."""
    Hq, Hkv, d = 8, 2, 128
    pool = Paged(dev, [400, 90], Hkv, d, 3, 3, 2, 16, seed=17)
    q = queries(np.random.default_rng(17), sum(q_lens), Hq, d, dev)
    for scale in (None, 1.0):
        out = pool.call(q, q_lens, softcap=softcap, scale=scale)
        tq.tq_sync_check()
        check(pool, out, q, q_lens, softcap=softcap, scale=scale)


# ---- nothing there -------------------------------------------------------------------------------

def test_calls_without_pages_or_table(dev):
    """Sequences without tokens need no pages, and rows that only pad the batch no table."""
    kv = tq.empty_paged(2, 2, 16, 64, 3, 3, device=dev)
    rot = rotation(64, dev)[2]
    for q_lens in ([1, 2], [200, 0]):
        q = queries(np.random.default_rng(0), sum(q_lens) + 1, 4, 64, dev)
        out = torch.full_like(q, 7.0)
        tq.tq_paged_attend(kv, q, i32(np.concatenate([[0], np.cumsum(q_lens)]), dev), i32([0, 0], dev),
                           torch.zeros(2, 0, dtype=torch.int32, device=dev), rot, out, max_q_len=max(q_lens), max_kv_len=0)
        assert torch.all(out[:-1] == 0) and torch.all(out[-1] == 7)
    x = torch.ones(3, 2, 64, device=dev)
    pad, none = i32([-1, -5, -1], dev), tq.tq_rope_table(0, 64)
    assert torch.equal(tq.tq_rope(x.clone(), pad, none), x)
    before = [t.clone() for t in kv.tensors]
    tq.tq_paged_append(kv, x, x, torch.full((3,), -1, dtype=torch.int64, device=dev), rot, positions=pad, table=none)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(before, kv.tensors))
    tq.tq_sync_check()


# ---- signs next to zero --------------------------------------------------------------------------

@pytest.mark.parametrize("log2_length", [0, 12])
@pytest.mark.parametrize("d", [64, 128])
def test_append_signs_next_to_zero(dev, d, log2_length):
    """Signs as in fp64, of vectors made so that one coordinate of S r vanishes but for the rounding of the vector to
    fp32, and whatever the length of S's rows (which changes no sign)."""
    Hkv, tokens, ps = 4, 2048, 64
    n = tokens * Hkv
    Pi, S = W.rotation(d), W.jl_matrix(d) * np.float32(2.0**log2_length)
    cb = lloyd_max(d, 2)
    rng = np.random.default_rng(d)
    x = rng.standard_normal((n, d))
    at = np.arange(n) % d
    for _ in range(5):                                           # the indices may move with x: again
        s = Q.encode_prod(x, Pi, S, cb)["s"][np.arange(n), at]
        row = S[at].astype(np.float64)
        x -= row * (s * np.linalg.norm(x, axis=1) / (row**2).sum(1))[:, None]
    x = x.astype(np.float32)
    e = Q.encode_prod(x.astype(np.float64), Pi, S, cb)
    close = np.abs(e["s"][np.arange(n), at]) < 1e-6 * 2.0**log2_length
    assert close.mean() > 0.3
    rot = tq.tq_rotation_prepare(torch.from_numpy(Pi).to(dev), torch.from_numpy(S).to(dev))
    kv = filled(dev, tokens // ps, Hkv, ps, d, 1, 3, 2)
    v = torch.from_numpy(x.reshape(tokens, Hkv, d)).to(dev)
    tq.tq_paged_append(kv, v, v, torch.arange(tokens, device=dev), rot)
    tq.tq_sync_check()
    got = Q.unpack_signs(np_u32(kv.tensors[4]).swapaxes(1, 2).reshape(n, d // 32))
    wrong = (got != e["z"]) & (np.abs(e["s"]) >= 1e-11 * 2.0**log2_length)
    assert not wrong.any(), int(wrong.sum())
