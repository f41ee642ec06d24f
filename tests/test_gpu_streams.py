"""Calls on a stream that is not the current one: the memory that a call makes for itself (a workspace, a table, a prepared
rotation) is in that stream's order (B200)."""
import numpy as np
import pytest

import workloads as W
from oracle import paged as OP
from test_gpu_paged import Paged, i32, queries, rotation

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("kv_cache_vector_encode_b200")

LATE = 40_000_000       # clock cycles by which a stream is behind: some 20 ms


@pytest.fixture(scope="module")
def dev(gpu_required):
    tq.lib()
    return torch.device("cuda")


def fill_what_is_free(sizes):
    """Overwrites blocks of these sizes that the current stream's pool gives out."""
    return [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("q_lens", [[1, 1], [300, 1]])
def test_paged_workspace_on_another_stream(dev, q_lens, raw):
    Hq, Hkv, d, lens = 8, 2, 128, [2000, 700]
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 64, seed=3)
    q = queries(np.random.default_rng(3), sum(q_lens), Hq, d, dev)
    want = pool.call(q, q_lens)
    args = [i32(a, dev) for a in (np.concatenate([[0], np.cumsum(q_lens)]), lens, pool.table)]
    need = tq.tq_paged_attend_workspace_bytes(pool.kv, 2, Hq, sum(q_lens), max(q_lens), max(lens))
    outs = [torch.zeros_like(q) for _ in range(3)]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for side in sides:
        with torch.cuda.stream(side):
            torch.cuda._sleep(LATE)
    for out, side in zip(outs, (sides[0], sides[1], sides[0])):   # two streams at once, one of them twice
        tq.tq_paged_attend(pool.kv, q, *args, rotation(d, dev)[2], out, max_q_len=max(q_lens), max_kv_len=max(lens),
                           stream=side.cuda_stream if raw else side)
    kept = fill_what_is_free([need])
    torch.cuda.synchronize()
    tq.tq_sync_check()
    assert all(torch.equal(out, want) for out in outs)
    del kept


def test_attend_decode_workspace_on_another_stream(dev):
    B, Hq, Hkv, T, d = 2, 8, 2, 3000, 128
    rng = np.random.default_rng(5)
    rot = rotation(d, dev)[2]
    cbk, cbv = tq.tq_codebook_init(d, 3), tq.tq_codebook_init(d, 2)
    n = B * Hkv * T
    kc, kn = tq.empty_mse(n, d, 3)
    vc, vn = tq.empty_mse(n, d, 2)
    x = torch.from_numpy(rng.standard_normal((n, d))).to(dev).to(torch.bfloat16)
    tq.tq_encode_mse(cbk, x, rot, kc, kn)
    tq.tq_encode_mse(cbv, x, rot, vc, vn)
    kn, vn = kn.view(B, Hkv, T), vn.view(B, Hkv, T)
    q = queries(rng, B, Hq, d, dev)
    want, out = (torch.zeros(B, Hq, d, device=dev) for _ in range(2))
    tq.tq_attend_decode(cbk, cbv, q, rot, kc, kn, vc, vn, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    tq.tq_attend_decode(cbk, cbv, q, rot, kc, kn, vc, vn, out, stream=side)
    kept = fill_what_is_free([tq.tq_attend_workspace_bytes(B, Hq, Hkv, T, d)])
    torch.cuda.synchronize()
    tq.tq_sync_check()
    assert torch.equal(out, want)
    del kept


def test_results_made_on_another_stream(dev):
    """A table and a rotation take no memory that work still waiting on the current stream writes."""
    n, rot_dim, d = 5000, 128, 128
    side = torch.cuda.Stream()
    Pi, S = (torch.from_numpy(a).to(dev) for a in (W.rotation(d), W.jl_matrix(d)))
    want = tq.tq_rotation_prepare(Pi, S)
    torch.cuda.synchronize()
    torch.cuda._sleep(LATE)
    late = [torch.empty(size, dtype=torch.uint8, device=dev) for size in (n * rot_dim * 4, tq.tq_rotation_bytes(d))]
    for t in late:
        t.fill_(255)
    del late, t
    table = tq.tq_rope_table(n, rot_dim, stream=side.cuda_stream)
    rot = tq.tq_rotation_prepare(Pi, S, stream=side)
    torch.cuda.synchronize()
    exact = OP.rope_table(n, OP.rope_freqs(rot_dim))
    assert np.max(np.abs(table.cpu().numpy() - exact)) <= 2.0**-24 + 1e-10
    used = slice(0, 8)                                           # header; then the fp32 matrices, 256 bytes in
    assert torch.equal(rot[used], want[used]) and torch.equal(rot[256:256 + 3 * d * d * 4], want[256:256 + 3 * d * d * 4])
