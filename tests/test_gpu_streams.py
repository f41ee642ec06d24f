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


@pytest.mark.parametrize("q_lens", [[1, 1], [180, 2]])
def test_a_captured_step_follows_its_inputs(dev, q_lens):
    """Turn, append and attend captured together on a stream of their own and replayed with other inputs, positions, slots
    and lengths in place; twice over, with a replay of each graph in turn."""
    Hq, Hkv, d, ps, pages = 8, 2, 128, 16, 30
    rng = np.random.default_rng(6)
    rot = rotation(d, dev)[2]
    table = tq.tq_rope_table(600, d)
    rows = sum(q_lens)
    order = rng.permutation(2 * pages).reshape(2, pages)
    start, page_table = i32(np.concatenate([[0], np.cumsum(q_lens)]), dev), i32(order, dev)
    caches = [tq.empty_paged(2 * pages, Hkv, ps, d, 3, 3, 2, device=dev) for _ in range(3)]
    for kv in caches:
        for t in kv.tensors:
            t.zero_()

    class Inputs:
        def __init__(self):
            self.qkv = torch.zeros(rows, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device=dev)
            self.pos, self.lens = torch.zeros(rows, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
            self.slots = torch.zeros(rows, dtype=torch.int64, device=dev)
            self.out = torch.zeros(rows, Hq, d, dtype=torch.bfloat16, device=dev)

        def fill(self, data, lens):
            pos = np.concatenate([n - m + np.arange(m) for n, m in zip(lens, q_lens)])
            seq = np.repeat(np.arange(2), q_lens)
            self.qkv.copy_(data)
            self.pos.copy_(i32(pos, dev))
            self.lens.copy_(i32(lens, dev))
            self.slots.copy_(torch.from_numpy(order[seq, pos // ps] * ps + pos % ps))

        def step(self, kv):
            q, k, v = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]
            tq.tq_rope(q, self.pos, table)
            tq.tq_paged_append(kv, k, v, self.slots, rot, positions=self.pos, table=table)
            tq.tq_paged_attend(kv, q, start, self.lens, page_table, rot, self.out, max_q_len=max(q_lens), max_kv_len=400)

    plain, held = Inputs(), [Inputs(), Inputs()]
    plain.step(caches[0])                                        # warm-up: nothing is loaded during the capture
    graphs = []
    for x, kv in zip(held, caches[1:]):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            x.step(kv)
        graphs.append(g)
    for kv in caches:
        for t in kv.tensors:
            t.zero_()
    for n in range(3):
        data, lens = queries(rng, rows, Hq + 2 * Hkv, d, dev), [200 + 31 * n, 190 + n]
        for x in (plain, *held):
            x.fill(data, lens)
        plain.step(caches[0])
        for g in graphs:
            g.replay()
        for x, kv in zip(held, caches[1:]):
            assert torch.equal(x.out, plain.out) and torch.equal(x.qkv, plain.qkv)
            assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(kv.tensors, caches[0].tensors))
    tq.tq_sync_check()


def test_calls_from_two_threads(dev):
    """Host threads with streams of their own, and each the message of its own failure."""
    import threading
    Hq, Hkv, d = 8, 2, 128
    pool = Paged(dev, [900, 333], Hkv, d, 3, 3, 2, 32, seed=8)
    jobs = [(queries(np.random.default_rng(8), sum(m), Hq, d, dev), m) for m in ([1, 1], [150, 7])]
    wants = [pool.call(q, m) for q, m in jobs]
    torch.cuda.synchronize()
    results, table = [[], []], tq.tq_rope_table(9, d)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                results[i].append(torch.equal(pool.call(*jobs[i]), wants[i]))
                try:
                    tq.tq_rope(jobs[i][0], i32(np.zeros(len(jobs[i][0])), dev), table, layout=5) if i else pool.call(*jobs[i], window=-1)
                except tq.TQError as e:
                    results[i].append(("layout" if i else "window") in str(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [len(r) for r in results] == [40, 40] and all(map(all, results))
    tq.tq_sync_check()
