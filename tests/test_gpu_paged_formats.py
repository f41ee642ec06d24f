"""tq_paged_attend in every packed format and form of its kernels, held to the bound of tests/paged_bound.py (B200).

A decode step's kernel exists per head size, key bits, value bits, algorithm and number of rows (up to four, more), the
chunks' per head size, key bits, value bits and algorithm: each runs here once at least."""
import math

import numpy as np
import pytest

import paged_bound as PB
from oracle import paged as OP
from test_gpu_paged import CASES, DTYPES, Paged, check_append, filled, heads_data, i32, queries, records, rotation

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("kv_cache_vector_encode_b200")


@pytest.fixture(scope="module")
def dev(gpu_required):
    tq.lib()
    return torch.device("cuda")


def check(pool, out, q, q_lens, scale=None, prefix=None, present=None, **kw):
    got, qs = out.double().cpu().numpy(), q.double().cpu().numpy()
    start = np.concatenate([[0], np.cumsum(q_lens)])
    assert np.all(np.isnan(got[start[-1]:]))                     # padding rows as they were
    Pi = rotation(pool.d, pool.dev)[0]
    for b, m in enumerate(q_lens):
        if not m:
            continue
        k, v = pool.sequence(b)
        here = None if present is None else present[b]
        if here is not None:
            k, v = (np.where(here[None, :, None], a, 0.0) for a in (k, v))
        rows = slice(start[b], start[b + 1])
        want, tol, sees = PB.bounds(qs[rows], k, v, Pi, pool.lens[b], scale or 1.0 / math.sqrt(pool.d),
                                    prefix=0 if prefix is None else prefix[b], present=here, **kw)
        err = np.linalg.norm(got[rows] - want, axis=-1)
        assert np.all(err <= tol), (b, float(np.max(err / np.maximum(tol, 1e-30))))
        assert np.all(got[rows][~sees] == 0)


@pytest.mark.parametrize("vb,alg", [(1, 1), (2, 1), (3, 1), (4, 1), (2, 2), (3, 2), (4, 2)])
@pytest.mark.parametrize("kb", [1, 2, 3, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_formats(dev, d, kb, vb, alg):
    number = 7 * kb + vb + 3 * alg + d // 64
    lens, Hq, Hkv = [150, 37], 8, 2
    pool = Paged(dev, lens, Hkv, d, kb, vb, alg, 16 << number % 7, seed=number)
    rng = np.random.default_rng(number)
    # four rows per KV head; eight of one sequence, and a chunk of 280 of another
    for q_lens in ([1, 1], [70, 2]):
        q = queries(rng, sum(q_lens) + 2, Hq, d, dev)
        for opt in ({}, dict(scale=0.3), dict(window=19, softcap=4.0)):
            out = pool.call(q, q_lens, pad=2, **opt)
            tq.tq_sync_check()
            check(pool, out, q, q_lens, **opt)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attend_closely(dev, case):
    lens, q_lens, Hq, Hkv, d, kb, vb, alg, ps, opt = CASES[case]
    rng = np.random.default_rng(case)
    pool = Paged(dev, lens, Hkv, d, kb, vb, alg, ps, seed=100 + case)
    q = queries(rng, sum(q_lens) + 2, Hq, d, dev)
    opt = dict(opt)
    if opt.pop("prefix", False):
        opt["prefix"] = [min(n, int(rng.integers(0, n + 1))) for n in lens]
    if opt.pop("slopes", False):
        opt["slopes"] = (2.0 ** (-8.0 * np.arange(1, Hq + 1) / Hq)).astype(np.float32)
    out = pool.call(q, q_lens, pad=2, **opt)
    tq.tq_sync_check()
    check(pool, out, q, q_lens, **opt)


def test_attend_long_context(dev):
    """One sequence alone, and contexts as long as the packed cache's other calls are measured at."""
    for lens, Hq, Hkv, ps in (([131072], 8, 2, 64), ([50001, 131000], 4, 1, 256)):
        pool = Paged(dev, lens, Hkv, 128, 3, 2, 2, ps, seed=9)
        q_lens = [1] * len(lens)
        q = queries(np.random.default_rng(9), len(lens), Hq, 128, dev)
        out = pool.call(q, q_lens)
        tq.tq_sync_check()
        check(pool, out, q, q_lens)


@pytest.mark.parametrize("Hq,Hkv,d,batch,q_len", [
    (128, 1, 128, 1, 1), (128, 1, 64, 40, 1), (256, 2, 128, 3, 2), (9, 3, 64, 2, 5), (10, 2, 128, 5, 60), (12, 1, 128, 2, 40),
])
def test_attend_head_groups(dev, Hq, Hkv, d, batch, q_len):
    """Up to 128 query heads per KV head (a single token then has as many rows as a chunk), and numbers that divide no
    block of rows."""
    rng = np.random.default_rng(Hq + batch)
    lens = [int(n) for n in rng.integers(q_len, 180, batch)]
    q_lens = [q_len] * batch
    pool = Paged(dev, lens, Hkv, d, 3, 3, 2, 32, seed=Hq)
    q = queries(rng, sum(q_lens) + 2, Hq, d, dev)
    out = pool.call(q, q_lens, pad=2, window=90)
    tq.tq_sync_check()
    check(pool, out, q, q_lens, window=90)


@pytest.mark.parametrize("most", [1, 3, 17])
def test_attend_many_sequences(dev, most):
    """More sequences than a block has threads, empty ones among them: single tokens, several, and chunks (more than 52
    query rows per KV head) beside them."""
    B, Hq, Hkv, d = 700, 8, 2, 64
    rng = np.random.default_rng(most)
    lens = rng.integers(0, 90, B)
    lens[rng.choice(B, 4, replace=False)] = 400, 333, 0, 1
    q_lens = np.minimum(lens, rng.integers(0, most + 1, B))
    lens, q_lens = [int(n) for n in lens], [int(n) for n in q_lens]
    pool = Paged(dev, lens, Hkv, d, 2, 3, 1, 16, seed=most)
    q = queries(rng, sum(q_lens) + 2, Hq, d, dev)
    for opt in ({}, dict(window=25)):
        out = pool.call(q, q_lens, pad=2, **opt)
        tq.tq_sync_check()
        check(pool, out, q, q_lens, **opt)


@pytest.mark.parametrize("rot,pairs", [(0, False), (64, False), (64, True), (22, False), (50, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [1, 2, 3, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_append_formats(dev, d, bits, dtype, rot, pairs):
    """Every width of both codebooks, head size and type, with the ways a key is turned."""
    rng = np.random.default_rng(10 * bits + d + rot)
    tokens, Hkv, ps, alg = 45, 3, 32, 1 if bits == 4 or pairs else 2
    kv = filled(dev, 4, Hkv, ps, d, 5 - bits, bits + (alg == 2), alg)
    before = records(kv)
    x = torch.from_numpy(np.stack([heads_data(rng, tokens, Hkv, d), heads_data(rng, tokens, Hkv, d)])).to(dev).to(DTYPES[dtype])
    slots, pos = rng.permutation(4 * ps)[:tokens], rng.integers(0, 900, tokens)
    slots[7] = -1
    table = tq.tq_rope_table(900, rot) if rot else None
    tq.tq_paged_append(kv, x[0], x[1], torch.from_numpy(slots).to(dev), rotation(d, dev)[2],
                       positions=i32(pos, dev) if rot else None, table=table, layout=int(pairs))
    tq.tq_sync_check()
    k = x[0].double().cpu().numpy()
    if rot:
        k = OP.rope(k, pos, table.cpu().numpy(), pairs)
    check_append(kv, before, k, x[1].double().cpu().numpy(), slots, dev, alg)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [100, 1, 90]])
def test_attend_shared_pages(dev, q_lens):
    """Sequences that begin with the same pages, and one that names a page twice."""
    Hq, Hkv, d, ps = 8, 2, 128, 32
    pool = Paged(dev, [300, 280, 260], Hkv, d, 3, 3, 2, ps, seed=30)
    pool.table[1, :5] = pool.table[0, :5]
    pool.table[2, 3:7] = pool.table[0, [0, 0, 8, 2]]
    q = queries(np.random.default_rng(30), sum(q_lens) + 2, Hq, d, dev)
    out = pool.call(q, q_lens, pad=2)
    tq.tq_sync_check()
    check(pool, out, q, q_lens)
