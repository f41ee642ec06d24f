"""A prepared rotation has no size in the C calls: the binding refuses what is not one for the call's d (B200; every
refusal comes before a launch)."""
import pytest

from test_gpu_paged import i32, rotation

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("kv_cache_vector_encode_b200")


@pytest.fixture(scope="module")
def dev(gpu_required):
    tq.lib()
    return torch.device("cuda")


def wrong_ones(dev):
    """Given as a rotation for d = 128: that for 64, for 96, its start, the matrix itself, every other byte of a buffer."""
    whole = rotation(128, dev)[2]
    return [rotation(64, dev)[2], rotation(96, dev)[2], whole[:-1], torch.eye(128, device=dev),
            torch.zeros(2 * whole.numel(), dtype=torch.uint8, device=dev)[::2], whole.cpu(), whole.view(torch.int32)]


def test_paged_calls_refuse_other_rotations(dev):
    kv = tq.empty_paged(4, 2, 16, 128, 3, 3, device=dev)
    x = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=dev)
    slots = torch.arange(2, device=dev)
    args = i32([0, 1, 2], dev), i32([5, 9], dev), i32([[0], [1]], dev)
    larger = torch.zeros(rotation(128, dev)[2].numel() + 256, dtype=torch.uint8, device=dev)
    for rot in wrong_ones(dev) + [larger]:
        with pytest.raises(ValueError, match="rot"):
            tq.tq_paged_append(kv, x, x, slots, rot)
        with pytest.raises(ValueError, match="rot"):
            tq.tq_paged_attend(kv, x, *args, rot, torch.empty_like(x), max_q_len=1, max_kv_len=16)
    tq.tq_paged_append(kv, x, x, slots, rotation(128, dev)[2])
    tq.tq_sync_check()


def test_other_calls_refuse_smaller_rotations(dev):
    d, n = 128, 64
    cb = tq.tq_codebook_init(d, 3)
    x, out = (torch.zeros(n, d, device=dev) for _ in range(2))
    codes, norms = tq.empty_mse(n, d, 3)
    codes2, signs, norms2, gammas = tq.empty_prod(n, d, 4)
    q, o = torch.zeros(1, 2, d, device=dev), torch.zeros(1, 2, d, device=dev)
    cache = codes.view(1, 1, n, 4, 3), norms.view(1, 1, n)
    for rot in wrong_ones(dev):
        for call in (lambda: tq.tq_encode_mse(cb, x, rot, codes, norms),
                     lambda: tq.tq_encode_prod(cb, x, rot, codes2, signs, norms2, gammas),
                     lambda: tq.tq_decode(cb, rot, codes, norms, out),
                     lambda: tq.tq_encode_mse_mixed([3, 3, 3, 3], x, rot, codes.view(n, 12), norms),
                     lambda: tq.tq_decode_mixed([3, 3, 3, 3], rot, codes.view(n, 12), norms, out),
                     lambda: tq.tq_scores(cb, q[0], rot, codes, norms, k=1, topk_ids=i32([[0], [0]], dev),
                                          topk_scores=torch.zeros(2, 1, device=dev)),
                     lambda: tq.tq_attend_decode(cb, cb, q, rot, *cache, *cache, o),
                     lambda: tq.tq_attend_decode_noalloc(cb, cb, q, rot, *cache, *cache, o),
                     lambda: tq.tq_attend_prefill(cb, cb, q[None], rot, *cache, *cache, o[None])):
            with pytest.raises(ValueError, match="rot"):
                call()
    Pi = torch.eye(d, device=dev)
    for a, b in ((Pi[:64], Pi), (Pi, Pi[:64]), (Pi, Pi[:, :64].contiguous())):
        with pytest.raises(ValueError):
            tq.tq_rotation_prepare(a, b)
    tq.tq_sync_check()
