"""The paged operators' calls at the edges of what their documentation allows (B200)."""
import pytest


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
