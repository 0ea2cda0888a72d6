"""What one stream's calls flag while another stream is synchronised is reported by one pic_sync or the next, never lost."""
import pytest
import torch

from .test_gpu_batch import pkl, nothing_flagged, sync  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

INVALID, RANGE = 1, 7


def pic_sync(stream):
    from position_independent_kv_link_gb300 import _lib as L
    return L.load().pic_sync(None, stream.cuda_stream)


def test_flags_raised_while_another_stream_is_synchronised(pkl):
    """The current stream's call has flagged a token; another stream's call flags a weight at a moment that sweeps over the
    other's pic_sync, from before it to after it. Whichever call of pic_sync sees it, one does."""
    x = torch.zeros(1, 64, device="cuda")
    wrong = torch.tensor([64], dtype=torch.int32, device="cuda")
    out = pkl.TokenLogprobs(torch.empty(1, device="cuda"), None, None, None)
    W = torch.full((1, 32), float("nan"), device="cuda")
    here, there = torch.cuda.current_stream(), torch.cuda.Stream()
    pkl.pack_weight4(W, 32, stream=there)
    assert pic_sync(there) == RANGE
    seen = {}
    for turn in range(4):
        for delay in range(0, 400000, 1000):                  # cycles: to 200 us and more
            pkl.token_logprobs(x, wrong, out=out)
            here.synchronize()
            with torch.cuda.stream(there):
                torch.cuda._sleep(delay)
            pkl.pack_weight4(W, 32, stream=there)
            a = pic_sync(here)
            b = pic_sync(there)
            assert (a, b) in ((RANGE, 0), (INVALID, RANGE)), (turn, delay, a, b)
            seen[a] = seen.get(a, 0) + 1
    assert len(seen) == 2, seen                               # before and after: the sweep crossed it


def test_one_event_is_reported_once(pkl):
    """By the first pic_sync, of whatever stream; events of both kinds together by the more severe one."""
    x, W = torch.zeros(1, 64, device="cuda"), torch.full((1, 32), float("nan"), device="cuda")
    wrong = torch.tensor([-2], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), s):
        pkl.token_logprobs(x, wrong)
        pkl.pack_weight4(W, 32)
        torch.cuda.synchronize()
        assert pic_sync(stream) == RANGE and pic_sync(s) == 0 and sync() == 0
        pkl.token_logprobs(x, wrong, stream=stream)
        assert pic_sync(stream) == INVALID and sync() == 0


@pytest.mark.parametrize("which,status", [(1, 4), (2, 4), (3, 7)])
def test_flags_of_the_store_are_reported_once(pkl, which, status):
    from position_independent_kv_link_gb300 import _lib as L
    s = torch.cuda.Stream()
    assert L.load().pic_debug_raise_device_flag(which) == 0
    torch.cuda.synchronize()
    assert pic_sync(s) == status and pic_sync(s) == 0 and sync() == 0
