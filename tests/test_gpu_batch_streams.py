"""The batched calls on a stream that is not the current one, with buffers of their own making."""
import pytest
import torch

from .test_gpu_batch import PAGE, Batch, i32, pkl, nothing_flagged  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.fixture
def given(monkeypatch):
    """Arguments of the C calls that the binding makes."""
    from position_independent_kv_link_gb300 import api
    calls, real = [], api._call

    def spy(idx, stream, f, *args):
        calls.append(args)
        real(idx, stream, f, *args)
    monkeypatch.setattr(api, "_call", spy)
    return calls


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("prefix", [0, 300])
def test_scratch_stays_with_the_stream(pkl, given, half, prefix):
    """The scratch that a call makes and drops is not given to the current stream, which does not wait for the call."""
    b = Batch(pkl, [900] * 5, [1, 40, 3, 300, 1], 8, 2, 128, half, seed=7, prefix=prefix)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for own_out in (True, False):
        b.out.fill_(7.0)
        torch.cuda.synchronize()
        args = dict(out=b.out) if own_out else {}
        if prefix:
            out = pkl.attention_prefix(b.q, b.row_start, b.pre_blocks, prefix, b.pages, b.k, b.v, b.rope, stream=s, **args)
        else:
            out = pkl.attention_window(b.q, b.row_start, b.pages, b.k, b.v, b.rope, 200, 4, stream=s, **args)
        scratch, nbytes = given[-1][-2:]
        taken = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(abs(x.data_ptr() - scratch) >= nbytes for x in taken)
        s.synchronize()
        b.check(out, *((0, 0) if prefix else (200, 4)))


def test_outputs_stay_with_the_stream(pkl):
    """block_tables and qk_norm_rope: results that are dropped at once are not given to the current stream."""
    s = torch.cuda.Stream()
    kv, new, table, free = i32([16, 30]), i32([1, 17]), i32([[4, -1, -1], [5, 6, -1]]), i32([9, 8])
    rope = torch.ones(64, 32, 2, device="cuda")
    k = torch.zeros(4, 1, PAGE, 64, device="cuda")
    x = torch.randn(3, 3 * 64, device="cuda")
    pos, slot = i32([0, 1, 2]), i32([1, 2, 3])
    torch.cuda.synchronize()
    r = pkl.block_tables(kv, new, table, free, 20, stream=s)
    at = r.kv_len.data_ptr()
    s.synchronize()
    assert r.counts.tolist() == [18, 2, 0] and r.kv_len.tolist() == [17, 47]
    del r
    q = pkl.qk_norm_rope(x, 1, 1, pos, slot, rope, k, k.clone(), stream=s)
    s.synchronize()
    turned = torch.cat([x[:, :32] - x[:, 32:64], x[:, 32:64] + x[:, :32]], -1)
    assert torch.equal(q[:, 0], turned)
    there = {at, q.data_ptr()}
    del q
    small = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (50, 50, 192, 192, 192)]
    assert not there & {t.data_ptr() for t in small}


def test_captured_on_the_given_stream(pkl):
    """A capture of calls that name their stream."""
    b = Batch(pkl, [300, 33], [1, 20], 8, 2, 128, True, seed=9)
    b.window(60, 2)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        out = pkl.attention_window(b.q, b.row_start, b.pages, b.k, b.v, b.rope, 60, 2, stream=s)
    for seed in range(3):
        b.q.copy_(torch.randn(b.q.shape, device="cuda").half())
        graph.replay()
        torch.cuda.synchronize()
        b.check(out, 60, 2)
