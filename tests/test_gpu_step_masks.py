"""Log probabilities where ids are masked in runs, and rows that a cluster shares are padding, or have tokens outside the vocabulary."""
import pytest
import torch

from .test_gpu_batch import pkl, nothing_flagged, sync  # noqa: F401  (fixtures)
from .test_gpu_step_rows import logits, near, reference

pytestmark = pytest.mark.gpu

NONE = -float("inf")


def held(pkl, x, top, tokens=None):
    tokens = torch.randint(0, x.shape[1], (x.shape[0],), device="cuda").int() if tokens is None else tokens
    lp, ent, ids, tops = reference(x, tokens, top)
    r = pkl.token_logprobs(x, tokens, top)
    near(r.logprob, lp), near(r.entropy, ent), near(r.top_logprobs, tops)
    assert torch.equal(r.top_ids, ids)


TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("mask", ["none", "lowest", "-1e4"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [1, 5, 320])                     # eight CTAs a row, and one
def test_runs_of_masked_ids(pkl, T, dtype, mask):
    """The first 1, 2 and 3 chunks of 32 KB (of the row, and of every eighth of it), all but the last ids, all but 3, and a run
    that ends in the middle of a chunk; by -inf, the type's lowest value, and another."""
    V, t = 128256, TYPES[dtype]
    value = dict(none=NONE, lowest=torch.finfo(t).min).get(mask, -1e4)
    chunk = 32768 // torch.empty(0, dtype=t).element_size()
    for masked in (lambda x: x[:, :chunk], lambda x: x[:, :chunk - 200], lambda x: x[:, :3 * chunk + 1], lambda x: x[:, :V - 700],
                   lambda x: x[:, 3:], lambda x: x[:, :V // 8 * 8].view(T, 8, V // 8)[:, :, :V // 9], lambda x: x[:, 100:]):
        x = logits("normal", T, V, t, seed=T)
        masked(x).fill_(value)
        for top in (1, 20, 32):
            held(pkl, x, top)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [2, 320])
def test_all_that_is_great_in_a_few_threads_columns(pkl, T, dtype):
    """In every 4 KB the first 1984 bytes, 31 threads' groups of 64, are above the rest: with 32 alternatives the bound is one of the rest's."""
    V, t = 100000, TYPES[dtype]
    size = torch.empty(0, dtype=t).element_size()
    x = logits("normal", T, V, torch.float32, seed=8)
    i = torch.arange(V, device="cuda") % (4096 // size)
    x[:, i < 1984 // size] += 40
    held(pkl, x.to(t), 32)


def passes(pkl, x, top):
    """GPU time of a call in microseconds: the least of 5 runs of 10."""
    out = pkl.token_logprobs(x, top=top)
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            pkl.token_logprobs(x, top=top, out=out)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_runs_are_not_searched_for_one_alternative_after_the_other(pkl, dtype):
    """Rows whose first chunk, first half or all but ten ids are masked, by -inf or a number, are read once or twice. (Searches of the
    share for each of the 32 alternatives took 30 to 50 times as long as ordinary rows.)"""
    T, V, t = 608, 128256, TYPES[dtype]
    x = logits("normal", T, V, t)
    plain = passes(pkl, x, 32)
    for value in (NONE, torch.finfo(t).min):
        for masked in (slice(0, 32768 // x.element_size()), slice(0, V // 2), slice(10, V)):
            y = x.clone()
            y[:, masked] = value
            us = passes(pkl, y, 32)
            assert us < (1.5 if value == NONE and masked.stop != V // 2 else 5) * plain, (value, masked, us, plain)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 4])
def test_padding_and_tokens_outside_in_rows_that_a_cluster_shares(pkl, T, dtype):
    V, top = 128256, 20
    x = logits("normal", T, V, dtype, seed=3)
    good = torch.randint(0, V, (T,), device="cuda").int()
    lp, ent, ids, tops = reference(x, good, top)
    for wrong, status in ((-1, 0), (V, 1), (-2 ** 31, 1)):
        for r in range(T):
            tokens = good.clone()
            tokens[r] = wrong
            out = pkl.TokenLogprobs(torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda"),
                                    torch.full((T, top), 7, dtype=torch.int32, device="cuda"), torch.full((T, top), 7.0, device="cuda"))
            pkl.token_logprobs(x, tokens, top, out=out)
            assert sync() == status
            live = tokens == good
            near(out.logprob[live], (lp[0][live], lp[1][live])), near(out.entropy[live], (ent[0][live], ent[1][live]))
            near(out.top_logprobs[live], (tops[0][live], tops[1][live]))
            assert torch.equal(out.top_ids[live], ids[live])
            for v in (out.logprob, out.entropy, out.top_ids, out.top_logprobs):
                assert (v[r] == 7).all()
    everything = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    out = pkl.token_logprobs(x, everything, top)
    assert sync() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_shares_with_more_candidates_than_the_list_holds(pkl, shift, dtype):
    """Rows of ties and rising rows, at addresses between 16-byte borders, in rows of one CTA and of a cluster."""
    for T in (2, 320):
        for kind in ("equal", "rising", "steps"):
            V = 100003
            wide = torch.full((T, V + 13), 80.0, device="cuda").to(dtype)
            x = wide[:, shift:shift + V]
            x.copy_(logits(kind, T, V, dtype, seed=shift))
            held(pkl, x, 32)
