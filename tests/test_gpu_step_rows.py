"""The residual's addition with the norm, and the log probabilities of tokens, on the GPU against 64 bits.

Norm. h + delta is one fp32 addition (compared for equality). The mean of squares: at most 32 squares in a thread, then 5 + 32 additions:
within 72 2^-24; its root's reciprocal within half of that and 2^-22; two more products: y is within e = (36 + 4 + 2) 2^-24 of itself,
then rounded: half a step of the type (eps / 2; fp16 below its normal range 2^-25). 8-bit: the scale is within e + 2^-24 of the greatest |y| / 448,
a value times the scale within 2^-4 of y (2^-10 of the scale below e4m3's normal range), and 2 e.

Log probabilities. d = x - m is within 2^-24, d log2(e) within 2^-23 more, the exponential 2^-22: a term e^d is within
t = 2^-22 + 3 2^-24 max |d| of itself, where max |d| need not count beyond 100 (what is smaller than e^-100 has no part in sums). Sums of terms: up to
600 in a row in a thread, and 30 joins: (640) 2^-24. So rest and e are within r = t + 640 2^-24 of themselves, log(n + rest) within
r rest / (n + rest) + 2^-22 |log|, and the entropy likewise with r times the sum of p |d| added. A log probability adds the
rounding of d and of the difference.
"""
import numpy as np
import pytest
import torch

from .test_gpu_batch import pkl, nothing_flagged, sync  # noqa: F401  (fixtures)
from .test_gpu_weight4 import randn

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
Y_ERR = 42 * 2.0 ** -24


def check_norm(y, scales, h, gain, eps, dtype):
    """y (and scales) against 64 bits of h."""
    x = h.double()
    ref = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (1 if gain is None else gain.double())
    if dtype is not E4M3:
        tol = ref.abs() * (Y_ERR + torch.finfo(dtype).eps / 2 * (1 + Y_ERR)) + (2.0 ** -25 if dtype is torch.float16 else 2.0 ** -140)
        assert ((y.double() - ref).abs() <= tol).all()
        return
    T, d = ref.shape
    a = torch.nn.functional.pad(ref, (0, -d % 128)).view(T, -1, 128).abs().amax(-1) / 448
    assert ((scales.double() - a).abs() <= a * (Y_ERR + 2.0 ** -23)).all()
    s = scales.double().repeat_interleave(128, dim=1)[:, :d]
    off = (y.double() * s - ref).abs()
    assert (off <= ref.abs() * (2.0 ** -4 + 2 * Y_ERR + 2.0 ** -22) + s * 2.0 ** -10 * (1 + 2.0 ** -20)).all()
    top = y.double().abs().view(T, d)
    assert (torch.nn.functional.pad(top, (0, -d % 128)).view(T, -1, 128).amax(-1)[a > 0] == 448).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, E4M3], ids=["f32", "f16", "e4m3"])
@pytest.mark.parametrize("T,d", [(1, 4), (1, 4096), (3, 36), (2, 128), (5, 132), (700, 256), (9, 4100), (400, 4096), (3, 8192), (310, 14336),
                                 (2, 16384), (400, 20480), (2, 32768)])
def test_norm(pkl, T, d, dtype):
    for with_delta in (False, True):
        for with_gain in (False, True):
            h, delta = 3 * randn(T, T, d), randn(d, T, d) if with_delta else None
            gain = 1 + 0.1 * randn(7, d) if with_gain else None
            before = h.clone()
            r = pkl.add_rms_norm(h, gain, delta, eps=1e-6, dtype=dtype)
            y, scales = r if dtype is E4M3 else (r, None)
            assert torch.equal(h, before if delta is None else before + delta)
            check_norm(y, scales, h, gain, 1e-6, dtype)


def test_norm_rows_that_lie_apart(pkl):
    """Rows of h and delta within wider ones: what is between them stays; out= and scales= are written, nothing beside them."""
    T, d = 7, 260
    wide, wider = torch.full((T, 300), 7.0, device="cuda"), torch.full((T, 400), float("nan"), device="cuda")
    h, delta = randn(1, T, d), randn(2, T, d)
    wide[:, 8:8 + d], wider[:, 100:100 + d] = h, delta
    out, scales = torch.full((T + 2, d), 5.0, device="cuda").to(E4M3), torch.full((T + 1, 3), 9.0, device="cuda")
    y = out[0:T]
    got = pkl.add_rms_norm(wide[:, 8:8 + d], None, wider[:, 100:100 + d], out=y, scales=scales[:T])
    assert got[0].data_ptr() == y.data_ptr()
    assert torch.equal(wide[:, 8:8 + d], h + delta)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[8:8 + d] = False
    assert (wide[:, keep] == 7).all() and (out[T:].float() == 5).all() and (scales[T:] == 9).all()
    check_norm(y, scales[:T], h + delta, None, 1e-5, E4M3)


def test_norm_of_zeros_and_small_rows(pkl):
    """Rows and groups of zeros have scale 0 and values 0; tiny rows are divided by the root of eps."""
    h = torch.zeros(4, 384, device="cuda")
    h[1, 128:256] = randn(1, 128)
    h[2] = randn(2, 384) * 1e-30
    h[3] = randn(3, 384) * 1e-12
    y, scales = pkl.add_rms_norm(h, dtype=E4M3)
    assert (y[0].float() == 0).all() and (scales[0] == 0).all() and (scales[1, [0, 2]] == 0).all() and (y[1, :128].float() == 0).all()
    check_norm(y, scales, h, None, 1e-5, E4M3)
    check_norm(pkl.add_rms_norm(h), None, h, None, 1e-5, torch.float16)
    z = torch.zeros(1, 128, device="cuda")
    z[0, 5] = 1e-42                                           # the scale is below fp32's normal range or 0
    y, scales = pkl.add_rms_norm(z, dtype=E4M3)
    assert torch.isfinite(scales).all() and torch.isfinite(y.float()).all()


@pytest.mark.parametrize("dtype,bad,flagged", [(torch.float16, 1e6, 7), (torch.float16, float("nan"), 7), (E4M3, float("inf"), 7),
                                               (E4M3, float("nan"), 7), (torch.float32, float("nan"), 0)], ids=str)
def test_norm_flags_what_does_not_fit(pkl, dtype, bad, flagged):
    h, gain = randn(1, 3, 256), torch.ones(256, device="cuda")
    if bad == 1e6:
        gain[3] = bad
    else:
        h[1, 9] = bad
    r = pkl.add_rms_norm(h, gain, dtype=dtype)
    assert sync() == flagged
    y = (r[0] if dtype is E4M3 else r)[0 if bad != 1e6 else 1:1 if bad != 1e6 else 2, 128:]
    assert torch.isfinite(y.float()).all()


# ----------------------------------------------------------------------------- log probabilities

def reference(x, tokens, top):
    """logprob, entropy, ids, top logprobs, and the bounds of the floats, in 64 bits by the definition."""
    x = x.double()
    bad = (x.isnan() | (x == float("inf"))).any(-1)
    o = torch.where(x.isnan(), -float("inf"), x)
    m = o.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), 0.0, m)
    d = o - m
    p = torch.where(x == float("inf"), 0.0, d.exp())
    total = p.sum(-1, keepdim=True)
    some = torch.where(total > 0, total, 1.0)
    e = -torch.where(p > 0, p * d, 0.0).sum(-1, keepdim=True) / some
    rest = torch.where(d < 0, p, 0.0).sum(-1, keepdim=True)
    n = torch.where(total > 0, (d == 0).sum(-1, keepdim=True).double(), 1.0)
    log_total = n.log() + torch.log1p(rest / n)               # some.log() would lose a rest below 2^-53
    none = torch.where(bad, float("nan"), 0.0)[:, None]
    far = torch.where(torch.isfinite(d), -d, 0.0).clamp(0, 100).amax(-1, keepdim=True)
    r = 2.0 ** -22 + 3 * 2.0 ** -24 * far + 640 * 2.0 ** -24
    log_err = r * rest / some + 2.0 ** -22 * log_total
    ent_err = log_err + 2 * r * e + 2.0 ** -23 * (log_total + e)
    lp = d - log_total + none
    lp_err = log_err + 2.0 ** -23 * (d.abs() + log_total)
    ids = torch.sort(o, dim=-1, descending=True, stable=True).indices[:, :top]
    pick = lambda v, i: v.gather(1, i)  # noqa: E731
    t = tokens.long()[:, None]
    return (pick(lp, t)[:, 0], pick(lp_err, t)[:, 0]), ((log_total + e + none)[:, 0], ent_err[:, 0]), ids.int(), (pick(lp, ids), pick(lp_err, ids))


def near(got, want):
    ref, err = want
    g = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(fine, torch.isfinite(g)) and torch.equal(ref.isnan(), g.isnan()) and torch.equal(ref == -float("inf"), g == -float("inf"))
    assert ((g - ref).abs()[fine] <= err[fine] + 2.0 ** -140).all(), ((g - ref).abs()[fine] / (err[fine] + 2.0 ** -140)).amax().item()


def logits(kind, T, V, dtype, seed=0):
    x = randn(seed + V, T, V) * 3
    if kind == "equal":
        x = torch.zeros(T, V, device="cuda")
        x[1, ::2] = -0.0
    elif kind == "masked":
        x = x.masked_fill(randn(seed + 1, T, V) < 2.3, -float("inf"))
    elif kind == "few":                                       # seven tokens allowed
        j = torch.randint(0, V, (T, 7), device="cuda")
        x = torch.full_like(x, -float("inf")).scatter_(1, j, x.gather(1, j))
    elif kind == "rising":
        x = torch.arange(V, device="cuda").float().expand(T, V) * (20.0 / V)
    elif kind == "falling":
        x = torch.arange(V, device="cuda").float().expand(T, V) * (-20.0 / V)
    elif kind == "nan":
        x[2, V // 2] = float("nan")
        x[3] = float("nan")
    elif kind == "inf":
        x[1, V // 3] = float("inf")
        x[2, 0] = x[2, V - 1] = float("inf")
    elif kind == "peaked":
        x[:, V // 2] = torch.tensor([20.0, 25.0, 30.0, 60.0, 500.0], device="cuda")[:T]
    elif kind == "empty":
        x[1] = x[3] = -float("inf")
    elif kind == "steps":                                     # many ties
        x = (x * 2).round() / 2
    return x.to(dtype)


KINDS = ["normal", "equal", "masked", "few", "rising", "falling", "nan", "inf", "peaked", "empty", "steps"]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_logprobs(pkl, kind, dtype):
    T = 5
    for V in (1, 2, 37, 700, 8191, 8192, 8193, 32003, 128256, 270001):
        x = logits(kind, T, V, dtype)
        tokens = torch.randint(0, V, (T,), device="cuda").int()
        if kind == "peaked":
            tokens[:4] = V // 2
        for top in sorted({0, 1, min(5, V), min(32, V)}):
            lp, ent, ids, tops = reference(x, tokens, max(top, 1))
            r = pkl.token_logprobs(x, tokens, top)
            near(r.logprob, lp)
            near(r.entropy, ent)
            if top:
                assert torch.equal(r.top_ids, ids[:, :top]), (V, top)
                near(r.top_logprobs, (tops[0][:, :top], tops[1][:, :top]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", range(9))
def test_logprobs_of_rows_at_any_address(pkl, dtype, shift):
    """Rows at every distance from a 16-byte border, apart from one another; what lies between them is not counted."""
    for T, V in ((3, 5), (4, 101), (3, 50001)):
        wide = torch.full((T, V + 13), 80.0, device="cuda").to(dtype)
        x = wide[:, shift:shift + V]
        x.copy_(logits("normal", T, V, dtype, seed=shift))
        tokens = torch.randint(0, V, (T,), device="cuda").int()
        lp, ent, ids, tops = reference(x, tokens, 5)
        r = pkl.token_logprobs(x, tokens, 5)
        near(r.logprob, lp), near(r.entropy, ent), near(r.top_logprobs, tops)
        assert torch.equal(r.top_ids, ids)


@pytest.mark.parametrize("T", [1, 2, 40, 77, 311, 1200])
def test_logprobs_by_rows(pkl, T):
    """As many CTAs a row as the rows leave room for."""
    V = 40013
    x = logits("normal", T, V, torch.float32, seed=T)
    tokens = x.argmax(-1).int()
    lp, ent, ids, tops = reference(x, tokens, 20)
    r = pkl.token_logprobs(x, tokens, 20)
    near(r.logprob, lp), near(r.entropy, ent), near(r.top_logprobs, tops)
    assert torch.equal(r.top_ids, ids)
    again = pkl.token_logprobs(x, tokens, 20)
    for a, b in ((r.logprob, again.logprob), (r.entropy, again.entropy), (r.top_ids, again.top_ids), (r.top_logprobs, again.top_logprobs)):
        assert torch.equal(a, b)


def test_logprobs_padding_and_tokens_outside(pkl):
    """Rows with token -1 are neither read nor written; tokens outside the vocabulary are flagged, their rows left alone."""
    T, V, top = 6, 1000, 3
    x = logits("normal", T, V, torch.float32)
    x[1] = float("nan")
    tokens = torch.tensor([5, -1, 999, -1, 0, 7], dtype=torch.int32, device="cuda")
    make = lambda: pkl.TokenLogprobs(torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda"),  # noqa: E731
                                     torch.full((T, top), 7, dtype=torch.int32, device="cuda"), torch.full((T, top), 7.0, device="cuda"))
    out = make()
    pkl.token_logprobs(x, tokens, top, out=out)
    lp, ent, ids, tops = reference(x, tokens.clamp(min=0), top)
    live = tokens >= 0
    near(out.logprob[live], (lp[0][live], lp[1][live]))
    assert torch.equal(out.top_ids[live], ids[live])
    for v in (out.logprob, out.entropy, out.top_ids, out.top_logprobs):
        assert (v[~live] == 7).all()
    assert sync() == 0
    for wrong in (V, -2, 2 ** 31 - 1, -2 ** 31):
        tokens[4] = wrong
        out = make()
        pkl.token_logprobs(x, tokens, top, out=out)
        assert sync() == 1                                    # PIC_ERR_INVALID_ARG, once
        assert out.logprob[4] == 7 and (out.top_ids[4] == 7).all() and out.logprob[5] != 7


def test_logprobs_of_what_is_asked_for(pkl):
    """Any of the outputs alone."""
    x = logits("normal", 4, 20000, torch.float32)
    tokens = torch.randint(0, 20000, (4,), device="cuda").int()
    full = pkl.token_logprobs(x, tokens, 4)
    r = pkl.token_logprobs(x)
    assert r.logprob is None and r.top_ids is None and torch.equal(r.entropy, full.entropy)
    r = pkl.token_logprobs(x, top=4)
    assert r.logprob is None and torch.equal(r.top_ids, full.top_ids) and torch.equal(r.top_logprobs, full.top_logprobs)
    r = pkl.token_logprobs(x, tokens, out=pkl.TokenLogprobs(torch.empty(4, device="cuda"), None, None, None))
    assert torch.equal(r.logprob, full.logprob)


def test_logprobs_behind_32_bits(pkl):
    """Logits behind 2^32 elements."""
    T, V = 34000, 128256
    x = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    tokens = torch.randint(0, V, (T,), device="cuda").int()
    r = pkl.token_logprobs(x, tokens, 5)
    at = torch.tensor([0, T // 2, T - 2, T - 1], device="cuda")
    lp, ent, ids, tops = reference(x[at], tokens[at], 5)
    near(r.logprob[at], lp), near(r.entropy[at], ent), near(r.top_logprobs[at], tops)
    assert torch.equal(r.top_ids[at], ids)
    del x
    torch.cuda.empty_cache()


def test_norm_behind_32_bits(pkl):
    T, d = 140000, 32768
    h = torch.empty(T, d, device="cuda")
    h.normal_()
    y, scales = pkl.add_rms_norm(h, dtype=E4M3)
    check_norm(y[-3:], scales[-3:], h[-3:], None, 1e-5, E4M3)
    check_norm(y[T // 2:T // 2 + 3], scales[T // 2:T // 2 + 3], h[T // 2:T // 2 + 3], None, 1e-5, E4M3)
    del h, y
    torch.cuda.empty_cache()
