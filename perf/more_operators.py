"""The steps of a captured decode loop between its attention calls, measured: what a serving program runs
for every layer and token beside the tables, q/k norms and attention of the batched calls.

  pack     4-bit codes with a scale and a zero for each group of columns, from weights at load time
  gemm     products of few rows with 4-bit weights: rows in fp16, or in 8 bits with scales
  norm     the residual's addition with the root-mean-square norm, to fp16, fp32, or 8 bits with scales
  logprob  log probabilities of given tokens, entropy, and the likeliest alternatives, from logits

A 4-bit weight is scale * (code - zero), code and zero in 0..15, the scale in fp16; a row in 8 bits is
e4m3 values times an fp32 scale for each 128 columns.
"""
import random

import torch

own = False

EPS = 1e-5
XGROUP = 128          # columns that share a scale in 8-bit rows
E4M3_MAX = 448.0
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # an 8B-shaped output projection, quantised at load time
        dict(name="pack_o", op="pack", N=4096, K=4096, group=128, dtype="bf16"),
        # the gate/up projection in finer groups
        dict(name="pack_gate_up_g64", op="pack", N=28672, K=4096, group=64, dtype="bf16"),
        # a small fp32 matrix of odd sizes
        dict(name="pack_f32_odd", op="pack", N=1001, K=1120, group=32, dtype="f32"),
        # one request decoding: the down projection, a long sum for few outputs
        dict(name="gemm_down_1", op="gemm", N=4096, K=14336, T=1, group=128, x="f16"),
        # a batch of 16 at the gate/up projection, the largest weights of a layer
        dict(name="gemm_gate_up_16", op="gemm", N=28672, K=4096, T=16, group=128, x="f16"),
        # the LM head of a 64-request batch, rows in 8 bits
        dict(name="gemm_head_64_e4m3", op="gemm", N=128256, K=4096, T=64, group=128, x="e4m3"),
        # a small model's projection: odd numbers of outputs and rows, groups that the columns do not fill
        dict(name="gemm_odd_3", op="gemm", N=1001, K=1120, T=3, group=64, x="f16"),
        # one decoding request's row: the latency case
        dict(name="norm_decode_1", op="norm", T=1, d=4096, out="f16", delta=True),
        # a long prompt's rows, to 8 bits
        dict(name="norm_prefill_8192_e4m3", op="norm", T=8192, d=4096, out="e4m3", delta=True),
        # the next token of one request with 20 alternatives
        dict(name="logprob_decode_1", op="logprob", T=1, V=128256, top=20, dtype="f32", masked=0.0, mix=1),
        # 32 requests' 32-token queries scored in one call, the 5 likeliest tokens of each
        dict(name="logprob_query_1024", op="logprob", T=1024, V=128256, top=5, dtype="f32", masked=0.0, mix=2),
        # an odd vocabulary in bf16, most of it masked (constrained decoding)
        dict(name="logprob_bf16_masked_77", op="logprob", T=77, V=32003, top=8, dtype="bf16", masked=0.9, mix=3),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["pack", "gemm", "gemm", "gemm", "norm", "logprob", "logprob"])
    if op in ("pack", "gemm"):
        K = 32 * _log(rng, 2, 512)
        N = _log(rng, 33, min(32768, (80 << 20) // K))
        group = rng.choice([32, 64, 128, 128])
        if op == "pack":
            return dict(op=op, N=N, K=K, group=group, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
        return dict(op=op, N=N, K=K, T=_log(rng, 1, 64), group=group, x=rng.choice(["f16", "f16", "e4m3"]))
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 8192), d=32 * _log(rng, 4, 256), out=rng.choice(["f16", "f16", "f32", "e4m3"]),
                    delta=rng.random() < 0.8)
    return dict(op=op, T=_log(rng, 1, 512), V=_log(rng, 700, 160000), top=rng.choice([0, 1, 5, 20, 32]),
                dtype=rng.choice(["f32", "f32", "bf16", "f16"]), masked=rng.choice([0.0, 0.0, 0.5, 0.99]),
                mix=rng.randrange(1 << 20))


# ----------------------------------------------------------------------------- inputs

def _spread(x, group, width):
    """[rows, groups] to [rows, width]: each group's value at its columns."""
    return x.repeat_interleave(group, dim=1)[:, :width]


def _quantise(W, group):
    """codes [N, K] and zeros [N, groups] (uint8) and scales (fp16). Which code is nearest is decided exactly: in 64 bits
    for 32-bit weights, whose quotients may lie next to a border; quotients of 16-bit weights by 16-bit scales do not."""
    N, K = W.shape
    w = torch.nn.functional.pad(W.double() if W.dtype is torch.float32 else W.float(), (0, -K % group)).view(N, -1, group)
    lo, hi = w.amin(-1).clamp(max=0).double(), w.amax(-1).clamp(min=0).double()
    s = ((hi - lo) / 15).float().half()
    d = torch.where(s > 0, s, 1).double()
    z = torch.where(s > 0, (-lo / d).round().clamp(0, 15), 0).to(w.dtype)
    c = (w.div_(d[..., None]).round_() + z[..., None]).clamp_(0, 15).mul_((s > 0)[..., None])
    return c.byte().view(N, -1)[:, :K].contiguous(), s, z.byte()


def _to_8bit(y):
    """e4m3 values of y [T, d] and the scales [T, ceil(d / 128)] that they are to be multiplied by."""
    T, d = y.shape
    a = torch.nn.functional.pad(y, (0, -d % XGROUP)).view(T, -1, XGROUP)
    s = a.abs().amax(-1) / E4M3_MAX
    q = torch.where((s > 0)[..., None], a / torch.where(s > 0, s, 1)[..., None], 0).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn).view(T, -1)[:, :d].contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(op=case["op"])
    if case["op"] in ("pack", "gemm"):
        N, K, group = case["N"], case["K"], case["group"]
        W = randn(N, K).mul_(K ** -0.5)
        s.update(group=group)
        if case["op"] == "pack":
            s.update(W=W.to(FLOATS[case["dtype"]]))
            return s
        x = randn(case["T"], K)
        x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")] *= 8      # a few loud channels
        codes, scales, zeros = _quantise(W.bfloat16(), group)
        s.update(codes=codes, scales=scales, zeros=zeros, x=x.half(), x_scales=None)
        if case["x"] == "e4m3":
            s["x"], s["x_scales"] = _to_8bit(x)
        if own:
            import position_independent_kv_link_gb300 as pkl
            s["w"] = pkl.pack_codes4(codes, scales, zeros, group)      # laid out once, as at load time
        return s
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        s.update(h=3 * randn(T, d), delta=randn(T, d) if case["delta"] else None, gain=1 + 0.1 * randn(d), out=case["out"])
        return s
    T, V = case["T"], case["V"]
    x = randn(T, V) * (0.5 + 4 * torch.rand(T, 1, generator=g, device="cuda"))                # flat rows and peaked ones
    if case["masked"] > 0:
        x.masked_fill_(torch.rand(T, V, generator=g, device="cuda") < case["masked"], float("-inf"))
    x = x.to(FLOATS[case["dtype"]])
    r = random.Random(case["mix"])
    sampled = torch.tensor([r.random() < 0.5 for _ in range(T)], device="cuda")
    tokens = torch.where(sampled, torch.randint(0, V, (T,), generator=g, device="cuda"), x.argmax(-1))
    s.update(logits=x, tokens=tokens.int(), top=case["top"])
    return s


# ----------------------------------------------------------------------------- the plain forms

def _values(codes, scales, zeros, group):
    K = codes.shape[1]
    return (codes.float() - _spread(zeros.float(), group, K)).mul_(_spread(scales.float(), group, K))


def _gemm_plain(s):
    x = s["x"].float()
    if s["x_scales"] is not None:
        x = x * _spread(s["x_scales"], XGROUP, x.shape[1])
    return torch.matmul(x, _values(s["codes"], s["scales"], s["zeros"], s["group"]).t())


def _norm_plain(s):
    h = s["h"]
    if s["delta"] is not None:
        h += s["delta"]
    y = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["gain"]
    if s["out"] != "e4m3":
        return dict(h=h, y=y.to(FLOATS[s["out"]]))
    q, scales = _to_8bit(y)
    return dict(h=h, y=q, scales=scales)


def _logprob_plain(s):
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    x = x - torch.where(m.isinf(), 0.0, m)
    p = x.exp()
    total = p.sum(-1)
    total = torch.where(total > 0, total, 1.0)          # a row without a token: -inf throughout, entropy 0
    log_total = total.log()
    weighted = torch.where(p > 0, p * x, 0).sum(-1)
    out = dict(logprob=x.gather(1, s["tokens"].long()[:, None])[:, 0] - log_total, entropy=log_total - weighted / total)
    if s["top"]:
        v, i = torch.sort(x, dim=-1, descending=True, stable=True)
        out.update(top_ids=i[:, :s["top"]].int(), top_logprobs=v[:, :s["top"]] - log_total[:, None])
    return out


def run(s):
    if not own:
        if s["op"] == "pack":
            return _values(*_quantise(s["W"], s["group"]), s["group"])
        return _gemm_plain(s) if s["op"] == "gemm" else _norm_plain(s) if s["op"] == "norm" else _logprob_plain(s)
    import position_independent_kv_link_gb300 as pkl
    if s["op"] == "pack":
        return pkl.unpack_weight4(pkl.pack_weight4(s["W"], s["group"]))
    if s["op"] == "gemm":
        return pkl.gemm_w4(s["w"], s["x"], s["x_scales"])
    if s["op"] == "norm":
        y = pkl.add_rms_norm(s["h"], s["gain"], s["delta"], eps=EPS, dtype=FLOATS[s["out"]])
        return dict(h=s["h"], y=y[0], scales=y[1]) if s["out"] == "e4m3" else dict(h=s["h"], y=y)
    r = pkl.token_logprobs(s["logits"], s["tokens"], s["top"])
    out = dict(logprob=r.logprob, entropy=r.entropy)
    if s["top"]:
        out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
    return out


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] in ("pack", "gemm"):
        N, K = case["N"], case["K"]
        if case["op"] == "pack":         # the values that the codes stand for are the result
            return {"bytes": N * K * (BYTES[case["dtype"]] + 4.0), "flops": 4.0 * N * K}
        T, e = case["T"], BYTES[case["x"]]
        rows = T * K * e + (4.0 * T * -(-K // XGROUP) if case["x"] == "e4m3" else 0.0)
        return {"bytes": N * K / 2 + 3.0 * N * -(-K // case["group"]) + rows + 4.0 * T * N, "flops": 2.0 * T * N * K}
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        b = T * d * ((12.0 if case["delta"] else 4.0) + BYTES[case["out"]]) + 4.0 * d
        return {"bytes": b + (4.0 * T * -(-d // XGROUP) if case["out"] == "e4m3" else 0.0), "flops": 5.0 * T * d}
    T, V = case["T"], case["V"]
    return {"bytes": T * (V * BYTES[case["dtype"]] + 12.0 + 8.0 * case["top"]), "flops": 5.0 * T * V}


# ----------------------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pack":
        N, K, group = case["N"], case["K"], case["group"]
        out = torch.empty(N, K, dtype=torch.float64, device="cuda")
        for a in range(0, K, group):
            w = s["W"][:, a:a + group].double()
            lo, hi = torch.clamp(w.min(1).values, max=0), torch.clamp(w.max(1).values, min=0)
            step = ((hi - lo) / 15).float().half().double()[:, None]       # rounded to 32 bits, then to 16
            some = step > 0
            zero = torch.clamp(torch.round(-lo[:, None] / step), 0, 15)
            code = torch.clamp(torch.round(w / step) + zero, 0, 15)
            out[:, a:a + group] = torch.where(some, step * (code - zero), 0.0)
        return out
    if case["op"] == "gemm":
        # group by group: scale * (sum of code x - zero * sum of x)
        x = s["x"].double()
        out = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
        for i in range(s["scales"].shape[1]):
            a, b = i * case["group"], min(case["K"], (i + 1) * case["group"])
            part = x[:, a:b]
            if s["x_scales"] is not None:
                part = part * s["x_scales"][:, a // XGROUP, None].double()
            sums = part @ s["codes"][:, a:b].t().double() - part.sum(1, keepdim=True) * s["zeros"][:, i].double()
            out += sums * s["scales"][:, i].double()
        return out
    if case["op"] == "norm":
        h = s["h"].double() if s["delta"] is None else (s["h"] + s["delta"]).double()
        y = s["gain"].double() * h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["d"] + EPS)
        if case["out"] != "e4m3":
            return dict(h=h, y=y)
        top = torch.stack([p.abs().max(1).values for p in y.split(XGROUP, dim=1)], dim=1) / E4M3_MAX
        return dict(h=h, y=torch.cat([p / top[:, i, None] for i, p in enumerate(y.split(XGROUP, dim=1))], dim=1), scales=top)
    logprob, entropy, ids, tops = [], [], [], []
    for a in range(0, case["T"], 64):
        x = s["logits"][a:a + 64].double()
        lse = torch.logsumexp(x, dim=-1, keepdim=True)
        lp = x - torch.where(lse.isinf(), 0.0, lse)         # all masked: -inf throughout
        seen = torch.isfinite(lp)
        logprob.append(lp[torch.arange(len(lp), device="cuda"), s["tokens"][a:a + 64].long()])
        entropy.append(-torch.where(seen, lp.exp() * lp, 0.0).sum(-1))
        if case["top"]:
            tops.append(torch.topk(lp, case["top"], dim=-1).values)
    out = dict(logprob=torch.cat(logprob), entropy=torch.cat(entropy))
    if case["top"]:
        out.update(top_ids=None, top_logprobs=torch.cat(tops))
    return out
