"""The batched decoding step's operators, measured: what a serving program that keeps its page
tables on the GPU runs for every layer and step beside the link.

  tables   block tables and slot maps built on the GPU from request lengths
  qk       per-head norms of q and k, the rotation of q, and the K/V rows into their pages
  window   attention over the paged pool with a sliding window and a few first tokens that stay
           visible
  prefix   attention of a batch of requests that share a long prefix, read once for all

K rows are kept unrotated in 16-token pages (block-major pools [blocks][G][16][D]), q is rotated;
pools and activations are bf16 and fp16, or fp32 throughout. A case's lengths follow from its own
values; block ids and data follow from the seed.
"""
import random

import torch

own = False

PAGE = 16
EPS = 1e-5
BASE = 500000.0


# ----------------------------------------------------------------------------- cases

def listed():
    big = dict(H=32, G=8, D=128, dtype="bf16")     # the 8B-shaped workloads' heads
    tiny = dict(H=4, G=4, D=64, dtype="f32")       # the tiny workload's heads
    return [
        # one decode step's bookkeeping of a 256-request batch, 512 to 16384 tokens each
        dict(name="tables_decode_256", op="tables", n=256, lo=512, hi=16384, new="one", ragged=False, mix=1),
        # a mixed step: decodes and prompt pieces of up to 600 tokens, pages of linked chunks (ragged tails)
        dict(name="tables_mixed_1024", op="tables", n=1024, lo=0, hi=9000, new="mixed", ragged=True, mix=2),
        # the rows of one decode step of a 64-request batch
        dict(name="qk_decode_64", op="qk", T=64, norm=True, mix=3, **big),
        # a long prompt's rows
        dict(name="qk_prefill_8192", op="qk", T=8192, norm=True, mix=4, **big),
        # an odd number of fp32 rows
        dict(name="qk_f32_1001", op="qk", T=1001, norm=True, mix=5, **tiny),
        # one request decoding after a long linked prompt (98 chunks of 512 and 64 query tokens)
        dict(name="window_decode_1", op="window", n=1, lo=50240, hi=50240, rows="one", window=1024, sinks=4,
             ragged=False, mix=6, **big),
        # a decode batch of long conversations
        dict(name="window_decode_32", op="window", n=32, lo=3000, hi=32000, rows="one", window=4096, sinks=16,
             ragged=False, mix=7, **big),
        # two whole prompts prefilled in one call
        dict(name="window_prefill_2x4096", op="window", n=2, lo=4096, hi=4096, rows="all", window=1024, sinks=4,
             ragged=False, mix=8, **big),
        # fp32, ragged chunk pages, single tokens and short pieces together
        dict(name="window_f32_mixed", op="window", n=5, lo=40, hi=900, rows="mixed", window=100, sinks=4,
             ragged=True, mix=9, **tiny),
        # four requests after a 98-chunk shared prompt: the latency case
        dict(name="prefix_decode_4", op="prefix", n=4, prefix=50176, lo=1, hi=300, rows="one", ragged=True, mix=10,
             **big),
        # a decode batch over one system prompt
        dict(name="prefix_decode_64", op="prefix", n=64, prefix=16384, lo=32, hi=1024, rows="one", ragged=False,
             mix=11, **big),
        # 32 requests' 32-token queries over the 8 chunks they all use
        dict(name="prefix_query_32x32", op="prefix", n=32, prefix=4096, lo=32, hi=32, rows="all", ragged=False,
             mix=12, **big),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["tables", "qk", "window", "window", "prefix", "prefix"])
    mix = rng.randrange(1 << 20)
    heads = rng.choice([(32, 8, 128), (32, 8, 128), (8, 2, 128), (16, 16, 128), (28, 4, 128), (16, 8, 64)])
    dtype = "bf16"
    if rng.random() < 0.15:
        heads, dtype = rng.choice([(4, 4, 64), (8, 2, 64), (8, 4, 128)]), "f32"
    H, G, D = heads
    shape = dict(H=H, G=G, D=D, dtype=dtype)
    if op == "tables":
        return dict(op=op, n=_log(rng, 1, 1024), lo=rng.choice([0, 1, 300]), hi=_log(rng, 301, 16384),
                    new=rng.choice(["one", "mixed"]), ragged=rng.random() < 0.5, mix=mix)
    if op == "qk":
        return dict(op=op, T=_log(rng, 1, 8192 if dtype == "bf16" else 2000), norm=rng.random() < 0.8, mix=mix, **shape)
    ragged = rng.random() < 0.4
    if op == "window":
        rows = rng.choice(["one", "one", "mixed", "all"])
        if dtype == "f32":
            n, hi = _log(rng, 1, 6), _log(rng, 60, 900)
        elif rows == "all":
            n, hi = rng.randint(1, 2), _log(rng, 300, 4000)
        else:
            n, hi = _log(rng, 1, 32), _log(rng, 300, 24000 if rows == "one" else 4000)
        return dict(op=op, n=n, lo=max(1, hi // 8), hi=hi, rows=rows, window=_log(rng, 33, 4096),
                    sinks=rng.choice([0, 1, 4, 16, 70]), ragged=ragged, mix=mix, **shape)
    rows = rng.choice(["one", "one", "mixed"])
    if dtype == "f32":
        n, prefix, hi = _log(rng, 1, 6), _log(rng, 33, 700), _log(rng, 2, 200)
    else:
        n, prefix, hi = _log(rng, 1, 64 if rows == "one" else 24), _log(rng, 300, 16384 if rows == "one" else 4096), \
            _log(rng, 2, 1024 if rows == "one" else 300)
    return dict(op=op, n=n, prefix=prefix, lo=1, hi=hi, rows=rows, ragged=ragged, mix=mix, **shape)


# ----------------------------------------------------------------------------- lengths (from the case alone)

def _pages_of(total, ragged, r):
    """Lengths of the pages of `total` tokens: full ones and a last one, or those of chunks of 30 to 512 tokens."""
    out, left = [], total
    while left > 0:
        chunk = min(left, r.randint(30, 512)) if ragged else left
        out += [PAGE] * (chunk // PAGE) + ([chunk % PAGE] if chunk % PAGE else [])
        left -= chunk
    return out


def _lengths(case):
    """Per request: keys before the step's end (or before it, for tables), rows of the step, page lengths."""
    r = random.Random(case["mix"])
    kv, rows, pages = [], [], []
    for _ in range(case["n"]):
        k = r.randint(case["lo"], max(case["lo"], case["hi"]))
        how = case["new"] if case["op"] == "tables" else case["rows"]
        if how == "one":
            m = 1
        elif how == "all":
            m = k
        else:
            m = 1 if r.random() < 0.7 else r.randint(2, 600 if case["op"] == "tables" else 90)
        if case["op"] != "tables":
            m = min(m, k)
        kv.append(k)
        rows.append(m)
        pages.append(_pages_of(k, case["ragged"], r))
    return kv, rows, pages


def _prefix_pages(case):
    return _pages_of(case["prefix"], case["ragged"], random.Random(case["mix"] + 1))


def _starts(lens, at=0):
    out = []
    for n in lens:
        out.append(at)
        at += n
    return out


# ----------------------------------------------------------------------------- inputs

def _i32(a, dev="cuda"):
    return torch.tensor(a, dtype=torch.int32).to(dev)


def _rope_table(n, D):
    theta = BASE ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * theta
    return torch.stack([a.cos(), a.sin()], dim=-1).float().contiguous()


def _tables(pages, stride, blocks, at=0, first=0):
    """block_table and page_pos [n][stride] (-1 and 2^30 in unused places) from page lengths and block ids."""
    n = len(pages)
    table = torch.full((n, stride), -1, dtype=torch.int32)
    pos = torch.full((n, stride), 1 << 30, dtype=torch.int32)
    for i, p in enumerate(pages):
        table[i, :len(p)] = blocks[at:at + len(p)]
        pos[i, :len(p)] = torch.tensor(_starts(p, first), dtype=torch.int32)
        at += len(p)
    return table.cuda(), pos.cuda(), at


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    s = dict(op=case["op"])
    if case["op"] == "tables":
        kv, rows, pages = _lengths(case)
        grown = [len(p) + -(-m // PAGE) + 1 for p, m in zip(pages, rows)]
        n_old, n_new = sum(map(len, pages)), sum(grown)
        ids = torch.randperm(n_old + n_new + 7, generator=cpu, dtype=torch.int32)
        stride = max(grown) + 3
        table, pos, at = _tables(pages, stride, ids)
        s.update(kv_len=_i32(kv), new_len=_i32(rows), block_table=table, free=ids[at:].cuda(),
                 max_rows=sum(rows) + 5, page_pos=pos if case["ragged"] else None,
                 n_pages=_i32([len(p) for p in pages]) if case["ragged"] else None)
        return s
    H, G, D = case["H"], case["G"], case["D"]
    half = case["dtype"] == "bf16"
    pool_t, act_t = (torch.bfloat16, torch.float16) if half else (torch.float32, torch.float32)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "qk":
        T = case["T"]
        r = random.Random(case["mix"])
        blocks = -(-T // PAGE) * 2 + 3
        slots = torch.randperm(blocks * PAGE, generator=cpu)[:T].to(torch.int32)
        pos = torch.tensor([r.randrange(50240) for _ in range(T)], dtype=torch.int32)
        s.update(H=H, G=G, D=D, half=half, norm=case["norm"], qkv=randn(T, (H + 2 * G) * D), q_gain=1 + 0.1 * randn(D),
                 k_gain=1 + 0.1 * randn(D), pos=pos.cuda(), slot=slots.cuda(), rope=_rope_table(50240, D),
                 k=randn(blocks, G, PAGE, D).to(pool_t), v=randn(blocks, G, PAGE, D).to(pool_t))
        return s
    kv, rows, pages = _lengths(case)
    first = case.get("prefix", 0)
    pre = _prefix_pages(case) if case["op"] == "prefix" else []
    blocks = sum(map(len, pages)) + len(pre) + 5
    ids = torch.randperm(blocks, generator=cpu, dtype=torch.int32)
    table, pos, at = _tables(pages, max(map(len, pages)) + 2, ids, first=first)
    s.update(H=H, G=G, D=D, half=half, q=(1.5 * randn(sum(rows), H, D)).to(act_t),
             row_start=_i32(_starts(rows) + [sum(rows)]), kv_len=_i32(kv), block_table=table,
             page_pos=pos if case["ragged"] else None, n_pages=_i32([len(p) for p in pages]) if case["ragged"] else None,
             rope=_rope_table(-(-(first + max(kv)) // PAGE) * PAGE + PAGE, D),
             k=randn(blocks, G, PAGE, D).to(pool_t), v=randn(blocks, G, PAGE, D).to(pool_t),
             max_rows=max(rows), max_kv=max(kv))
    if case["op"] == "window":
        s.update(window=case["window"], sinks=case["sinks"], max_span=min(max(kv), case["window"] - 1 + max(rows)))
    else:
        s.update(prefix_blocks=ids[at:at + len(pre)].cuda(), prefix_len=first,
                 prefix_pos=_i32(_starts(pre)) if case["ragged"] else None)
    return s


# ----------------------------------------------------------------------------- the plain forms

def _tables_plain(s):
    kv, new, table = s["kv_len"].long(), s["new_len"].long(), s["block_table"]
    n, stride = table.shape
    dev = table.device
    if s["page_pos"] is None:
        n_pages = (kv + PAGE - 1) // PAGE
        last = (n_pages - 1) * PAGE
    else:
        n_pages = s["n_pages"].long()
        last = s["page_pos"].long().gather(1, (n_pages - 1).clamp(min=0)[:, None])[:, 0]
    room = torch.where(n_pages > 0, last + PAGE, 0)            # the position after the last page's last row
    more = ((kv + new - room).clamp(min=0) + PAGE - 1) // PAGE
    took = more.cumsum(0) - more
    col = torch.arange(stride, device=dev)
    k = col - n_pages[:, None]
    fresh = (k >= 0) & (k < more[:, None])
    free = s["free"]
    ids = free[(took[:, None] + k).clamp(0, len(free) - 1)]
    table = torch.where(fresh, ids, table)
    end = new.cumsum(0)
    t = torch.arange(s["max_rows"], device=dev)
    r = torch.searchsorted(end, t, right=True).clamp(max=n - 1)
    live = t < end[-1]
    pos = kv[r] + t - (end - new)[r]
    over = pos - room[r]
    page = torch.where(over >= 0, n_pages[r] + over.clamp(min=0) // PAGE, n_pages[r] - 1)
    row = torch.where(over >= 0, over.clamp(min=0) % PAGE, pos - last[r])
    slot = table[r, page.clamp(0, stride - 1)].long() * PAGE + row
    out = dict(block_table=table, kv_len=(kv + new).int(), n_pages=(n_pages + more).int(),
               row_start=torch.cat([torch.zeros_like(end[:1]), end]).int(), row_pos=torch.where(live, pos, 0).int(),
               row_slot=torch.where(live, slot, -1).int(), counts=torch.stack([end[-1], more.sum()]).int())
    if s["page_pos"] is not None:
        out["page_pos"] = torch.where(fresh, room[:, None] + PAGE * k, s["page_pos"].long()).int()
    return out


def _rotate(x, cs):
    """x [..., heads, D] by the rows cs [..., D / 2, 2] of the table, halves paired."""
    c, n = cs[..., 0][..., None, :], cs[..., 1][..., None, :]
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * c - b * n, b * c + a * n], dim=-1)


def _qk_plain(s):
    H, G, D = s["H"], s["G"], s["D"]
    T = len(s["pos"])
    q, k, v = s["qkv"].view(T, H + 2 * G, D).split([H, G, G], dim=1)
    if s["norm"]:
        q = q * (q.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["q_gain"]
        k = k * (k.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["k_gain"]
    q = _rotate(q, s["rope"][s["pos"].long()])
    slot = s["slot"].long()
    s["k"][slot // PAGE, :, slot % PAGE] = k.to(s["k"].dtype)
    s["v"][slot // PAGE, :, slot % PAGE] = v.to(s["v"].dtype)
    return dict(q=q.to(torch.float16 if s["half"] else torch.float32), k=s["k"], v=s["v"])


def _gather(s, blk, row, pos):
    """fp32 K (rotated to pos) and V of the given places [..., G, D]."""
    blk, row = blk.long().clamp(min=0), row.clamp(0, PAGE - 1)
    k, v = s["k"][blk, :, row].float(), s["v"][blk, :, row].float()
    return _rotate(k, s["rope"][pos.clamp(0, len(s["rope"]) - 1)]), v


def _own_keys(s, pos, first):
    """K, V of positions pos [n, L] of every request, out of its own pages."""
    if s["page_pos"] is None:
        page, row = (pos - first) // PAGE, (pos - first) % PAGE
    else:
        start = s["page_pos"].long()
        page = (torch.searchsorted(start, pos, right=True) - 1).clamp(0, start.shape[1] - 1)
        row = pos - start.gather(1, page)
    blk = s["block_table"].gather(1, page.clamp(0, s["block_table"].shape[1] - 1))
    return _gather(s, blk, row, pos)


def _attend(s, q, parts):
    """q [n, R, H, D] against parts of (K, V, visible), joined by one softmax; rows with no key give zeros."""
    n, R, H, D = q.shape
    G, rep = s["G"], H // s["G"]
    q = q.view(n, R, G, rep, D).permute(0, 2, 1, 3, 4).reshape(n, G, R * rep, D)
    x = []
    for k, _, seen in parts:
        y = torch.matmul(q, k.permute(0, 2, 3, 1)).view(n, G, R, rep, -1) * D ** -0.5
        x.append(y.masked_fill_(~seen[:, None, :, None, :], float("-inf")))
    top = torch.stack([y.amax(-1) for y in x]).amax(0).clamp(min=-1e30)[..., None]
    o, l = 0.0, 0.0
    for y, (_, v, _) in zip(x, parts):
        p = y.sub_(top).exp_()
        l = l + p.sum(-1)
        o = o + torch.matmul(p.view(n, G, R * rep, -1), v.permute(0, 2, 1, 3)).view(n, G, R, rep, D)
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    return o.permute(0, 2, 1, 3, 4).reshape(n, R, H, D)


def _attention_plain(s):
    start, kv = s["row_start"].long(), s["kv_len"].long()
    dev, R = kv.device, s["max_rows"]
    first = s.get("prefix_len", 0)
    m = start.diff()
    i = torch.arange(R, device=dev)
    q = s["q"].float()[(start[:-1, None] + i).clamp(max=len(s["q"]) - 1)]        # [n, R, H, D]
    at = (first + kv - m)[:, None] + i                                          # [n, R] row positions
    end = (first + kv)[:, None, None]
    if s["op"] == "window":
        W, S = s["window"], s["sinks"]
        lo = (kv - m - W + 1).clamp(min=0)
        pos = torch.cat([torch.arange(S, device=dev).expand(len(kv), S),
                         lo[:, None] + torch.arange(s["max_span"], device=dev)], dim=1)
        p, a = pos[:, None, :], at[:, :, None]
        sink = torch.arange(pos.shape[1], device=dev) < S
        seen = (p <= a) & (p < end) & torch.where(sink, True, (p > a - W) & (p >= S))
        parts = [(*_own_keys(s, pos, 0), seen)]
    else:
        pos = first + torch.arange(s["max_kv"], device=dev).expand(len(kv), -1)
        own_seen = (pos[:, None, :] <= at[:, :, None]) & (pos[:, None, :] < end)
        p0 = torch.arange(first, device=dev)
        if s["prefix_pos"] is None:
            page, row = p0 // PAGE, p0 % PAGE
        else:
            page = torch.searchsorted(s["prefix_pos"].long(), p0, right=True) - 1
            row = p0 - s["prefix_pos"].long()[page]
        k, v = _gather(s, s["prefix_blocks"][page], row, p0)
        seen = torch.ones(1, 1, 1, dtype=torch.bool, device=dev).expand(len(kv), R, first)
        parts = [(k[None], v[None], seen), (*_own_keys(s, pos, first), own_seen)]
    o = _attend(s, q, parts)
    t = torch.arange(len(s["q"]), device=dev)
    r = torch.searchsorted(start, t, right=True) - 1
    return o[r, t - start[r]].to(s["q"].dtype)


def run(s):
    if not own:
        return _tables_plain(s) if s["op"] == "tables" else _qk_plain(s) if s["op"] == "qk" else _attention_plain(s)
    import position_independent_kv_link_gb300 as pkl
    if s["op"] == "tables":
        r = pkl.block_tables(s["kv_len"], s["new_len"], s["block_table"], s["free"], s["max_rows"],
                             page_pos=s["page_pos"], n_pages=s["n_pages"])
        out = dict(block_table=s["block_table"], kv_len=r.kv_len, n_pages=r.n_pages, row_start=r.row_start,
                   row_pos=r.row_pos, row_slot=r.row_slot, counts=r.counts[:2])
        if s["page_pos"] is not None:
            out["page_pos"] = s["page_pos"]
        return out
    if s["op"] == "qk":
        gains = dict(q_gain=s["q_gain"], k_gain=s["k_gain"]) if s["norm"] else {}
        q = pkl.qk_norm_rope(s["qkv"], s["H"], s["G"], s["pos"], s["slot"], s["rope"], s["k"], s["v"], eps=EPS, **gains)
        return dict(q=q, k=s["k"], v=s["v"])
    pages = pkl.BatchPages(s["kv_len"], s["block_table"], s["page_pos"], s["n_pages"])
    if s["op"] == "window":
        return pkl.attention_window(s["q"], s["row_start"], pages, s["k"], s["v"], s["rope"], s["window"], s["sinks"])
    return pkl.attention_prefix(s["q"], s["row_start"], s["prefix_blocks"], s["prefix_len"], pages, s["k"], s["v"],
                                s["rope"], prefix_pos=s["prefix_pos"])


# ----------------------------------------------------------------------------- what a pass cannot do without

def _window_pairs(kv, m, W, S):
    """(visible pairs, distinct visible keys) of a request's last m of kv positions."""
    pairs = 0
    for a in range(kv - m, kv):
        lo = max(0, a - W + 1)
        pairs += a - lo + 1 + min(S, lo)
    lo = max(0, kv - m - W + 1)
    return pairs, kv - lo + min(S, lo)


def work(case):
    if case["op"] == "tables":
        kv, rows, pages = _lengths(case)
        new = 0
        for k, m, p in zip(kv, rows, pages):
            room = PAGE - p[-1] if p else 0
            new += -(-max(0, m - room) // PAGE)
        per_req = 5 + (2 if case["ragged"] else 0) + 1     # lengths in and out, page counts, row starts, the last page
        return {"bytes": 4.0 * (per_req * case["n"] + 2 * (sum(rows) + 5) + new * (3 if case["ragged"] else 2)),
                "flops": 0.0}
    H, G, D = case["H"], case["G"], case["D"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "qk":
        T = case["T"]
        return {"bytes": T * ((H + 2 * G) * D * (4 + e) + 8 + D * 4.0) + (8.0 * D if case["norm"] else 0.0),
                "flops": T * (H * D * 7.0 + G * D * 4.0)}
    kv, rows, pages = _lengths(case)
    T = sum(rows)
    if case["op"] == "window":
        pairs, keys = map(sum, zip(*[_window_pairs(k, m, case["window"], case["sinks"]) for k, m in zip(kv, rows)]))
    else:
        pairs = sum(m * (case["prefix"] + k) - m * (m - 1) // 2 for k, m in zip(kv, rows))
        keys = case["prefix"] + sum(kv)
    return {"bytes": 2.0 * T * H * D * e + 2.0 * keys * G * D * e + keys / PAGE * 4.0 + 12.0 * case["n"],
            "flops": 4.0 * pairs * H * D}


# ----------------------------------------------------------------------------- in 64 bits, from the definitions

def _turned(x, pos, table):
    """Complex rotation of x [n, heads, D] (64 bits) by the table's rows, halves as real and imaginary parts."""
    z = torch.complex(x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:])
    w = torch.view_as_complex(table[pos].double().contiguous())
    z = z * w[:, None, :]
    return torch.cat([z.real, z.imag], dim=-1)


def _places(lens, blocks):
    """(block, row) of every token of pages of the given lengths."""
    b = torch.repeat_interleave(blocks[:len(lens)].long().cpu(), torch.tensor(lens))
    r = torch.cat([torch.arange(n) for n in lens]) if lens else torch.zeros(0, dtype=torch.long)
    return b.cuda(), r.cuda()


def exact(case, seed):
    if case["op"] == "tables":
        return None                      # whole numbers only
    s = prepare(case, seed)
    H, G, D = case["H"], case["G"], case["D"]
    if case["op"] == "qk":
        T = case["T"]
        x = s["qkv"].double().reshape(T, H + 2 * G, D)
        q, k, v = x[:, :H], x[:, H:H + G], x[:, H + G:]
        if case["norm"]:
            q = q / torch.sqrt((q * q).sum(-1, keepdim=True) / D + EPS) * s["q_gain"].double()
            k = k / torch.sqrt((k * k).sum(-1, keepdim=True) / D + EPS) * s["k_gain"].double()
        kp, vp = s["k"].double().transpose(1, 2).reshape(-1, G, D), s["v"].double().transpose(1, 2).reshape(-1, G, D)
        kp[s["slot"].long()] = k
        vp[s["slot"].long()] = v
        back = lambda t: t.view(-1, PAGE, G, D).transpose(1, 2).contiguous()  # noqa: E731
        return dict(q=_turned(q, s["pos"].long(), s["rope"]), k=back(kp), v=back(vp))
    kv, rows, pages = _lengths(case)
    first = case.get("prefix", 0)
    shared = _places(_prefix_pages(case), s["prefix_blocks"]) if case["op"] == "prefix" else None
    out = torch.zeros(sum(rows), H, D, dtype=torch.float64, device="cuda")
    t0 = 0
    for r in range(case["n"]):
        blk, row = _places(pages[r], s["block_table"][r])
        if shared is not None:
            blk, row = torch.cat([shared[0], blk]), torch.cat([shared[1], row])
        N = first + kv[r]
        p = torch.arange(N, device="cuda")
        if case["op"] == "window":       # keys that no row of the request sees are left out
            near = (p < case["sinks"]) | (p > N - rows[r] - case["window"])
            blk, row, p = blk[near], row[near], p[near]
        K = _turned(s["k"][blk, :, row].double(), p, s["rope"])
        V = s["v"][blk, :, row].double()
        for a in range(0, rows[r], 512):
            b = min(rows[r], a + 512)
            at = torch.arange(N - rows[r] + a, N - rows[r] + b, device="cuda")
            seen = p[None, :] <= at[:, None]
            if case["op"] == "window":
                seen = seen & ((p[None, :] > at[:, None] - case["window"]) | (p[None, :] < case["sinks"]))
            some = seen.any(0)
            Q = s["q"][t0 + a:t0 + b].double().view(b - a, G, H // G, D)
            x = torch.einsum("tgrd,kgd->grtk", Q, K[some]) / D ** 0.5
            x = torch.softmax(x.masked_fill(~seen[:, some], float("-inf")), dim=-1)
            out[t0 + a:t0 + b] = torch.einsum("grtk,kgd->tgrd", x, V[some]).reshape(b - a, H, D)
        t0 += rows[r]
    return out
