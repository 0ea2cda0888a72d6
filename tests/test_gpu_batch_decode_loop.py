"""The operators together as a serving program runs them, each held to the formula on what it was given: a captured decode
loop, requests in different company, the pages of a linked request.

Attention over bf16 pools is compared from the rotated q and the pools as they are stored (so that their own roundings,
checked apart, do not widen its bound): each element within half a step of fp16 of a number within E of the formula,
  E = (2 es + 2^-16 + 2^-20 + (N + 40) 2^-24) sum_u p_u |v_u|,  es = ((2 D + 8) 2^-24 + 2^-22) A + 2^-25 |q|
with A the largest sum of |q k| (rotated K in two fp16 numbers, fp32 sums of 2 D terms, weights in two bf16 numbers, the
exponential). fp32: es = (D + 8) 2^-24 A, E = (2 es + 2^-20 + (N + 40) 2^-24) sum_u p_u |v_u|, one rounding. Weights in one
bf16 number or rotated K in one fp16 number, which the norm's bound would show, are off by 1.7e-3 of the norm.
"""
import numpy as np
import pytest
import torch

from .test_gpu_batch import PAGE, Batch, i32, pkl, nothing_flagged, rope_table, rotated, sync  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def hold(out, q, K, V, seen, half):
    """out, q [m, H, D], K (rotated) and V [N, G, D] in 64 bits, seen [m, N]."""
    m, H, D = q.shape
    N, G, _ = K.shape
    Q = q.double().view(m, G, H // G, D)
    w = torch.softmax((torch.einsum("tgrd,kgd->grtk", Q, K) / D ** 0.5).masked_fill(~seen, float("-inf")), -1)
    ref = torch.einsum("grtk,kgd->tgrd", w, V).reshape(m, H, D)
    size = torch.einsum("grtk,kgd->tgrd", w, V.abs()).reshape(m, H, D)
    A = (torch.einsum("tgrd,kgd->grtk", Q.abs(), K.abs()) / D ** 0.5).amax().item()
    if half:
        es = ((2 * D + 8) * 2.0 ** -24 + 2.0 ** -22) * A + 2.0 ** -25 * (Q.abs().sum(-1).amax() / D ** 0.5).item()
        E = (2 * es + 2.0 ** -16 + 2.0 ** -20 + (N + 40) * 2.0 ** -24) * size
        tol = E + 2.0 ** -11 * (ref.abs() + E) + 2.0 ** -25
    else:
        E = (2 * (D + 8) * 2.0 ** -24 * A + 2.0 ** -20 + (N + 40) * 2.0 ** -24) * size
        tol = E + 2.0 ** -24 * (ref.abs() + E)
    off = (out.double() - ref).abs()
    assert (off <= tol).all(), (off / tol).amax().item()
    # rounding to fp16 alone is off by 2^-11 / sqrt 3 of the norm at most, about 2.1e-4 on average over a binade
    rel = (off.norm() / ref.norm()).item()
    assert rel < (2.0 ** -11 / 3 ** 0.5 + 2.0 ** -14 if half else 2e-6), rel


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("prefix", [0, 213])
def test_captured_decode_loop(pkl, half, prefix):
    """block_tables, qk_norm_rope and attention of two layers captured as one step and replayed over lengths that only the
    device knows: slots against a loop, q, K and V rows against 64 bits, attention against 64 bits of those."""
    H, G, D, n, window, sinks, layers = 8, 2, 128, 3, 40, 4, 2
    steps = [[30, 1, 17], [1, 1, 1], [1, 0, 1], [1, 1, 1], [2, 1, 0]] + [[1, 1, 1]] * 3
    max_rows, pool = 50, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    pool_t, act_t = (torch.bfloat16, torch.float16) if half else (torch.float32, torch.float32)
    k = torch.randn(layers, pool, G, PAGE, D, generator=g, device="cuda").to(pool_t)
    v = torch.randn(layers, pool, G, PAGE, D, generator=g, device="cuda").to(pool_t)
    table, rope = i32(np.full((n, 6), -1)), rope_table(prefix + 200, D)
    gq, gk = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    n_pre = -(-prefix // PAGE)
    pre = torch.arange(n_pre, dtype=torch.int32, device="cuda")
    free = torch.arange(n_pre, pool, dtype=torch.int32, device="cuda").flip(0).contiguous()
    kv, new = i32([0] * n), i32([0] * n)
    qkv = torch.zeros(layers, max_rows, (H + 2 * G) * D, device="cuda")
    bt = pkl.BlockTables(kv, i32([0] * n), i32([0] * (n + 1)), i32([0] * max_rows), i32([-1] * max_rows), i32([0, 0, 0]))
    q = torch.zeros(layers, max_rows, H, D, dtype=act_t, device="cuda")
    out = torch.full_like(q, 7.0)

    def step():
        pkl.block_tables(kv, new, table, free, max_rows, free_used=bt.counts[1:2], first=prefix, out=bt)
        for l in range(layers):
            pkl.qk_norm_rope(qkv[l], H, G, bt.row_pos, bt.row_slot, rope, k[l], v[l], gq, gk, q_out=q[l])
            pages = pkl.BatchPages(kv, table)
            if prefix:
                pkl.attention_prefix(q[l], bt.row_start, pre, prefix, pages, k[l], v[l], rope, out=out[l])
            else:
                pkl.attention_window(q[l], bt.row_start, pages, k[l], v[l], rope, window, sinks, out=out[l])
    step()                                          # no rows: nothing happens, modules load
    assert sync() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    norm = lambda x, gain: x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * gain.double()  # noqa: E731
    ids, used, slots = free.tolist(), 0, [[] for _ in range(n)]
    work = (D / 4 + 16) * 2.0 ** -24                # of the norm and the rotation in fp32
    for lens in steps:
        new.copy_(i32(lens))
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        out.fill_(7.0)
        graph.replay()
        assert sync() == 0
        t = 0
        for r, m in enumerate(lens):
            for _ in range(m):
                if len(slots[r]) % PAGE == 0:
                    page, used = ids[used], used + 1
                    slots[r].append(page * PAGE)
                else:
                    slots[r].append(slots[r][-1] + 1)
            assert bt.row_slot[t:t + m].tolist() == slots[r][len(slots[r]) - m:]
            if m == 0:
                continue
            N = prefix + len(slots[r])
            at = torch.arange(N - m, N, device="cuda")
            u = torch.arange(N, device="cuda")
            seen = u[None] <= at[:, None]
            if not prefix:
                seen &= (u[None] > at[:, None] - window) | (u[None] < sinks)
            place = torch.cat([torch.arange(prefix, device="cuda"), torch.tensor(slots[r]).cuda()])
            for l in range(layers):
                x = qkv[l, t:t + m].double().view(m, H + 2 * G, D)
                K, V = (p[l][place // PAGE, :, place % PAGE].double() for p in (k, v))
                for got, ref, ty in ((q[l, t:t + m].double(), rotated(norm(x[:, :H], gq), at, rope), act_t),
                                     (K[N - m:], norm(x[:, H:H + G], gk), pool_t), (V[N - m:], x[:, H + G:], pool_t)):
                    size = (ref.square() + ref.roll(D // 2, -1).square()).sqrt()
                    tol = 1.5 * work * size + torch.finfo(ty).eps / 2 * (1 + work) * ref.abs() + (2.0 ** -25 if ty is torch.float16 else 0.0)
                    assert ((got - ref).abs() <= tol).all()
                hold(out[l, t:t + m], q[l, t:t + m], rotated(K, u, rope), V, seen, half)
            t += m
        assert (out[:, t:] == 7.0).all()
    assert bt.counts.tolist() == [sum(steps[-1]), used, 0]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("prefix", [0, 700])
def test_other_company(pkl, half, prefix):
    """The same requests (one of one row, one of several) beside others of other numbers, lengths and rows: the rows are within
    the bound of the formula in each company, and within two roundings of each other."""
    mine, rows = [900, 330], [1, 33]
    first = None
    for others, theirs in (([], []), ([5], [1]), ([1500, 64, 800], [1, 64, 700]), ([40] * 200, [1] * 200), ([3000], [2500])):
        b = Batch(pkl, mine + others, rows + theirs, 8, 2, 128, half, ragged=True, prefix=prefix, seed=5)
        if first is None:
            first = b
        else:          # the first batch's q, and its K and V at this batch's places
            b.q[:34] = first.q[:34]
            for r in range(2):
                for p, f in ((b.k, first.k), (b.v, first.v)):
                    p[b.places[r][0], :, b.places[r][1]] = f[first.places[r][0], :, first.places[r][1]]
            for p, f in ((b.k, first.k), (b.v, first.v)):
                p[b.pre_place[0], :, b.pre_place[1]] = f[first.pre_place[0], :, first.pre_place[1]]
        out = b.shared() if prefix else b.window(200, 4)
        b.check(out, *((0, 0) if prefix else (200, 4)))
        if b is first:
            want = out[:34].double().clone()
            continue
        off = ((out[:34].double() - want).norm() / want.norm()).item()
        # two roundings, each off by 2^-11 / sqrt 3 of the norm at most
        assert off < (2.0 ** -11 if half else 2e-6), off


def test_pages_of_a_linked_request_against_the_formula(pkl):
    """The pages of linked requests (ragged chunk pages) attended to by the batched call, against 64 bits of the same pools."""
    import pic_inputs as pi
    spec = pi.SMALL_BF16
    wl = pi.make_workload("batch pages", spec, 3, [50, 64, 37], 20, 8)
    model = pkl.PicModel(spec, pi.gen_weights(spec))
    store = pkl.PicStore(model, num_blocks=64, max_rows=512, max_requests=4, max_positions=1024)
    cids = store.compile(wl.chunks)
    res = store.link([([cids[c] for c in r.chunk_ids], r.query) for r in wl.requests], wl.k)
    store.sync()
    H, G, D = spec.n_heads, spec.n_kv_heads, spec.head_dim
    rope = pkl.rope_table(1024, D, spec.rope_base)
    info = store.request_info(res.requests[0])
    pos, ln, pt = (np.asarray(info[x]) for x in ("page_pos", "page_len", "page_table"))
    assert (pos[1:] - pos[:-1] == ln[:-1]).all() and (ln < PAGE).any()
    n, m = int(pos[-1] + ln[-1]), 9
    blk = torch.tensor(np.repeat(pt, ln)).cuda().long()
    row = torch.tensor(np.concatenate([np.arange(x) for x in ln])).cuda()
    u, at = torch.arange(n, device="cuda"), torch.arange(n - m, n, device="cuda")
    q = torch.randn(m, H, D, device="cuda").half()
    for l in range(spec.n_layers):
        kl, vl = store.k_pool[l], store.v_pool[l]
        pages = pkl.BatchPages(i32([n]), i32(pt[None]), i32(pos[None]), i32([len(pos)]))
        out = pkl.attention_window(q, i32([0, m]), pages, kl, vl, rope, 0)
        hold(out, q, rotated(kl[blk, :, row].double(), u, rope), vl[blk, :, row].double(), u[None] <= at[:, None], True)
    store.close()
    model.close()
