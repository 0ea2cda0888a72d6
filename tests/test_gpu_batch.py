"""GPU parity of the batched calls on device-resident lengths (block tables, per-head q/k norms with
the rotation, windowed attention with sinks, shared-prefix attention) against plain 64-bit
implementations, at the lengths and masks where they can go wrong: single tokens and single keys,
ragged chunk pages, windows that end inside a page, sinks that meet the window, requests without
rows, NaN in every place that must not be read, rows and tables that must stay as they were.

Tolerances are worst cases of the roundings (half a step: eps / 2 of the type, relative):
* fp32: a dot product of D terms is within (D + 8) 2^-24 sum|q k|; a softmax weight's relative error
  is twice that of its score, and the output adds (N + 8) 2^-24 for N keys.
* bf16 pools: rotated K is held as two fp16 numbers (each term within 2^-22, or within 2^-25 where the second one
  is below fp16's normal range), the weights as two bf16 numbers (2^-16) or one fp16 number (2^-11), which enters
  the product with V but not the denominator, the output in fp16 (2^-11).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 16
BIG = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def pkl():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.set_device(0)
    import position_independent_kv_link_gb300 as pkg
    pkg.load()
    return pkg


@pytest.fixture(autouse=True)
def nothing_flagged(pkl):
    yield
    assert sync() == 0


def sync():
    from position_independent_kv_link_gb300 import _lib as L
    return L.load().pic_sync(None, torch.cuda.current_stream().cuda_stream)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def page_lengths(total, ragged, rng):
    out = []
    while total > 0:
        chunk = min(total, int(rng.integers(1, 130))) if ragged else total
        out += [PAGE] * (chunk // PAGE) + ([chunk % PAGE] if chunk % PAGE else [])
        total -= chunk
    return out


def rope_table(n, D, base=10000.0):
    theta = base ** (-np.arange(0, D, 2) / D)
    a = np.arange(n)[:, None] * theta
    return torch.tensor(np.stack([np.cos(a), np.sin(a)], -1), dtype=torch.float32).cuda()


def rotated(x, pos, table):
    """x [n, heads, D] in 64 bits turned as complex numbers by the table's rows."""
    h = x.shape[-1] // 2
    z = torch.complex(x[..., :h], x[..., h:]) * torch.view_as_complex(table[pos].double().contiguous())[:, None, :]
    return torch.cat([z.real, z.imag], -1)


class Batch:
    """Requests over a pool in which every row that holds no key is NaN."""

    def __init__(self, pkl, kv, rows, H, G, D, half, ragged=False, prefix=0, seed=0, spare_rows=0, scale=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.pkl, self.kv, self.rows, self.H, self.G, self.D, self.half, self.prefix = pkl, kv, rows, H, G, D, half, prefix
        self.pool_t, self.act_t = (torch.bfloat16, torch.float16) if half else (torch.float32, torch.float32)
        self.T = sum(rows) + spare_rows
        lens = [page_lengths(k, ragged, rng) for k in kv]
        pre = page_lengths(prefix, ragged, rng)
        n_pages = sum(map(len, lens)) + len(pre)
        pool = n_pages + 3
        ids = rng.permutation(pool)
        stride = max(map(len, lens)) + 2
        table, pos = np.full((len(kv), stride), -7), np.full((len(kv), stride), BIG)
        self.k = torch.full((pool, G, PAGE, D), float("nan"), dtype=self.pool_t, device="cuda")
        self.v = self.k.clone()

        def fill(blocks, ln):
            b = np.repeat(blocks, ln)
            r = np.concatenate([np.arange(n) for n in ln]) if ln else np.zeros(0, int)
            b, r = torch.tensor(b).cuda().long(), torch.tensor(r).cuda().long()
            self.k[b, :, r] = torch.randn(len(b), G, D, generator=g, device="cuda").to(self.pool_t)
            self.v[b, :, r] = torch.randn(len(b), G, D, generator=g, device="cuda").to(self.pool_t)
            return b, r
        at, self.places = 0, []
        for r, p in enumerate(lens):
            blk = ids[at:at + len(p)]
            table[r, :len(p)] = blk
            if p:
                pos[r, :len(p)] = prefix + np.concatenate([[0], np.cumsum(p)[:-1]])
            self.places.append(fill(blk, p))
            at += len(p)
        blk = ids[at:at + len(pre)]
        self.pre_place = fill(blk, pre)
        self.pre_blocks = i32(blk)
        self.pre_pos = i32(np.concatenate([[0], np.cumsum(pre)[:-1]])) if ragged and pre else None
        self.row_start = i32(np.concatenate([[0], np.cumsum(rows)]))
        self.pages = pkl.BatchPages(i32(kv), i32(table), i32(pos) if ragged else None,
                                    i32([len(p) for p in lens]) if ragged else None)
        self.rope = rope_table(prefix + max(kv) + PAGE, D)
        self.q = (scale * torch.randn(self.T, H, D, generator=g, device="cuda")).to(self.act_t)
        self.out = torch.full((self.T, H, D), 7.0, dtype=self.act_t, device="cuda")

    def window(self, window, sinks, **kw):
        return self.pkl.attention_window(self.q, self.row_start, self.pages, self.k, self.v, self.rope, window, sinks,
                                         out=self.out, **kw)

    def shared(self, **kw):
        return self.pkl.attention_prefix(self.q, self.row_start, self.pre_blocks, self.prefix, self.pages, self.k, self.v,
                                         self.rope, prefix_pos=self.pre_pos, out=self.out, **kw)

    def check(self, out, window=0, sinks=0, left=()):
        """Every row against 64 bits, within the worst case of its roundings; requests `left` alone keep their 7.0."""
        rep, t0 = self.H // self.G, 0
        for r, (kv, m) in enumerate(zip(self.kv, self.rows)):
            if r in left:
                assert (out[t0:t0 + m] == 7.0).all()
                t0 += m
                continue
            if m == 0:
                continue
            N = self.prefix + kv
            blk, row = (torch.cat(x) for x in zip(self.pre_place, self.places[r]))
            u = torch.arange(N, device="cuda")
            K = rotated(self.k[blk, :, row].double(), u, self.rope)
            V = self.v[blk, :, row].double()
            p = torch.arange(N - m, N, device="cuda")
            seen = u[None] <= p[:, None]
            if window:
                seen &= (u[None] > p[:, None] - window) | (u[None] < sinks)
            Q = self.q[t0:t0 + m].double().view(m, self.G, rep, self.D)
            x = torch.einsum("tgrd,kgd->grtk", Q, K) / self.D ** 0.5
            w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
            ref = torch.einsum("grtk,kgd->tgrd", w, V).reshape(m, self.H, self.D)
            A = (torch.einsum("tgrd,kgd->grtk", Q.abs(), K.abs()) / self.D ** 0.5 * seen).amax().item()
            vmax = V.abs().amax().item()
            es = (self.D + 8) * 2.0 ** -24 * A
            if self.half:
                qmax = Q.abs().sum(-1).amax().item() / self.D ** 0.5
                tol = (2 * (es + 2.0 ** -22 * A + 2.0 ** -25 * qmax) + 2 * 2.0 ** -11 + (N + 8) * 2.0 ** -24) * vmax
            else:
                tol = (2 * es + (N + 8) * 2.0 ** -24) * vmax
            err = (out[t0:t0 + m].double() - ref).abs().amax().item()
            assert err <= tol, (r, kv, m, err, tol)
            # and on average nowhere near it: a wrong key or page would show
            rel = ((out[t0:t0 + m].double() - ref).norm() / ref.norm()).item()
            assert rel < (7e-4 if self.half else 2e-5), (r, kv, m, rel)
            t0 += m
        assert (out[t0:] == 7.0).all()          # rows behind the last sequence


WINDOW_CASES = [
    # kv, rows, window, sinks, ragged
    ([1], [1], 5, 0, False),
    ([1, 2, 16, 17], [1, 1, 1, 1], 1, 0, False),
    ([1, 2, 16, 17], [1, 2, 16, 17], 1, 1, False),
    ([33, 0, 40, 129], [33, 0, 1, 40], 16, 4, False),
    ([500, 77, 300, 1], [1, 1, 1, 1], 100, 20, True),
    ([500, 77, 300, 64], [130, 77, 5, 64], 33, 70, True),
    ([700, 260], [700, 3], 0, 0, False),
    ([700, 260], [300, 260], 128, 16, True),
    ([2100], [1], 1000, 4, False),
    ([64] * 37, [1] * 37, 64, 0, False),
    ([100, 300, 50, 700], [4, 3, 1, 2], 60, 5, True),        # a few rows each
    ([200] * 20 + [90], [1] * 20 + [40], 0, 0, False),       # and one request of many
    ([40, 50], [16, 9], 20, 2, False),
]
SHAPES = [(4, 4, 64, False), (8, 2, 128, False), (8, 2, 128, True), (8, 8, 128, True), (7, 1, 128, True), (8, 2, 64, True),
          (16, 1, 128, True)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("case", WINDOW_CASES, ids=str)
def test_window_attention(pkl, shape, case):
    kv, rows, window, sinks, ragged = case
    b = Batch(pkl, kv, rows, *shape, ragged=ragged, seed=len(kv) + window, spare_rows=3)
    b.check(b.window(window, sinks), window, sinks)


PREFIX_CASES = [
    # kv, rows, prefix, ragged
    ([1], [1], 1, False),
    ([1, 5, 16], [1, 1, 1], 15, False),
    ([17, 0, 40, 3], [17, 0, 9, 1], 16, False),
    ([30, 1, 77, 160], [1, 1, 1, 1], 500, True),
    ([64] * 33, [1] * 33, 1030, False),
    ([20] * 12, [20] * 12, 333, True),
    ([300, 7], [1, 7], 0, True),
    ([300, 290], [300, 1], 700, False),
    ([2] * 3, [1] * 3, 4000, False),
    ([9, 33], [2, 2], 3000, True),
    ([90, 64, 200, 77], [90, 64, 64, 77], 1500, True),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("case", PREFIX_CASES, ids=str)
def test_prefix_attention(pkl, shape, case):
    kv, rows, prefix, ragged = case
    b = Batch(pkl, kv, rows, *shape, ragged=ragged, prefix=prefix, seed=len(kv) + prefix, spare_rows=2)
    b.check(b.shared())


@pytest.mark.parametrize("rows,prefix,rep", [(1, 0, 4), (20, 0, 4), (20, 300, 4), (1, 300, 4), (1, 300, 8)])
def test_many_requests(pkl, rows, prefix, rep):
    """More items than CTAs several times over (none is cut then, or, next to long ones of a prefix, some)."""
    b = Batch(pkl, [30 + rows] * 420, [rows] * 420, 2 * rep, 2, 128, True, prefix=prefix, seed=rows + prefix + rep)
    b.check(b.shared() if prefix else b.window(25, 3), 0 if prefix else 25, 0 if prefix else 3)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("spare", [1, 3, 700])
def test_batches_without_rows(pkl, half, spare):
    """Room for rows that no request has: nothing is written, whichever form the shapes ask for."""
    for prefix in (0, 300):
        b = Batch(pkl, [5, 0, 70], [0, 0, 0], 8, 2, 128, half, prefix=prefix, seed=spare, spare_rows=spare)
        b.check(b.shared() if prefix else b.window(9, 2))
        assert (b.out == 7.0).all()


@pytest.mark.parametrize("T", range(1, 10))
def test_fewer_rows_than_a_box(pkl, T):
    """1 to 9 rows of one request, 16 query heads a KV head (a box of q holds 8)."""
    b = Batch(pkl, [40 + T], [T], 16, 1, 128, True, seed=T)
    b.check(b.window(30, 1), 30, 1)


@pytest.mark.parametrize("n,prefix", [(310, 9000), (1300, 3000)])
def test_many_rows_of_many_parts(pkl, n, prefix):
    """One KV head: few long items behind a prefix, each cut into about eight parts (or few) for many rows."""
    b = Batch(pkl, [5] * n, [1] * n, 16, 1, 128, True, prefix=prefix, seed=n)
    b.check(b.shared())


@pytest.mark.parametrize("H,G,D", [(6, 2, 128), (10, 2, 64), (12, 1, 128), (15, 1, 64)])
def test_heads_that_do_not_fill_a_tile(pkl, H, G, D):
    """Groups of 3, 5, 12 and 15 query heads: single rows, as many as fit one small item, one more, and many."""
    n = 16 // (H // G)
    for rows in ([1, 1, 1], [n, n, 1], [n + 1, n, n], [70, 130, 1], [300, 257, 9]):
        kv = [r + 40 * i + 3 for i, r in enumerate(rows)]
        b = Batch(pkl, kv, rows, H, G, D, True, ragged=True, prefix=150, seed=sum(rows), spare_rows=1)
        b.check(b.shared())
        b = Batch(pkl, kv, rows, H, G, D, True, ragged=True, seed=sum(rows) + 1, spare_rows=1)
        b.check(b.window(30, 7), 30, 7)


def test_rows_and_blocks_behind_2_to_the_32(pkl):
    """A pool of more than 2^32 elements whose last blocks are used: written by qk_norm_rope, read by the attention."""
    G, H, D, far = 2, 8, 128, (1 << 32) // (2 * PAGE * 128) + 40
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    small = Batch(pkl, [100, 33, 700], [1, 1, 300], H, G, D, True, seed=17)
    pool = small.k.shape[0]
    k = torch.empty((far, G, PAGE, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    # the same rows, through the norm-less call, into blocks at the pool's end
    N = pool * PAGE
    qkv = torch.zeros(N, (H + 2 * G) * D, device="cuda")
    rows = qkv.view(N, H + 2 * G, D)
    rows[:, H:H + G] = small.k.transpose(1, 2).reshape(N, G, D).float().nan_to_num(0.0)
    rows[:, H + G:] = small.v.transpose(1, 2).reshape(N, G, D).float().nan_to_num(0.0)
    slot = i32(np.arange(N) + (far - pool) * PAGE)
    pkl.qk_norm_rope(qkv, H, G, torch.zeros_like(slot), slot, small.rope, k, v)
    assert torch.equal(k[far - pool:], small.k.nan_to_num(0.0)) and torch.equal(v[far - pool:], small.v.nan_to_num(0.0))
    want = small.window(90, 4).clone()
    t = small.pages.block_table
    t += (t >= 0) * (far - pool)
    small.k, small.v = k, v
    small.out.fill_(0)
    assert torch.equal(small.window(90, 4), want)
    del qkv, rows


@pytest.mark.parametrize("half", [False, True])
def test_large_scores_and_far_positions(pkl, half):
    """Scores of some hundreds (the running maximum moves by far more than any threshold) at positions up to 40000."""
    b = Batch(pkl, [40000, 900], [2, 300], 8, 2, 128, half, seed=3, scale=20.0)
    b.check(b.window(3000, 4), 3000, 4)


def test_scores_of_minus_infinity_and_nan_pass_through(pkl):
    """An infinite q component makes its row NaN as the formula does, and no other row."""
    b = Batch(pkl, [100, 90], [1, 1], 8, 2, 128, True, seed=4)
    ref = b.window(50, 0).clone()
    b.q[0, 3, 5] = float("inf")
    out = b.window(50, 0)
    assert torch.isnan(out[0, 3]).all()
    keep = torch.ones(2, 8, dtype=torch.bool)
    keep[0, 3] = False
    assert torch.equal(out[keep.cuda()], ref[keep.cuda()])


def test_results_do_not_depend_on_the_company_kept(pkl):
    """The same call twice gives the same bits (no order of arrival in any sum)."""
    for half in (False, True):
        b = Batch(pkl, [900, 33, 1500, 64], [3, 33, 1, 64], 8, 2, 128, half, ragged=True, prefix=700, seed=5)
        first = b.shared().clone()
        for _ in range(5):
            b.out.fill_(0)
            assert torch.equal(b.shared(), first)


@pytest.mark.parametrize("half", [False, True])
def test_captured_calls_follow_the_lengths(pkl, half):
    """One capture, replayed with other lengths, tables and rows in the same tensors, between eager calls."""
    small = Batch(pkl, [40, 300, 90], [1, 1, 1], 8, 2, 128, half, seed=6, prefix=200)
    small.shared()                               # modules loaded before the capture
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        small.shared()
    for lens in ([40, 300, 90], [39, 8, 89], [1, 33, 1], [5, 0, 17]):
        small.kv = lens
        small.pages.kv_len.copy_(i32(lens))
        small.rows = [min(1, k) for k in lens]
        small.row_start.copy_(i32(np.concatenate([[0], np.cumsum(small.rows)])))
        keep = small.places
        small.places = [(p[0][:n], p[1][:n]) for p, n in zip(keep, lens)]
        small.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        small.check(small.out)
        small.places = keep


def test_two_streams_with_scratch_of_their_own(pkl):
    a = Batch(pkl, [900] * 9, [1] * 9, 8, 2, 128, True, seed=7)
    b = Batch(pkl, [333] * 5, [40] * 5, 8, 2, 128, True, seed=8)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                x.window(200, 4)
    torch.cuda.synchronize()
    a.check(a.out, 200, 4)
    b.check(b.out, 200, 4)


def test_bad_device_metadata_is_skipped_and_reported(pkl):
    """Lengths, blocks and positions that only the device sees (test_batch_plan_host.py shows on the CPU that they
    lead nowhere out of bounds): the request is left alone or the page is empty, pic_sync says so once."""
    from position_independent_kv_link_gb300 import _lib as L
    for half in (False, True):
        b = Batch(pkl, [100, 90, 80], [1, 1, 1], 8, 2, 128, half, seed=9)
        good = b.window(0, 0).clone()
        assert sync() == 0
        kv = b.pages.kv_len.clone()
        b.pages.kv_len[1] = 10 ** 6
        b.out.fill_(7.0)
        out = b.window(0, 0)
        assert sync() == L.PIC_ERR_INVALID_ARG and sync() == 0
        # the others are right; not bit for bit `good`, as the work is cut elsewhere without request 1
        b.check(out, left=(1,))
        b.pages.kv_len.copy_(kv)
        table = b.pages.block_table.clone()
        b.pages.block_table[0, :7] = torch.tensor([-1, 10 ** 6, -5, 2 ** 31 - 1, 99999, -2 ** 31, 10 ** 5], dtype=torch.int32)
        out = b.window(0, 0)
        assert sync() == L.PIC_ERR_INVALID_ARG
        assert (out[0] == 0).all() and torch.equal(out[1:], good[1:])      # no page left: zeros
        b.pages.block_table.copy_(table)
        assert torch.equal(b.window(0, 0), good)


# ----------------------------------------------------------------------------- q/k norms

@pytest.mark.parametrize("H,G,D,half", [(32, 8, 128, True), (4, 4, 64, False), (7, 1, 64, True), (3, 1, 128, False),
                                        (40, 40, 128, True)])
@pytest.mark.parametrize("T", [1, 2, 37, 700])
@pytest.mark.parametrize("norm", ["both", "q", "none"])
def test_qk_norm_rope(pkl, H, G, D, half, T, norm):
    """q, K and V rows in 64 bits; padding rows, other slots and the columns behind the heads untouched.
    fp32: 2^-24 per operation of about 10 on the way (the norm's sum of D: D / 4 + 6 additions); then one rounding
    to the output type."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    N, extra = (H + 2 * G) * D, 8
    qkv = torch.randn(T, N + extra, generator=g, device="cuda") * torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
    qkv[0, :D] = 0.0                              # a head of zeros: eps keeps it finite
    qkv[:, N:] = float("nan")
    pool_t, act_t = (torch.bfloat16, torch.float16) if half else (torch.float32, torch.float32)
    blocks = T // 8 + 2
    k = torch.full((blocks, G, PAGE, D), 5.0, dtype=pool_t, device="cuda")
    v = torch.full_like(k, 6.0)
    rng = np.random.default_rng(T)
    slot = rng.permutation(blocks * PAGE)[:T]
    if T > 2:
        slot[1] = -1
    pos = rng.integers(0, 5000, T)
    table = rope_table(5000, D)
    gains = [None if norm == "none" else 1 + 0.2 * torch.randn(D, generator=g, device="cuda"),
             None if norm != "both" else 1 + 0.2 * torch.randn(D, generator=g, device="cuda")]
    q = torch.full((T, H, D), 7.0, dtype=act_t, device="cuda")
    out = pkl.qk_norm_rope(qkv[:, :N + 4], H, G, i32(pos), i32(slot), table, k, v, *gains, eps=1e-5, q_out=q)
    assert out is q
    x = qkv[:, :N].double().view(T, H + 2 * G, D)
    xq, xk, xv = x.split([H, G, G], 1)
    if gains[0] is not None:
        xq = xq / (xq.square().mean(-1, keepdim=True) + 1e-5).sqrt() * gains[0].double()
    if gains[1] is not None:
        xk = xk / (xk.square().mean(-1, keepdim=True) + 1e-5).sqrt() * gains[1].double()
    xq = rotated(xq, torch.tensor(pos).cuda(), table)
    live = torch.tensor(slot >= 0).cuda()
    s = torch.tensor(slot).cuda().clamp(min=0)
    rows_k, rows_v = k[s // PAGE, :, s % PAGE], v[s // PAGE, :, s % PAGE]
    work = (D / 4 + 16) * 2.0 ** -24
    for got, ref, t in ((q, xq, act_t), (rows_k, xk, pool_t), (rows_v, xv, pool_t)):
        step = torch.finfo(t).eps / 2
        # a rotated pair mixes two values, each off by `work` of its own size; fp16 has steps of 2^-24 near zero
        size = (ref.square() + ref.roll(D // 2, -1).square()).sqrt()
        tol = (1.5 * work * size + step * (1 + work) * ref.abs() + (2.0 ** -25 if t is torch.float16 else 0.0))
        assert ((got.double() - ref).abs() <= tol)[live].all()
    assert (q[~live] == 7.0).all()
    used = torch.zeros(blocks * PAGE, dtype=torch.bool)
    used[slot[slot >= 0]] = True
    free = ~used.view(blocks, PAGE).cuda()
    assert (k.transpose(1, 2)[free] == 5.0).all() and (v.transpose(1, 2)[free] == 6.0).all()


def test_qk_norm_rope_flags(pkl):
    """Slots and positions outside the pool and the table are skipped, values beyond fp16 flagged."""
    from position_independent_kv_link_gb300 import _lib as L
    k = torch.zeros(4, 1, PAGE, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    x = torch.randn(3, 3 * 64, device="cuda")
    table = rope_table(100, 64)
    q = torch.full((3, 1, 64), 7.0, dtype=torch.float16, device="cuda")
    pkl.qk_norm_rope(x, 1, 1, i32([5, 100, -1]), i32([64, 3, 4]), table, k, v, q_out=q)
    assert sync() == L.PIC_ERR_INVALID_ARG and sync() == 0
    assert (q == 7.0).all() and (k == 0).all() and (v == 0).all()
    x[1, 64] = 5e4                                 # k
    pkl.qk_norm_rope(x, 1, 1, i32([5, 6, 7]), i32([1, 2, 3]), table, k, v, q_out=q)
    assert sync() == L.PIC_ERR_RANGE and sync() == 0


# ----------------------------------------------------------------------------- block tables

def tables_reference(kv, new, pages, table, free, used, max_rows, first, pos):
    """The step's bookkeeping as a loop."""
    kv, table, pos = list(kv), table.copy(), None if pos is None else pos.copy()
    start, row_pos, slot, n_pages = [0], [], [], []
    for r, m in enumerate(new):
        starts = [int(p) for p in pos[r, :pages[r]]] if pos is not None else [first + PAGE * p for p in range(pages[r])]
        for _ in range(m):
            at = first + kv[r]
            if not starts or at >= starts[-1] + PAGE:
                starts.append(at)
                table[r, len(starts) - 1] = free[used]
                if pos is not None:
                    pos[r, len(starts) - 1] = at
                used += 1
            row_pos.append(at)
            slot.append(int(table[r, len(starts) - 1]) * PAGE + at - starts[-1])
            kv[r] += 1
        start.append(start[-1] + m)
        n_pages.append(len(starts))
    n = len(row_pos)
    return dict(kv_len=kv, n_pages=n_pages, row_start=start, row_pos=row_pos + [0] * (max_rows - n),
                row_slot=slot + [-1] * (max_rows - n), counts=[n, used, 0]), table, pos


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("n,kv_hi,new_hi,first,used", [(1, 1, 1, 0, 0), (1, 40, 3000, 0, 3), (5, 40, 0, 7, 0), (300, 200, 2, 0, 0),
                                                       (700, 90, 70, 33, 1), (5000, 20, 3, 0, 0), (12288, 3, 2, 0, 0)])
def test_block_tables(pkl, ragged, n, kv_hi, new_hi, first, used):
    rng = np.random.default_rng(n)
    kv = rng.integers(0, kv_hi + 1, n).tolist()
    new = rng.integers(0, new_hi + 1, n).tolist()
    lens = [page_lengths(k, ragged, rng) for k in kv]
    pages = [len(p) for p in lens]
    stride = max(p + -(-m // PAGE) for p, m in zip(pages, new)) + 1
    table, pos = np.full((n, stride), -3), np.full((n, stride), BIG)
    at = 0
    for r, p in enumerate(lens):
        table[r, :len(p)] = np.arange(at, at + len(p))
        if p:
            pos[r, :len(p)] = first + np.concatenate([[0], np.cumsum(p)[:-1]])
        at += len(p)
    need = sum(-(-max(0, m - (PAGE - p[-1] if p else 0)) // PAGE) for m, p in zip(new, lens))
    free = rng.permutation(at + need + 40)[:used + need].tolist()
    max_rows = max(1, sum(new) + 3)
    ref, rt, rp = tables_reference(kv, new, pages, table, free, used, max_rows, first, pos if ragged else None)
    d_table, d_pos, d_np = i32(table), i32(pos) if ragged else None, i32(pages) if ragged else None
    r = pkl.block_tables(i32(kv), i32(new), d_table, i32(free), max_rows, page_pos=d_pos, n_pages=d_np,
                         free_used=i32([used]), first=first)
    for key, want in ref.items():
        assert getattr(r, key).tolist() == want, key
    assert np.array_equal(d_table.cpu().numpy(), rt)
    if ragged:
        assert np.array_equal(d_pos.cpu().numpy(), rp)


@pytest.mark.parametrize("max_rows", [1, 1023, 1024, 1025, 4096, 24575, 24576, 24577, 40000])
@pytest.mark.parametrize("n", [1, 1024, 1025])
def test_block_tables_row_counts(pkl, n, max_rows):
    """One request has all the rows (or every row of max_rows is one of its own), the others none."""
    new = [0] * n
    new[n // 2] = max_rows
    kv = [7] * n
    table = np.full((n, -(-(7 + max_rows) // PAGE)), -3)
    table[:, 0] = np.arange(n)
    free = list(range(n, n + -(-(7 + max_rows) // PAGE)))
    ref, rt, _ = tables_reference(list(kv), new, [1] * n, table, free, 0, max_rows, 5, None)
    d = i32(table)
    r = pkl.block_tables(i32(kv), i32(new), d, i32(free), max_rows, first=5)
    for key, want in ref.items():
        assert getattr(r, key).tolist() == want, key
    assert np.array_equal(d.cpu().numpy(), rt)


@pytest.mark.parametrize("max_rows", [40, 9000, 30000])
def test_block_tables_in_place(pkl, max_rows):
    """The lengths, page counts and used entries updated in place, twice in a row and captured."""
    kv, new, table = i32([0, 17, 40]), i32([5, 0, 30]), i32(np.arange(300).reshape(3, 100) + 1000)
    free, used = i32(np.arange(50)), i32([3])
    out = pkl.BlockTables(kv, torch.empty_like(kv), i32(np.zeros(4)), i32(np.zeros(max_rows)), i32(np.zeros(max_rows)),
                          torch.zeros(3, dtype=torch.int32, device="cuda"))
    call = lambda: pkl.block_tables(kv, new, table, free, max_rows, free_used=out.counts[1:2], out=out)
    out.counts[1:2] = used
    call()
    assert kv.tolist() == [5, 17, 70] and out.counts.tolist() == [35, 6, 0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    assert kv.tolist() == [10, 17, 100] and out.counts.tolist() == [35, 8, 0]
    assert out.row_start.tolist() == [0, 5, 5, 35] and out.row_pos[:5].tolist() == [5, 6, 7, 8, 9]
    assert table[0, 0] == 3 and table[2, 3:7].tolist() == [4, 5, 6, 7]


def test_block_tables_all_or_nothing(pkl):
    from position_independent_kv_link_gb300 import _lib as L
    table = i32([[4, -1, -1], [5, 6, -1]])
    kv, new, free = i32([16, 30]), i32([1, 17]), i32([9, 8])

    def call(kv=kv, new=new, free=free, max_rows=20, **kw):
        t = table.clone()
        return pkl.block_tables(kv, new, t, free, max_rows, **kw), t
    r, t = call()
    assert r.counts.tolist() == [18, 2, 0] and t.tolist() == [[4, 9, -1], [5, 6, 8]] and sync() == 0
    for kw, status in ((dict(free=i32([9])), L.PIC_ERR_OUT_OF_BLOCKS), (dict(free_used=i32([1])), L.PIC_ERR_OUT_OF_BLOCKS),
                       (dict(free_used=i32([-1])), L.PIC_ERR_OUT_OF_BLOCKS),
                       (dict(max_rows=17), L.PIC_ERR_CAPACITY), (dict(new=i32([1, 19])), L.PIC_ERR_CAPACITY),
                       (dict(new=i32([1, -1])), L.PIC_ERR_INVALID_ARG), (dict(kv=i32([-4, 30])), L.PIC_ERR_INVALID_ARG),
                       (dict(page_pos=i32([[0, 0, 0], [0, 16, 0]]), n_pages=i32([1, 1])), L.PIC_ERR_INVALID_ARG)):
        r, t = call(**kw)
        assert torch.equal(t, table), kw
        assert r.counts[0] == 0 and r.counts[2] != 0 and r.row_start.tolist() == [0, 0, 0]
        assert (r.row_slot == -1).all() and r.kv_len.tolist() == kw.get("kv", kv).tolist()
        assert sync() == status and sync() == 0


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("prefix", [0, 213])
def test_decode_loop_captured(pkl, half, prefix):
    """Block tables, norms with rotation and attention as one captured step, replayed over steps whose lengths only
    the device knows (a prompt piece, then single tokens; one request pauses), against a 64-bit recomputation from
    the rows of qkv alone."""
    H, G, D, n, window, sinks = 8, 2, 128, 3, 40, 4
    steps = [[30, 1, 17], [1, 1, 1], [1, 0, 1], [1, 1, 1], [2, 1, 0], [1, 1, 1]]
    max_rows, pool = 50, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    pool_t, act_t = (torch.bfloat16, torch.float16) if half else (torch.float32, torch.float32)
    k = torch.zeros(pool, G, PAGE, D, dtype=pool_t, device="cuda")
    v = torch.zeros_like(k)
    table, rope = i32(np.full((n, 6), -1)), rope_table(prefix + 200, D)
    gq, gk = (1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    n_pre = -(-prefix // PAGE)
    pre = torch.arange(n_pre, dtype=torch.int32, device="cuda")
    hist = [[] for _ in range(n)]                   # (k, v) rows in 64 bits
    pre_k = torch.randn(prefix, G, D, generator=g, device="cuda").to(pool_t)
    pre_v = torch.randn(prefix, G, D, generator=g, device="cuda").to(pool_t)
    p = torch.arange(prefix, device="cuda")
    k[p // PAGE, :, p % PAGE], v[p // PAGE, :, p % PAGE] = pre_k, pre_v
    free = torch.arange(n_pre, pool, dtype=torch.int32, device="cuda").flip(0).contiguous()
    kv, new, qkv = i32([0] * n), i32([0] * n), torch.zeros(max_rows, (H + 2 * G) * D, device="cuda")
    bt = pkl.BlockTables(kv, i32([0] * n), i32([0] * (n + 1)), i32([0] * max_rows), i32([-1] * max_rows), i32([0, 0, 0]))
    q = torch.zeros(max_rows, H, D, dtype=act_t, device="cuda")
    out = torch.zeros_like(q)

    def step():
        pkl.block_tables(kv, new, table, free, max_rows, free_used=bt.counts[1:2], first=prefix, out=bt)
        pkl.qk_norm_rope(qkv, H, G, bt.row_pos, bt.row_slot, rope, k, v, gq, gk, q_out=q)
        pages = pkl.BatchPages(kv, table)
        if prefix:
            pkl.attention_prefix(q, bt.row_start, pre, prefix, pages, k, v, rope, out=out)
        else:
            pkl.attention_window(q, bt.row_start, pages, k, v, rope, window, sinks, out=out)
    step()                                          # no rows: nothing happens, modules load
    assert sync() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    norm = lambda x, gain: x / (x.square().mean(-1, keepdim=True) + 1e-5).sqrt() * gain.double()  # noqa: E731
    for lens in steps:
        new.copy_(i32(lens))
        qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda"))
        graph.replay()
        assert sync() == 0
        t = 0
        for r, m in enumerate(lens):
            x = qkv[t:t + m].double().view(m, H + 2 * G, D)
            for i in range(m):
                hist[r].append((norm(x[i, H:H + G], gk).to(pool_t).double(), x[i, H + G:].to(pool_t).double()))
            if m:
                K = torch.cat([pre_k.double(), torch.stack([a for a, _ in hist[r]])])
                V = torch.cat([pre_v.double(), torch.stack([b for _, b in hist[r]])])
                N = len(K)
                u = torch.arange(N, device="cuda")
                at = torch.arange(N - m, N, device="cuda")
                Q = rotated(norm(x[:, :H], gq), at, rope).view(m, G, H // G, D)
                y = torch.einsum("tgrd,kgd->grtk", Q, rotated(K, u, rope)) / D ** 0.5
                seen = u[None] <= at[:, None]
                if not prefix:
                    seen &= (u[None] > at[:, None] - window) | (u[None] < sinks)
                w = torch.softmax(y.masked_fill(~seen, float("-inf")), -1)
                ref = torch.einsum("grtk,kgd->tgrd", w, V).reshape(m, H, D)
                rel = ((out[t:t + m].double() - ref).norm() / ref.norm()).item()
                # fp32 norms and sums; with bf16 pools also q and rotated K in fp16, weights in bf16
                assert rel < (1.2e-2 if half else 2e-5), (r, m, rel)
            t += m
    assert bt.counts.tolist()[1] == sum(-(-len(h) // PAGE) for h in hist)


def test_pages_of_a_linked_request(pkl):
    """The page table of a linked request (ragged chunk pages) taken over by the batched call gives what the
    single-sequence attention gives over the same pages."""
    import pic_inputs as pi
    spec = pi.SMALL_BF16
    wl = pi.make_workload("batch pages", spec, 3, [50, 64, 37], 20, 8)
    model = pkl.PicModel(spec, pi.gen_weights(spec))
    store = pkl.PicStore(model, num_blocks=64, max_rows=512, max_requests=4, max_positions=1024)
    cids = store.compile(wl.chunks)
    res = store.link([([cids[c] for c in r.chunk_ids], r.query) for r in wl.requests], wl.k)
    store.sync()
    info = store.request_info(res.requests[0])
    H, G, D = spec.n_heads, spec.n_kv_heads, spec.head_dim
    n = int(info["page_pos"][-1] + info["page_len"][-1])
    m = 9
    q = torch.randn(m, H, D, device="cuda")
    rope = pkl.rope_table(1024, D, spec.rope_base)
    at = np.arange(n - m, n, dtype=np.int32)
    kl, vl = store.k_pool[1], store.v_pool[1]
    ref = pkl.attention(q, at, kl, vl, (info["page_table"], info["page_pos"], info["page_len"]), rope, G)
    pages = pkl.BatchPages(i32([n]), i32(info["page_table"][None]), i32(info["page_pos"][None]), i32([len(info["page_pos"])]))
    turned = rotated(q.double(), torch.tensor(at).cuda().long(), rope).half()
    got = pkl.attention_window(turned, i32([0, m]), pages, kl, vl, rope, 0)
    # both within the roundings of fp16 operands and bf16 weights of the same numbers
    assert ((got.double() - ref.double()).norm() / ref.double().norm()).item() < 1.5e-2
    store.close()
    model.close()


def test_refusals(pkl):
    from position_independent_kv_link_gb300 import _lib as L
    b = Batch(pkl, [40], [1], 8, 2, 128, True, seed=1)
    with pytest.raises(ValueError):
        pkl.attention_window(b.q.float(), b.row_start, b.pages, b.k, b.v, b.rope, 5)
    with pytest.raises(ValueError):
        pkl.attention_window(b.q, b.row_start, b.pages, b.k, b.v[:-1], b.rope, 5)
    with pytest.raises(ValueError):
        pkl.attention_window(b.q, b.row_start.long(), b.pages, b.k, b.v, b.rope, 5)
    with pytest.raises(ValueError):
        pkl.attention_window(b.q, b.row_start, b.pages, b.k.transpose(1, 2), b.v, b.rope, 5)
    for args in ((-1, 0), (5, -1)):
        with pytest.raises(L.PicError) as e:
            b.window(*args)
        assert e.value.status == L.PIC_ERR_INVALID_ARG
    with pytest.raises(L.PicError) as e:
        b.window(5, 0, scratch=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == L.PIC_ERR_INVALID_ARG
    wide = Batch(pkl, [40], [1], 17, 1, 64, True, seed=1)
    with pytest.raises(L.PicError) as e:
        wide.window(5, 0)
    assert e.value.status == L.PIC_ERR_UNSUPPORTED
    with pytest.raises(L.PicError):
        pkl.attention_prefix(b.q, b.row_start, i32([0]), 17, b.pages, b.k, b.v, b.rope)   # 17 positions in one page
    with pytest.raises(L.PicError):
        pkl.qk_norm_rope(torch.zeros(1, 12 * 128 + 1, device="cuda"), 8, 2, i32([0]), i32([0]), b.rope, b.k, b.v)  # stride % 4
