"""4-bit weights on the GPU: packing against the definition in 64 bits, the layout as documented, and the product of few rows against
64 bits, at the row counts, sizes, groups and strides where its forms change.

Packing is exact: scales, zeros and codes are compared for equality.

Product: a group's sum consists of n <= 256 products (8-bit rows: codes and zeros apart), each exact; adding them in fp32, the tensor
cores' additions truncating, is off by at most n 2^-23 of B = sum (code + zero) |x|; then comes one product with the scales (2^-23 for both)
and one addition per group, split over at most 16 partial sums: (G + 16) 2^-24 of the sum of magnitudes. So each element is within
  ((256 + 2) 2^-23 + (G + 16) 2^-24) sum_g s B_g.
Mistakes of a smaller size show in the norm: independent errors of G additions, and of some 64 in a group whose partial sums are
up to 5 times the result's (code + zero against code - zero, which has a spread of 4.6), leave it within 2^-24 (sqrt(G) + 5 * 8) of the
result's norm for rows without a common sign.
"""
import numpy as np
import pytest
import torch

from .test_gpu_batch import pkl, nothing_flagged, sync  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def spread(x, group, K):
    return x.repeat_interleave(group, dim=1)[:, :K]


def quantised(W, group):
    """Scales (fp16), zeros, codes [N, groups or K] by the definition, in 64 bits. A group with a NaN stands for zeros."""
    N, K = W.shape
    w = torch.nn.functional.pad(W.double(), (0, -K % group)).view(N, -1, group)
    w = torch.where(w.isnan().any(-1, keepdim=True), 0.0, w)
    lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15).float().half()
    d = torch.where(s > 0, s.double(), 1.0)
    z = torch.where(s > 0, torch.round(-lo / d).clamp(0, 15), 0.0)
    c = torch.where(s[..., None] > 0, (torch.round(w / d[..., None]) + z[..., None]).clamp(0, 15), 0.0)
    return s, z, c.view(N, -1)[:, :K]


def unpacked_by_the_document(w):
    """codes [N, K], scales and zeros [N, groups], read out of the packed bytes as include/pic.h states the layout."""
    N, K, group = w.N, w.K, w.group
    nt, kt, per = -(-N // 128), -(-K // 128), 128 // group
    t = w.data.cpu().numpy().reshape(nt, kt, 8192 + per * 384)
    r, q = np.arange(128)[:, None], np.arange(4)[None, :]
    at = 64 * r + 16 * (q ^ (r // 2 % 4))
    codes = np.zeros((nt, kt, 128, 128), np.uint8)
    words = t[..., :8192].reshape(nt, kt, -1, 4).copy().view(np.uint32)[..., 0]
    for j in range(4):
        x = words[:, :, at // 4 + j]                                       # [nt, kt, 128, 4 pieces]
        for e in range(8):
            codes[..., 32 * j + e::8][..., :4] = x >> (4 * (e // 2 + 4 * (e % 2))) & 15
    place = r[:, 0] // 32 * 32 + r[:, 0] % 8 * 4 + r[:, 0] // 8 % 4
    s = t[..., 8192:8192 + per * 256].reshape(nt, kt, per, 256).copy().view(np.float16)[..., place]
    z = t[..., 8192 + per * 256:].reshape(nt, kt, per, 128)[..., place]
    flat = lambda x: torch.tensor(x.transpose(0, 3, 1, 2).reshape(nt * 128, kt * per)[:N, :-(-K // group)])  # noqa: E731
    return torch.tensor(codes.transpose(0, 2, 1, 3).reshape(nt * 128, kt * 128)[:N, :K]), flat(s), flat(z)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (128, 128, 128), (129, 160, 64), (77, 1120, 32), (300, 4096, 128), (5, 96, 128)])
def test_packing_is_the_definition(pkl, dtype, N, K, group):
    W = (randn(N + K, N, K) * K ** -0.5).to(TYPES[dtype])
    w = pkl.pack_weight4(W, group)
    s, z, c = quantised(W, group)
    codes, scales, zeros = unpacked_by_the_document(w)
    assert torch.equal(scales, s.cpu()) and torch.equal(zeros.double(), z.cpu()) and torch.equal(codes.double(), c.cpu())
    values = pkl.unpack_weight4(w)
    assert torch.equal(values.double(), spread(s.double(), group, K) * (c - spread(z, group, K)))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_packing_next_to_the_borders(pkl, dtype):
    """Weights that lie halfway between two codes, or one bit beside that, in every code of scales of eleven bits."""
    rows, group = 64, 32
    rng = np.random.default_rng(3)
    W = np.zeros((rows, 4 * group), np.float64)
    for r in range(rows):
        for g in range(4):
            s = float(np.float16(rng.uniform(0.01, 0.02)))
            zero = int(rng.integers(0, 16))
            lo, hi = -zero * s, (15 - zero) * s
            x = (rng.integers(0, 15, group) - zero + 0.5) * s
            x[:2] = lo, hi
            W[r, g * group:(g + 1) * group] = x
    t = torch.tensor(W).to(TYPES[dtype]).cuda()
    if dtype == "f32":                                       # one bit up, one bit down (a NaN where a group ends in 0), and as they are
        bits = t.view(torch.int32)
        bits[0::3, 2:] += 1
        bits[1::3, 2:] -= 1
    w = pkl.pack_weight4(t, group)
    s, z, c = quantised(t, group)
    codes, scales, zeros = unpacked_by_the_document(w)
    assert torch.equal(scales, s.cpu()) and torch.equal(zeros.double(), z.cpu()) and torch.equal(codes.double(), c.cpu())
    assert sync() == (7 if t.isnan().any() else 0)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_packing_of_weights_at_any_16_bytes(pkl, dtype):
    """Weights that begin between two 32-byte borders are loaded in smaller pieces."""
    N, K, t = 130, 160, TYPES[dtype]
    each = 16 // torch.empty(0, dtype=t).element_size()
    buf = randn(4, N * K + each).to(t)
    apart = buf[each:].view(N, K)
    assert apart.data_ptr() % 32 == 16
    for group in (32, 64, 128):
        a, b = pkl.pack_weight4(apart, group), pkl.pack_weight4(apart.clone(), group)
        assert torch.equal(a.data, b.data)


def test_packing_of_special_groups(pkl):
    """Zeros (and -0), one sign only, scales below fp16's normal range and below its least number, the greatest ones."""
    W = torch.zeros(8, 64, device="cuda")
    W[0] = -0.0
    W[1] = torch.linspace(1, 5, 64)
    W[2] = -torch.linspace(1, 5, 64)
    W[3] = randn(1, 64) * 3e-6
    W[4] = randn(2, 64) * 1e-8
    W[5, 7] = 15 * 65504.0
    W[6] = randn(3, 64) * 1e5
    W[7, 0], W[7, 1] = 1e-40, -1e-40
    s, z, c = quantised(W, 64)
    w = pkl.pack_weight4(W, 64)
    codes, scales, zeros = unpacked_by_the_document(w)
    assert torch.equal(scales, s.cpu()) and torch.equal(zeros.double(), z.cpu()) and torch.equal(codes.double(), c.cpu())
    assert scales[4, 0] == 0 and torch.isfinite(scales).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 2e6])
def test_packing_flags_what_has_no_scale(pkl, bad):
    W = randn(4, 130, 256)
    want = quantised(W, 128)
    W[129, 200] = bad
    w = pkl.pack_weight4(W)
    assert sync() == 7                                       # PIC_ERR_RANGE, once
    values = pkl.unpack_weight4(w)
    assert (values[129, 128:] == 0).all()
    s, z, c = want
    whole = (spread(s.double(), 128, 256) * (c - spread(z, 128, 256)))
    assert torch.equal(values[:129].double(), whole[:129]) and torch.equal(values[129, :128].double(), whole[129, :128])


@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (130, 160, 64), (257, 1120, 128), (128, 96, 32)])
def test_codes_of_another_quantiser(pkl, N, K, group):
    rng = np.random.default_rng(N)
    codes = torch.tensor(rng.integers(0, 16, (N, K)), dtype=torch.uint8).cuda()
    scales = torch.tensor(rng.standard_normal((N, -(-K // group)))).half().cuda()          # negative ones too
    zeros = torch.tensor(rng.integers(0, 16, (N, -(-K // group))), dtype=torch.uint8).cuda()
    for z in (zeros, None):
        w = pkl.pack_codes4(codes, scales, z, group)
        got = unpacked_by_the_document(w)
        zz = torch.full_like(zeros, 8) if z is None else z
        assert torch.equal(got[0], codes.cpu()) and torch.equal(got[1], scales.cpu()) and torch.equal(got[2], zz.cpu())
        values = spread(scales.double(), group, K) * (codes.double() - spread(zz.double(), group, K))
        assert torch.equal(pkl.unpack_weight4(w).double(), values)


def test_codes_above_15_are_flagged(pkl):
    codes = torch.full((3, 64), 7, dtype=torch.uint8, device="cuda")
    scales, zeros = torch.ones(3, 1, dtype=torch.float16, device="cuda"), torch.full((3, 1), 8, dtype=torch.uint8, device="cuda")
    codes[1, 5] = 0x35
    w = pkl.pack_codes4(codes, scales, zeros, 64)
    assert sync() == 1
    assert pkl.unpack_weight4(w)[1, 5] == 5 - 8
    codes[1, 5], zeros[2, 0] = 5, 0x18
    pkl.pack_codes4(codes, scales, zeros, 64)
    assert sync() == 1


# ----------------------------------------------------------------------------- product

def weights(pkl, N, K, group, seed=0):
    rng = np.random.default_rng(seed + N + K)
    codes = torch.tensor(rng.integers(0, 16, (N, K)), dtype=torch.uint8).cuda()
    scales = torch.tensor(rng.uniform(0.5, 2.0, (N, -(-K // group)))).half().cuda()
    zeros = torch.tensor(rng.integers(0, 16, (N, -(-K // group))), dtype=torch.uint8).cuda()
    return pkl.pack_codes4(codes, scales, zeros, group), codes, scales, zeros


def rows(T, K, e4m3, seed=1):
    x = randn(seed, T, K)
    if not e4m3:
        return x.half(), None
    a = torch.nn.functional.pad(x, (0, -K % 128)).view(T, -1, 128)
    s = a.abs().amax(-1) / 448 * (1 + 0.3 * randn(seed + 1, T, a.shape[1]).abs())
    return (a / s[..., None]).view(T, -1)[:, :K].contiguous().to(torch.float8_e4m3fn), s


def hold(y, codes, scales, zeros, group, x, x_scales):
    K = codes.shape[1]
    s, z = spread(scales.double(), group, K), spread(zeros.double(), group, K)
    X = x.double() if x_scales is None else x.double() * spread(x_scales.double(), 128, K)
    ref = X @ ((codes.double() - z) * s).t()
    size = X.abs() @ ((codes.double() + z) * s).t()
    G = scales.shape[1]
    tol = ((256 + 2) * 2.0 ** -23 + (G + 16) * 2.0 ** -24) * size
    off = (y.double() - ref).abs()
    assert (off <= tol).all(), (off / tol).amax().item()
    rel = (off.norm() / ref.norm()).item()
    assert rel <= 2.0 ** -24 * (G ** 0.5 + 40), rel


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130])
@pytest.mark.parametrize("N,K,group", [(257, 416, 64), (128, 128, 128)])
def test_product_by_rows(pkl, T, N, K, group, e4m3):
    w, *parts = weights(pkl, N, K, group)
    x, sx = rows(T, K, e4m3)
    hold(pkl.gemm_w4(w, x, sx), *parts, group, x, sx)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 16, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 32), (3, 96), (127, 160), (129, 1120), (1001, 128), (300, 14336), (40, 16416), (2305, 64)])
def test_product_by_shape(pkl, T, group, N, K, e4m3):
    w, *parts = weights(pkl, N, K, group)
    x, sx = rows(T, K, e4m3)
    hold(pkl.gemm_w4(w, x, sx), *parts, group, x, sx)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [17, 33, 64, 200])
def test_product_of_many_blocks(pkl, T, group, e4m3):
    """More blocks than the narrow form takes, an odd number of tiles; bands in turn (N 40961) and bands shared by clusters."""
    for N, K in ((40961, 1760), (1153, 65536)):
        w, *parts = weights(pkl, N, K, group)
        x, sx = rows(T, K, e4m3)
        hold(pkl.gemm_w4(w, x, sx), *parts, group, x, sx)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,N,K,group", [(1, 89500, 256, 128), (5, 90000, 160, 32), (16, 70000, 288, 64), (128, 12000, 256, 128),
                                         (64, 43520, 256, 128), (50, 43300, 416, 64), (20, 43001, 1120, 32), (130, 30000, 512, 32),
                                         (190, 30000, 512, 128), (64, 39000, 128, 128), (64, 6144, 4096, 128), (33, 4200, 4096, 64)])
def test_product_of_what_a_turn_leaves(pkl, T, N, K, group, e4m3):
    """Somewhat more bands than CTAs that run at once (pairs share the rest; with one block in a band they cannot), and clusters that
    need not all find room."""
    w, *parts = weights(pkl, N, K, group)
    x, sx = rows(T, K, e4m3)
    y = pkl.gemm_w4(w, x, sx)
    hold(y, *parts, group, x, sx)
    assert torch.equal(pkl.gemm_w4(w, x, sx), y)


@pytest.mark.parametrize("e4m3", [False, True])
def test_product_again_and_in_place(pkl, e4m3):
    """The same bits again; out= written whole, nothing beside it; rows of X that lie apart, NaN between them."""
    T, N, K = 11, 300, 544
    w, *parts = weights(pkl, N, K, 128)
    x, sx = rows(T, K, e4m3)
    first = pkl.gemm_w4(w, x, sx)
    apart = torch.full((T, K + 32), float("nan"), device="cuda").to(x.dtype)
    apart[:, 16:16 + K] = x if not e4m3 else x
    buf = torch.full((T + 2, N), 7.0, device="cuda")
    again = pkl.gemm_w4(w, apart[:, 16:16 + K], sx, out=buf[1:T + 1]) if (buf[1:].data_ptr() % 16 == 0) else None
    assert again is not None and torch.equal(again, first) and (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert torch.equal(pkl.gemm_w4(w, x, sx), first)


@pytest.mark.parametrize("T", [3, 40])
def test_product_keeps_rows_apart(pkl, T):
    """NaN and infinity in one row of X, and in one row of weights' scales, stay there."""
    N, K = 300, 4096 if T == 3 else 65536
    w, codes, scales, zeros = weights(pkl, N, K, 128)
    x, _ = rows(T, K, False)
    clean = pkl.gemm_w4(w, x)
    x[1, 100], x[2, 5] = float("nan"), float("inf")
    y = pkl.gemm_w4(w, x)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[3:], clean[3:]) and y[1].isnan().all() and not torch.isfinite(y[2]).any()
    scales[7, 3] = float("inf")
    y = pkl.gemm_w4(pkl.pack_codes4(codes, scales, zeros, 128), rows(T, K, False)[0])
    keep = torch.arange(N, device="cuda") != 7
    assert torch.equal(y[:, keep], clean[:, keep]) and not torch.isfinite(y[:, 7]).any()


@pytest.mark.parametrize("T,N,K", [(3, 300, 1120), (40, 300, 65536)])
def test_product_keeps_8_bit_rows_apart(pkl, T, N, K):
    """The same for 8-bit rows, and for their scales."""
    w, *_ = weights(pkl, N, K, 128)
    x, sx = rows(T, K, True)
    clean = pkl.gemm_w4(w, x, sx)
    x[1, 100] = float("nan")
    sx[2, 3] = float("inf")
    y = pkl.gemm_w4(w, x, sx)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[3:], clean[3:]) and y[1].isnan().all() and not torch.isfinite(y[2]).any()


def test_rows_of_one_sign(pkl):
    """Rows with a common sign, where the codes' part and the zeros' part are much larger than their difference: within the
    element's bound (the norm's is for rows without one)."""
    T, N, K = 20, 300, 2048
    for e4m3 in (False, True):
        w, codes, scales, zeros = weights(pkl, N, K, 128)
        x, sx = rows(T, K, e4m3)
        x = x.float().abs().to(x.dtype)
        y = pkl.gemm_w4(w, x, sx)
        X = x.double() if sx is None else x.double() * spread(sx.double(), 128, K)
        s, z = spread(scales.double(), 128, K), spread(zeros.double(), 128, K)
        ref, size = X @ ((codes.double() - z) * s).t(), X @ ((codes.double() + z) * s).t()
        assert ((y.double() - ref).abs() <= (258 * 2.0 ** -23 + 32 * 2.0 ** -24) * size).all()


def test_packed_and_multiplied(pkl):
    """pack_weight4 and the product against the values that unpack_weight4 gives."""
    for dtype in TYPES.values():
        W = (randn(5, 640, 1056) * 0.03).to(dtype)
        w = pkl.pack_weight4(W, 64)
        x = randn(6, 5, 1056).half()
        ref = x.double() @ pkl.unpack_weight4(w).double().t()
        assert ((pkl.gemm_w4(w, x).double() - ref).norm() / ref.norm()).item() < 2.0 ** -24 * (17 ** 0.5 + 40)


def test_offsets_behind_32_bits(pkl):
    """More than 2^32 weights, and results behind 2^32 elements."""
    N, K = 262145, 16416
    codes = torch.randint(0, 16, (N, K), dtype=torch.uint8, device="cuda")
    scales = torch.ones(N, -(-K // 128), dtype=torch.float16, device="cuda")
    w = pkl.pack_codes4(codes, scales)
    x = rows(2, K, False)[0]
    y = pkl.gemm_w4(w, x)
    for n in (0, N // 2, N - 1):
        ref = x.double() @ (codes[n].double() - 8)
        assert ((y[:, n].double() - ref).abs() < 1e-3 * K ** 0.5).all()
    values = pkl.unpack_weight4(w, out=torch.empty(N, K, device="cuda"))
    assert torch.equal(values[N - 1], codes[N - 1].float() - 8)
    del codes, values, y, w
    torch.cuda.empty_cache()
    T, N, K = 40000, 110000, 32
    w, codes, scales, zeros = weights(pkl, N, K, 32)
    x = rows(T, K, False)[0]
    y = pkl.gemm_w4(w, x)
    hold(y[-2:], codes, scales, zeros, 32, x[-2:], None)
    hold(y[T // 2:T // 2 + 2], codes, scales, zeros, 32, x[T // 2:T // 2 + 2], None)
    del y
    torch.cuda.empty_cache()
