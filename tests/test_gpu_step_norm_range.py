"""The norm of rows whose squares, or their sum, fp32 does not hold, against 64 bits (the bounds of test_gpu_step_rows.py: the scaled
sum has as many roundings as the plain one, and scaling by powers of two has none)."""
import pytest
import torch

from .test_gpu_batch import pkl, nothing_flagged, sync  # noqa: F401  (fixtures)
from .test_gpu_step_rows import E4M3, check_norm
from .test_gpu_weight4 import randn

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.float16, E4M3], ids=["f32", "f16", "e4m3"])
LARGEST = torch.finfo(torch.float32).max


def norm(pkl, h, gain, delta, eps, dtype):
    r = pkl.add_rms_norm(h, gain, delta, eps=eps, dtype=dtype)
    return r if dtype is E4M3 else (r, None)


@TYPES
@pytest.mark.parametrize("d", [4, 132, 4096, 32768])
def test_rows_whose_squares_overflow(pkl, d, dtype):
    """One large value, large ones throughout, the largest, and ordinary rows beside them, which are the same as without."""
    h, gain = randn(d, 7, d), 1 + 0.1 * randn(1, d)
    plain = norm(pkl, h.clone(), gain, None, 1e-5, dtype)
    h[1, d // 2] = 1e20
    h[2] *= 1e30
    h[3] = LARGEST
    h[4] = -LARGEST
    h[5] *= 2.0 ** 63 / (d ** 0.5)                             # squares that fit, about the border of their sum
    y, scales = norm(pkl, h, gain, None, 1e-5, dtype)
    check_norm(y, scales, h, gain, 1e-5, dtype)
    for r in (0, 6):
        assert torch.equal(y[r].float(), plain[0][r].float())
    assert sync() == 0


@TYPES
@pytest.mark.parametrize("rows", [3, 700])
def test_sums_with_delta_that_overflow_when_squared(pkl, rows, dtype):
    h, delta = randn(1, rows, 516), randn(2, rows, 516)
    delta[::2] *= 2.0 ** 70
    want = h + delta
    y, scales = norm(pkl, h, None, delta, 1e-5, dtype)
    assert torch.equal(h, want)
    check_norm(y, scales, h, None, 1e-5, dtype)


@TYPES
def test_infinite_rows_are_flagged_as_before(pkl, dtype):
    h = randn(3, 3, 256)
    h[1, 7], h[1, 9] = 1e25, float("inf")
    y, _ = norm(pkl, h, None, None, 1e-5, dtype)
    assert sync() == (0 if dtype is torch.float32 else 7)
    assert torch.isfinite(y[0].float()).all() and torch.isfinite(y[2].float()).all()
    if dtype is not E4M3:
        assert y[1, 9].isnan()


@TYPES
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 2.0 ** -100, 1e20])
def test_eps_beside_rows_of_any_size(pkl, eps, dtype):
    """Rows from fp32's least numbers to its largest with an eps that counts, or does not, beside their squares."""
    d = 260
    h = torch.stack([randn(5 + i, d) * 2.0 ** e for i, e in enumerate((-135, -128, -100, -75, -70, -64, -50, -48, -45, -20, 0, 33, 60, 64, 90, 120))])
    y, scales = norm(pkl, h, None, None, eps, dtype)
    eps32 = torch.tensor(eps, dtype=torch.float32).double().item()
    x = h.double()
    ref = x / (x.square().mean(-1, keepdim=True) + eps32).sqrt()
    kept = ref.abs().amax(-1) > 2.0 ** -100                    # others give nothing but zeros in most types
    check_norm(y[kept], None if scales is None else scales[kept], h[kept], None, eps32, dtype)
    rest = y[~kept].double() * (1 if scales is None else scales[~kept].double().repeat_interleave(128, dim=1)[:, :d])
    assert (rest.abs() < 2.0 ** -99).all()
    assert sync() == 0
