"""Batches whose plan does not fit 31 bits whatever a tile costs, and more rows x heads than the merge counts, are refused
(C ABI, no GPU needed: nothing is launched)."""
import pytest

from position_independent_kv_link_gb300 import _lib as L

from .test_batch_refusals import A, lib, window  # noqa: F401  (fixture)

FAR = 1 << 50     # an output that does not overlap q


@pytest.mark.parametrize("dtype", [L.PIC_BF16, L.PIC_F32])
@pytest.mark.parametrize("kw", [dict(n=60000, stride=100_000), dict(n=1, T=2_000_000, stride=1_000_000), dict(T=1 << 28),
                                dict(n=2 ** 31 - 1),
                                dict(n=1, T=2 ** 31 - 1, stride=2 ** 31 - 1), dict(n=8, stride=2 ** 31 - 1)], ids=str)
def test_refused(lib, dtype, kw):
    assert window(lib, dtype=dtype, out=FAR, **kw) == L.PIC_ERR_CAPACITY
    assert b"too large" in lib.pic_last_error()
    H, G, D, n, T, stride = 8, 2, 128, kw.get("n", 1), kw.get("T", 1), kw.get("stride", 4)
    assert lib.pic_op_attention_batch_scratch_bytes(dtype, T, n, H, G, D, stride, 0, 0) == 0
