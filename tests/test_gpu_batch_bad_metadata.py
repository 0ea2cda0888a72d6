"""Lengths and tables that only the device sees and that do not fit together (tests/test_batch_walk_host.py shows on the
CPU that they lead nowhere): what they concern is skipped and reported once, the other requests' rows are right."""
import pytest
import torch

from .test_gpu_batch import Batch, i32, pkl, nothing_flagged, sync  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows", [[3, 2, 1], [30, 20, 10], [700, 90, 80]], ids=str)
@pytest.mark.parametrize("prefix", [0, 300])
def test_rows_behind_the_last_start(pkl, half, rows, prefix):
    """row_start that falls at its end: the first request stays, the second one's rows lie behind row_start[n]."""
    from position_independent_kv_link_gb300 import _lib as L
    b = Batch(pkl, [m + 20 for m in rows], rows, 8, 2, 128, half, prefix=prefix, seed=rows[0])
    run = b.shared if prefix else lambda: b.window(25, 3)
    window = (0, 0) if prefix else (25, 3)
    for bad in ([0, rows[0], rows[0] + rows[1], rows[0] + 1], [0, rows[0], rows[0] + rows[1], rows[0]]):
        b.row_start.copy_(i32(bad))
        b.out.fill_(7.0)
        out = run()
        assert sync() == L.PIC_ERR_INVALID_ARG and sync() == 0
        b.check(out, *window, left=(1, 2))
    for bad in ([0, rows[0], sum(rows), 0], [0, rows[0], 5, -1]):
        b.row_start.copy_(i32(bad))
        b.out.fill_(7.0)
        run()
        assert sync() == L.PIC_ERR_INVALID_ARG
        assert (b.out == 7.0).all()
