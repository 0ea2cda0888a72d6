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


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows", [[1, 1, 1, 1], [1, 100, 180, 60], [300, 800, 900, 700]], ids=str)
@pytest.mark.parametrize("window", [0, 20])
def test_page_positions_that_do_not_ascend(pkl, half, rows, window):
    """Two requests' page_pos in another order: the others' rows are right, whatever these give."""
    from position_independent_kv_link_gb300 import _lib as L
    b = Batch(pkl, [m + 90 for m in rows], rows, 8, 2, 128, half, ragged=True, seed=rows[1])
    keep = b.pages.page_pos.clone()
    t = torch.tensor([0] + rows).cumsum(0).tolist()
    for turn in range(4):
        b.pages.page_pos.copy_(keep)
        for r in (1, 3):
            n = int(b.pages.n_pages[r]) - 1
            b.pages.page_pos[r, :n] = keep[r, :n].roll(turn) if turn else keep[r, :n].flip(0)
        b.out.fill_(7.0)
        out = b.window(window, 3)
        assert sync() in ((L.PIC_ERR_INVALID_ARG,) if window == 0 else (L.PIC_OK, L.PIC_ERR_INVALID_ARG))
        for r in (1, 3):
            out[t[r]:t[r + 1]] = 7.0
        b.check(out, window, 3, left=(1, 3))
