"""Page tables so wide that the plan's cost axis would pass 31 bits: items then cost one unit a tile, and only what does not
fit even so is refused (before anything is launched: tests/test_batch_wide_tables.py)."""
import pytest
import torch

from .test_gpu_batch import Batch, pkl, nothing_flagged  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("half,kv,rows,stride", [
    (True, [90, 3000], [1, 1], 70_000_000),                 # narrow: 2 blocks x 8 heads x (32 + 8 x 17.5 M)
    (True, [1100, 1300], [1100, 1100], 2_000_000),          # 70 blocks x 8 heads x 8 x 0.5 M
    (False, [1100, 1300], [1100, 1100], 1_000_000),         # 552 blocks x 8 heads x 2 x 0.25 M
], ids=["narrow", "one tile", "fp32"])
@pytest.mark.parametrize("prefix", [0, 100])
def test_wide_tables(pkl, half, kv, rows, stride, prefix):
    b = Batch(pkl, kv, rows, 32, 8, 128, half, seed=stride, prefix=prefix)
    table = torch.full((len(kv), stride), -7, dtype=torch.int32, device="cuda")
    table[:, :b.pages.block_table.shape[1]] = b.pages.block_table
    b.pages.block_table = table
    b.check(b.shared() if prefix else b.window(70, 3), *((0, 0) if prefix else (70, 3)))
