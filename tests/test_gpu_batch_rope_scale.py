"""RoPE tables whose rows carry a factor (an attention factor of 1.25, one per pair of dims) or begin at another position:
every form of the batched attention turns a key by its own row of the table, once."""
import numpy as np
import pytest
import torch

from .test_gpu_batch import Batch, pkl, nothing_flagged  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

TABLES = ["factor", "per pair", "shifted"]


def table(b, kind):
    n, h = b.rope.shape[0], b.D // 2
    if kind == "shifted":
        a = (np.arange(n)[:, None] + 37) * 10000.0 ** (-np.arange(h) / h)
        return torch.tensor(np.stack([np.cos(a), np.sin(a)], -1), dtype=torch.float32).cuda()
    s = torch.full((h, 1), 1.25) if kind == "factor" else 0.5 + torch.rand(h, 1, generator=torch.Generator().manual_seed(1))
    return (b.rope.double() * s.double().cuda()).float().contiguous()


@pytest.mark.parametrize("kind", TABLES)
@pytest.mark.parametrize("half,H,G,D", [(True, 8, 2, 128), (True, 8, 2, 64), (True, 16, 1, 128), (False, 8, 2, 128)])
@pytest.mark.parametrize("kv,rows", [([90, 1, 40], [1, 1, 1]), ([60, 135], [60, 35]), ([800, 790], [800, 780])], ids=str)
def test_window(pkl, kind, half, H, G, D, kv, rows):
    b = Batch(pkl, kv, rows, H, G, D, half, ragged=True, seed=sum(rows))
    b.rope = table(b, kind)
    b.check(b.window(50, 3), 50, 3)


@pytest.mark.parametrize("kind", TABLES)
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("kv,rows", [([3, 1], [1, 1]), ([6] * 60, [1] * 60), ([30] * 20, [30] * 20)],
                         ids=["few", "60 single", "20 of 30"])
def test_prefix(pkl, kind, half, kv, rows):
    b = Batch(pkl, kv, rows, 8, 2, 128, half, seed=sum(rows), prefix=700)
    b.rope = table(b, kind)
    b.check(b.shared())
