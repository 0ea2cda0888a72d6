"""sync(): what the batched calls met on the device reaches a program that has no store."""
import pytest
import torch

import position_independent_kv_link_gb300 as pkg

from .test_gpu_batch import Batch, i32, pkl, nothing_flagged  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def raised(stream=None):
    with pytest.raises(pkg.PicError) as e:
        pkg.sync(stream)
    pkg.sync(stream)                                   # once
    return e.value


def test_what_the_calls_met_is_raised(pkl):
    from position_independent_kv_link_gb300 import _lib as L
    assert "sync" in pkl.__all__
    pkl.sync()
    b = Batch(pkl, [100, 90, 80], [1, 1, 1], 8, 2, 128, True, seed=9)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.window(0, 0, stream=s)
    pkl.sync(s)
    b.check(b.out)
    b.pages.kv_len[1] = 10 ** 6
    torch.cuda.synchronize()
    b.window(0, 0, stream=s)
    e = raised(s)
    assert e.status == L.PIC_ERR_INVALID_ARG and "lengths" in str(e)
    pkl.block_tables(i32([16, 30]), i32([1, 17]), i32([[4, -1, -1], [5, 6, -1]]), i32([9]), 20)
    assert raised().status == L.PIC_ERR_OUT_OF_BLOCKS
    pkl.block_tables(i32([16, 30]), i32([1, 17]), i32([[4, -1, -1], [5, 6, -1]]), i32([9, 8]), 17)
    assert raised().status == L.PIC_ERR_CAPACITY
    k = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.full((1, 192), 5e4, device="cuda")
    rope = torch.tensor([1.0, 0.0], device="cuda").expand(16, 32, 2).contiguous()
    pkl.qk_norm_rope(x, 1, 1, i32([0]), i32([0]), rope, k, k.clone())
    assert raised().status == L.PIC_ERR_RANGE
