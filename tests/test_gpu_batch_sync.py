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


COPIES = """
import torch
from torch.profiler import ProfilerActivity, profile
import position_independent_kv_link_gb300 as pkl

def copies():
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        pkl.sync()
        torch.cuda.synchronize()
    return sum(e.count for e in p.key_averages() if "Memcpy DtoH" in e.key)

torch.zeros(1, device="cuda")
copies()
before = copies()
i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
pkl.block_tables(i(3), i(1), i(7).view(1, 1), i(8), 2)
print("copies", before, copies())
"""


def test_programs_without_batched_calls_read_no_flag_of_theirs(pkl):
    """pic_sync reads three words of the store's kernels, and a fourth only once a batched call has been made."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", COPIES], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "copies 3 4" in r.stdout, r.stdout
