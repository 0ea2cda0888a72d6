"""Captures that nothing has warmed up, two captured graphs over one scratch, and rows before the first request's."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from .test_gpu_batch import Batch, i32, pkl, nothing_flagged  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

FIRST = """
import torch
from tests.test_gpu_batch import Batch, i32, rope_table
import position_independent_kv_link_gb300 as pkl
half = %r
b = Batch(pkl, [40, 3000, 900], %r, 8, 2, 128, half, seed=6, prefix=%d)
if not b.prefix:
    kv, new, table, free = i32([16, 30]), i32([1, 17]), i32([[4, -1, -1], [5, 6, -1]]), i32([9, 8])
    x, pos, slot, rope = torch.randn(2, 3 * 64, device="cuda"), i32([0, 1]), i32([3, 4]), rope_table(16, 64)
    k = torch.zeros(4, 1, 16, 64, dtype=b.pool_t, device="cuda")
    v = torch.zeros_like(k)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    if b.prefix:
        b.shared()
    else:
        b.window(70, 3)
        r = pkl.block_tables(kv, new, table, free, 20)
        q = pkl.qk_norm_rope(x, 1, 1, pos, slot, rope, k, v)
graph.replay()
pkl.sync()
b.check(b.out, *((0, 0) if b.prefix else (70, 3)))
if not b.prefix:
    assert r.counts.tolist() == [18, 2, 0] and torch.equal(v[0, 0, 3:5], x[:, 128:].to(v.dtype))
print("captured")
"""


@pytest.mark.parametrize("half,rows,prefix", [(True, [1, 1, 1], 0), (True, [20, 2900, 800], 300), (True, [20, 100, 30], 300),
                                              (False, [1, 20, 1], 0), (False, [1, 1, 1], 100)], ids=str)
def test_first_calls_of_a_process_captured(pkl, half, rows, prefix):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % (half, rows, prefix)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_graphs_over_one_scratch(pkl):
    """Two captured calls of other shapes with one scratch and one out each, replayed in turn."""
    a = Batch(pkl, [900] * 9, [1] * 9, 8, 2, 128, True, seed=7)
    b = Batch(pkl, [2333] * 2, [2000] * 2, 8, 2, 128, True, seed=8, prefix=3000)
    scratch = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    a.window(200, 4, scratch=scratch)
    b.shared(scratch=scratch)
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: a.window(200, 4, scratch=scratch), lambda: b.shared(scratch=scratch)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(3):
        for x in (a, b):
            x.out.fill_(7.0)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        a.check(a.out, 200, 4)
        b.check(b.out)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rows", [[1, 1, 30], [700, 5, 800]], ids=str)
@pytest.mark.parametrize("prefix", [0, 500])
def test_rows_before_the_first_request(pkl, half, rows, prefix):
    """row_start[0] > 0: the rows before it belong to no request and stay as they were."""
    skip = 37
    b = Batch(pkl, [m + 11 for m in rows], rows, 8, 2, 128, half, seed=rows[0], prefix=prefix, ragged=True, spare_rows=skip)
    want = (b.shared() if prefix else b.window(60, 2)).clone()
    n = sum(rows)
    b.check(want, *((0, 0) if prefix else (60, 2)))
    q = b.q
    b.q = torch.cat([q[n:], q[:n]])
    b.row_start.copy_(i32(skip + np.concatenate([[0], np.cumsum(rows)])))
    b.out.fill_(7.0)
    out = b.shared() if prefix else b.window(60, 2)
    assert (out[:skip] == 7.0).all()
    b.q = q                                        # as check() counts the rows
    b.check(torch.cat([out[skip:], out[:skip]]), *((0, 0) if prefix else (60, 2)))
