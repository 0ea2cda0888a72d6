"""What the batched attention over bf16 pools loses besides rounding its fp16 result: every form (narrow, one MMA tile,
two MMA tiles) holds the softmax weights to 16 bits or more.

Queries are small, so that scores are near 0, errors of scores count for little, and a handful of keys of about equal
weight make each result: rounding the weights to 11 bits would be off by up to 2^-11 of sum p |v|, twenty times what is allowed here.

Each element of the result is within half a step of fp16 (2^-11 relative, 2^-25 below its normal range) of a number that is
within E of the formula:
  E = (2 es + 2^-16 + 2^-20 + (N + 40) 2^-24) sum_u p_u |v_u|
  es  a score's error: rotated K in two fp16 numbers (2^-22 of each term, 2^-25 |q| below fp16's normal range) and the fp32
      sum of 2 D terms; a weight's relative error is at most twice that (its own, and through the denominator)
  2^-16  weights in two bf16 numbers (each half a step of 2^-8), 2^-20 the exponential (2 units of 2^-22, numerator and denominator)
  (N + 40) 2^-24  fp32 sums over N keys, normalizations and the join of a prefix with own pages.
"""
import numpy as np
import pytest
import torch

from .test_gpu_batch import Batch, pkl, nothing_flagged, rotated  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def hold(b, out, window=0, sinks=0):
    t0, rep, D = 0, b.H // b.G, b.D
    for r, (kv, m) in enumerate(zip(b.kv, b.rows)):
        N = b.prefix + kv
        blk, row = (torch.cat(x) for x in zip(b.pre_place, b.places[r]))
        u = torch.arange(N, device="cuda")
        K, V = rotated(b.k[blk, :, row].double(), u, b.rope), b.v[blk, :, row].double()
        p = torch.arange(N - m, N, device="cuda")
        seen = u[None] <= p[:, None]
        if window:
            seen &= (u[None] > p[:, None] - window) | (u[None] < sinks)
        Q = b.q[t0:t0 + m].double().view(m, b.G, rep, D)
        x = torch.einsum("tgrd,kgd->grtk", Q, K) / D ** 0.5
        w = torch.softmax(x.masked_fill(~seen, float("-inf")), -1)
        ref = torch.einsum("grtk,kgd->tgrd", w, V).reshape(m, b.H, D)
        size = torch.einsum("grtk,kgd->tgrd", w, V.abs()).reshape(m, b.H, D)
        A = (torch.einsum("tgrd,kgd->grtk", Q.abs(), K.abs()) / D ** 0.5).amax().item()
        qsum = (Q.abs().sum(-1).amax() / D ** 0.5).item()
        es = ((2 * D + 8) * 2.0 ** -24 + 2.0 ** -22) * A + 2.0 ** -25 * qsum
        tol = (2 * es + 2.0 ** -16 + 2.0 ** -20 + (N + 40) * 2.0 ** -24) * size
        tol += 2.0 ** -11 * (ref.abs() + tol) + 2.0 ** -25
        off = (out[t0:t0 + m].double() - ref).abs()
        assert (off <= tol).all(), (r, (off / tol).max().item(), (off > tol).float().mean().item())
        t0 += m


@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (8, 2, 64), (16, 1, 128), (6, 2, 128)])
@pytest.mark.parametrize("kv,rows,window,sinks", [
    ([9, 1, 40], [1, 1, 1], 12, 1),                 # narrow
    ([60, 35], [60, 35], 10, 2),                    # one MMA tile
    ([800, 790], [800, 780], 6, 1),                 # two, K rotated ahead
    ([1100], [1100], 20, 0),
])
def test_window_weights(pkl, H, G, D, kv, rows, window, sinks):
    b = Batch(pkl, kv, rows, H, G, D, True, seed=sum(rows), scale=0.02)
    hold(b, b.window(window, sinks), window, sinks)


@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (8, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("kv,rows,prefix", [
    ([3, 1], [1, 1], 20),                           # narrow
    ([6] * 60, [1] * 60, 9),                        # one MMA tile
    ([5] * 600, [1] * 600, 11),                     # two for the prefix, narrow for the own pages
    ([20] * 30, [20] * 30, 17),                     # or one tile
    ([30] * 20, [30] * 20, 700),                    # both in one plan
])
def test_prefix_weights(pkl, H, G, D, kv, rows, prefix):
    b = Batch(pkl, kv, rows, H, G, D, True, seed=sum(rows) + prefix, prefix=prefix, scale=0.02)
    hold(b, b.shared())


@pytest.mark.parametrize("H,G,D", [(8, 2, 128), (8, 8, 128), (8, 4, 64)])
@pytest.mark.parametrize("kv,rows,window,sinks,ragged", [
    ([2500, 2300, 0], [2500, 2300, 0], 0, 0, False),
    ([2600, 3000], [2049, 2900], 700, 70, True),    # windows and sinks that end inside pages, holes between them
    ([2400, 2100], [2400, 2050], 33, 1, True),
])
def test_many_rows(pkl, H, G, D, kv, rows, window, sinks, ragged):
    """Masks, ragged pages and requests without rows where every KV head's keys meet thousands of rows."""
    kv, rows = (kv, rows) if H > G else ([kv[0]], [rows[0]])
    b = Batch(pkl, kv, rows, H, G, D, True, ragged=ragged, seed=sum(rows) + window, spare_rows=2)
    b.check(b.window(window, sinks), window, sinks)
    again = b.out.clone()
    b.out.fill_(7.0)
    assert torch.equal(b.window(window, sinks), again)


@pytest.mark.parametrize("kv,rows,prefix,ragged", [
    ([700, 90, 0, 80], [700, 90, 0, 33], 1500, True),       # own pages with the prefix
    ([3] * 900, [1] * 900, 2000, True),                     # apart
])
def test_many_rows_behind_a_prefix(pkl, kv, rows, prefix, ragged):
    b = Batch(pkl, kv, rows, 8, 2, 128, True, ragged=ragged, prefix=prefix, seed=sum(rows), spare_rows=5)
    b.check(b.shared())
