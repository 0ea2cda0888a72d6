"""Inconsistent device lengths and tables on the CPU, walked as the kernels walk their plan: the other requests' tiles
are all done, once, nothing else is, and the merge of a prefix batch looks up no prefix block that the plan lacks."""
import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest

from .test_batch_plan_host import BAD_LENGTHS, ROOT, batch


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    so = str(tmp_path_factory.mktemp("walk") / "walk.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "position_independent_kv_link_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "batch_walk_host.cpp")], check=True)
    lib = C.CDLL(so)
    i32 = lambda a: None if a is None else np.ascontiguousarray(a, dtype=np.int32)
    ptr = lambda a: None if a is None else a.ctypes.data_as(C.POINTER(C.c_int32))

    def run(b, window=2 ** 31 - 1, sinks=0, mrows=256, kpages=4, costs=(24, 8, 6), grid=152, G=2, rep=4):
        p = i32([b["T"], G, rep, b["table"].shape[1], b["pre_len"], len(b["pre_blocks"]), window, sinks, b["pool"],
                 b["rope"], mrows, kpages, *costs, grid, len(b["kv"])])
        arrs = [i32(b[k]) for k in ("row_start", "kv", "table", "page_pos", "n_pages", "pre_blocks", "pre_pos")]
        blocks, done, beyond = np.zeros((9000, 5), np.int32), np.zeros((9000, G), np.int32), np.zeros((9000, G), np.int32)
        counts = np.zeros(4, np.int32)
        assert lib.batch_walk_host(ptr(p), *[ptr(a) for a in arrs], ptr(blocks), ptr(done), ptr(beyond), len(blocks),
                                   ptr(counts)) == 0
        n = counts[0]
        return blocks[:n], done[:n], beyond[:n], counts[1:].tolist()
    return run


def check(walk, b, **kw):
    """Every block's tiles once each, and no others. Returns the blocks, the flags and the prefix blocks that are missing."""
    blocks, done, beyond, (n_pre, bad, lost) = walk(b, **kw)
    assert (beyond == 0).all()
    assert (blocks[:, 3] >= 1).all() and (blocks[:, 4] >= 1).all()
    assert (done == blocks[:, 3:4]).all()
    return blocks, bad, lost


@pytest.mark.parametrize("row_start", [[0, 64, 4], [60, 64, 0], [0, 10, 5], [0, 64, -1], [5, 64, 64], [0, 40, 64], [0, 70, 64]],
                         ids=str)
@pytest.mark.parametrize("mrows", [16, 128])
def test_rows_behind_the_last_start_are_refused(walk, row_start, mrows):
    """row_start that falls again at its end: the prefix is planned for the rows before row_start[n] alone."""
    b = batch([70, 70], [64, 0], prefix=90, seed=1)
    b["row_start"] = np.array(row_start)
    blocks, bad, lost = check(walk, b, mrows=mrows)
    assert lost == 0
    good = row_start in ([5, 64, 64], [0, 40, 64])
    assert bool(bad & BAD_LENGTHS) != good
    own = blocks[blocks[:, 0] >= 0]
    live = max(0, min(row_start[-1], b["T"]))
    assert (own[:, 1] + own[:, 2] <= live).all()
    assert bool(len(own)) == good


def test_garbage_row_starts(walk):
    for seed in range(200):
        rng = np.random.default_rng(seed)
        b = batch([100, 200, 300, 40], [5, 200, 1, 7], prefix=90, seed=seed)
        a = np.array(b["row_start"], dtype=np.int64)
        hit = rng.random(a.shape) < 0.5
        a[hit] = rng.choice([-2 ** 31, -1, 0, 1, 3, 50, 205, 213, 214, 2 ** 31 - 1], size=int(hit.sum()))
        b["row_start"] = a
        _, _, lost = check(walk, b, mrows=16)
        assert lost == 0


@pytest.mark.parametrize("window,sinks", [(20, 0), (20, 40), (2 ** 31 - 1, 0), (90, 3)])
@pytest.mark.parametrize("costs,grid", [((32, 8, 8), 152), ((17, 8, 8), 5), ((1, 2, 2), 304), ((24, 8, 6), 1)], ids=str)
def test_page_positions_that_do_not_ascend(walk, window, sinks, costs, grid):
    """Requests with page_pos in any order between good ones: each has some tiles of its own, the good ones have all of
    theirs, and what the shuffled ones list is flagged where it does not fit."""
    flagged = 0
    for seed in range(60):
        rng = np.random.default_rng(seed)
        b = batch([180, 150, 200, 90, 170], [1, 100, 180, 60, 9], ragged=True, prefix=33, seed=seed)
        good, *_ = check(walk, b, window=window, sinks=sinks, mrows=16, costs=costs, grid=grid)
        for r in (1, 3):
            n = b["n_pages"][r]
            b["page_pos"][r, :n - 1] = rng.permutation(b["page_pos"][r, :n - 1]) + rng.integers(-5, 6, n - 1)
        got, bad, _ = check(walk, b, window=window, sinks=sinks, mrows=16, costs=costs, grid=grid)
        keep = lambda x: x[~np.isin(x[:, 0], (1, 3))].tolist()
        assert keep(got) == keep(good)
        flagged += bool(bad & BAD_LENGTHS)
    if window > 200:
        assert flagged == 60               # every page is listed there


def test_pages_whose_positions_do_not_fit_are_flagged(walk):
    for i, x in ((2, 20), (2, 16), (2, 50), (3, 95)):        # of 0 16 32 48 64 80
        b = batch([96], [1], prefix=0, seed=2)
        b["page_pos"], b["n_pages"] = np.zeros_like(b["table"]), [6]
        b["page_pos"][0, :6] = 16 * np.arange(6)
        assert check(walk, b)[1] == 0
        b["page_pos"][0, i] = x
        assert check(walk, b)[1] == BAD_LENGTHS
    b = batch([5], [1], ragged=True, prefix=96, seed=2)
    b["pre_pos"], b["pre_blocks"] = np.array([0, 16, 32, 64, 80]), b["pre_blocks"][:5]
    assert check(walk, b)[1] == BAD_LENGTHS                  # positions 48 to 63 in no page
