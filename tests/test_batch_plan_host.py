"""The batched attention's work plan, on the CPU: the scalar functions of csrc/batch_plan.h (which
the kernels evaluate on the GPU from device lengths) compiled for the host and checked against the
definition. Every tile of every item belongs to exactly one CTA, parts have slots of their own,
a block's pages hold every key its rows see and none is listed twice, and inconsistent lengths,
blocks and positions are skipped and flagged."""
import ctypes as C
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PAGE = 16
BAD_LENGTHS, BAD_BLOCK, BAD_POSITION = 1, 2, 4


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "position_independent_kv_link_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "batch_plan_host.cpp")], check=True)
    lib = C.CDLL(so)
    i32 = lambda a: None if a is None else np.ascontiguousarray(a, dtype=np.int32)
    ptr = lambda a: None if a is None else a.ctypes.data_as(C.POINTER(C.c_int32))

    def run(b, window=2 ** 31 - 1, sinks=0, mrows=256, kpages=8, costs=(4, 8, 5), grid=152, G=2, rep=4):
        p = i32([b["T"], G, rep, b["table"].shape[1], b["pre_len"], len(b["pre_blocks"]), window, sinks, b["pool"],
                 b["rope"], mrows, kpages, *costs, grid, len(b["kv"])])
        arrs = [i32(b[k]) for k in ("row_start", "kv", "table", "page_pos", "n_pages", "pre_blocks", "pre_pos")]
        items, pages = np.zeros((200000, 12), np.int32), np.zeros((400000, 5), np.int32)
        counts = np.zeros(5, np.int32)
        assert lib.batch_plan_host(ptr(p), *[ptr(a) for a in arrs], ptr(items), len(items), ptr(pages), len(pages),
                                   ptr(counts)) == 0
        assert counts[4] == 0          # owner() agrees with the shares
        return items[:counts[0]], pages[:counts[1]], counts[2], counts[3]
    return run


def positions(start, mask):
    return start + np.array([i for i in range(PAGE) if mask >> i & 1], dtype=int)


def page_lengths(total, ragged, rng):
    out = []
    while total > 0:
        chunk = min(total, int(rng.integers(1, 100))) if ragged else total
        out += [PAGE] * (chunk // PAGE) + ([chunk % PAGE] if chunk % PAGE else [])
        total -= chunk
    return out


def batch(kv, rows, ragged=False, prefix=0, seed=0, spare=3):
    rng = np.random.default_rng(seed)
    pages = [page_lengths(k, ragged, rng) for k in kv]
    pre = page_lengths(prefix, ragged, rng)
    stride = max(1, max((len(p) for p in pages), default=0)) + spare
    pool = sum(map(len, pages)) + len(pre) + 2
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((len(kv), stride), -7, np.int32)
    pos = np.full((len(kv), stride), -9, np.int32)
    at = 0
    for r, p in enumerate(pages):
        table[r, :len(p)] = ids[at:at + len(p)]
        pos[r, :len(p)] = prefix + np.concatenate([[0], np.cumsum(p)[:-1]]) if p else 0
        at += len(p)
    return dict(T=sum(rows), kv=kv, rows=rows, row_start=np.concatenate([[0], np.cumsum(rows)]), table=table,
                page_pos=pos if ragged else None, n_pages=[len(p) for p in pages] if ragged else None,
                pre_blocks=ids[at:at + len(pre)], pre_len=prefix,
                pre_pos=np.concatenate([[0], np.cumsum(pre)[:-1]]) if ragged and pre else None, pool=pool,
                rope=prefix + max(list(kv) + [1]) + 16)


CASES = [
    (batch([1], [1]), {}),
    (batch([50240], [1]), dict(window=1024, sinks=4)),
    (batch([17, 0, 5, 300], [1, 0, 5, 17]), dict(window=16, sinks=1)),
    (batch([4096, 4096], [4096, 4096]), dict(window=1000, sinks=70)),
    (batch([900, 33, 1, 640], [90, 1, 1, 64], ragged=True, seed=1), dict(window=100, sinks=4)),
    (batch([900, 33, 1, 640], [90, 33, 1, 64], ragged=True, seed=2), dict(window=33, sinks=40, mrows=16, kpages=4)),
    (batch([300] * 40, [1] * 40, prefix=5000, seed=3), {}),
    (batch([31, 40, 1], [31, 2, 1], ragged=True, prefix=777, seed=4), dict(grid=7)),
    (batch([9, 9], [9, 1], prefix=3, seed=5), dict(grid=1000)),
    (batch([64] * 700, [1] * 700, seed=6), dict(rep=3, G=1)),
    (batch([2000, 1, 2000], [2000, 1, 1], seed=7), dict(rep=16, costs=(0, 1, 1), grid=13)),
    (batch([0, 0], [0, 0]), {}),
    (batch([20] * 400, [9] * 400, prefix=9000, seed=9), dict(kpages=4, costs=(28, 8, 6))),       # many items, some of them long
    (batch([90] * 900, [1] * 900, ragged=True, seed=10), dict(mrows=16, kpages=4, costs=(32, 8, 8), window=50, sinks=3)),   # none long
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_plan_covers_the_work_once(plan, i):
    b, kw = CASES[i]
    G, rep, window, sinks = kw.get("G", 2), kw.get("rep", 4), kw.get("window", 2 ** 31 - 1), kw.get("sinks", 0)
    rb = kw.get("mrows", 256) // rep
    items, pages, n_blocks, bad = plan(b, **kw)
    assert bad == 0
    blocks = {}
    slots = set()
    for cta, req, row0, nrows, pos0, g, j0, j1, nt, slot, blk, sp in items.tolist():
        assert 0 <= j0 < j1 <= nt and nrows <= rb
        e = blocks.setdefault(blk, dict(req=req, row0=row0, nrows=nrows, pos0=pos0, nt=nt, tiles={}))
        seen = e["tiles"].setdefault(g, np.zeros(nt, int))
        seen[j0:j1] += 1
        assert (slot >= 0) == (j1 - j0 < nt)
        if slot >= 0:
            assert slot not in slots and slot // 2 == cta
            slots.add(slot)
    assert len(blocks) == n_blocks
    rows_own, rows_pre = np.zeros(b["T"], int), np.zeros(b["T"], int)
    for blk, e in blocks.items():
        assert sorted(e["tiles"]) == list(range(G)) and all((t == 1).all() for t in e["tiles"].values())
        (rows_pre if e["req"] < 0 else rows_own)[e["row0"]:e["row0"] + e["nrows"]] += 1
        pg = pages[pages[:, 0] == blk]
        assert -(-len(pg) // kw.get("kpages", 8)) == e["nt"]
        assert len(set(pg[:, 2].tolist())) == len(pg)                # no page twice
        have = np.concatenate([positions(p, m) for _, _, _, p, m in pg.tolist()])
        assert len(set(have.tolist())) == len(have)
        if e["req"] < 0:
            assert np.array_equal(np.sort(have), np.arange(b["pre_len"]))
            continue
        r, first = e["req"], b["pre_len"]
        i0 = e["row0"] - b["row_start"][r]
        assert e["pos0"] == first + b["kv"][r] - b["rows"][r] + i0
        qp = e["pos0"] + np.arange(e["nrows"])[:, None]
        u = np.arange(first, first + b["kv"][r])[None]
        need = u[0, ((u <= qp) & ((u > qp - window) | (u < sinks))).any(0)]
        assert np.array_equal(np.sort(have), need)                   # no key that nobody sees
        assert (pg[:, 4] != 0).all()                                 # and no page without one
    assert (rows_own == 1).all() and (rows_pre == (1 if b["pre_len"] else 0)).all()


def test_inconsistent_lengths_skip_the_request(plan):
    def change(**kw):
        b = batch([40, 50, 60], [2, 3, 4], ragged=kw.pop("ragged", False), seed=8)
        for k, (i, x) in kw.items():
            b[k] = np.array(b[k])
            b[k][i] = x
        return b
    for b, lost in ((change(kv=(1, 2)), {1}), (change(kv=(1, -5)), {1}), (change(kv=(2, 10 ** 9)), {2}),
                    (change(row_start=(1, -3)), {0, 1}), (change(row_start=(3, 1000)), {2}),
                    (change(row_start=(1, 9)), {1}),
                    (change(n_pages=(0, 0), ragged=True), {0}), (change(n_pages=(0, 99), ragged=True), {0}),
                    (change(page_pos=((1, slice(None)), 49), ragged=True), set())):
        items, _, _, bad = plan(b)
        got = set(items[:, 1].tolist())
        if lost:
            assert bad & BAD_LENGTHS and not got & lost, (bad, got, lost)
        rows = items[:, 2:4]
        assert (rows[:, 0] >= 0).all() and (rows.sum(1) <= b["T"]).all()


def test_bad_blocks_and_positions_are_empty_pages(plan):
    b = batch([40, 50], [1, 1], ragged=True, seed=9)
    b["table"][0, 0], b["table"][1, 1] = 10 ** 6, -1
    b["page_pos"][1, 0] = -4
    _, pages, _, bad = plan(b)
    assert bad == BAD_BLOCK | BAD_POSITION
    assert (pages[:, 2] >= 0).all() and (pages[:, 2] < b["pool"]).all()
    assert all(0 <= p and (m == 0 or positions(p, m).max() < b["rope"]) for p, m in pages[:, 3:].tolist())
    assert (pages[:, 4] == 0).sum() == 3


def test_garbage_tables_stay_in_bounds(plan):
    """Random positions, blocks and lengths: everything that would be read lies in the arrays."""
    for seed in range(30):
        rng = np.random.default_rng(seed)
        b = batch([100, 200, 300, 40], [5, 200, 1, 7], ragged=True, prefix=90, seed=seed)
        for k in ("page_pos", "table", "n_pages", "kv", "row_start", "pre_pos", "pre_blocks"):
            a = np.array(b[k], dtype=np.int64)
            hit = rng.random(a.shape) < 0.2
            a[hit] = rng.choice([-2 ** 31, -1, 0, 1, 3, 50, 10 ** 6, 2 ** 31 - 1, 2 ** 31 - 20], size=int(hit.sum()))
            b[k] = a
        items, pages, _, _ = plan(b, window=50, sinks=4, mrows=16, kpages=4)
        assert (pages[:, 2] >= 0).all() and (pages[:, 2] < b["pool"]).all()
        assert all(0 <= m < 1 << 16 and 0 <= p and (m == 0 or positions(p, m).max() < b["rope"])
                   for p, m in pages[:, 3:].tolist())
        assert (items[:, 2] >= 0).all() and (items[:, 2] + items[:, 3] <= b["T"]).all()
