"""The packed layout of 4-bit weights on the CPU: csrc/weight4.cuh against the layout as include/pic.h states it, and the banks of
shared memory that its readers meet."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def w4(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    so = str(tmp_path_factory.mktemp("w4") / "w4.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "position_independent_kv_link_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "weight4_host.cpp")], check=True)
    return C.CDLL(so)


def test_layout_as_documented(w4):
    for r in range(128):
        for q in range(4):
            assert w4.piece(r, q) == 64 * r + 16 * (q ^ (r // 2 % 4))
        assert w4.place(r) == r // 32 * 32 + r % 8 * 4 + r // 8 % 4
    for e in range(8):
        assert w4.shift(e) == 4 * (e // 2 + 4 * (e % 2))
    for g in (32, 64, 128):
        assert w4.tile_bytes(1, 32, g) == 8192 + 128 // g * 384


def test_every_code_has_a_place_of_its_own(w4):
    places = {(w4.piece(r, q) + 4 * j, w4.shift(e)) for r in range(128) for q in range(4) for j in range(4) for e in range(8)}
    assert len(places) == 128 * 128 and all(0 <= b < 8192 and b % 4 == 0 and 0 <= s <= 28 for b, s in places)
    assert sorted(w4.place(r) for r in range(128)) == list(range(128))


def test_readers_meet_every_bank_once(w4):
    """Sixteen-byte reads go by eight lanes: rows of one piece, and four pieces of two rows, lie in different 16 bytes of 128."""
    for r0 in range(0, 128, 8):
        for q in range(4):
            assert len({w4.piece(r0 + i, q) % 128 for i in range(8)}) == 8
        for r in range(r0, r0 + 8, 2):
            assert len({w4.piece(r + i, q) % 128 for i in range(2) for q in range(4)}) == 8
    # rows 8 apart: 512 bytes apart, and their scales side by side
    for r in range(128 - 8):
        assert all(w4.piece(r + 8, q) - w4.piece(r, q) == 512 for q in range(4))
    assert all(w4.place(r + 8 * i) == w4.place(r) + i for r in range(8) for i in range(4))
