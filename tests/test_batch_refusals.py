"""Refusals of the batched calls that need no GPU: wrong devices in the binding, wrong shapes, pointers and
alignments in the C ABI (nothing is launched; the addresses are never followed)."""
import pytest
import torch

import position_independent_kv_link_gb300 as pkl
from position_independent_kv_link_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    import os

    from position_independent_kv_link_gb300 import _build
    if not os.path.exists(L.LIB_PATH):
        _build.build()
    return L.load()


A = 4096    # an aligned address that nothing reads


def window(lib, dtype=L.PIC_BF16, T=1, H=8, G=2, D=128, q=A, row_start=A, n=1, kv=A, table=A, stride=4, page_pos=None,
           n_pages=None, w=5, sinks=0, k=A, v=A, pool=4, rope=A, positions=64, out=A, scratch=A, size=1 << 40):
    return lib.pic_op_attention_window(dtype, T, H, G, D, q, row_start, n, kv, table, stride, page_pos, n_pages, w, sinks, k,
                                       v, pool, rope, positions, out, scratch, size, None)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(T=0), dict(H=7), dict(G=0), dict(D=96), dict(q=None), dict(row_start=None),
                                dict(n=0), dict(kv=None), dict(table=None), dict(stride=0), dict(page_pos=A),
                                dict(n_pages=A), dict(w=-1), dict(sinks=-1), dict(k=None), dict(v=None), dict(pool=0),
                                dict(rope=None), dict(positions=15), dict(out=None), dict(scratch=None), dict(size=100),
                                dict(q=A + 8), dict(k=A + 2), dict(out=A + 16), dict(scratch=A + 16)], ids=str)
def test_window_refuses(lib, kw):
    assert window(lib, **kw) == L.PIC_ERR_INVALID_ARG
    assert lib.pic_last_error()


def test_too_many_heads_for_a_kv_head(lib):
    assert window(lib, H=34, G=2) == L.PIC_ERR_UNSUPPORTED
    assert lib.pic_op_attention_batch_scratch_bytes(L.PIC_BF16, 1, 1, 34, 2, 128, 4, 0, 0) == 0


@pytest.mark.parametrize("kw", [dict(n_len=-1), dict(blocks=None), dict(pages=1), dict(n_len=100), dict(pages=18, pos=A),
                                dict(pages=1, pos=A)], ids=str)
def test_prefix_refuses(lib, kw):
    n_len, pages = kw.get("n_len", 17), kw.get("pages", 2)
    assert lib.pic_op_attention_prefix(L.PIC_BF16, 1, 8, 2, 128, A, A, kw.get("blocks", A), kw.get("pos"), pages, n_len, 1, A,
                                       A, 4, None, None, A, A, 4, A, 64, A, A, 1 << 40, None) == L.PIC_ERR_INVALID_ARG


@pytest.mark.parametrize("i,x", [(0, 0), (1, None), (2, None), (3, None), (4, 0), (5, A), (6, A), (8, -1), (10, -1), (11, 0),
                                 (12, None), (13, None), (14, None), (15, None), (16, None), (17, None)])
def test_block_tables_refuse(lib, i, x):
    args = [1, A, A, A, 4, None, None, A, 4, None, 0, 8, A, A, A, A, A, A, None]
    args[i] = x
    assert lib.pic_op_block_tables(*args) == L.PIC_ERR_INVALID_ARG


def test_block_tables_capacity(lib):
    assert lib.pic_op_block_tables(12289, A, A, A, 4, None, None, A, 4, None, 0, 8, A, A, A, A, A, A, None) == L.PIC_ERR_CAPACITY
    assert lib.pic_op_block_tables(1, A, A, A, 1 << 26, None, None, A, 4, None, 0, 8, A, A, A, A, A, A, None) == L.PIC_ERR_CAPACITY


@pytest.mark.parametrize("i,x", [(0, 5), (1, 0), (2, 0), (3, 0), (4, 32), (5, None), (5, A + 4), (6, 100), (6, 1538), (7, A + 4),
                                 (9, -1.0), (9, float("nan")), (10, None), (11, None), (12, None), (13, 0), (14, None),
                                 (15, None), (16, None), (17, 0)])
def test_qk_norm_rope_refuses(lib, i, x):
    args = [L.PIC_BF16, 1, 8, 2, 128, A, 1536, None, None, 1e-5, A, A, A, 64, A, A, A, 4, None]
    args[i] = x
    assert lib.pic_op_qk_norm_rope(*args) == L.PIC_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(1, 8, 128, dtype=torch.float16)
    k = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    rope = torch.zeros(16, 64, 2)
    with pytest.raises(ValueError, match="device"):
        pkl.attention_window(x, i, pkl.BatchPages(i[:1], i[None]), k, k, rope, 4)
    with pytest.raises(ValueError, match="device"):
        pkl.block_tables(i, i, i[None], i, 4)
    with pytest.raises(ValueError, match="device"):
        pkl.qk_norm_rope(torch.zeros(1, 1536), 8, 2, i[:1], i[:1], rope, k, k)
