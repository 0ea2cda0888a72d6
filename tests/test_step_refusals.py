"""Refusals of the decode-step calls that need no GPU: wrong shapes, pointers, alignments and overlaps in the C ABI (nothing is
launched; the addresses are never followed), wrong devices, types and shapes in the binding."""
import os

import pytest
import torch

import position_independent_kv_link_gb300 as pkl
from position_independent_kv_link_gb300 import _lib as L


@pytest.fixture(scope="module")
def lib():
    from position_independent_kv_link_gb300 import _build
    if not os.path.exists(L.LIB_PATH):
        _build.build()
    return L.load()


A, B, C, D, E = (4096 + (i << 32) for i in range(5))     # aligned addresses far apart that nothing reads
INVALID = L.PIC_ERR_INVALID_ARG


def refused(lib, f, args, i, x, status=INVALID):
    args = list(args)
    args[i] = x
    assert getattr(lib, f)(*args) == status, (f, i, x)
    assert lib.pic_last_error()


def test_weight4_bytes(lib):
    assert lib.pic_op_weight4_bytes(128, 128, 128) == 8192 + 384
    assert lib.pic_op_weight4_bytes(129, 160, 64) == 4 * (8192 + 768)
    assert lib.pic_op_weight4_bytes(1, 32, 32) == 8192 + 1536
    for n, k, g in ((0, 128, 128), (128, 0, 128), (128, 100, 128), (128, 16, 32), (128, 128, 96), (128, 128, 0),
                    (-1, 128, 128), (128, 128, 256), (2 ** 31 - 1, 128, 128), (2 ** 30, 2 ** 30, 128)):
        assert lib.pic_op_weight4_bytes(n, k, g) == 0


@pytest.mark.parametrize("i,x", [(0, L.PIC_E4M3), (0, 9), (1, None), (1, A + 8), (2, None), (2, B + 64), (2, A + 128), (3, 0),
                                 (4, 48), (4, 0), (5, 100)])
def test_pack_weight4_refuses(lib, i, x):
    refused(lib, "pic_op_pack_weight4", (L.PIC_BF16, A, B, 200, 256, 128, None), i, x)


@pytest.mark.parametrize("i,x", [(0, None), (0, A + 4), (1, None), (1, B + 1), (3, None), (3, C + 16), (3, A), (3, B), (3, D),
                                 (4, 0), (5, 40), (6, 31)])
def test_pack_codes4_refuses(lib, i, x):
    refused(lib, "pic_op_pack_codes4", (A, B, D, C, 200, 256, 128, None), i, x)


@pytest.mark.parametrize("i,x", [(0, None), (0, A + 16), (1, None), (1, B + 16), (1, A), (2, -1), (3, 33), (4, 129)])
def test_unpack_weight4_refuses(lib, i, x):
    refused(lib, "pic_op_unpack_weight4", (A, B, 200, 256, 128, None), i, x)


@pytest.mark.parametrize("i,x", [(0, L.PIC_F32), (0, L.PIC_BF16), (0, L.PIC_E4M3), (1, None), (1, A + 64), (2, None), (2, B + 8),
                                 (3, 255), (3, 260), (3, 1 << 38), (3, -256), (4, D), (5, None), (5, C + 4), (5, A), (5, B), (6, 0),
                                 (7, 250), (8, 0), (8, -3), (9, 16)])
def test_gemm_w4_refuses(lib, i, x):
    refused(lib, "pic_op_gemm_w4", (L.PIC_F16, A, B, 256, None, C, 200, 256, 5, 128, None), i, x)


def test_gemm_w4_refuses_8_bit_rows(lib):
    args = (L.PIC_E4M3, A, B, 256, D, C, 200, 256, 5, 128, None)
    for i, x in ((4, None), (4, D + 2), (4, C), (3, 264), (0, L.PIC_F16)):
        refused(lib, "pic_op_gemm_w4", args, i, x)
    refused(lib, "pic_op_gemm_w4", args, 8, (1 << 20) + 1, L.PIC_ERR_CAPACITY)


@pytest.mark.parametrize("i,x", [(0, L.PIC_BF16), (0, L.PIC_E4M3), (1, 0), (2, 0), (2, 130), (3, None), (3, A + 8), (3, B), (3, C),
                                 (4, 124), (4, 130), (4, 1 << 38), (5, B + 4), (5, C), (6, 124), (6, 129), (7, D + 4), (7, C), (7, A), (8, -1.0),
                                 (8, float("nan")), (9, None), (9, C + 8), (10, E)])
def test_add_rms_norm_refuses(lib, i, x):
    refused(lib, "pic_op_add_rms_norm", (L.PIC_F16, 3, 128, A, 128, B, 128, D, 1e-5, C, None, None), i, x)


def test_add_rms_norm_refuses_scales_and_wide_rows(lib):
    args = (L.PIC_E4M3, 3, 128, A, 128, None, 0, None, 1e-5, C, E, None)
    for i, x in ((10, None), (10, E + 4), (10, A), (10, C), (0, L.PIC_F32)):
        refused(lib, "pic_op_add_rms_norm", args, i, x)
    wide = (L.PIC_F16, 3, 32772, A, 32772, None, 0, None, 1e-5, C, None, None)
    assert lib.pic_op_add_rms_norm(*wide) == L.PIC_ERR_UNSUPPORTED


@pytest.mark.parametrize("i,x", [(0, L.PIC_E4M3), (0, 7), (1, 0), (2, 0), (2, 4), (3, None), (3, A + 2), (4, 99), (4, 1 << 38), (5, None),
                                 (5, B + 2), (6, -1), (6, 33), (6, 0), (7, None), (7, A), (7, B), (8, A + 396), (8, C), (9, None),
                                 (9, D), (10, None), (10, E + 2)])
def test_token_logprobs_refuses(lib, i, x):
    refused(lib, "pic_op_token_logprobs", (L.PIC_F32, 3, 100, A, 100, B, 5, C, D, E, E + 4096, None), i, x)


def test_token_logprobs_refuses_nothing_to_do(lib):
    assert lib.pic_op_token_logprobs(L.PIC_F32, 3, 100, A, 100, None, 0, None, None, None, None, None) == INVALID
    assert lib.pic_op_token_logprobs(L.PIC_F32, 2 ** 30, 1, A, 1, None, 0, None, 1 << 50, None, None, None) == L.PIC_ERR_CAPACITY


def test_binding_refuses_host_tensors_and_sizes():
    w = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (lambda: pkl.pack_weight4(w), lambda: pkl.pack_codes4(w.byte(), w.half()), lambda: pkl.add_rms_norm(w.float()),
              lambda: pkl.token_logprobs(w), lambda: pkl.gemm_w4(pkl.Weight4(w, 4, 64, 64), w.half()),
              lambda: pkl.unpack_weight4(pkl.Weight4(w, 4, 64, 64))):
        with pytest.raises(ValueError, match="device"):
            f()


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on device 0."""

    def get_device(self):
        return 0


def d(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def calls(monkeypatch):
    from position_independent_kv_link_gb300 import api
    made = []
    monkeypatch.setattr(api, "_call", lambda idx, stream, f, *args: made.append(args))
    return made


def test_binding_refuses_shapes_and_types(lib, calls):
    w = pkl.Weight4(d(lib.pic_op_weight4_bytes(200, 256, 128), dtype=torch.uint8), 200, 256, 128)
    x, half = d(5, 256), torch.float16
    bad = [lambda: pkl.pack_weight4(d(4, 64, dtype=torch.float64)), lambda: pkl.pack_weight4(d(4, 64).t()),
           lambda: pkl.pack_weight4(d(4, 60)), lambda: pkl.pack_weight4(d(4, 64), group=48), lambda: pkl.pack_weight4(d(64)),
           lambda: pkl.pack_codes4(d(4, 64, dtype=torch.uint8), d(4, 2, dtype=half)),
           lambda: pkl.pack_codes4(d(4, 64, dtype=torch.uint8), d(4, 1)),
           lambda: pkl.pack_codes4(d(4, 64, dtype=torch.uint8), d(4, 1, dtype=half), d(4, 1)),
           lambda: pkl.gemm_w4(w, x), lambda: pkl.gemm_w4(w, d(5, 128, dtype=half)), lambda: pkl.gemm_w4(w, x.half(), d(5, 2)),
           lambda: pkl.gemm_w4(w, x.to(torch.float8_e4m3fn)), lambda: pkl.gemm_w4(w, x.to(torch.float8_e4m3fn), d(5, 3)),
           lambda: pkl.gemm_w4(w, x.half(), out=d(5, 201)), lambda: pkl.gemm_w4(pkl.Weight4(w.data, 200, 256, 64), x.half()),
           lambda: pkl.gemm_w4(w, d(256, 5, dtype=half).t()),
           lambda: pkl.add_rms_norm(d(5, 256, dtype=half)), lambda: pkl.add_rms_norm(x, d(255)), lambda: pkl.add_rms_norm(x, None, d(4, 256)),
           lambda: pkl.add_rms_norm(x, None, d(5, 252)), lambda: pkl.add_rms_norm(x, dtype=torch.int8), lambda: pkl.add_rms_norm(x, dtype=torch.bfloat16, out=d(5, 256, dtype=torch.bfloat16)),
           lambda: pkl.add_rms_norm(x, scales=d(5, 2)), lambda: pkl.add_rms_norm(x, dtype=torch.float8_e4m3fn, scales=d(5, 3)),
           lambda: pkl.add_rms_norm(x.t()), lambda: pkl.add_rms_norm(d(256)),
           lambda: pkl.token_logprobs(x, d(5)), lambda: pkl.token_logprobs(x, d(4, dtype=torch.int32)), lambda: pkl.token_logprobs(x, top=33),
           lambda: pkl.token_logprobs(d(5, 7), top=8), lambda: pkl.token_logprobs(x, top=-1), lambda: pkl.token_logprobs(d(5, 7, dtype=torch.int32)),
           lambda: pkl.token_logprobs(x, top=2, out=pkl.TokenLogprobs(None, d(5), d(5, 3, dtype=torch.int32), d(5, 3))),
           lambda: pkl.token_logprobs(x.t())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    assert not calls


@pytest.mark.parametrize("x", [2 ** 31, 2 ** 32 + 128, -2 ** 40])
def test_binding_refuses_integers_beyond_32_bits(lib, calls, x):
    with pytest.raises(ValueError):
        pkl.pack_weight4(d(4, 64), group=x)
    with pytest.raises(ValueError):
        pkl.unpack_weight4(pkl.Weight4(d(9, dtype=torch.uint8), x, 64, 64))
    with pytest.raises(ValueError):
        pkl.token_logprobs(d(5, 256), top=x)
    assert not calls


def test_one_row_of_any_stride(lib, calls):
    """The distance of rows does not matter when there is one."""
    w = pkl.Weight4(d(lib.pic_op_weight4_bytes(200, 256, 128), dtype=torch.uint8), 200, 256, 128)
    pkl.gemm_w4(w, d(256, 1, dtype=torch.float16).t().as_subclass(OnDevice), out=d(1, 200))
    assert calls[-1][3] == 256
    pkl.add_rms_norm(d(3, 259)[1:2, :256], out=d(1, 256), dtype=torch.float32)
    assert calls[-1][4] == 256
