"""Outputs of the batched calls that overlap the inputs they are computed from are refused (C ABI, no GPU needed: nothing is
launched and no address is followed; a scratch of 100 bytes is refused last, so its message shows that nothing else was)."""
import pytest

from position_independent_kv_link_gb300 import _lib as L

from .test_batch_refusals import lib  # noqa: F401  (fixture)

MB = 1 << 20
S = dict(k=64 * MB, v=65 * MB, rope=66 * MB, rest=67 * MB, scratch=68 * MB)


def attention(lib, prefix, dtype, q, out, T=3, H=8):
    r, n = S["rest"], 2
    head = (dtype, T, H, 2, 128, q, r)
    tail = (n, r, r, 4, None, None)
    end = (S["k"], S["v"], 4, S["rope"], 64, out, S["scratch"], 100, None)
    if prefix:
        return lib.pic_op_attention_prefix(*head, r, None, 2, 32, *tail, *end)
    return lib.pic_op_attention_window(*head, *tail, 5, 0, *end)


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("dtype,e", [(L.PIC_BF16, 2), (L.PIC_F32, 4)])
def test_attention_output_over_q(lib, prefix, dtype, e):
    size, q = 3 * 8 * 128 * e, 32 * MB
    for out in (q, q + 32, q - 32, q + size - 32, q - size + 32):
        assert attention(lib, prefix, dtype, q, out) == L.PIC_ERR_INVALID_ARG
        assert b"overlap" in lib.pic_last_error()
    for out in (q + size, q - size):
        assert attention(lib, prefix, dtype, q, out) == L.PIC_ERR_INVALID_ARG
        assert b"scratch too small" in lib.pic_last_error()


@pytest.mark.parametrize("dtype,e", [(L.PIC_BF16, 2), (L.PIC_F32, 4)])
def test_rotated_q_over_qkv(lib, dtype, e):
    T, stride, qkv, r = 3, 12 * 128 + 8, 32 * MB, S["rest"]
    rows, size = ((T - 1) * stride + 12 * 128) * 4, T * 8 * 128 * e
    for out in (qkv, qkv + rows - 16, qkv - size + 16, qkv + 4 * stride):
        assert lib.pic_op_qk_norm_rope(dtype, T, 8, 2, 128, qkv, stride, None, None, 1e-5, r, r, S["rope"], 64, out, S["k"],
                                       S["v"], 4, None) == L.PIC_ERR_INVALID_ARG
        assert b"overlap" in lib.pic_last_error()
