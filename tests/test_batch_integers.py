"""Integers that do not fit 32 bits are refused by the binding of the batched calls: ctypes would drop their upper bits
(a window of 2^32 would arrive as 0, every key). On the CPU: a stand-in for device tensors, nothing is launched."""
import pytest
import torch

import position_independent_kv_link_gb300 as pkl
from position_independent_kv_link_gb300 import api


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on device 0."""

    def get_device(self):
        return 0


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(api, "_call", lambda idx, stream, f, *args: made.append(args))
    monkeypatch.setattr(api, "_attention_scratch", lambda idx, *shape: made.append(shape) or 256)
    monkeypatch.setattr(api.L, "load", lambda: type("lib", (), {"__getattr__": lambda s, n: n})())
    return made


def d(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


FAR = [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, -2 ** 40]


def attention_args():
    k, rope = d(4, 2, 16, 128, dtype=torch.bfloat16), d(64, 64, 2, dtype=torch.float32)
    return d(3, 8, 128, dtype=torch.float16), d(3), pkl.BatchPages(d(2), d(2, 4)), k, k.clone().as_subclass(OnDevice), rope


@pytest.mark.parametrize("x", FAR)
def test_window(calls, x):
    q, start, *rest = attention_args()
    out = q.clone().as_subclass(OnDevice)
    pkl.attention_window(q, start, *rest, 2 ** 31 - 1, 2 ** 31 - 1, out=out)
    assert len(calls) == 2
    for window, sinks in ((x, 0), (5, x)):
        with pytest.raises(ValueError, match="32 bits"):
            pkl.attention_window(q, start, *rest, window, sinks, out=out)
    assert len(calls) == 2


@pytest.mark.parametrize("x", FAR)
def test_prefix(calls, x):
    q, start, *rest = attention_args()
    out = q.clone().as_subclass(OnDevice)
    pkl.attention_prefix(q, start, d(2), 32, *rest, out=out)
    with pytest.raises(ValueError, match="32 bits"):
        pkl.attention_prefix(q, start, d(2), x, *rest, out=out)
    assert len(calls) == 2


@pytest.mark.parametrize("x", FAR)
def test_block_tables(calls, x):
    out = pkl.BlockTables(d(2), d(2), d(3), d(8), d(8), d(3))
    args = d(2), d(2), d(2, 4), d(5)
    pkl.block_tables(*args, 8, first=2 ** 31 - 1, out=out)
    with pytest.raises(ValueError, match="32 bits"):
        pkl.block_tables(*args, 8, first=x, out=out)
    for o in (out, None):
        with pytest.raises(ValueError, match="32 bits"):
            pkl.block_tables(*args, x, out=o)
    assert len(calls) == 1


@pytest.mark.parametrize("x", FAR)
def test_qk_norm_rope(calls, x):
    k, rope = d(4, 2, 16, 128, dtype=torch.bfloat16), d(64, 64, 2, dtype=torch.float32)
    for heads in ((x, 2), (8, x)):
        with pytest.raises(ValueError):
            pkl.qk_norm_rope(d(3, 1536, dtype=torch.float32), *heads, d(3), d(3), rope, k, k)
    assert not calls
