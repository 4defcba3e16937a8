"""Host checks of the operators around the attention of recent tokens (no GPU): bad arguments are refused with their
code before anything touches CUDA, and empty calls that need no launch return at once."""
import ctypes

import pytest

from deepseek_v4_sparse_c128_gb300 import binding, build
from test_abi_host import FAKE, _t
from test_serving_host import _call

I32, I64, F32, U8, BF16 = (binding.C128_I32, binding.C128_I64, binding.C128_F32, binding.C128_U8, binding.C128_BF16)
NULL, DTYPE, SHAPE, STRIDE, ALIGN, UNSUPPORTED, ARG = 1, 2, 3, 4, 5, 6, 7


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.load()


def _rope(**over):
    r = binding.rope(scaling="yarn", factor=4.0)
    for k, v in over.items():
        setattr(r, k, v)
    return r


@pytest.mark.parametrize("rope,first,table,code", [
    (None, 0, _t([9, 64], F32), NULL), (_rope(), 0, None, NULL), (_rope(), 0, _t([9, 64], F32, data=None), NULL),
    (_rope(), 0, _t([9, 64], BF16), DTYPE), (_rope(), 0, _t([64], F32), SHAPE),
    (_rope(), 0, _t([9, 64], F32, strides=[128, 2]), STRIDE), (_rope(), 0, _t([9, 64], F32, strides=[63, 1]), STRIDE),
    (_rope(), 0, _t([9, 64], F32, data=FAKE + 2), ALIGN),
    (_rope(), 0, _t([9, 0], F32), UNSUPPORTED), (_rope(), 0, _t([9, 63], F32), UNSUPPORTED), (_rope(), 0, _t([9, 514], F32), UNSUPPORTED),
    (_rope(scaling=3), 0, _t([9, 64], F32), UNSUPPORTED), (_rope(scaling=-1), 0, _t([9, 64], F32), UNSUPPORTED),
    (_rope(theta=1.0), 0, _t([9, 64], F32), ARG), (_rope(theta=float("nan")), 0, _t([9, 64], F32), ARG),
    (_rope(theta=float("inf")), 0, _t([9, 64], F32), ARG), (_rope(reserved=1), 0, _t([9, 64], F32), ARG),
    (_rope(magnitude=float("nan")), 0, _t([9, 64], F32), ARG), (_rope(magnitude=1e39), 0, _t([9, 64], F32), ARG),
    (_rope(factor=0.0), 0, _t([9, 64], F32), ARG), (_rope(scaling=1, factor=-1.0), 0, _t([9, 64], F32), ARG),
    (_rope(original_positions=0.0), 0, _t([9, 64], F32), ARG), (_rope(beta_fast=float("inf")), 0, _t([9, 64], F32), ARG),
    (_rope(beta_slow=-1.0), 0, _t([9, 64], F32), ARG),
    (_rope(), -1, _t([9, 64], F32), ARG), (_rope(), (1 << 32) - 8, _t([9, 64], F32), ARG), (_rope(), 1 << 62, _t([0, 64], F32), ARG),
    (_rope(), 0, _t([0, 64], F32), 0), (_rope(scaling=0, factor=0.0, beta_fast=0.0), 1 << 32, _t([0, 64], F32), 0),
])
def test_build_cos_sin_refuses(L, rope, first, table, code):
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    assert L.c128_build_cos_sin(ref(rope), first, ref(table), None) == code


ROTATE = ("x", "pos", "cs", "first", "layout", "inverse", "out")


@pytest.mark.parametrize("over,code", [
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(pos=None), NULL), (dict(cs=None), NULL),
    (dict(x=_t([3, 5, 96], BF16, data=None)), NULL), (dict(out=_t([3, 5, 96], BF16, data=None)), NULL),
    (dict(x=_t([3, 5, 96], I32)), DTYPE), (dict(out=_t([3, 5, 96], F32)), DTYPE), (dict(pos=_t([3], I32)), DTYPE),
    (dict(cs=_t([9, 64], BF16)), DTYPE),
    (dict(x=_t([15, 96], BF16)), SHAPE), (dict(pos=_t([4], I64)), SHAPE), (dict(out=_t([3, 6, 96], BF16)), SHAPE),
    (dict(x=_t([3, 5, 96], BF16, strides=[960, 192, 2])), STRIDE), (dict(x=_t([3, 5, 96], BF16, strides=[480, 0, 1])), STRIDE),
    (dict(out=_t([3, 5, 96], BF16, strides=[96, 96, 1])), STRIDE), (dict(out=_t([3, 5, 96], BF16, strides=[470, 96, 1])), STRIDE),
    (dict(out=_t([3, 5, 96], BF16, strides=[960, 192, 1])), STRIDE),  # x itself, with other strides
    (dict(pos=_t([3], I64, strides=[2])), STRIDE),
    (dict(x=_t([3, 5, 96], BF16, data=FAKE + 1)), ALIGN), (dict(out=_t([3, 5, 96], BF16, data=FAKE + 1)), ALIGN),
    (dict(cs=_t([9, 65], F32)), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(layout=-1), UNSUPPORTED),
    (dict(inverse=2), ARG), (dict(first=-1), ARG), (dict(first=33), ARG), (dict(first=1 << 40), ARG),
    (dict(cs=_t([9, 128], F32)), ARG),
    (dict(x=_t([1, 1 << 20, 1 << 12], BF16), out=_t([1, 1 << 20, 1 << 12], BF16), pos=_t([1], I64)), ARG),
    (dict(x=_t([0, 5, 96], BF16), out=_t([0, 5, 96], BF16), pos=_t([0], I64)), 0),
    (dict(x=_t([3, 0, 96], BF16), out=_t([3, 0, 96], BF16)), 0),
])
def test_rotate_refuses(L, over, code):
    args = dict(x=_t([3, 5, 96], BF16), pos=_t([3], I64), cs=_t([9, 64], F32), first=32, layout=0, inverse=0,
                out=_t([3, 5, 96], BF16))
    assert _call(L, "c128_rotate", ROTATE, args, over) == code


NORM = ("pos", "slot", "eps", "cs", "q", "q_w", "q_out", "k", "k_w", "cache", "block")


@pytest.mark.parametrize("over,code", [
    (dict(pos=None), NULL), (dict(slot=None), NULL), (dict(cs=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL),
    (dict(k=None), NULL), (dict(cache=None), NULL), (dict(q=None, q_out=None, q_w=None, k=None, cache=None, k_w=None), NULL),
    (dict(q=None, q_out=None), NULL), (dict(k=None, cache=None), NULL), (dict(q=_t([3, 5, 512], BF16, data=None)), NULL),
    (dict(q=_t([3, 5, 512], U8)), DTYPE), (dict(k=_t([3, 512], I32)), DTYPE), (dict(pos=_t([3], I32)), DTYPE),
    (dict(q_w=_t([512], BF16)), DTYPE), (dict(cache=_t([4, 2, 584], I32)), DTYPE), (dict(q_out=_t([3, 5, 512], F32)), DTYPE),
    (dict(slot=_t([4], I64)), SHAPE), (dict(q=_t([4, 5, 512], BF16)), SHAPE), (dict(q_out=_t([3, 4, 512], BF16)), SHAPE),
    (dict(k=_t([2, 512], BF16)), SHAPE), (dict(k_w=_t([448], F32)), SHAPE), (dict(cache=_t([4, 2, 583], U8)), SHAPE),
    (dict(q=_t([3, 5, 512], BF16, strides=[5120, 1024, 2])), STRIDE), (dict(q_out=_t([3, 5, 512], BF16, strides=[512, 512, 1])), STRIDE),
    (dict(q_out=_t([3, 5, 512], BF16, strides=[5120, 1024, 1])), STRIDE),  # q itself, with other strides
    (dict(k=_t([3, 512], BF16, strides=[256, 1])), STRIDE), (dict(cs=_t([9, 64], F32, strides=[32, 1])), STRIDE),
    (dict(q_w=_t([512], F32, strides=[2])), STRIDE),
    (dict(q=_t([3, 5, 512], BF16, data=FAKE + 8)), ALIGN), (dict(k=_t([3, 512], BF16, strides=[516, 1])), ALIGN),
    (dict(q_w=_t([512], F32, data=FAKE + 4)), ALIGN), (dict(k_w=_t([512], F32, data=FAKE + 8)), ALIGN),
    (dict(cache=_t([4, 2, 584], U8, data=FAKE + 8)), ALIGN), (dict(cache=_t([4, 1, 588], U8), block=1), ALIGN),
    (dict(q=_t([3, 5, 128], BF16)), UNSUPPORTED), (dict(k=_t([3, 256], BF16)), UNSUPPORTED), (dict(cs=_t([9, 32], F32)), UNSUPPORTED),
    (dict(block=3), ARG), (dict(block=0), ARG),
    (dict(pos=_t([1 << 30], I64), slot=_t([1 << 30], I64), q=_t([1 << 30, 5, 512], BF16), q_out=_t([1 << 30, 5, 512], BF16),
          k=_t([1 << 30, 512], BF16)), ARG),
    (dict(pos=_t([0], I64), slot=_t([0], I64), q=_t([0, 5, 512], BF16), q_out=_t([0, 5, 512], BF16), k=_t([0, 512], BF16)), 0),
    (dict(q=_t([3, 0, 512], BF16), q_out=_t([3, 0, 512], BF16), k=None, k_w=None, cache=None), 0),
])
def test_norm_rope_store_refuses(L, over, code):
    args = dict(pos=_t([3], I64), slot=_t([3], I64), eps=1e-6, cs=_t([9, 64], F32), q=_t([3, 5, 512], BF16), q_w=_t([512], F32),
                q_out=_t([3, 5, 512], BF16), k=_t([3, 512], BF16), k_w=_t([512], F32), cache=_t([4, 2, 584], U8), block=2)
    assert _call(L, "c128_norm_rope_store", NORM, args, over) == code


WINDOW = ("q", "cache", "block", "table", "req", "pos", "slot", "window", "first", "scale", "sink", "out", "lse", "ws")


@pytest.mark.parametrize("over,code", [
    (dict(q=None), NULL), (dict(ws=None), NULL), (dict(table=None), NULL), (dict(req=None), NULL), (dict(pos=None), NULL),
    (dict(slot=None), NULL), (dict(out=None), NULL), (dict(cache=_t([4, 2, 584], U8, data=None)), NULL),
    (dict(q=_t([3, 5, 512], F32)), DTYPE), (dict(out=_t([3, 5, 512], U8)), DTYPE), (dict(req=_t([3], I64)), DTYPE),
    (dict(pos=_t([3], I32)), DTYPE), (dict(slot=_t([3], I32)), DTYPE), (dict(table=_t([2, 9], I64)), DTYPE),
    (dict(lse=_t([3, 5], BF16)), DTYPE),
    (dict(out=_t([3, 4, 512], BF16)), SHAPE), (dict(req=_t([2], I32)), SHAPE), (dict(pos=_t([4], I64)), SHAPE),
    (dict(slot=_t([2], I64)), SHAPE), (dict(sink=_t([4], F32)), SHAPE), (dict(lse=_t([5, 3], F32)), SHAPE), (dict(table=_t([9], I32)), SHAPE),
    (dict(q=_t([3, 5, 512], BF16, strides=[512, 0, 1])), STRIDE), (dict(out=_t([3, 5, 512], BF16, strides=[512, 512, 1])), STRIDE),
    (dict(lse=_t([3, 5], F32, strides=[1, 1])), STRIDE), (dict(table=_t([2, 9], I32, strides=[8, 1])), STRIDE),
    (dict(pos=_t([3], I64, strides=[2])), STRIDE),
    (dict(q=_t([3, 5, 512], BF16, data=FAKE + 8)), ALIGN), (dict(pos=_t([3], I64, data=FAKE + 4)), ALIGN),
    (dict(ws=_t([1 << 30], U8, data=FAKE + 128)), ALIGN), (dict(cache=_t([4, 2, 584], U8, data=FAKE + 8)), ALIGN),
    (dict(q=_t([3, 5, 256], BF16)), UNSUPPORTED), (dict(q=_t([3, 1025, 512], BF16)), UNSUPPORTED),
    (dict(block=4), ARG), (dict(window=0), ARG), (dict(window=1 << 31), ARG), (dict(first=-1), ARG), (dict(first=1 << 31), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=3e38), ARG),
    (dict(q=_t([0, 5, 512], BF16), out=_t([0, 5, 512], BF16), req=_t([0], I32), pos=_t([0], I64), slot=_t([0], I64),
          lse=_t([0, 5], F32)), 0),
])
def test_window_attention_refuses(L, over, code):
    args = dict(q=_t([3, 5, 512], BF16), cache=_t([4, 2, 584], U8), block=2, table=_t([2, 9], I32), req=_t([3], I32), pos=_t([3], I64),
                slot=_t([3], I64), window=128, first=4, scale=0.1, sink=_t([5], F32), out=_t([3, 5, 512], BF16), lse=_t([3, 5], F32),
                ws=_t([1 << 30], U8))
    assert _call(L, "c128_window_attention", WINDOW, args, over) == code


def test_window_attention_refuses_more_tiles_than_it_counts(L):
    """T * (min(MB*bs, window + first) / 64 + 2) has to be below 2^31."""
    T = 1 << 16
    args = dict(q=_t([T, 5, 512], BF16), cache=_t([4, 2, 584], U8), block=2, table=_t([2, 1 << 20], I32), req=_t([T], I32),
                pos=_t([T], I64), slot=_t([T], I64), window=(1 << 31) - 1, first=0, scale=0.1, sink=None, out=_t([T, 5, 512], BF16),
                lse=None, ws=_t([1 << 30], U8))
    assert _call(L, "c128_window_attention", WINDOW, args, {}) == ARG  # 2^16 * 32770


def test_binding_refuses():
    import torch
    with pytest.raises(ValueError, match="scaling"):
        binding.rope(scaling="ntk")
    with pytest.raises(ValueError, match="CUDA"):
        binding.build_cos_sin(binding.rope(), 0, torch.zeros(3, 64))
    with pytest.raises(ValueError, match="CUDA"):
        binding.rotate(torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int64), torch.zeros(9, 64))
    with pytest.raises(ValueError, match="CUDA"):
        binding.norm_rope_store(torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int64), 1e-6, torch.zeros(9, 64),
                                q=torch.zeros(3, 2, 512))
