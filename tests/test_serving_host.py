"""Host checks of the operators around the compressor (no GPU): bad arguments are refused with their
code before anything touches CUDA, and empty calls that need no launch return at once."""
import ctypes

import pytest

from deepseek_v4_sparse_c128_gb300 import binding, build
from test_abi_host import FAKE, _t

I32, I64, F32, U8, BF16 = (binding.C128_I32, binding.C128_I64, binding.C128_F32, binding.C128_U8, binding.C128_BF16)
NULL, DTYPE, SHAPE, STRIDE, ALIGN, UNSUPPORTED, ARG = 1, 2, 3, 4, 5, 6, 7


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.load()


def _ref(x):
    return ctypes.byref(x) if isinstance(x, binding.Tensor) else x


def _call(L, name, order, args, over):
    a = dict(args, **over)
    return getattr(L, name)(*[_ref(a[k]) for k in order], None)


EXTEND = ("seq_lens", "held", "table", "free", "taken", "ratio", "block", "held_out", "taken_out")


@pytest.mark.parametrize("over,code", [
    (dict(seq_lens=None), NULL), (dict(held=_t([5], I32, data=None)), NULL), (dict(taken=None), NULL),
    (dict(seq_lens=_t([5], I64)), DTYPE), (dict(taken=_t([1], I32)), DTYPE), (dict(table=_t([5, 9], I64)), DTYPE),
    (dict(held=_t([4], I32)), SHAPE), (dict(table=_t([6, 9], I32)), SHAPE), (dict(taken=_t([2], I64)), SHAPE),
    (dict(held_out=_t([5, 1], I32)), SHAPE),
    (dict(table=_t([5, 9], I32, strides=[9, 2])), STRIDE), (dict(table=_t([5, 9], I32, strides=[8, 1])), STRIDE),
    (dict(seq_lens=_t([5], I32, strides=[2])), STRIDE),
    (dict(free=_t([9], I32, data=FAKE + 2)), ALIGN), (dict(taken=_t([1], I64, data=FAKE + 4)), ALIGN),
    (dict(ratio=0), ARG), (dict(block=0), ARG), (dict(block=1 << 31), ARG), (dict(ratio=-4), ARG),
    (dict(free=_t([1 << 31], I32)), ARG), (dict(held_out=_t([5], I32, data=FAKE + 4)), ARG),
])
def test_extend_block_tables_refuses(L, over, code):
    args = dict(seq_lens=_t([5], I32), held=_t([5], I32), table=_t([5, 9], I32), free=_t([40], I32), taken=_t([1], I64),
                ratio=1, block=8, held_out=_t([5], I32, data=FAKE + 64), taken_out=_t([1], I64))
    assert _call(L, "c128_extend_block_tables", EXTEND, args, over) == code


MAPS = ("seq_lens", "query_lens", "state_table", "state_block", "kv_table", "kv_block", "ratio", "query_start", "req",
        "pos", "slot", "kv_slot", "kv_lens")


@pytest.mark.parametrize("over,code", [
    (dict(query_lens=None), NULL), (dict(pos=_t([7], I64, data=None)), NULL),
    (dict(query_lens=_t([5], I64)), DTYPE), (dict(pos=_t([7], I32)), DTYPE), (dict(req=_t([7], I64)), DTYPE),
    (dict(query_start=_t([5], I32)), SHAPE), (dict(slot=_t([8], I64)), SHAPE), (dict(kv_table=_t([4, 9], I32)), SHAPE),
    (dict(kv_lens=_t([6], I32)), SHAPE), (dict(state_table=_t([9], I32)), SHAPE),
    (dict(kv_slot=_t([7], I64, strides=[2])), STRIDE), (dict(kv_table=_t([5, 9], I32, strides=[3, 1])), STRIDE),
    (dict(pos=_t([7], I64, data=FAKE + 4)), ALIGN),
    (dict(ratio=0), ARG), (dict(state_block=0), ARG), (dict(kv_block=-1), ARG),
])
def test_build_slot_maps_refuses(L, over, code):
    args = dict(seq_lens=_t([5], I32), query_lens=_t([5], I32), state_table=_t([5, 9], I32), state_block=8,
                kv_table=_t([5, 9], I32), kv_block=64, ratio=128, query_start=_t([6], I32), req=_t([7], I32),
                pos=_t([7], I64), slot=_t([7], I64), kv_slot=_t([7], I64), kv_lens=_t([5], I32))
    assert _call(L, "c128_build_slot_maps", MAPS, args, over) == code


DECODE = ("q", "cache", "block", "table", "lens", "scale", "sink", "out", "lse", "ws")


@pytest.mark.parametrize("over,code", [
    (dict(q=None), NULL), (dict(ws=None), NULL), (dict(cache=_t([4, 2, 584], U8, data=None)), NULL),
    (dict(q=_t([3, 5, 512], F32)), DTYPE), (dict(out=_t([3, 5, 512], U8)), DTYPE), (dict(lens=_t([3], I64)), DTYPE),
    (dict(cache=_t([4, 2, 584], I32)), DTYPE), (dict(lse=_t([3, 5], BF16)), DTYPE),
    (dict(out=_t([3, 4, 512], BF16)), SHAPE), (dict(lens=_t([2], I32)), SHAPE), (dict(sink=_t([4], F32)), SHAPE),
    (dict(lse=_t([5, 3], F32)), SHAPE), (dict(cache=_t([4, 2, 583], U8)), SHAPE), (dict(table=_t([2, 9], I32)), SHAPE),
    (dict(q=_t([3, 512], BF16)), SHAPE),
    (dict(q=_t([3, 5, 512], BF16, strides=[5120, 1024, 2])), STRIDE),
    (dict(q=_t([3, 5, 512], BF16, strides=[512, 0, 1])), STRIDE),
    (dict(out=_t([3, 5, 512], BF16, strides=[256, 512, 1])), STRIDE),
    (dict(cache=_t([4, 2, 584], U8, strides=[1160, 584, 1])), STRIDE),
    (dict(lse=_t([3, 5], F32, strides=[0, 1])), STRIDE),
    (dict(q=_t([3, 5, 512], BF16, data=FAKE + 8)), ALIGN),
    (dict(q=_t([3, 5, 512], BF16, strides=[2564, 512, 1])), ALIGN),
    (dict(out=_t([3, 5, 512], F32, strides=[2562, 512, 1])), ALIGN),
    (dict(cache=_t([4, 2, 584], U8, data=FAKE + 8)), ALIGN),
    (dict(cache=_t([4, 1, 588], U8), block=1), ALIGN), (dict(ws=_t([1 << 30], U8, data=FAKE + 128)), ALIGN),
    (dict(q=_t([3, 5, 256], BF16)), UNSUPPORTED), (dict(out=_t([3, 5, 128], BF16)), UNSUPPORTED),
    (dict(q=_t([3, 1025, 512], BF16)), UNSUPPORTED),
    (dict(block=4), ARG), (dict(block=0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(q=_t([0, 5, 512], BF16), out=_t([0, 5, 512], BF16), lens=_t([0], I32), table=_t([0, 9], I32),
          lse=_t([0, 5], F32)), 0),
])
def test_decode_attention_refuses(L, over, code):
    args = dict(q=_t([3, 5, 512], BF16), cache=_t([4, 2, 584], U8), block=2, table=_t([3, 9], I32), lens=_t([3], I32),
                scale=0.1, sink=_t([5], F32), out=_t([3, 5, 512], BF16), lse=_t([3, 5], F32), ws=_t([1 << 30], U8))
    assert _call(L, "c128_decode_attention", DECODE, args, over) == code


def test_decode_workspace_refuses(L):
    n = ctypes.c_int64(0)
    assert L.c128_decode_attention_workspace(5, None) == NULL
    assert L.c128_decode_attention_workspace(0, ctypes.byref(n)) == UNSUPPORTED
    assert L.c128_decode_attention_workspace(1025, ctypes.byref(n)) == UNSUPPORTED


MERGE = ("part", "part_lse", "out", "lse")


@pytest.mark.parametrize("over,code", [
    (dict(part=None), NULL), (dict(out=_t([3, 5, 512], BF16, data=None)), NULL),
    (dict(part=_t([2, 3, 5, 512], U8)), DTYPE), (dict(part_lse=_t([2, 3, 5], BF16)), DTYPE),
    (dict(part_lse=_t([3, 3, 5], F32)), SHAPE), (dict(out=_t([5, 3, 512], BF16)), SHAPE), (dict(lse=_t([3, 4], F32)), SHAPE),
    (dict(part=_t([3, 5, 512], BF16)), SHAPE),
    (dict(part=_t([2, 3, 5, 512], BF16, strides=[0, 2560, 512, 1])), STRIDE),
    (dict(out=_t([3, 5, 512], F32, strides=[5120, 1024, 2])), STRIDE),
    (dict(out=_t([3, 5, 512], BF16, data=FAKE + 4)), ALIGN),
    (dict(part=_t([2, 3, 5, 512], F32, strides=[7682, 2560, 512, 1])), ALIGN),
    (dict(part=_t([2, 3, 5, 256], BF16)), UNSUPPORTED),
    (dict(part=_t([0, 3, 5, 512], BF16), part_lse=_t([0, 3, 5], F32)), ARG),
    (dict(part=_t([2, 0, 5, 512], BF16), part_lse=_t([2, 0, 5], F32), out=_t([0, 5, 512], BF16), lse=None), 0),
])
def test_merge_attention_refuses(L, over, code):
    args = dict(part=_t([2, 3, 5, 512], BF16), part_lse=_t([2, 3, 5], F32), out=_t([3, 5, 512], BF16), lse=_t([3, 5], F32))
    assert _call(L, "c128_merge_attention", MERGE, args, over) == code


def test_binding_refuses_host_tensors_and_other_types():
    import torch
    a = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.extend_block_tables(a, a, torch.zeros(3, 4, dtype=torch.int32), a, torch.zeros(1, dtype=torch.int64), 1, 8)
    with pytest.raises(ValueError, match="CUDA"):
        binding.merge_attention(torch.zeros(2, 1, 1, 512), torch.zeros(2, 1, 1), torch.zeros(1, 1, 512))
    with pytest.raises(TypeError):
        binding.describe(torch.zeros(3, dtype=torch.float16))


def test_decode_attention_refuses_more_tiles_than_it_counts(L):
    """R * (MB*bs / 64 + 2) has to be below 2^31, and scale * log2(e) finite."""
    args = dict(q=_t([3, 5, 512], BF16), cache=_t([4, 2, 584], U8), block=2, table=_t([3, 9], I32), lens=_t([3], I32),
                scale=0.1, sink=_t([5], F32), out=_t([3, 5, 512], BF16), lse=_t([3, 5], F32), ws=_t([1 << 30], U8))
    R = 1 << 16
    many = dict(q=_t([R, 5, 512], BF16), out=_t([R, 5, 512], BF16), lens=_t([R], I32), lse=_t([R, 5], F32))
    assert _call(L, "c128_decode_attention", DECODE, args, dict(many, table=_t([R, 1 << 20], I32))) == ARG  # 2^16 * 32770
    assert _call(L, "c128_decode_attention", DECODE, args, dict(scale=3e38)) == ARG
