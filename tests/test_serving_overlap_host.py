"""Results whose rows share elements are refused (no GPU): many CTAs store them at once, in no order."""
import ctypes

import pytest

from deepseek_v4_sparse_c128_gb300 import binding, build
from test_abi_host import FAKE, _t

I32, F32, U8, BF16 = binding.C128_I32, binding.C128_F32, binding.C128_U8, binding.C128_BF16
SHAPE, STRIDE, ALIGN = 3, 4, 5


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.load()


def _ref(x):
    return ctypes.byref(x) if isinstance(x, binding.Tensor) else x


REFUSED = [
    dict(out=_t([3, 5, 512], BF16, strides=[512, 512, 1])), dict(out=_t([3, 5, 512], BF16, strides=[2048, 512, 1])),
    dict(out=_t([3, 5, 512], BF16, strides=[2560 - 8, 512, 1])), dict(out=_t([3, 5, 512], F32, strides=[512, 1024, 1])),
    dict(out=_t([3, 5, 512], F32, strides=[512, 1536 - 4, 1])), dict(lse=_t([3, 5], F32, strides=[1, 1])),
    dict(lse=_t([3, 5], F32, strides=[4, 1])), dict(lse=_t([3, 5], F32, strides=[2, 4])),
]
TAKEN = [
    dict(), dict(out=_t([3, 5, 512], F32, strides=[512, 1536, 1])), dict(out=_t([3, 5, 512], F32, strides=[1024, 4096, 1])),
    dict(out=_t([3, 5, 512], BF16, strides=[2560, 512, 1])), dict(lse=_t([3, 5], F32, strides=[1, 3])),
    dict(lse=_t([3, 5], F32, strides=[2, 5])), dict(lse=_t([3, 5], F32, strides=[2, 6])), dict(lse=_t([3, 5], F32, strides=[1 << 40, 1 << 33])),
]


@pytest.mark.parametrize("over,code", [(o, STRIDE) for o in REFUSED] + [(o, ALIGN) for o in TAKEN])
def test_decode_attention_refuses_results_that_overlap(L, over, code):
    """(The last check, behind that of the results, stops the others: the workspace is not aligned.)"""
    a = dict(dict(q=_t([3, 5, 512], BF16), cache=_t([4, 2, 584], U8), block=2, table=_t([3, 9], I32), lens=_t([3], I32),
                  scale=0.1, sink=None, out=_t([3, 5, 512], BF16), lse=None, ws=_t([1 << 30], U8, data=FAKE + 128)), **over)
    order = ("q", "cache", "block", "table", "lens", "scale", "sink", "out", "lse", "ws")
    assert L.c128_decode_attention(*[_ref(a[k]) for k in order], None) == code


@pytest.mark.parametrize("over", REFUSED)
def test_merge_attention_refuses_results_that_overlap(L, over):
    a = dict(dict(out=_t([3, 5, 512], BF16), lse=None), **over)
    args = (_t([2, 3, 5, 512], BF16), _t([2, 3, 5], F32), a["out"], a["lse"])
    assert L.c128_merge_attention(*[_ref(x) for x in args], None) == STRIDE


@pytest.mark.parametrize("R,H", [(1, 4), (4, 1), (1, 1)])
def test_the_stride_of_a_single_index_does_not_matter(L, R, H):
    """(Stopped behind the check of `out`: lse has one column too many.)"""
    args = (_t([2, R, H, 512], BF16), _t([2, R, H], F32), _t([R, H, 512], BF16, strides=[512, 512, 1]), _t([R, H + 1], F32))
    assert L.c128_merge_attention(*[_ref(x) for x in args], None) == SHAPE
