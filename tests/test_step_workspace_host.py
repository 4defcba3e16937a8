"""Host checks of the size of window attention's workspace (no GPU)."""
import ctypes

import pytest

from deepseek_v4_sparse_c128_gb300 import binding, build

NULL, UNSUPPORTED, ARG = 1, 6, 7


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.load()


@pytest.mark.parametrize("heads,window,first,code", [
    (0, 128, 0, UNSUPPORTED), (1025, 128, 0, UNSUPPORTED), (-1, 128, 0, UNSUPPORTED), (5, 0, 0, ARG), (5, -3, 0, ARG), (5, 1 << 31, 0, ARG),
    (5, 128, -1, ARG), (5, 128, 1 << 31, ARG), (5, (1 << 63) - 1, (1 << 63) - 1, ARG)])
def test_size_refuses(L, heads, window, first, code):
    n = ctypes.c_int64(-5)
    assert L.c128_window_attention_workspace(heads, window, first, ctypes.byref(n)) == code
    assert n.value == -5


def test_short_windows_take_none(L):
    n = ctypes.c_int64(-5)
    assert L.c128_window_attention_workspace(5, 128, 8, None) == NULL
    for heads, window, first in ((1, 1, 0), (64, 128, 8), (1024, 1, 135), (5, 136, 0)):
        n.value = -5
        assert L.c128_window_attention_workspace(heads, window, first, ctypes.byref(n)) == 0 and n.value == 0
    assert binding.window_attention_workspace(64, 128, 4) == 0
