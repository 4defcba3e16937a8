"""Host checks of the steps of rotations (no GPU)."""
import ctypes
import math

import pytest

from deepseek_v4_sparse_c128_gb300 import binding, build
from test_abi_host import _t

F32 = binding.C128_F32
ARG, OK = 7, 0


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.load()


def _status(L, rows, **rope):
    """Of a table of no rows, which needs no GPU, unless `rows` says otherwise."""
    return L.c128_build_cos_sin(ctypes.byref(binding.rope(**rope)), 0, ctypes.byref(_t([rows, 64], F32)), None)


@pytest.mark.parametrize("scaling,factor", [(s, f) for s in ("linear", "yarn") for f in (5e-324, 1e-310, 1e-300, 1e-20)] + [("linear", 1e-8)])
def test_factors_that_make_steps_without_a_fraction_are_refused(L, factor, scaling):
    """1 / factor radians per position and more: infinite, or so many turns that doubles hold no part of one."""
    assert _status(L, 9, scaling=scaling, factor=factor) == ARG
    assert _status(L, 0, scaling=scaling, factor=factor) == ARG


def test_the_largest_step(L):
    """The first pair's step is 1 radian: up to 2^20 turns of it."""
    most = 1 / (2 * math.pi * 2.0 ** 20)
    assert _status(L, 0, scaling="linear", factor=most * 1.001) == OK
    assert _status(L, 0, scaling="linear", factor=most * 0.999) == ARG
    for factor in (1e-3, 0.5, 1.0, 1e300):
        assert _status(L, 0, scaling="linear", factor=factor) == OK
    # (yarn stretches the slow pairs only: the fastest of them by 1 / factor is 1.8e4 radians, 2.9e3 turns)
    assert _status(L, 0, scaling="yarn", factor=1e-8) == OK
    # without a scaling the factor is not used
    assert _status(L, 0, factor=1e-310) == OK
