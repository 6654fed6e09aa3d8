"""Refusals of the sequence mixers' plans at the limits of fp32 (no GPU needed)."""
import ctypes

import pytest

from fft_long_convolution_causal_b200 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("eps,status", [(0.0, 0), (1e-45, 0), (1e-46, 1), (5e-324, 1), (3.4e38, 0), (3.5e38, 1), (1e300, 1)])
def test_norm_eps_in_fp32(lib, eps, status):
    h = ctypes.c_void_p()
    got = lib.fftconv_norm_plan_create(ctypes.byref(h), 4, 8, 1, 1, ctypes.byref(ctypes.c_double(eps)))
    assert got == status and bool(h.value) == (status == 0)
    lib.fftconv_norm_plan_destroy(h)
