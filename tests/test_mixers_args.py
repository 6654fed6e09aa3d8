"""Refusals of the operators around the convolution that need no GPU: sizes,
types and argument blocks are checked on the host before anything is launched."""
import ctypes
import math

import pytest
import torch

from fft_long_convolution_causal_b200 import binding, build, mixers


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def linattn(lib, B=1, H=2, N=64, dk=64, dv=64, dtype=1, log_decay=(-0.1, -0.2)):
    h = ctypes.c_void_p()
    g = None if log_decay is None else (ctypes.c_double * len(log_decay))(*log_decay)
    return lib.fftconv_linattn_plan_create(ctypes.byref(h), B, H, N, dk, dv, dtype, g)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(H=0, log_decay=()), 1), (dict(N=0), 1), (dict(dtype=2), 1), (dict(log_decay=None), 1),
    (dict(log_decay=(-0.1, 0.5)), 1), (dict(log_decay=(math.nan, 0.0)), 1), (dict(dk=0), 2), (dict(dk=4), 2),
    (dict(dk=60), 2), (dict(dk=136), 2), (dict(dv=7), 2), (dict(dv=256), 2), (dict(B=65536), 2)])
def test_linattn_plan_refusals(lib, bad, status):
    assert linattn(lib, **bad) == status


def test_null_plans_and_blocks(lib):
    assert lib.fftconv_linattn_plan_create(None, 1, 1, 1, 8, 8, 1, None) == 1
    for call, n in (("linattn_fwd", 3), ("linattn_bwd", 3), ("linattn_step", 2), ("rotary_apply", 2)):
        assert getattr(lib, "fftconv_" + call)(None, *[None] * n) == 1
    assert lib.fftconv_norm_fwd(None, 1, *[None] * 7) == 1
    assert lib.fftconv_norm_bwd(None, 1, *[None] * 10) == 1
    assert lib.fftconv_linattn_device_status(None, None) == 1
    assert lib.fftconv_linattn_set_wait_limit(None, 5) == 1
    for kind in ("linattn", "rotary", "norm"):
        assert getattr(lib, f"fftconv_{kind}_plan_destroy")(None) == 0
    assert lib.fftconv_linattn_workspace_bytes(None, 0) == 0
    assert lib.fftconv_norm_bwd_workspace_bytes(None) == 0


def rotary(lib, dtype=1, **over):
    o = dict(dim=64, rot=64, interleaved=0, scaling=0, base=10000.0, factor=1.0, context=4096.0)
    o.update(over)
    size = o.pop("size", ctypes.sizeof(mixers._RotaryOptions))
    h, opts = ctypes.c_void_p(), mixers._RotaryOptions(size, *o.values())
    return lib.fftconv_rotary_plan_create(ctypes.byref(h), dtype, ctypes.byref(opts))


@pytest.mark.parametrize("bad,status", [
    (dict(rot=0), 1), (dict(rot=7), 1), (dict(rot=66), 1), (dict(scaling=4), 1), (dict(scaling=-1), 1),
    (dict(base=1.0), 1), (dict(base=math.inf), 1), (dict(base=math.nan), 1), (dict(factor=0.5), 1),
    (dict(factor=math.nan), 1), (dict(scaling=3, context=0.0), 1), (dict(scaling=2, rot=2, dim=8), 1),
    (dict(dtype=3), 1), (dict(size=8), 1), (dict(dim=2048), 2)])
def test_rotary_plan_refusals(lib, bad, status):
    bad = dict(bad)
    assert rotary(lib, bad.pop("dtype", 1), **bad) == status


@pytest.mark.parametrize("rows,C,groups,dtype,eps,status", [
    (0, 8, 1, 1, 1e-5, 1), (4, 0, 1, 1, 1e-5, 1), (4, 8, 3, 1, 1e-5, 1), (4, 8, 0, 1, 1e-5, 1), (4, 8, 1, 5, 1e-5, 1),
    (4, 8, 1, 1, -1.0, 1), (4, 8, 1, 1, math.nan, 1), (4, 20000, 1, 1, 1e-5, 2), (1 << 31, 8, 1, 1, 1e-5, 2),
    (4, 8, 2, 1, 1e-5, 0)])
def test_norm_plan_refusals(lib, rows, C, groups, dtype, eps, status):
    h = ctypes.c_void_p()
    got = lib.fftconv_norm_plan_create(ctypes.byref(h), rows, C, groups, dtype, ctypes.byref(ctypes.c_double(eps)))
    assert got == status and bool(h.value) == (status == 0)
    lib.fftconv_norm_plan_destroy(h)


def test_norm_refuses_host_tensors_and_bad_rows():
    plan = mixers.LayerNormPlan(4, 8, groups=2)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        plan.fwd(x, torch.ones(2, 8), torch.zeros(2, 8))
    with pytest.raises(ValueError):
        plan.fwd(x[:, :4], torch.ones(2, 8), torch.zeros(2, 8))
    with pytest.raises(ValueError):
        plan.fwd([1.0], torch.ones(2, 8), torch.zeros(2, 8))


def test_python_side_counts():
    with pytest.raises(ValueError):
        mixers.LinearAttentionPlan(1, 3, 64, 64, 64, [-0.1, -0.2])
    with pytest.raises(KeyError):
        mixers.RotaryPlan(64, layout="other")
    with pytest.raises(KeyError):
        mixers.RotaryPlan(64, scaling="other")


@pytest.mark.parametrize("name", ["LinearAttentionPlan", "RotaryPlan", "LayerNormPlan", "RetentionPlan"])
def test_exported(name):
    import fft_long_convolution_causal_b200 as pkg
    assert getattr(pkg, name) is getattr(mixers, name)
