"""Edges of the sequence mixers: what lies around a tensor, long runs of a state, strides off the beaten track.
Tolerances as in test_gpu_mixers.py unless a test derives its own."""
import math

import pytest
import torch

import test_gpu_mixers as base
from test_gpu_mixers import TORCH, gen, mixers, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fft_long_convolution_causal_b200 import binding
    binding.load_library()


def inside(t, room=64):
    """t's values in the middle of a buffer of NaN, and the buffer."""
    buf = torch.full((2 * room + t.numel(),), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[room:room + t.numel()].view(t.shape)
    view.copy_(t)
    return view, buf


def around_is_nan(buf, n, room=64):
    return bool(torch.isnan(buf[:room]).all() and torch.isnan(buf[room + n:]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2, 3, 5, 11, 1000])
@pytest.mark.parametrize("C", range(1, 8))
def test_layernorm_narrow_rows(C, rows, dtype):
    """Rows narrower than a 16-byte piece, inside a buffer of NaN that stays as it was."""
    base.test_layernorm(rows, C, 1, dtype)
    g, dt = gen(10 * C + rows), TORCH[dtype]
    x, dy = normal(g, rows, C, dtype=dt), normal(g, rows, C, dtype=dt)
    w, b = 1 + 0.3 * normal(g, 1, C), normal(g, 1, C)
    plan = mixers().LayerNormPlan(rows, C, dtype=dtype, eps=1e-2)
    y, mean, rstd = plan.fwd(x, w, b, statistics=True)
    dx, dw, db = plan.bwd(dy, x, w, mean, rstd)
    vx, bx = inside(x)
    vy, by = inside(torch.zeros_like(x))
    vd, bd = inside(dy)
    plan.fwd(vx, w, b, y=vy)
    assert torch.equal(vy, y) and torch.equal(vx, x) and around_is_nan(by, y.numel()) and around_is_nan(bx, x.numel())
    got = plan.bwd(vd, vx, w, mean, rstd)
    assert all(torch.equal(s, t) for s, t in zip(got, (dx, dw, db))) and around_is_nan(bd, dy.numel())
    plan.fwd(vx, w, b, y=vx)
    assert torch.equal(vx, y) and around_is_nan(bx, x.numel())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C", [(5, 1), (1000, 5), (700, 37), (333, 557), (200, 768), (60, 5001)])
def test_layernorm_gradient_in_place(rows, C, dtype):
    """dx may be dy."""
    g, dt = gen(C), TORCH[dtype]
    x, dy = normal(g, rows, C, dtype=dt), normal(g, rows, C, dtype=dt)
    w, b = 1 + 0.3 * normal(g, 1, C), normal(g, 1, C)
    plan = mixers().LayerNormPlan(rows, C, dtype=dtype, eps=1e-2)
    _, mean, rstd = plan.fwd(x, w, b, statistics=True)
    want = plan.bwd(dy, x, w, mean, rstd)
    vd, bd = inside(dy)
    dw, db = torch.empty(1, C, device="cuda"), torch.empty(1, C, device="cuda")
    ws = torch.empty(plan._bytes, dtype=torch.uint8, device="cuda")
    status = plan.lib.fftconv_norm_bwd(plan._handle, rows, vd.data_ptr(), x.data_ptr(), w.data_ptr(), mean.data_ptr(),
                                       rstd.data_ptr(), vd.data_ptr(), dw.data_ptr(), db.data_ptr(), ws.data_ptr(),
                                       plan._stream(None))
    assert status == 0
    assert all(torch.equal(s, t) for s, t in zip((vd, dw, db), want)) and around_is_nan(bd, dy.numel())
