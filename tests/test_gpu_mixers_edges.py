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


# neither powers of two nor near them; the last two nearer to one than fp32 holds
SLOW = [-0.0123, -3.35e-4, -1e-5, -4.1e-8, -2e-8]


def recurrence(k, v, log_decay, state=None):
    """S_t = a S_{t-1} + k_t^T v_t in 64 bits, token by token: the last state."""
    B, H, N, dk = k.shape
    a = torch.exp(torch.tensor(log_decay, dtype=torch.float64, device="cuda"))[:, None, None]
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64, device="cuda") if state is None else state.double()
    for t in range(N):
        S = torch.baddbmm((a * S).flatten(0, 1), k[:, :, t].double().flatten(0, 1)[..., None],
                          v[:, :, t].double().flatten(0, 1)[:, None]).view_as(S)
    return S


def off(got, want):
    """Relative 2-norm of the difference, for each head."""
    d = (got.double() - want).transpose(0, 1).flatten(1).norm(dim=1)
    return (d / want.transpose(0, 1).flatten(1).norm(dim=1)).tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linattn_single_tokens_do_not_drift(dtype):
    """Thousands of single tokens with slow decays.  A step rounds the new state, off by at most 2^-24 of it and to
    either side, and the state grows with the root of the steps: T of them add up to at most sqrt(T) 2^-24 in the 2-norm.
    (One-signed errors of a decay rounded to fp32, 2^-25 a step, would reach T / 2 times that: 6e-5.)
    "To either side" needs low bits to round: a product of two bf16 numbers has 16, so that with |s| up to 2^8 times the
    products the sum of a step lies on fp32's grid but for the decay's part, |log a| |s|.  Where that is below half the
    grid's spacing (at most 2^-24 |s|), rounding to nearest drops it in every step, whatever the decay's precision: what
    a token adds misses at most T |log a|."""
    g, dt = gen(60), TORCH[dtype]
    B, H, T, d = 2, len(SLOW), 4096, 64
    q, k, v = (normal(g, B, H, T, d, dtype=dt) for _ in range(3))
    plan = mixers().LinearAttentionPlan(B, H, 1, d, d, SLOW, dtype=dtype)
    state = torch.zeros(B, H, d, d, device="cuda")
    for t in range(T):
        plan.step(q[:, :, t], k[:, :, t], v[:, :, t], state)
    rel = off(state, recurrence(k, v, SLOW))
    bound = [T ** 0.5 * 2.0 ** -24 + (T * -x if dtype == "bf16" and -x < 2.0 ** -24 else 0.0) for x in SLOW]
    assert all(r <= b for r, b in zip(rel, bound)), (rel, bound)


def test_linattn_single_tokens_keep_infinite_states():
    g = gen(61)
    q, k, v = (normal(g, 1, 3, 64) for _ in range(3))
    state = normal(g, 1, 3, 64, 64)
    state[0, :, 3, 5], state[0, :, 4, 6], state[0, :, 5, 7] = math.inf, -math.inf, math.nan
    plan = mixers().LinearAttentionPlan(1, 3, 1, 64, 64, [-0.1, -1e-5, 0.0], dtype="f32")
    plan.step(q, k, v, state)
    assert (state[0, :, 3, 5] == math.inf).all() and (state[0, :, 4, 6] == -math.inf).all()
    assert torch.isnan(state).sum() == 3 and torch.isnan(state[0, :, 5, 7]).all()
