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


# Relative 2-norms.  A sum's roundings to fp32 are off by at most 2^-24 of the partial sum each, to either side, and a
# partial sum grows with the root of its terms: n of them add up to at most sqrt(n) 2^-24.  What has one sign is the
# tensor core's truncation inside a partial sum that starts from zero: at most 16 accumulations on top of a sum of its
# final size (states in bf16: of 24 products of a chunk the first eight are those of the small terms), 2^-24 each in the
# mean, so 2^-20 of what a chunk adds; fp32 has at most 4 of them, 2^-22, and drops products of two small parts (up to 2^-22, of either sign, 4e-8 in the mean).
# One of three bf16 terms lost would cost 2.5e-6 of the states, one accumulator for all chunks 4e-6 to 7e-6.
def state_bound(dtype, N):
    if dtype == "bf16":
        return math.ceil(N / 128) ** 0.5 * 2.0 ** -24 + 2.0 ** -20
    return (math.ceil(N / 64) * (64 // 16 + 1)) ** 0.5 * 2.0 ** -24 + 2.0 ** -22


def output_bound(N, d):  # fp32: sums over d and 64 tokens in steps of 16, and the state's
    return state_bound("f32", N) + (d / 8 + 4) ** 0.5 * 2.0 ** -24 + 2.0 ** -22


def last_state(k, v, log_decay, state=None):
    """The last state by the direct sum in 64 bits: k, v [H, N, d]."""
    N = k.shape[1]
    left = torch.arange(N - 1, -1, -1, device="cuda").double()
    g = torch.tensor(log_decay, dtype=torch.float64, device="cuda")[:, None]
    S = (k.double() * torch.exp(g * left)[..., None]).transpose(1, 2) @ v.double()
    return S if state is None else S + torch.exp(g * N)[..., None] * state.double()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [59, 1])
def test_linattn_long_rows_do_not_drift(rows, dtype):
    """Hundreds of chunks of rows that run whole (59 x 5 of them fill the GPU once) and in segments (5), from large
    states, with slow decays; the fourth's power over a chunk lies halfway between two fp32 numbers (an error of 2^-25 a
    chunk, always to one side, would reach 4e-6 in bf16, 8e-6 in fp32)."""
    g, dt = gen(62), TORCH[dtype]
    H, N, d = 5, 32768, 64
    lg = [-0.0123, -3.35e-4, -1e-5, -100.5 * 2.0 ** -24 / (128 if dtype == "bf16" else 64), -2e-8]
    q, k, v = (normal(g, 1, H, N, d, dtype=dt) for _ in range(3))
    s0 = 64 * normal(g, 1, H, d, d)
    plan = mixers().LinearAttentionPlan(rows, H, N, d, d, lg, dtype=dtype)
    many = [t.expand(rows, H, N, d) for t in (q, k, v)]
    o, s = plan.fwd(*many, state=s0.expand(rows, H, d, d).contiguous(), final_state=True)
    want = last_state(k[0], v[0], lg, s0[0])[None]
    assert torch.equal(s, s[:1].expand_as(s))
    rel = off(s[:1], want)
    assert max(rel) <= state_bound(dtype, N), (rel, state_bound(dtype, N))
    if dtype == "f32":  # the last outputs, from the state before them
        end = N - 200
        before = last_state(k[0, :, :end], v[0, :, :end], lg, s0[0])
        last, _ = base.linattn(*(t[:, :, end:] for t in (q, k, v)), lg, plan.scale, before[None])
        rel = off(o[:1, :, end:], last)
        assert max(rel) <= output_bound(N, d), (rel, output_bound(N, d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,N,dk,dv,layout", [s for s in base.SIZES if s[0] * s[1] * s[3] * s[4] >= 1000])
def test_linattn_norms(B, H, N, dk, dv, layout, dtype):
    """States and, in fp32, outputs and gradients by their 2-norm, which sees the loss of one small term."""
    g, dt = gen(N + dk + dv), TORCH[dtype]
    q, k, v, do = (base.tokens(g, B, H, N, d, dt, layout) for d in (dk, dk, dv, dv))
    s0, ds = normal(g, B, H, dk, dv), normal(g, B, H, dk, dv)
    lg = base.decays(H, "slow")
    plan = mixers().LinearAttentionPlan(B, H, N, dk, dv, lg, dtype=dtype)
    o, s1 = plan.fwd(q, k, v, state=s0, final_state=True)
    want = base.linattn(q, k, v, lg, plan.scale, s0)
    got = plan.bwd(do, q, k, v, state=s0, dstate=ds)
    grads = base.gradients((q, k, v, s0), do, ds, lg, plan.scale, None)
    pairs = [("state", s1, want[1]), ("dstate", got["dstate"], grads[3])]
    if dtype == "f32":
        pairs += [("o", o, want[0])] + [(n, got[n], t) for n, t in zip(("dq", "dk", "dv"), grads)]
    for name, x, y in pairs:
        rel = float((x.double() - y).norm() / y.norm())
        bound = state_bound(dtype, N) if "state" in name else output_bound(N, max(dk, dv))
        assert rel <= bound, (name, rel, bound)


def odd_views(g, kind, B, H, N, dims, dt):
    """[B, H, N, d] views for each d whose strides are no multiples of one another (or whose rows overlap), and the
    buffers they lie in."""
    if kind == "fused":  # one projection of all of them
        buf = normal(g, B, N, H * sum(dims), dtype=dt)
        views, at = [], 0
        for d in dims:
            views.append(buf[..., at:at + H * d].view(B, N, H, d).transpose(1, 2))
            at += H * d
        return views, [buf] * len(dims)
    if kind == "padded heads":  # a head's tokens side by side, eight elements between heads
        bufs = [normal(g, B * (H * (N * d + 8)) + 8, dtype=dt) for d in dims]
        return [b.as_strided((B, H, N, d), (H * (N * d + 8), N * d + 8, d, 1)) for b, d in zip(bufs, dims)], bufs
    assert kind == "windows"  # token t starts eight elements behind token t - 1
    bufs = [normal(g, B, H, 8 * N + d, dtype=dt) for d in dims]
    return [b.as_strided((B, H, N, d), (H * (8 * N + d), 8 * N + d, 8, 1)) for b, d in zip(bufs, dims)], bufs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["fused", "padded heads", "windows"])
@pytest.mark.parametrize("B,H,N,dk,dv", [(2, 3, 1, 64, 96), (2, 3, 130, 64, 96), (2, 3, 700, 40, 104), (1, 5, 1000, 128, 72),
                                         (60, 5, 300, 64, 40)])
def test_linattn_strides_that_are_no_multiples(B, H, N, dk, dv, kind, dtype):
    """The same bits as dense copies give, and outputs that touch only their elements."""
    g, dt = gen(N + dv), TORCH[dtype]
    (q, k, v, do), _ = odd_views(g, kind, B, H, N, (dk, dk, dv, dv), dt)
    dense = [t.clone(memory_format=torch.contiguous_format) for t in (q, k, v, do)]
    lg = base.decays(H)
    plan = mixers().LinearAttentionPlan(B, H, N, dk, dv, lg, dtype=dtype)
    lengths = torch.randint(0, N + 1, (B,), generator=g, device="cuda").int()
    for n in (None, lengths):
        o, s = plan.fwd(*dense[:3], lengths=n, final_state=True)
        got, end = plan.fwd(q, k, v, lengths=n, final_state=True)
        assert torch.equal(got, o) and torch.equal(end, s)
        if kind != "windows":
            (_, _, out, _), bufs = odd_views(g, kind, B, H, N, (dk, dk, dv, dv), dt)
            bufs[2].fill_(7.0)
            plan.fwd(*dense[:3], lengths=n, o=out)
            assert torch.equal(out, o)
            out.fill_(7.0)
            assert (bufs[2] == 7.0).all()
        want = plan.bwd(dense[3], *dense[:3], lengths=n)
        got = plan.bwd(do, q, k, v, lengths=n)
        assert all(torch.equal(got[x], want[x]) for x in ("dq", "dk", "dv"))
    assert plan.device_status() == 0


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_retention_runs_no_other_kernels(layout):
    """Every step is one of the library's: torch allocates and makes views, whatever order the tokens are stored in."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Record(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.names = set()

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.add(func.overloadpacket.__name__)
            return func(*args, **(kwargs or {}))

    g = gen(70)
    B, H, N, dk, dv = 2, 3, 150, 64, 96
    q, k, v = (base.tokens(g, B, H, N, d, torch.bfloat16, layout) for d in (dk, dk, dv))
    w, b, at = 1 + 0.2 * normal(g, H, dv), 0.2 * normal(g, H, dv), torch.arange(N, device="cuda")
    plan = mixers().RetentionPlan(B, H, N, dk, dv)
    state, dy = normal(g, B, H, dk, dv), normal(g, B, N, H, dv, dtype=torch.bfloat16)
    with Record() as seen:
        y, end, saved = plan.fwd(q, k, v, w, b, at, state=state, final_state=True, save=True)
        plan.bwd(dy, saved, w)
        plan.step(q[:, :, 0], k[:, :, 0], v[:, :, 0], w, b, at[:B], end)
    assert seen.names <= {"empty", "empty_like", "empty_strided", "view", "transpose", "unsqueeze", "squeeze", "select",
                          "slice", "detach", "alias", "as_strided"}, seen.names
    qr, kr = plan.rotary.apply(q, k, positions=at)
    o = plan.attention.fwd(qr, kr, v, state=state)
    assert torch.equal(y, plan.norm.fwd(o.transpose(1, 2).contiguous(), w, b))


def test_linattn_range_of_values():
    """fp32 values from 2^-114 (a second tf32 part is whole down to there) to 3.4019e38 (the first is finite up to there);
    states in bf16 for keys from 2^-110 on (the third of their terms)."""
    g = gen(71)
    B, H, N, d = 1, 2, 200, 64
    lg = [-0.01, -0.1]
    q, k, v = (normal(g, B, H, N, d) for _ in range(3))
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, lg, dtype="f32")
    for small in ((q * 2.0 ** -114, k, v), (q, k * 2.0 ** -114, v), (q, k, v * 2.0 ** -114)):
        o, s = plan.fwd(*small, final_state=True)
        want = base.linattn(*small, lg, plan.scale)
        assert max(off(o, want[0])) <= output_bound(N, d) and max(off(s, want[1])) <= state_bound("f32", N)
    w = v.clone()
    w[:, :, 50, 3], w[:, :, 60, 4] = 3.4019e38, -3.4019e38
    low = (q * 2.0 ** -6, k * 2.0 ** -6, w)
    o, s = plan.fwd(*low, final_state=True)
    want = base.linattn(*low, lg, plan.scale)
    assert torch.isfinite(o).all() and max(off(o, want[0])) <= output_bound(N, d)
    half = mixers().LinearAttentionPlan(B, H, N, d, d, lg)
    keys, values = (k * 2.0 ** -110).bfloat16(), v.bfloat16()
    _, s = half.fwd(q.bfloat16(), keys, values, final_state=True)
    _, want = base.linattn(q.bfloat16(), keys, values, lg, half.scale)
    assert max(off(s, want)) <= state_bound("bf16", N)


def test_linattn_negative_strides():
    """Tokens stored backwards, through the C call: read and (fp32) written so; bf16 outputs are refused before anything runs."""
    g, m = gen(72), mixers()
    B, H, N, d = 1, 2, 150, 64
    for dtype in ("f32", "bf16"):
        q, k, v = (normal(g, B, H, N, d, dtype=TORCH[dtype]) for _ in range(3))
        plan = m.LinearAttentionPlan(B, H, N, d, d, [-0.1, -0.01], dtype=dtype)
        want = plan.fwd(q, k, v)
        back = q.flip(2)  # token t of q is row N - 1 - t
        forth, reverse = (0, N * d, d), (0, N * d, -d)
        last = (N - 1) * d * q.element_size()

        def call(out, so, end):
            a = m._FWD.pack(m._FWD.size, B, N, plan.scale, back.data_ptr() + last, k.data_ptr(), v.data_ptr(), *reverse,
                            *forth, *forth, 0, 0, out.data_ptr() + end, *so, 0)
            ws = plan._workspace(0)
            return plan.lib.fftconv_linattn_fwd(plan._handle, a, ws.data_ptr(), plan._stream(None))

        o = torch.full_like(v, 7.0)
        assert call(o, forth, 0) == 0 and torch.equal(o, want)
        o.fill_(7.0)
        status = call(o, reverse, last)
        if dtype == "f32":
            assert status == 0 and torch.equal(o.flip(2), want)
        else:
            assert status == 2 and (o == 7.0).all()
