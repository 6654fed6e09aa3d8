"""Linear attention with a decay per head, rotary positions and layer norm
against plain forms in 64 bits.

Tolerances.  Let u be half a step of the output's type (bf16 2^-8, fp32 2^-24)
and A the operator applied to the absolute values (every product and decay
positive), which bounds the effect of relative errors in its terms.
bf16: the result is rounded once (u |o|), the scores once and the state's copy
once (each at most 2^-8 of A): |error| <= 2^-8 (|o| + 2 A), and in the mean over
many outputs three independent roundings, uniform within half a step (rms
2^-8 / sqrt 3 each): relative 2-norm <= 2^-8.
fp32 (and the fp32 states of either type): each sum of n terms is off by at most
n 2^-24 of the sum of absolute values; a term passes through at most dk + 2
chunks of 128 terms and a product per chunk of the row: |error| <= n 2^-24 A."""
import math

import pytest
import torch

from mixer_reference import layernorm, linattn, rotary

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fft_long_convolution_causal_b200 import binding
    binding.load_library()


def mixers():
    from fft_long_convolution_causal_b200 import mixers as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def decays(H, kind="mixed"):
    if kind == "mixed":  # none, forgetful, the token alone, and slow ones
        return ([0.0, -3.0, -math.inf] + [math.log1p(-2.0 ** -(5 + h)) for h in range(H)])[:H]
    return [math.log1p(-2.0 ** -(5 + 7 * h / max(1, H - 1))) for h in range(H)]


def tokens(g, B, H, N, d, dtype, layout):
    """A [B, H, N, d] tensor in one of the layouts a program has."""
    if layout == "bhnd":
        return normal(g, B, H, N, d, dtype=dtype)
    if layout == "bnhd":
        return normal(g, B, N, H, d, dtype=dtype).transpose(1, 2)
    if layout == "slice":  # a part of a wider projection, rows of a longer buffer
        return normal(g, B, N + 3, H, d + 16, dtype=dtype)[:, 2:N + 2, :, 8:8 + d].transpose(1, 2)
    assert layout == "shared"  # one head for all
    return normal(g, B, 1, N, d, dtype=dtype).expand(B, H, N, d)


def chain(N, d):
    return d + 2 * 128 + 2 * math.ceil(N / 64) + 16


def check(got, want, absolute, dtype, N, d, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    err = (got - want).abs()
    if dtype == "bf16":
        bound = U["bf16"] * (want.abs() + 2 * absolute)
        norm = want.norm()
        # the norm's statement is one on many outputs
        if want.numel() >= 1000:
            assert err.norm() <= U["bf16"] * norm, (what, float(err.norm() / norm))
    else:
        bound = chain(N, d) * U["f32"] * absolute
    worst = (err - bound - 1e-30).max()
    assert worst <= 0, (what, float(worst), float(err.max()))


def absolutes(ts):
    return [None if t is None else t.double().abs() for t in ts]


SIZES = [  # B, H, N, dk, dv, layout
    (1, 1, 1, 8, 8, "bhnd"), (2, 3, 2, 16, 24, "bnhd"), (1, 4, 63, 64, 64, "bhnd"), (2, 3, 64, 128, 128, "bnhd"),
    (1, 5, 65, 72, 104, "slice"), (3, 2, 127, 128, 8, "bhnd"), (2, 4, 128, 64, 128, "bnhd"),
    (1, 3, 129, 128, 64, "slice"), (2, 2, 200, 40, 64, "shared"), (1, 5, 513, 64, 64, "bnhd"),
    (2, 6, 1000, 128, 128, "bnhd"), (40, 8, 300, 64, 64, "bhnd"), (19, 16, 260, 128, 120, "bnhd")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,H,N,dk,dv,layout", SIZES)
def test_linattn_forward(B, H, N, dk, dv, layout, state, dtype):
    g, dt = gen(N + dk), TORCH[dtype]
    q, k, v = (tokens(g, B, H, N, d, dt, layout) for d in (dk, dk, dv))
    s0 = normal(g, B, H, dk, dv) if state else None
    lg = decays(H)
    plan = mixers().LinearAttentionPlan(B, H, N, dk, dv, lg, dtype=dtype)
    o, s1 = plan.fwd(q, k, v, state=s0, final_state=True)
    want = linattn(q, k, v, lg, plan.scale, s0)
    big = linattn(*absolutes((q, k, v)), lg, plan.scale, *absolutes((s0,)))
    check(o, want[0], big[0], dtype, N, dk, "o")
    check(s1, want[1], big[1], "f32", N, dk, "state")
    alone = plan.fwd(q, k, v, state=s0)  # the states not asked for
    check(alone, want[0], big[0], dtype, N, dk, "o alone")
    assert plan.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,N,dk,dv", [(6, 3, 300, 64, 64), (5, 2, 700, 128, 96), (64, 6, 200, 64, 64)])
def test_linattn_lengths(B, H, N, dk, dv, dtype):
    """Rows behind a length may hold anything; o is zero there and the states are those at the length."""
    g, dt = gen(B), TORCH[dtype]
    lengths = torch.tensor(([0, N, 1, N // 2, 128, N + 9, -3] + list(range(B)))[:B], dtype=torch.int32, device="cuda")
    dead = torch.arange(N, device="cuda") >= lengths[:, None]
    ts = []
    for d in (dk, dk, dv, dv):
        t = tokens(g, B, H, N, d, dt, "bnhd")
        t.masked_fill_(dead[:, None, :, None], float("nan"))
        ts.append(t)
    q, k, v, do = ts
    q.masked_fill_((dead & (torch.arange(N, device="cuda") % 2 == 0))[:, None, :, None], float("inf"))
    s0, ds = normal(g, B, H, dk, dv), normal(g, B, H, dk, dv)
    lg = decays(H)
    plan = mixers().LinearAttentionPlan(B, H, N, dk, dv, lg, dtype=dtype)
    o, s1 = plan.fwd(q, k, v, state=s0, lengths=lengths, final_state=True)
    want = linattn(q, k, v, lg, plan.scale, s0, lengths)
    big = linattn(*absolutes((q, k, v)), lg, plan.scale, s0.abs(), lengths)
    check(o, want[0], big[0], dtype, N, dk, "o")
    check(s1, want[1], big[1], "f32", N, dk, "state")
    assert (o.masked_select(dead[:, None, :, None]) == 0).all()
    assert torch.equal(s1[0], s0[0])  # an empty row keeps its state
    got = plan.bwd(do, q, k, v, state=s0, dstate=ds, lengths=lengths)
    compare_gradients(got, (q, k, v, s0), do, ds, lg, plan.scale, lengths, dtype, N)
    for n in ("dq", "dk", "dv"):
        assert (got[n].masked_select(dead[:, None, :, None]) == 0).all()


def gradients(ts, do, ds, lg, scale, lengths):
    """dq, dk, dv, dstate by automatic differentiation of the plain form in 64 bits."""
    N = do.shape[2]
    n = None if lengths is None else lengths.long().clamp(0, N)
    live = 1 if n is None else (torch.arange(N, device="cuda") < n[:, None])[:, None, :, None]
    leaves = [None if t is None else (t if t.dim() < 4 or n is None or t.shape[2] != N else
                                      torch.where(live, t.double(), 0.0)).double().clone().requires_grad_() for t in ts]
    o, s = linattn(*leaves[:3], lg, scale, leaves[3], lengths)
    loss = (o * (do.double() if n is None else torch.where(live, do.double(), 0.0))).sum()
    if ds is not None:
        loss = loss + (s * ds.double()).sum()
    wrt = [t for t in leaves if t is not None]
    return torch.autograd.grad(loss, wrt)


def compare_gradients(got, ts, do, ds, lg, scale, lengths, dtype, N):
    want = gradients(ts, do, ds, lg, scale, lengths)
    # absolute values everywhere: all terms positive, so the gradients bound the terms
    big = gradients(absolutes(ts), do.double().abs(), *absolutes((ds,)), lg, scale, lengths)
    for name, w, b in zip(("dq", "dk", "dv", "dstate"), want, big):
        check(got[name], w, b, "f32" if name == "dstate" else dtype, N, 128, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,H,N,dk,dv,layout", SIZES)
def test_linattn_backward(B, H, N, dk, dv, layout, state, dtype):
    g, dt = gen(N + dv), TORCH[dtype]
    q, k, v, do = (tokens(g, B, H, N, d, dt, layout) for d in (dk, dk, dv, dv))
    s0, ds = (normal(g, B, H, dk, dv), normal(g, B, H, dk, dv)) if state else (None, None)
    lg = decays(H)
    plan = mixers().LinearAttentionPlan(B, H, N, dk, dv, lg, dtype=dtype)
    got = plan.bwd(do, q, k, v, state=s0, dstate=ds)
    compare_gradients(got, (q, k, v, s0), do, ds, lg, plan.scale, None, dtype, N)
    assert (got["dstate"] is None) == (not state)
    assert plan.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linattn_rows_whole_and_split(dtype):
    """A few rows more than fill the GPU: most run whole, the rest in segments."""
    g, dt = gen(50), TORCH[dtype]
    B, H, N, d = 50, 3, 1500, 128
    q, k, v, do = (tokens(g, B, H, N, d, dt, "bnhd") for _ in range(4))
    lg = decays(H, "slow")
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, lg, dtype=dtype)
    s0, ds = normal(g, B, H, d, d), normal(g, B, H, d, d)
    o, s1 = plan.fwd(q, k, v, state=s0, final_state=True)
    got = plan.bwd(do, q, k, v, state=s0, dstate=ds)
    for b in (0, 31, 48, 49):  # rows of either kind
        one = [t[b:b + 1] for t in (q, k, v)]
        want = linattn(*one, lg, plan.scale, s0[b:b + 1])
        big = linattn(*absolutes(one), lg, plan.scale, s0[b:b + 1].abs())
        check(o[b:b + 1], want[0], big[0], dtype, N, d, "o")
        check(s1[b:b + 1], want[1], big[1], "f32", N, d, "state")
        compare_gradients({n: t[b:b + 1] for n, t in got.items()}, (*one, s0[b:b + 1]), do[b:b + 1], ds[b:b + 1], lg,
                          plan.scale, None, dtype, N)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linattn_one_tensor_for_all_and_one_token_for_all(dtype):
    """q, k and v the same memory; a token repeated by a stride of zero; the same memory with two strides."""
    g, dt = gen(51), TORCH[dtype]
    B, H, N, d = 2, 3, 300, 64
    x = tokens(g, B, H, N, d, dt, "bnhd")
    one = normal(g, B, H, 1, d, dtype=dt).expand(B, H, N, d)
    heads = x[:, :1].expand(B, H, N, d)
    lg = decays(H)
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, lg, dtype=dtype)
    for q, k, v in ((x, x, x), (one, x, one), (x, heads, x), (heads, x, heads)):
        o, s = plan.fwd(q, k, v, final_state=True)
        want, big = linattn(q, k, v, lg, plan.scale), linattn(*absolutes((q, k, v)), lg, plan.scale)
        check(o, want[0], big[0], dtype, N, d, "o")
        check(s, want[1], big[1], "f32", N, d, "state")
        got = plan.bwd(x, q, k, v)
        compare_gradients(got, (q, k, v, None), x, None, lg, plan.scale, None, dtype, N)


def test_linattn_far_strides():
    """Tokens 2^25 elements apart: offsets past 32 bits, in elements and in bytes."""
    N, d, far = 140, 64, 1 << 25
    buf = torch.empty(N * far, dtype=torch.bfloat16, device="cuda")
    g = gen(52)
    base = normal(g, 1, 1, N, d, dtype=torch.bfloat16)
    views = [buf.as_strided((1, 1, N, d), (0, 0, far, 1), 64 * i) for i in range(4)]
    for t in views[:3]:
        t.copy_(base)
    plan = mixers().LinearAttentionPlan(1, 1, N, d, d, [-0.01])
    plan.fwd(*views[:3], o=views[3])
    assert torch.equal(views[3], plan.fwd(base, base, base))
    turn = mixers().RotaryPlan(d)
    pos = torch.arange(N, device="cuda")
    turn.apply(views[0], positions=pos, inplace=True)
    assert torch.equal(views[0], turn.apply(base, positions=pos))


def test_linattn_no_decay_and_full_decay():
    """a = 1 over thousands of tokens, and a = 0: o_t = scale (q_t . k_t) v_t."""
    g = gen(53)
    B, H, N, d = 1, 2, 5000, 64
    for dtype in ("bf16", "f32"):
        q, k, v = (tokens(g, B, H, N, d, TORCH[dtype], "bhnd") for _ in range(3))
        plan = mixers().LinearAttentionPlan(B, H, N, d, d, [0.0, -math.inf], dtype=dtype)
        o, s = plan.fwd(q, k, v, final_state=True)
        want, big = linattn(q, k, v, [0.0, -math.inf], plan.scale), linattn(*absolutes((q, k, v)), [0.0, -math.inf],
                                                                           plan.scale)
        check(o, want[0], big[0], dtype, N, d, "o")
        check(s, want[1], big[1], "f32", N, d, "state")


def test_linattn_wait_that_runs_out():
    """No probe allowed: the call gives up, says so once, and the plan works again afterwards."""
    g = gen(54)
    for B, H, N, d in ((1, 2, 1000, 128), (2, 8, 700, 64)):
        q, k, v = (tokens(g, B, H, N, d, torch.bfloat16, "bnhd") for _ in range(3))
        plan = mixers().LinearAttentionPlan(B, H, N, d, d, decays(H, "slow"))
        want = plan.fwd(q, k, v, final_state=True)
        assert plan.device_status() == 0
        plan.set_wait_limit(0)
        plan.fwd(q, k, v, final_state=True)
        assert plan.device_status() == 6 and plan.device_status() == 0
        plan.set_wait_limit(65536)
        got = plan.fwd(q, k, v, final_state=True)
        assert plan.device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_linattn_state_in_place_and_streams_at_once():
    """The final states may replace the initial ones; two streams use one plan at the same time."""
    import ctypes
    g = gen(55)
    B, H, N, d = 40, 4, 256, 64  # one segment: the states' kernel runs beside the outputs'
    m = mixers()
    plan = m.LinearAttentionPlan(B, H, N, d, d, decays(H, "slow"))
    q, k, v = (tokens(g, B, H, N, d, torch.bfloat16, "bnhd") for _ in range(3))
    s0 = normal(g, B, H, d, d)
    o, s1 = plan.fwd(q, k, v, state=s0, final_state=True)
    for _ in range(5):
        st, out = s0.clone(), torch.empty_like(v)
        shape = (B, H, N, d)
        a = m._FWD.pack(m._FWD.size, B, N, plan.scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                        *plan._view(q, "q", shape), *plan._view(k, "k", shape), *plan._view(v, "v", shape), 0,
                        st.data_ptr(), out.data_ptr(), *plan._view(out, "o", shape), st.data_ptr())
        assert plan.lib.fftconv_linattn_fwd(plan._handle, a, plan._workspace(0).data_ptr(), plan._stream(None)) == 0
        assert torch.equal(out, o) and torch.equal(st, s1)
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for s in side:
            with torch.cuda.stream(s):
                outs.append((plan.fwd(q, k, v, state=s0, final_state=True), plan.bwd(v, q, k, v, state=s0)))
    torch.cuda.synchronize()
    first = plan.bwd(v, q, k, v, state=s0)
    for (a, b), grads in outs:
        assert torch.equal(a, o) and torch.equal(b, s1)
        assert all(torch.equal(grads[n], first[n]) for n in first)


def test_linattn_backward_against_differences():
    """The operator is linear in each of q, k, v and the state: a central difference with step 1 is exact but for rounding."""
    g = gen(5)
    B, H, N, d = 2, 3, 150, 64
    ts = [normal(g, B, H, N, d) for _ in range(3)] + [normal(g, B, H, d, d)]
    do, ds = normal(g, B, H, N, d), normal(g, B, H, d, d)
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, decays(H, "slow"), dtype="f32")
    got = plan.bwd(do, *ts[:3], state=ts[3], dstate=ds)

    def loss(args):
        o, s = plan.fwd(*args[:3], state=args[3], final_state=True)
        return (o.double() * do).sum() + (s.double() * ds).sum()

    for i, name in enumerate(("dq", "dk", "dv", "dstate")):
        e = normal(g, *ts[i].shape)
        up, down = ([t + s * e if j == i else t for j, t in enumerate(ts)] for s in (1, -1))
        want = (loss(up) - loss(down)) / 2
        have = (got[name].double() * e).sum()
        # losses of thousands of terms of order sqrt(N d), each off by some 2^-24 of its sums
        terms = (got[name].double() * e).abs().sum()
        assert abs(want - have) <= 2.0 ** -24 * chain(N, d) * terms, (name, float(want), float(have))


def test_linattn_long_row():
    """Many chunks and segments, a slow decay: the last rows against a window of the plain form."""
    g = gen(9)
    B, H, N, d = 1, 2, 20000, 64
    q, k, v = (tokens(g, B, H, N, d, torch.bfloat16, "bnhd") for _ in range(3))
    lg = [math.log1p(-2.0 ** -6), 0.0]
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, lg)
    o, s = plan.fwd(q, k, v, final_state=True)
    # the window's first state by the plain form's state over what comes before
    cut = N - 700
    t = torch.arange(cut, device="cuda")
    w = torch.stack([torch.exp(x * (cut - 1 - t).double()) for x in torch.tensor(lg, dtype=torch.float64)])
    s0 = (k[:, :, :cut].double() * w[..., None]).transpose(-1, -2) @ v[:, :, :cut].double()
    a0 = (k[:, :, :cut].double().abs() * w[..., None]).transpose(-1, -2) @ v[:, :, :cut].double().abs()
    part = [x[:, :, cut:] for x in (q, k, v)]
    want, big = linattn(*part, lg, plan.scale, s0), linattn(*absolutes(part), lg, plan.scale, a0)
    check(o[:, :, cut:], want[0], big[0], "bf16", N, d, "o")
    check(s, want[1], big[1], "f32", N, d, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linattn_runs_agree_and_reuse(dtype):
    """Repeated calls agree bit for bit; a plan serves smaller calls; the state goes on from call to call."""
    g, dt = gen(3), TORCH[dtype]
    B, H, N, d = 3, 4, 500, 64
    q, k, v = (tokens(g, B, H, N, d, dt, "bnhd") for _ in range(3))
    lg = decays(H, "slow")
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, lg, dtype=dtype)
    o, s = plan.fwd(q, k, v, final_state=True)
    o2, s2 = plan.fwd(q, k, v, final_state=True)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    one, mid = plan.fwd(q[:, :, :201], k[:, :, :201], v[:, :, :201], final_state=True)
    two, end = plan.fwd(q[:, :, 201:], k[:, :, 201:], v[:, :, 201:], state=mid, final_state=True)
    want = linattn(q, k, v, lg, plan.scale)
    big = linattn(*absolutes((q, k, v)), lg, plan.scale)
    check(torch.cat((one, two), 2), want[0], big[0], dtype, N, d, "o in parts")
    check(end, want[1], big[1], "f32", N, d, "state in parts")


def test_linattn_writes_only_its_rows():
    """An output inside a larger buffer: nothing around it changes."""
    g = gen(4)
    B, H, N, d = 2, 3, 130, 64
    q, k, v = (tokens(g, B, H, N, d, torch.bfloat16, "bhnd") for _ in range(3))
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, decays(H))
    buf = torch.full((B, N + 2, H, d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    o = buf[:, 1:N + 1, :, 8:8 + d].transpose(1, 2)
    plan.fwd(q, k, v, o=o)
    assert torch.equal(o, plan.fwd(q, k, v))
    o.fill_(7.0)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 8, 8), (4, 12, 64, 64), (7, 3, 72, 104), (33, 4, 128, 128),
                                       (5, 2, 128, 8), (3, 2, 8, 128)])
def test_linattn_step(B, H, dk, dv, dtype):
    g, dt = gen(B), TORCH[dtype]
    wide = normal(g, B, H, 2 * dk + dv + 1, dtype=dt)  # one projection, odd strides
    q, k, v = wide[..., :dk], wide[..., dk:2 * dk], wide[..., 2 * dk:-1]
    pool = normal(g, B + 3, H, dk, dv)
    slots = torch.randperm(B + 3, generator=g, device="cuda")[:B].int()
    if B > 2:
        slots[1], slots[2] = -1, B + 3  # idle rows
    lg = decays(H)
    plan = mixers().LinearAttentionPlan(B, H, 1, dk, dv, lg, dtype=dtype)
    before, at = pool.clone(), slots.long().clamp(0, B + 2)
    idle = (slots < 0) | (slots >= B + 3)
    o = plan.step(q, k, v, pool, slots=slots)
    want = linattn(*(x.unsqueeze(2) for x in (q, k, v)), lg, plan.scale, before[at])
    big = linattn(*absolutes(x.unsqueeze(2) for x in (q, k, v)), lg, plan.scale, before[at].abs())
    keep = ~idle
    check(o[keep], want[0][keep].squeeze(2), big[0][keep].squeeze(2), dtype, 1, dk, "o")
    check(pool[slots[keep].long()], want[1][keep], big[1][keep], "f32", 1, dk, "state")
    assert (o[idle] == 0).all()
    untouched = torch.ones(B + 3, dtype=torch.bool, device="cuda")
    untouched[slots[keep].long()] = False
    assert torch.equal(pool[untouched], before[untouched])


def test_linattn_step_same_slot_in_row_order():
    g = gen(8)
    B, H, d = 300, 2, 64
    q, k, v = (normal(g, B, H, d) for _ in range(3))
    slots = torch.randint(0, 40, (B,), generator=g, device="cuda").int()
    pool = normal(g, 40, H, d, d)
    plan = mixers().LinearAttentionPlan(B, H, 1, d, d, decays(H, "slow"), dtype="f32")
    one, o = pool.clone(), []
    for b in range(B):
        o.append(plan.step(q[b:b + 1], k[b:b + 1], v[b:b + 1], one, slots=slots[b:b + 1]))
    got = plan.step(q, k, v, pool, slots=slots)
    assert torch.equal(got, torch.cat(o)) and torch.equal(pool, one)


def test_linattn_steps_follow_a_prompt():
    """A prompt's states, then single tokens: the whole row's outputs."""
    g = gen(2)
    B, H, N, d, more = 3, 4, 100, 64, 5
    q, k, v = (normal(g, B, H, N + more, d, dtype=torch.bfloat16) for _ in range(3))
    lg = decays(H, "slow")
    plan = mixers().LinearAttentionPlan(B, H, N, d, d, lg)
    _, state = plan.fwd(q[:, :, :N], k[:, :, :N], v[:, :, :N], final_state=True)
    got = torch.stack([plan.step(q[:, :, t], k[:, :, t], v[:, :, t], state) for t in range(N, N + more)], 2)
    want, big = linattn(q, k, v, lg, plan.scale), linattn(*absolutes((q, k, v)), lg, plan.scale)
    check(got, want[0][:, :, N:], big[0][:, :, N:], "bf16", N + more, d, "o")
    check(state, want[1], big[1], "f32", N + more, d, "state")


def test_linattn_is_a_state_space_filter():
    """Constant queries and keys turned by rotary positions: the filter Re sum_j c_j lam_j^t with
    lam_j = a e^{i theta_j}, which the state-space plan computes by FFT convolutions."""
    from fft_long_convolution_causal_b200 import binding
    B, H, N, rot, dv = 2, 3, 4096, 32, 8
    g = gen(1)
    lg = [math.log1p(-2.0 ** -(6 + h)) for h in range(H)]
    u = normal(g, B, H, N, dv)
    pairs = rot // 2
    theta = 10000.0 ** (-2.0 * torch.arange(pairs, dtype=torch.float64) / rot)
    lam = torch.exp(torch.tensor(lg, dtype=torch.float64))[:, None] * torch.polar(torch.ones_like(theta), theta)
    c = torch.linspace(0.2, 1.0, pairs, dtype=torch.float64).expand(H, pairs)
    m = mixers()
    turn = m.RotaryPlan(rot, dtype="f32")
    # q holds (c, 0), k holds (1, 0): q_t . k_s = sum_j c_j cos(theta_j (t - s))
    q = torch.zeros(1, 1, N, rot, device="cuda")
    k = torch.zeros(1, 1, N, rot, device="cuda")
    q[..., :pairs], k[..., :pairs] = c[0].cuda().float(), 1.0
    q, k = turn.apply(q, k, positions=torch.arange(N, device="cuda"))
    plan = m.LinearAttentionPlan(B, H, N, rot, dv, lg, dtype="f32", scale=1.0)
    o = plan.fwd(q.expand(B, H, N, rot), k.expand(B, H, N, rot), u)
    ssm = binding.SSMPlan(B, H, N, "f32", d_state=pairs, chunk=1024)
    khat = ssm.set_filters(lam, c.to(torch.complex128))
    for j in range(dv):
        want = ssm.fwd(u[..., j].contiguous(), khat)
        # the poles reach the state-space plan rounded to fp32: lam^t drifts by t 2^-24, weighed by the decay
        # (t a^t has its mean at 1 / (1 - a) <= 256): 256 2^-24 = 1.5e-5, and its own tolerance of 1e-5
        err = (o[..., j] - want).norm() / want.norm()
        assert err <= 2.6e-5, float(err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,H,H2,N,dim,rot", [(1, 1, 0, 1, 8, 8), (2, 4, 2, 33, 64, 64), (3, 5, 5, 7, 128, 96),
                                              (2, 3, 1, 40, 80, 54), (2, 2, 0, 9, 10, 6), (1, 32, 8, 260, 128, 128),
                                              (16, 12, 4, 1, 64, 32)])
def test_rotary(B, H, H2, N, dim, rot, layout, dtype):
    g, dt = gen(dim), TORCH[dtype]
    x = normal(g, B, N, H, dim, dtype=dt).transpose(1, 2)
    x2 = normal(g, B, H2, N, dim, dtype=dt) if H2 else None
    pos = torch.randint(0, 1 << 20, (B, N), generator=g, device="cuda")
    if N > 2:
        pos[0, 0], pos[0, 1], pos[0, 2] = 0, -5, (1 << 31) + 7
    for scaling, factor, inverse in (("none", 1.0, False), ("linear", 4.0, True), ("base", 8.0, False),
                                     ("parts", 8.0, True)):
        plan = mixers().RotaryPlan(dim, rot_dim=rot, layout=layout, dtype=dtype, scaling=scaling, factor=factor)
        got = plan.apply(x, x2, positions=pos, inverse=inverse)
        for y, t in zip(got if H2 else (got,), (x, x2)):
            want = rotary(t, pos, rot, layout, scaling=scaling, factor=factor, inverse=inverse)
            # one rounding of the result; before it the sine and cosine (angle off by at most 2^-25 of half a
            # turn, about 1e-7, two units in the last place of the functions, one of m) and three products
            size = want.abs() + 0
            pair = t.double().abs().amax(-1, keepdim=True) * 2 * (0.1 * math.log(factor) + 1)
            assert ((y.double() - want).abs() <= U[dtype] * size + 8 * 2.0 ** -24 * pair).all()
            assert torch.equal(y[..., rot:], t[..., rot:])


def test_rotary_in_place_shared_positions_and_back():
    g = gen(6)
    x = normal(g, 2, 3, 50, 64)
    pos = torch.arange(1000, 1050, device="cuda")
    plan = mixers().RotaryPlan(64, rot_dim=48, dtype="f32")
    want = plan.apply(x, positions=pos.expand(2, 50).contiguous())
    y = x.clone()
    assert plan.apply(y, positions=pos, inplace=True) is y
    assert torch.equal(y, want)
    back = plan.apply(y, positions=pos, inverse=True)
    # two rotations, each within 8 units of the pair's size
    assert ((back - x).abs() <= 16 * 2.0 ** -24 * 2 * x.abs().amax(-1, keepdim=True)).all()
    buf = torch.zeros(2, 3, 50, 80, device="cuda")  # a view inside a wider buffer
    buf[..., 8:72] = x
    plan.apply(buf[..., 8:72], positions=pos, inplace=True)
    assert torch.equal(buf[..., 8:72], want) and (buf[..., :8] == 0).all() and (buf[..., 72:] == 0).all()


def test_rotary_gradient_against_differences():
    """Linear in x: <R x, dy> = <x, R^T dy>."""
    g = gen(7)
    x, dy = normal(g, 2, 3, 50, 64), normal(g, 2, 3, 50, 64)
    pos = torch.randint(0, 1 << 18, (2, 50), generator=g, device="cuda")
    plan = mixers().RotaryPlan(64, dtype="f32", scaling="parts", factor=4.0, layout="interleaved")
    a = (plan.apply(x, positions=pos).double() * dy).sum()
    b = (plan.apply(dy, positions=pos, inverse=True).double() * x).sum()
    assert abs(a - b) <= 16 * 2.0 ** -24 * 2 * (x.abs() * dy.abs()).double().sum() * 2


ROWS = [(1, 1, 1), (3, 7, 1), (24, 64, 12), (5, 65, 1), (70, 128, 5), (33, 768, 1), (6, 1000, 2), (9, 2047, 1),
        (4, 4096, 1), (3, 8192, 1), (3, 5001, 3), (2, 16384, 1), (2, 16383, 1), (5000, 96, 10), (700, 256, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C,G", ROWS)
def test_layernorm(rows, C, G, dtype):
    g, dt = gen(C), TORCH[dtype]
    x = (normal(g, rows, C) * 2 + 5 * normal(g, rows, 1)).to(dt)
    dy = normal(g, rows, C, dtype=dt)
    w, b = 1 + 0.3 * normal(g, G, C), normal(g, G, C)
    eps = 1e-2  # keeps rows of one or two elements well conditioned
    plan = mixers().LayerNormPlan(rows, C, dtype=dtype, groups=G, eps=eps)
    y, mean, rstd = plan.fwd(x, w, b, statistics=True)
    leaves = [t.double().clone().requires_grad_() for t in (x, w, b)]
    want = layernorm(*leaves, eps)
    # x - mean is off by some log2(C) 2^-24 of the row's largest value, then scaled by rstd w
    steps = math.ceil(math.log2(C)) + 16
    x64 = x.double()
    wide = w.double().abs().repeat(rows // G, 1)
    rs = 1 / (x64.var(-1, unbiased=False, keepdim=True) + eps).sqrt()
    rel = steps * 2.0 ** -24 * (1 + x64.abs().amax(-1, keepdim=True) * rs)
    xh = (x64 - x64.mean(-1, keepdim=True)) * rs
    err = (y.double() - want.detach()).abs()
    bound = U[dtype] * want.detach().abs() + rel * (wide * (1 + xh.abs()) + b.double().abs().repeat(rows // G, 1))
    assert (err <= bound).all(), float((err - bound).max())
    assert torch.equal(y, plan.fwd(x, w, b))
    dx, dw, db = plan.bwd(dy, x, w, mean, rstd)
    wx, ww, wb = torch.autograd.grad(want, leaves, dy.double())
    gr = (dy.double() * w.double().repeat(rows // G, 1)).abs()
    size = gr + gr.mean(-1, keepdim=True) + xh.abs() * (gr * xh.abs()).mean(-1, keepdim=True)
    bound = U[dtype] * wx.abs() + 4 * rel * rs * (size + gr.amax(-1, keepdim=True))
    assert ((dx.double() - wx).abs() <= bound).all(), float(((dx.double() - wx).abs() - bound).max())
    # sums over rows in 32 bits: a few hundred additions in line, then blocks
    n = (rows // G) / 296 + 64 + steps
    bw = (n * 2.0 ** -24 * dy.double().abs() * xh.abs() + rel * dy.double().abs()).unflatten(0, (-1, G)).sum(0)
    assert ((dw.double() - ww).abs() <= bw).all()
    bb = n * 2.0 ** -24 * dy.double().abs().unflatten(0, (-1, G)).sum(0)
    assert ((db.double() - wb).abs() <= bb).all()
    again = plan.bwd(dy, x, w, mean, rstd)
    assert all(torch.equal(s, t) for s, t in zip((dx, dw, db), again))


def test_layernorm_far_mean_and_shapes():
    """A mean a thousand times the spread (no cancellation in the variance); [..., C] shapes; a [C] weight."""
    g = gen(11)
    x = 1000 + normal(g, 4, 5, 6, 256)
    plan = mixers().LayerNormPlan(4 * 5 * 6, 256, dtype="f32", eps=0.0)
    w, b = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
    y = plan.fwd(x, w, b)
    want = layernorm(x.reshape(-1, 256), w[None], b[None], 0.0).reshape(x.shape)
    # x itself is exact; the mean is off by at most 24 2^-24 of 1000
    assert (y.double() - want).abs().max() <= 24 * 2.0 ** -24 * 1000 * 1.5
    one = plan.fwd(x[0, 0], w, b)
    assert torch.equal(one, y[0, 0])


def test_layernorm_against_differences():
    g = gen(12)
    x, dy = normal(g, 6, 200), normal(g, 6, 200)
    w, b = 1 + 0.3 * normal(g, 2, 200), normal(g, 2, 200)
    plan = mixers().LayerNormPlan(6, 200, dtype="f32", groups=2)
    _, mean, rstd = plan.fwd(x, w, b, statistics=True)
    got = plan.bwd(dy, x, w, mean, rstd)
    for i, t in enumerate((x, w, b)):
        e, h = normal(g, *t.shape), 2.0 ** -6
        loss = [(plan.fwd(*[u + s * h * e if j == i else u for j, u in enumerate((x, w, b))]).double() * dy).sum()
                for s in (1, -1)]
        want, have = (loss[0] - loss[1]) / (2 * h), (got[i].double() * e).sum()
        # 1200 terms rounded at 2^-23, over 2h; the third derivative's h^2 / 6 on a row of unit spread
        assert abs(want - have) <= 1200 ** 0.5 * 16 * 2.0 ** -23 / (2 * h) + 4 * h * h * (dy.norm() * e.norm()) / 6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_retention_together(dtype):
    """Rotary, attention and norm as a layer runs them: forward, gradients, then single tokens."""
    g, dt = gen(21), TORCH[dtype]
    B, H, N, dk, dv, more = 2, 4, 150, 64, 64, 3
    q, k, v = (normal(g, B, N + more, H, d, dtype=dt).transpose(1, 2) for d in (dk, dk, dv))
    w, b = 1 + 0.2 * normal(g, H, dv), 0.2 * normal(g, H, dv)
    pos = torch.arange(N + more, device="cuda").expand(B, N + more).contiguous() + 7
    plan = mixers().RetentionPlan(B, H, N, dk, dv, dtype=dtype, rotary=dict(scaling="linear", factor=2.0))
    lg = [math.log1p(-2.0 ** (-5.0 - h)) for h in range(H)]

    def plain(q, k, v, w, b, pos):
        qr, kr = (rotary(t, pos, dk, scaling="linear", factor=2.0) for t in (q, k))
        o, s = linattn(qr, kr, v, lg, dk ** -0.5)
        B, H, N, _ = o.shape
        rows = o.transpose(1, 2).reshape(-1, dv)
        return layernorm(rows, w, b, 1e-5).reshape(B, N, H, dv), s

    cut = [t[:, :, :N] for t in (q, k, v)]
    y, state, saved = plan.fwd(*cut, w, b, pos[:, :N].contiguous(), final_state=True, save=True)
    leaves = [t.double().clone().requires_grad_() for t in (*cut, w, b)]

    class Double(torch.autograd.Function):  # rotary's plain form copies in place: its transpose by hand
        @staticmethod
        def forward(ctx, t, pos):
            ctx.pos = pos
            return rotary(t, pos, dk, scaling="linear", factor=2.0)

        @staticmethod
        def backward(ctx, d):
            return rotary(d, ctx.pos, dk, scaling="linear", factor=2.0, inverse=True), None

    qr, kr = (Double.apply(t, pos[:, :N]) for t in leaves[:2])
    o, s = linattn(qr, kr, leaves[2], lg, dk ** -0.5)
    want = layernorm(o.transpose(1, 2).reshape(-1, dv), leaves[3], leaves[4], 1e-5).reshape(B, N, H, dv)
    # in the 2-norm: bf16 rounds q, k, the scores, the state's copy, o and y, each rms 2^-8 / sqrt 3, and the
    # gradients twice as many; fp32 sums a few hundred terms
    tol = 2.0 ** -8 * (12 / 3) ** 0.5 * 2 if dtype == "bf16" else 2.0 ** -24 * 64

    def near(x, y, what):
        rel = float((x.double() - y).norm() / y.norm())
        assert rel <= tol, (what, rel)

    near(y, want.detach(), "y")
    near(state, s.detach(), "state")
    dy = normal(g, B, N, H, dv, dtype=dt)
    got = plan.bwd(dy, saved, w)
    for name, t in zip(("dq", "dk", "dv", "dweight", "dbias"),
                       torch.autograd.grad(want, leaves, dy.double())):
        near(got[name], t, name)
    full, _ = plain(q, k, v, w, b, pos)
    for t in range(N, N + more):
        yt = plan.step(q[:, :, t], k[:, :, t], v[:, :, t], w, b, pos[:, t].contiguous(), state)
        near(yt, full[:, t], "step")


def test_capture_and_streams():
    """Captured forward, backward and step calls replay on new inputs; two captured graphs and an eager call on
    a side stream share no scratch memory."""
    g = gen(31)
    B, H, N, d = 2, 4, 400, 64
    m = mixers()
    lg = decays(H, "slow")
    plan = m.LinearAttentionPlan(B, H, N, d, d, lg)
    turn, norm = m.RotaryPlan(d), m.LayerNormPlan(B * N * H, d, groups=H)
    w, b = torch.ones(H, d, device="cuda"), torch.zeros(H, d, device="cuda")
    pos = torch.arange(N, device="cuda")

    def inputs():
        return [normal(g, B, N, H, d, dtype=torch.bfloat16).transpose(1, 2) for _ in range(4)]

    def body(q, k, v, do):
        qr, kr = turn.apply(q, k, positions=pos)
        o, s = plan.fwd(qr, kr, v, final_state=True)
        rows = o.transpose(1, 2).contiguous()
        y, mean, rstd = norm.fwd(rows, w, b, statistics=True)
        dx, dw, db = norm.bwd(do.transpose(1, 2).contiguous(), rows, w, mean, rstd)
        grads = plan.bwd(dx.transpose(1, 2), qr, kr, v)
        st = s.clone()
        last = plan.step(q[:, :, 0], k[:, :, 0], v[:, :, 0], st)
        return [y, s, dx, dw, db, grads["dq"], grads["dk"], grads["dv"], last, st]

    a, c = inputs(), inputs()
    body(*a)
    torch.cuda.synchronize()
    graphs = []
    for x in (a, c):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = body(*x)
        graphs.append((gr, x, out))
    for gr, x, _ in graphs:
        for t in x:
            t.copy_(normal(g, B, N, H, d, dtype=torch.bfloat16).transpose(1, 2))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
            extra = body(*graphs[0][1])
    torch.cuda.synchronize()
    for gr, x, out in graphs:
        assert all(torch.equal(s, t) for s, t in zip(out, body(*x)))
    assert all(torch.equal(s, t) for s, t in zip(extra, graphs[0][2]))
    # the stream argument: work and allocations on it
    torch.cuda.synchronize()
    o = plan.fwd(*a[:3], stream=side)
    side.synchronize()
    assert torch.equal(o, plan.fwd(*a[:3]))


def test_refusals_on_the_device():
    m = mixers()
    from fft_long_convolution_causal_b200 import binding
    plan = m.LinearAttentionPlan(2, 3, 64, 64, 64, decays(3))
    x = torch.zeros(2, 3, 64, 64, dtype=torch.bfloat16, device="cuda")
    bad = [(x.float(), x, x), (x, x[:1], x), (x[:, :2], x[:, :2], x[:, :2]), (x[..., :32], x, x),
           (x.cpu(), x.cpu(), x.cpu()), (torch.cat((x, x)),) * 3, (torch.cat((x, x), 2),) * 3,
           (x.transpose(2, 3), x, x)]
    for q, k, v in bad:
        with pytest.raises(ValueError):
            plan.fwd(q, k, v)
    wide = torch.zeros(2, 3, 64, 68, dtype=torch.bfloat16, device="cuda")
    for t in (wide[..., 2:66], wide[..., :64]):  # not on 16 bytes; strides of 68 elements
        with pytest.raises(binding.FFTConvError) as e:
            plan.fwd(t, x, x)
        assert e.value.status == 1
    with pytest.raises(binding.FFTConvError):  # an output that is an input
        plan.fwd(x, x.clone(), x.clone(), o=x)
    with pytest.raises(binding.FFTConvError):  # an output shared by the heads
        plan.fwd(x, x, x, o=x[:, :1].expand(2, 3, 64, 64))
    with pytest.raises(ValueError):
        plan.fwd(x, x, x, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        plan.fwd(x, x, x, state=torch.zeros(2, 3, 64, 32, device="cuda"))
    with pytest.raises(ValueError):
        plan.step(x[:, :, 0], x[:, :, 0], x[:, :, 0], torch.zeros(1, 3, 64, 64, device="cuda"))
    with pytest.raises(ValueError):
        plan.step(x[:, :, 0], x[:, :, 0], x[:, :, 0], torch.zeros(2, 3, 64, 64, device="cuda").transpose(2, 3))
    turn = m.RotaryPlan(64)
    with pytest.raises(ValueError):
        turn.apply(x)
    with pytest.raises(ValueError):
        turn.apply(x, positions=torch.zeros(2, 64, dtype=torch.int32, device="cuda"))
    with pytest.raises(binding.FFTConvError):  # in place, a head shared by all
        turn.apply(x[:, :1].expand(2, 3, 64, 64), positions=torch.arange(64, device="cuda"), inplace=True)
    norm = m.LayerNormPlan(12, 64, groups=3)
    y = torch.zeros(12, 64, dtype=torch.bfloat16, device="cuda")
    for rows in (y[:4], torch.cat((y, y)), y.t().contiguous().t()):
        with pytest.raises(ValueError):
            norm.fwd(rows, torch.ones(3, 64, device="cuda"), torch.zeros(3, 64, device="cuda"))
    with pytest.raises(ValueError):
        norm.fwd(y, torch.ones(64, device="cuda"), torch.zeros(64, device="cuda"))


def test_refusals_of_scales_and_of_one_tensor_turned_twice():
    m = mixers()
    from fft_long_convolution_causal_b200 import binding
    x = torch.zeros(2, 3, 64, 64, dtype=torch.bfloat16, device="cuda")
    plan = m.LinearAttentionPlan(2, 3, 64, 64, 64, decays(3), scale=1e39)  # finite, but not in fp32
    with pytest.raises(binding.FFTConvError):
        plan.fwd(x, x, x)
    with pytest.raises(binding.FFTConvError):
        plan.bwd(x, x, x, x)
    with pytest.raises(binding.FFTConvError):
        plan.step(x[:, :, 0], x[:, :, 0], x[:, :, 0], torch.zeros(2, 3, 64, 64, device="cuda"))
    turn, at = m.RotaryPlan(64), torch.arange(64, device="cuda")
    with pytest.raises(binding.FFTConvError):
        turn.apply(x, x, positions=at, inplace=True)
    a, b = turn.apply(x, x, positions=at)  # to two outputs
    assert a.data_ptr() != b.data_ptr()


def test_nonfinite_values_stay_in_their_row_and_behind_their_chunk():
    """A NaN in v reaches its own row and head from its chunk on, nothing else."""
    m = mixers()
    for dtype, chunk in (("bf16", 128), ("f32", 64)):
        t = torch.bfloat16 if dtype == "bf16" else torch.float32
        g = torch.Generator().manual_seed(5)
        q, k, v = (torch.randn(2, 2, 400, 64, generator=g).to(t).cuda() for _ in range(3))
        plan = m.LinearAttentionPlan(2, 2, 400, 64, 64, decays(2), dtype=dtype)
        clean = plan.fwd(q, k, v)
        at = chunk + 7
        v[1, 0, at] = float("nan")
        o = plan.fwd(q, k, v)
        assert torch.equal(o[0], clean[0]) and torch.equal(o[1, 1], clean[1, 1])
        assert torch.equal(o[1, 0, :chunk], clean[1, 0, :chunk])
        assert torch.isnan(o[1, 0, at:]).all()


UNALIGNED = [(1, 1, 1), (7, 3, 7), (39999, 21, 3), (4000, 13, 1000), (5000, 55, 1), (1776 * 3, 131, 1), (14 * 300, 557, 14),
             (2000, 761, 1), (900, 762, 1), (12 * 75, 1021, 12), (601, 1018, 1), (333, 2042, 1), (23 * 20, 1541, 23),
             (310, 3058, 1), (160, 8185, 1), (170, 8186, 1), (23 * 9, 5001, 23), (150, 16383, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,C,G", UNALIGNED)
def test_layernorm_rows_off_16_bytes(rows, C, G, dtype):
    """Rows that start anywhere in a 16-byte piece, walked in several steps, on one and on several warps."""
    test_layernorm(rows, C, G, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layernorm_in_place_and_within_its_rows(dtype):
    g, dt = gen(31), TORCH[dtype]
    for rows, C in ((700, 37), (300, 557), (200, 768), (150, 2050)):
        room = torch.full((rows * C + 64,), 7.0, dtype=dt, device="cuda")
        x = normal(g, rows, C, dtype=dt)
        w, b = 1 + 0.3 * normal(g, 1, C), normal(g, 1, C)
        plan = mixers().LayerNormPlan(rows, C, dtype=dtype)
        y = plan.fwd(x, w, b)
        at = room[:rows * C].view(rows, C)
        assert plan.fwd(x, w, b, y=at) is at and torch.equal(at, y) and (room[rows * C:] == 7).all()
        z = x.clone()
        assert torch.equal(plan.fwd(z, w, b, y=z), y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot", [(8, 2), (8, 6), (16, 10), (16, 14)] + [(40, r) for r in range(2, 41, 2)]
                         + [(128, 90), (128, 92), (128, 126), (256, 30), (256, 254)])
def test_rotary_parts_of_a_head(dim, rot, layout, dtype):
    """Rotated parts that end, or have their half, inside a 16-byte piece; in place the same, the rest as it was."""
    if rot > 2:  # one pair has no scaled base
        test_rotary(2, 9, 2, 17, dim, rot, layout, dtype)
    g, dt = gen(rot), TORCH[dtype]
    x = normal(g, 2, 9, 17, dim, dtype=dt)
    if rot < dim:
        x[..., rot], x[..., -1] = float("inf"), float("nan")
    pos = torch.arange(17, device="cuda") + 5
    plan = mixers().RotaryPlan(dim, rot_dim=rot, layout=layout, dtype=dtype)
    y = plan.apply(x, positions=pos)
    bits = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(y[..., rot:].view(bits), x[..., rot:].view(bits)) and torch.isfinite(y[..., :rot]).all()
    z = x.clone()
    plan.apply(z, positions=pos, inplace=True)
    assert torch.equal(z.view(bits), y.view(bits))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layernorm_more_weight_rows_than_sms(dtype):
    for rows, C, G in ((400, 64, 200), (600, 2048, 300), (1200, 67, 600)):
        test_layernorm(rows, C, G, dtype)
