"""Cases of the sequence-mixer operators: linear attention with a decay for each head (prompts, single tokens,
gradients), rotary positions and layer norm.

`listed()` gives fixed cases, `draw(rng)` more of the same ranges; `prepare` makes the inputs a program holds before
the call, `run` makes one pass: with `own` false in elementary torch operations in 32 bits, with `own` true through
the package's plans.  `exact` is the definition in 64 bits."""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
CHUNK = 64  # tokens a chunk of the plain form


def listed():
    return [
        # a chat turn of a few dozen tokens, one request: latency
        dict(name="prompt_short_bf16", op="la_fwd", B=1, H=12, N=37, dk=64, dv=64, dtype="bf16", heads_first=False,
             state=False, ragged=False),
        # one long document: few rows, many tokens
        dict(name="prompt_long_bf16", op="la_fwd", B=1, H=16, N=32768, dk=128, dv=128, dtype="bf16",
             heads_first=False, state=False, ragged=False),
        # a padded batch of prompts that go on from saved states
        dict(name="prompt_ragged_bf16", op="la_fwd", B=8, H=12, N=4096, dk=64, dv=64, dtype="bf16",
             heads_first=False, state=True, ragged=True),
        # the same layer in single precision
        dict(name="prompt_f32", op="la_fwd", B=2, H=12, N=4096, dk=64, dv=64, dtype="f32", heads_first=True,
             state=False, ragged=False),
        # a training step's gradients
        dict(name="train_bf16", op="la_bwd", B=4, H=16, N=4096, dk=128, dv=128, dtype="bf16", heads_first=False,
             state=False, ragged=False),
        # gradients at odd sizes, in single precision, with states and a padded batch
        dict(name="train_odd_f32", op="la_bwd", B=3, H=5, N=1023, dk=40, dv=104, dtype="f32", heads_first=True,
             state=True, ragged=True),
        # single tokens: a few streams, where latency counts
        dict(name="step_few_bf16", op="la_step", B=4, H=12, dk=64, dv=64, dtype="bf16", pool=4, idle=0.0),
        # single tokens: a full server, rows spread over a pool of states, some idle
        dict(name="step_many_bf16", op="la_step", B=256, H=16, dk=128, dv=128, dtype="bf16", pool=320, idle=0.05),
        # queries and keys of a training batch
        dict(name="rotary_train_bf16", op="rotary", B=4, N=4096, H=16, Hk=16, D=128, rot=128, layout="half",
             scaling="none", factor=1.0, far=0, inverse=False, dtype="bf16"),
        # single tokens at far positions, scaled for a long context, part of the head
        dict(name="rotary_far_f32", op="rotary", B=16, N=1, H=12, Hk=4, D=64, rot=32, layout="interleaved",
             scaling="parts", factor=8.0, far=1 << 20, inverse=False, dtype="f32"),
        # a block's norm, forward and backward, over a training batch
        dict(name="norm_train_bf16", op="norm_train", rows=32768, C=768, groups=1, dtype="bf16"),
        # the norm behind each head, in single precision
        dict(name="norm_heads_f32", op="norm_fwd", rows=4096 * 12, C=64, groups=12, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_step", "rotary", "norm_fwd", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("la_fwd", "la_bwd"):
        most = 16 * 32768 * 128 if op == "la_fwd" else 4 * 16 * 4096 * 128
        if dtype == "f32":
            most //= 8
        while True:
            B, H, N = _log(rng, 1, 16), _log(rng, 1, 32), _log(rng, 1, 32768)
            dk, dv = 8 * rng.randint(2, 16), 8 * rng.randint(2, 16)
            if B * H * N * max(dk, dv) <= most:
                break
        return dict(op=op, B=B, H=H, N=N, dk=dk, dv=dv, dtype=dtype, heads_first=rng.random() < 0.5,
                    state=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "la_step":
        B = _log(rng, 1, 256)
        return dict(op=op, B=B, H=_log(rng, 1, 16), dk=8 * rng.randint(2, 16), dv=8 * rng.randint(2, 16),
                    dtype=dtype, pool=B + rng.randint(0, 64), idle=rng.choice([0.0, 0.1, 0.3]))
    if op == "rotary":
        while True:
            B, N, H = _log(rng, 1, 16), _log(rng, 1, 8192), _log(rng, 1, 32)
            Hk, D = max(1, H // rng.choice([1, 2, 4])), 8 * rng.randint(2, 32)
            if B * N * (H + Hk) * D * SIZE[dtype] <= 4 * 4096 * 32 * 128 * 2:
                break
        return dict(op=op, B=B, N=N, H=H, Hk=Hk, D=D, rot=2 * rng.randint(2, D // 2),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "parts"]), factor=rng.choice([2.0, 4.0, 32.0]),
                    far=rng.choice([0, 100000, 1 << 24]), inverse=rng.random() < 0.5, dtype=dtype)
    groups = rng.choice([1, 1, rng.randint(2, 32)])
    while True:
        rows, C = _log(rng, 1, 1 << 17), _log(rng, 16, 8192)
        if rows * C * SIZE[dtype] <= 32768 * 768 * 2:
            break
    return dict(op=op, rows=max(1, rows // groups) * groups, C=C, groups=groups, dtype=dtype)


def _log_decay(H):
    """Decays 1 - 2^-5 ... 1 - 2^-12, spread over the heads."""
    return [math.log1p(-2.0 ** (-5.0 - 7.0 * h / max(1, H - 1))) for h in range(H)]


def _frequencies(case):
    """Radians per position of each pair, and the factor on the rotated values."""
    rot, factor, base, context = case["rot"], case["factor"], 10000.0, 4096
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "base":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":
        # turns over the trained context: above 32 kept, below 1 interpolated, a ramp over the index between
        at = [rot * math.log(context / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(0.0, math.floor(at[0])), min(rot - 1.0, math.ceil(at[1]))
        keep = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, t=dtype, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)

    s = dict(case=case)
    op = case["op"]
    if op in ("la_fwd", "la_bwd"):
        B, H, N, dk, dv = (case[n] for n in ("B", "H", "N", "dk", "dv"))

        def tokens(d):
            return normal(B, H, N, d) if case["heads_first"] else normal(B, N, H, d).transpose(1, 2)

        s.update(q=tokens(dk), k=tokens(dk), v=tokens(dv), scale=dk ** -0.5, log_decay=_log_decay(H))
        s["g"] = torch.tensor(s["log_decay"], dtype=torch.float64, device="cuda")
        s["state"] = normal(B, H, dk, dv, t=torch.float32) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = torch.tensor([N] + [rng.randint(0, N) for _ in range(B - 1)], dtype=torch.int32,
                                        device="cuda")
        if op == "la_bwd":
            s["do"] = tokens(dv)
            s["dstate"] = normal(B, H, dk, dv, t=torch.float32) if case["state"] else None
        if own:
            from fft_long_convolution_causal_b200 import LinearAttentionPlan
            s["plan"] = LinearAttentionPlan(B, H, N, dk, dv, s["log_decay"], dtype=case["dtype"])
    elif op == "la_step":
        B, H, dk, dv, pool = (case[n] for n in ("B", "H", "dk", "dv", "pool"))
        s.update(q=normal(B, H, dk), k=normal(B, H, dk), v=normal(B, H, dv), scale=dk ** -0.5,
                 log_decay=_log_decay(H), state=normal(pool, H, dk, dv, t=torch.float32))
        s["g"] = torch.tensor(s["log_decay"], dtype=torch.float64, device="cuda")
        rows = rng.sample(range(pool), B)
        s["slots"] = torch.tensor([-1 if rng.random() < case["idle"] else r for r in rows], dtype=torch.int32,
                                  device="cuda")
        if own:
            from fft_long_convolution_causal_b200 import LinearAttentionPlan
            s["plan"] = LinearAttentionPlan(B, H, 1, dk, dv, s["log_decay"], dtype=case["dtype"])
    elif op == "rotary":
        B, N, H, Hk, D = (case[n] for n in ("B", "N", "H", "Hk", "D"))
        s.update(q=normal(B, N, H, D).transpose(1, 2), k=normal(B, N, Hk, D).transpose(1, 2))
        first = torch.tensor([rng.randint(0, case["far"]) for _ in range(B)], dtype=torch.int64, device="cuda")
        s["positions"] = first[:, None] + torch.arange(N, device="cuda")
        s["frequencies"], s["magnitude"] = _frequencies(case)
        s["frequencies"] = s["frequencies"].cuda()
        if own:
            from fft_long_convolution_causal_b200 import RotaryPlan
            s["plan"] = RotaryPlan(D, rot_dim=case["rot"], layout=case["layout"], dtype=case["dtype"],
                                   scaling=case["scaling"], factor=case["factor"], context=4096)
    else:
        rows, C, G = case["rows"], case["C"], case["groups"]
        x = normal(rows, C, t=torch.float32)
        # activations as a block meets them: each column with a spread and an offset of its own
        x = x * (0.5 + torch.rand(C, generator=g, device="cuda")) + normal(C, t=torch.float32)
        s["x"] = x.to(dtype)
        s["weight"] = 1 + normal(G, C, t=torch.float32, scale=0.1)
        s["bias"] = normal(G, C, t=torch.float32, scale=0.1)
        s["eps"] = 1e-5
        if op == "norm_train":
            s["dy"] = normal(rows, C)
        if own:
            from fft_long_convolution_causal_b200 import LayerNormPlan
            s["plan"] = LayerNormPlan(rows, C, dtype=case["dtype"], groups=G, eps=1e-5)
    return s


# ---------------------------------------------------------------- plain forms
def _powers(g, exponents):
    """a_h^e = exp(g_h e) as [H, ...] for integer exponents e >= 0, by 64-bit exponents."""
    return torch.exp(g.reshape(-1, *([1] * exponents.dim())) * exponents.double()).float()


def _mix(x, y, z, g):
    """sum_{s <= t} a^(t-s) (x_t . y_s) z_s for [B, H, N, d] in chunks: masked scores inside a chunk, chunk states
    joined over the chunks by one lower-triangular product."""
    B, H, N, _ = x.shape
    n = -(-N // CHUNK)
    x, y, z = (torch.nn.functional.pad(t, (0, 0, 0, n * CHUNK - N)).reshape(B, H, n, CHUNK, -1) for t in (x, y, z))
    i = torch.arange(CHUNK, device="cuda")
    c = torch.arange(n, device="cuda")
    inside = (_powers(g, (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i))[:, None]
    out = (x @ y.transpose(-1, -2) * inside) @ z
    if n > 1:
        ends = (y * _powers(g, CHUNK - 1 - i)[:, None, :, None]).transpose(-1, -2) @ z
        join = _powers(g, (CHUNK * (c[:, None] - 1 - c)).clamp(min=0)) * (c[:, None] > c)
        states = (join @ ends.reshape(B, H, n, -1)).reshape(ends.shape)
        out = out + (x @ states) * _powers(g, i + 1)[:, None, :, None]
    return out.reshape(B, H, n * CHUNK, -1)[:, :, :N]


def _masked(s, names):
    """The named tensors in 32 bits with the rows behind each length zero, and the lengths."""
    N = s["q"].shape[2]
    lengths = s["lengths"] if s["lengths"] is not None else torch.full((s["q"].shape[0],), N, device="cuda")
    live = (torch.arange(N, device="cuda") < lengths[:, None])[:, None, :, None]
    return [torch.where(live, s[n].float(), 0.0) for n in names], lengths, live


def _run_fwd(s):
    (q, k, v), lengths, live = _masked(s, "qkv")
    t = torch.arange(q.shape[2], device="cuda")
    to_end = _powers(s["g"], (lengths[:, None] - 1 - t).clamp(min=0)).transpose(0, 1)  # [B, H, N]
    o = _mix(q, k, v, s["g"])
    state = (k * to_end[..., None]).transpose(-1, -2) @ v
    if s["state"] is not None:
        o = o + (q @ s["state"]) * _powers(s["g"], t + 1)[None, ..., None]
        state = state + _powers(s["g"], lengths).transpose(0, 1)[..., None, None] * s["state"]
    return {"o": (o * s["scale"]).to(s["q"].dtype), "state": state}


def _run_bwd(s):
    (q, k, v, do), lengths, live = _masked(s, ["q", "k", "v", "do"])
    t = torch.arange(q.shape[2], device="cuda")
    do = do * s["scale"]
    dq = _mix(do, v, k, s["g"])
    dk = _mix(v.flip(2), do.flip(2), q.flip(2), s["g"]).flip(2)
    dv = _mix(k.flip(2), q.flip(2), do.flip(2), s["g"]).flip(2)
    from_start = _powers(s["g"], t + 1)[None, ..., None]
    out = {}
    if s["state"] is not None:
        to_end = _powers(s["g"], (lengths[:, None] - 1 - t).clamp(min=0)).transpose(0, 1)[..., None] * live
        dq = dq + from_start * (do @ s["state"].transpose(-1, -2))
        dk = dk + to_end * (v @ s["dstate"].transpose(-1, -2))
        dv = dv + to_end * (k @ s["dstate"])
        out["dstate"] = (q * from_start).transpose(-1, -2) @ do + \
            _powers(s["g"], lengths).transpose(0, 1)[..., None, None] * s["dstate"]
    dtype = s["q"].dtype
    return {"dq": dq.to(dtype), "dk": dk.to(dtype), "dv": dv.to(dtype), **out}


def _run_step(s):
    slots, state = s["slots"].long(), s["state"]
    q, k, v = (s[n].float() for n in "qkv")
    hit = torch.arange(state.shape[0], device="cuda")[:, None] == slots  # [pool, B]
    live, row = hit.any(1)[:, None, None, None], hit.int().argmax(1)
    decay = _powers(s["g"], torch.ones((), device="cuda"))[:, None, None]
    state.copy_(torch.where(live, decay * state + k[row][..., None] * v[row][..., None, :], state))
    o = (q[..., None, :] @ state[slots.clamp(min=0)])[..., 0, :] * s["scale"]
    return {"o": torch.where((slots >= 0)[:, None, None], o, 0.0).to(s["q"].dtype), "state": state}


def _rotated(x, cos, sin, case):
    rot = case["rot"]
    x, rest = x.float()[..., :rot], x[..., rot:]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((y.to(rest.dtype), rest), -1)


def _run_rotary(s):
    # positions reach millions of radians: the angle in 64 bits
    angle = s["positions"][:, None, :, None].double() * s["frequencies"]
    cos, sin = (angle.cos() * s["magnitude"]).float(), (angle.sin() * s["magnitude"]).float()
    if s["case"]["inverse"]:
        sin = -sin
    return {n: _rotated(s[n], cos, sin, s["case"]) for n in "qk"}


def _run_norm(s):
    x = s["x"].float()
    rows, C = x.shape
    w, b = s["weight"], s["bias"]
    G = w.shape[0]
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"])
    xh = c * rstd
    y = (xh.reshape(-1, G, C) * w + b).reshape(rows, C).to(s["x"].dtype)
    if "dy" not in s:
        return {"y": y}
    dy = s["dy"].float()
    gr = (dy.reshape(-1, G, C) * w).reshape(rows, C)
    dx = rstd * (gr - gr.mean(-1, keepdim=True) - xh * (gr * xh).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(s["x"].dtype), "dweight": (dy * xh).reshape(-1, G, C).sum(0),
            "dbias": dy.reshape(-1, G, C).sum(0)}


def _run_own(s):
    op, plan = s["case"]["op"], s["plan"]
    if op == "la_fwd":
        o, state = plan.fwd(s["q"], s["k"], s["v"], state=s["state"], lengths=s["lengths"], final_state=True)
        return {"o": o, "state": state}
    if op == "la_bwd":
        got = plan.bwd(s["do"], s["q"], s["k"], s["v"], state=s["state"], dstate=s["dstate"], lengths=s["lengths"])
        return {n: t for n, t in got.items() if t is not None}
    if op == "la_step":
        return {"o": plan.step(s["q"], s["k"], s["v"], s["state"], slots=s["slots"]), "state": s["state"]}
    if op == "rotary":
        q, k = plan.apply(s["q"], s["k"], positions=s["positions"], inverse=s["case"]["inverse"])
        return {"q": q, "k": k}
    if op == "norm_fwd":
        return {"y": plan.fwd(s["x"], s["weight"], s["bias"])}
    y, mean, rstd = plan.fwd(s["x"], s["weight"], s["bias"], statistics=True)
    dx, dw, db = plan.bwd(s["dy"], s["x"], s["weight"], mean, rstd)
    return {"y": y, "dx": dx, "dweight": dw, "dbias": db}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "la_fwd":
        return _run_fwd(state)
    if op == "la_bwd":
        return _run_bwd(state)
    if op == "la_step":
        return _run_step(state)
    if op == "rotary":
        return _run_rotary(state)
    return _run_norm(state)


def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op in ("la_fwd", "la_bwd"):
        B, H, N, dk, dv = (case[n] for n in ("B", "H", "N", "dk", "dv"))
        # a padded batch's lengths are spread evenly, the first row full
        live = H * ((N + (B - 1) * N / 2) if case["ragged"] else B * N)
        states = B * H * dk * dv * 4
        if op == "la_fwd":
            # rows behind a length are written as zeros
            return {"bytes": e * (live * (2 * dk + dv) + B * H * N * dv) + states * (2 if case["state"] else 1),
                    "flops": 4 * dk * dv * live}
        return {"bytes": e * (live * (2 * dk + 2 * dv) + B * H * N * (2 * dk + dv)) + states * (3 if case["state"] else 0),
                "flops": 10 * dk * dv * live}
    if op == "la_step":
        B, H, dk, dv = (case[n] for n in ("B", "H", "dk", "dv"))
        live = B * (1 - case["idle"])
        return {"bytes": H * (live * (8 * dk * dv + e * (2 * dk + dv)) + B * e * dv), "flops": 5 * live * H * dk * dv}
    if op == "rotary":
        n = case["B"] * case["N"] * (case["H"] + case["Hk"])
        return {"bytes": 2 * e * n * case["D"] + 8 * case["B"] * case["N"], "flops": 3 * n * case["rot"]}
    n = case["rows"] * case["C"]
    if op == "norm_fwd":
        return {"bytes": 2 * e * n + 8 * case["groups"] * case["C"], "flops": 8 * n}
    return {"bytes": 4 * e * n + 16 * case["groups"] * case["C"], "flops": 20 * n}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("la_fwd", "la_bwd"):
        # token by token, the state carried
        N = case["N"]
        a = s["g"].exp()[None, :, None, None]
        q, k, v = (s[n].double() for n in "qkv")
        lengths = s["lengths"] if s["lengths"] is not None else torch.full((case["B"],), N, device="cuda")
        S = s["state"].double() if s["state"] is not None else \
            torch.zeros(case["B"], case["H"], case["dk"], case["dv"], dtype=torch.float64, device="cuda")
        o, dq = torch.zeros_like(v), torch.zeros_like(q)
        do = s["do"].double() if op == "la_bwd" else None
        for t in range(N):
            on = (t < lengths)[:, None, None, None]
            S = torch.where(on, a * S + k[:, :, t, :, None] * v[:, :, t, None, :], S)
            if op == "la_fwd":
                o[:, :, t] = torch.where(on[..., 0], torch.einsum("bhi,bhij->bhj", q[:, :, t], S), 0) * s["scale"]
            else:
                dq[:, :, t] = torch.where(on[..., 0], torch.einsum("bhj,bhij->bhi", do[:, :, t], S), 0) * s["scale"]
        if op == "la_fwd":
            return {"o": o, "state": S}
        R = s["dstate"].double() if s["dstate"] is not None else torch.zeros_like(S)
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        for t in reversed(range(N)):
            on = (t < lengths)[:, None, None, None]
            R = torch.where(on, R + s["scale"] * q[:, :, t, :, None] * do[:, :, t, None, :], R)
            dk[:, :, t] = torch.where(on[..., 0], torch.einsum("bhij,bhj->bhi", R, v[:, :, t]), 0)
            dv[:, :, t] = torch.where(on[..., 0], torch.einsum("bhi,bhij->bhj", k[:, :, t], R), 0)
            R = torch.where(on, a * R, R)
        got = {"dq": dq, "dk": dk, "dv": dv}
        if s["state"] is not None:
            got["dstate"] = R
        return got
    if op == "la_step":
        a = s["g"].exp()
        state, o = s["state"].double(), torch.zeros(case["B"], case["H"], case["dv"], dtype=torch.float64, device="cuda")
        for b, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                state[slot] = a[:, None, None] * state[slot] + torch.einsum("hi,hj->hij", s["k"][b].double(), s["v"][b].double())
                o[b] = torch.einsum("hi,hij->hj", s["q"][b].double(), state[slot]) * s["scale"]
        return {"o": o, "state": state}
    if op == "rotary":
        turn = torch.polar(torch.tensor(s["magnitude"], dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None, :, None] * s["frequencies"] * (-1 if case["inverse"] else 1))
        got, half = {}, case["rot"] // 2
        for n in "qk":
            x = s[n].double()
            part = x[..., :2 * half]
            pairs = part.unflatten(-1, (2, half)).transpose(-1, -2) if case["layout"] == "half" else part.unflatten(-1, (half, 2))
            y = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn)
            y = y.transpose(-1, -2) if case["layout"] == "half" else y
            got[n] = torch.cat((y.flatten(-2), x[..., 2 * half:]), -1)
        return got
    x = s["x"].double().requires_grad_()
    w, b = s["weight"].double().requires_grad_(), s["bias"].double().requires_grad_()
    c = x.unflatten(0, (-1, case["groups"]))
    y = (c - c.mean(-1, keepdim=True)) / (c.var(-1, unbiased=False, keepdim=True) + s["eps"]).sqrt() * w + b
    y = y.flatten(0, 1)
    if op == "norm_fwd":
        return {"y": y.detach()}
    dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].double())
    return {"y": y.detach(), "dx": dx, "dweight": dw, "dbias": db}
