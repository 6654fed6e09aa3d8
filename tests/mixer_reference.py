"""Plain forms, in 64 bits, of the operators around the convolution."""
import math

import torch


def powers(log_decay, e):
    """exp(log_decay[h] e) for integer e >= 0 (1 for e = 0, also where the decay is zero)."""
    g = torch.tensor(log_decay, dtype=torch.float64, device=e.device).reshape(-1, *([1] * e.dim()))
    return torch.where(e == 0, 1.0, torch.exp(g * e.clamp(min=1).double()))


def linattn(q, k, v, log_decay, scale, state=None, lengths=None):
    """(o, final states) by the full N x N sum."""
    B, H, N, _ = q.shape
    t = torch.arange(N, device=q.device)
    n = torch.full((B,), N, device=q.device) if lengths is None else lengths.long().clamp(0, N)
    live = (t < n[:, None])[:, None, :, None]
    q, k, v = (torch.where(live, x.double(), 0.0) for x in (q, k, v))
    D = powers(log_decay, (t[:, None] - t).clamp(min=0)) * (t[:, None] >= t)
    o = (q @ k.transpose(-1, -2) * D) @ v
    to_end = powers(log_decay, (n[:, None] - 1 - t).clamp(min=0)).transpose(0, 1)[..., None] * live
    S = (k * to_end).transpose(-1, -2) @ v
    if state is not None:
        o = o + torch.where(live, powers(log_decay, t + 1)[None, ..., None] * (q @ state.double()), 0.0)
        S = S + powers(log_decay, n).transpose(0, 1)[..., None, None] * state.double()
    return o * scale, S


def rotary(x, positions, rot, layout="half", base=10000.0, scaling="none", factor=1.0, context=4096, inverse=False):
    """x [B, H, N, d] rotated by positions [B, N]."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f, m = base ** (-2.0 * i / rot), 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        at = [rot * math.log(context / (2 * math.pi * n)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(0.0, math.floor(at[0])), min(rot - 1.0, math.ceil(at[1]))
        keep = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f, m = f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    a = positions[:, None, :, None].double() * f.to(x.device)
    cos, sin = m * a.cos(), m * a.sin() * (-1 if inverse else 1)
    y = x.double().clone()
    one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    x1, x2 = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return y


def layernorm(x, w, b, eps):
    """x [rows, C], w, b [G, C]: row r with weight r mod G."""
    x = x.double().unflatten(0, (-1, w.shape[0]))
    c = x - x.mean(-1, keepdim=True)
    y = c / (c.square().mean(-1, keepdim=True) + eps).sqrt() * w.double() + b.double()
    return y.flatten(0, 1)
