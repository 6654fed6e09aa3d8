"""Plans of the operators around the convolution: linear attention with a decay
per head, rotary positions, layer norm, and the retention core that runs the
three together.

Argument marshalling only, as in binding.py: every step runs in the CUDA
library.  Token tensors are [B, H, N, d] views whose last dimension is
contiguous (pass x.transpose(1, 2) for [B, N, H, d] storage); linear attention
takes strides that are multiples of 16 bytes, rotary any.  An output given as an
argument overlaps no input, and tensors rotated in place not each other.  Work
goes to `stream` (default: torch's current stream of the plan's device), outputs
and workspaces come from torch's allocator on that stream, so calls on several
streams and captured graphs never share scratch memory.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import struct
from typing import Optional

import torch

from .binding import DTYPES, TORCH_DTYPES, _check, load_library

_vp = ctypes.c_void_p


# Argument blocks of include/fftconv.h, packed in the C layout (a tenth of a ctypes structure's time); the library
# checks their sizes.  3q: the strides of a tensor.
_FWD = struct.Struct("@Niqd PPP 3q3q3q PP P3q P")
_BWD = struct.Struct("@Niqd PPPP 3q3q3q3q PPP PPP 3q3q3q P")
_STEP = struct.Struct("@Niid PPP 3q3q3q PP P3q")
_ROTARY = struct.Struct("@Niqii Pqi PPPP 3q3q3q3q")


class _RotaryOptions(ctypes.Structure):
    _fields_ = [("size", ctypes.c_size_t), ("dim", ctypes.c_int), ("rot", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("scaling", ctypes.c_int), ("base", ctypes.c_double),
                ("factor", ctypes.c_double), ("context", ctypes.c_double)]


SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}  # fftconv_rotary_scaling
LAYOUTS = {"half": 0, "interleaved": 1}


# the raw handle of the current stream of a device: a fraction of the time of building a Stream object
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _data(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


class _Mixer:
    """A plan's handle, device and argument checks."""
    _handle: ctypes.c_void_p
    _destroy = ""

    def __del__(self):
        h = getattr(self, "_handle", None)
        if h is not None and h.value:
            getattr(self.lib, self._destroy)(h)
            self._handle = None

    def destroy(self):
        self.__del__()

    def _make(self, create: str, *args):
        self.lib = load_library()
        h = ctypes.c_void_p()
        self._index = torch.cuda.current_device() if torch.cuda.is_available() else 0
        self.device = torch.device("cuda", self._index)
        _check(getattr(self.lib, create)(ctypes.byref(h), *args), create)
        self._handle = h

    def _need(self, t, name: str, shape, dtype, contiguous: bool = True):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.get_device() != self._index:
            raise ValueError(f"{name} is on {t.device}, the plan on {self.device}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _view(self, t, name: str, shape):
        """Strides of a [B, H, N, d] view of the plan's type (0 where a dimension has one element: its stride means
        nothing)."""
        self._need(t, name, shape, self.torch_dtype, False)
        b, h, n, d = t.stride()
        if d != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        B, H, N, _ = shape
        return b if B > 1 else 0, h if H > 1 else 0, n if N > 1 else 0

    def _stream(self, stream) -> int:
        return _current_raw(self._index) if stream is None else stream.cuda_stream

    def _on(self, stream):
        """Allocations belong to the stream the work runs on."""
        return _HERE if stream is None else torch.cuda.stream(stream)


_HERE = contextlib.nullcontext()


class LinearAttentionPlan(_Mixer):
    """Linear attention with a decay exp(log_decay[h]) for each head:

        S_t = a_h S_{t-1} + k_t^T v_t,    o_t = scale q_t S_t

    for up to B rows of up to N tokens, H heads of dk (queries, keys) and dv
    (values) elements, both multiples of 8 up to 128.  log_decay: H numbers <= 0,
    constants of the plan.  scale defaults to dk^-0.5."""
    _destroy = "fftconv_linattn_plan_destroy"

    def __init__(self, B: int, H: int, N: int, dk: int, dv: int, log_decay, dtype: str = "bf16",
                 scale: Optional[float] = None):
        if isinstance(log_decay, torch.Tensor):
            log_decay = log_decay.detach().double().cpu().tolist()
        log_decay = [float(x) for x in log_decay]
        if len(log_decay) != H:
            raise ValueError(f"log_decay has {len(log_decay)} values, expected {H}")
        self.B, self.H, self.N, self.dk, self.dv, self.dtype = B, H, N, dk, dv, dtype
        self.torch_dtype = TORCH_DTYPES[dtype]
        self.scale = float(dk) ** -0.5 if scale is None else float(scale)
        self._make("fftconv_linattn_plan_create", B, H, N, dk, dv, DTYPES[dtype], (ctypes.c_double * H)(*log_decay))
        self._bytes = [int(self.lib.fftconv_linattn_workspace_bytes(self._handle, i)) for i in (0, 1)]

    def set_wait_limit(self, probes: int):
        """Probes per bounded device wait (0: give up at the first check)."""
        _check(self.lib.fftconv_linattn_set_wait_limit(self._handle, int(probes)), "fftconv_linattn_set_wait_limit")

    def device_status(self, stream=None) -> int:
        """Synchronise the stream; 0, or 6 (timed out) once after a launch whose device wait gave up."""
        return int(self.lib.fftconv_linattn_device_status(self._handle, self._stream(stream)))

    def _tokens(self, q):
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError("q must be [B, H, N, dk]")
        B, _, N, _ = q.shape
        if B > self.B or N > self.N or B < 1 or N < 1:
            raise ValueError(f"q has {B} rows of {N} tokens, the plan {self.B} of {self.N}")
        return B, N

    def _optional(self, B, lengths, **states):
        if lengths is not None:
            self._need(lengths, "lengths", (B,), torch.int32)
        for name, t in states.items():
            if t is not None:
                self._need(t, name, (B, self.H, self.dk, self.dv), torch.float32)

    def _workspace(self, backward: int):
        n = self._bytes[backward]
        return torch.empty(n, dtype=torch.uint8, device=self.device) if n else None

    def fwd(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, state: Optional[torch.Tensor] = None,
            lengths: Optional[torch.Tensor] = None, final_state: bool = False, o: Optional[torch.Tensor] = None,
            stream=None):
        """o [B, H, N, dv]; with final_state, (o, the states after each row's last token).

        q, k [B, H, N, dk], v [B, H, N, dv]; state [B, H, dk, dv] fp32: the states
        before the first token (None: zero); lengths [B] int32: tokens of each row,
        o is zero behind them."""
        B, N = self._tokens(q)
        H, dk, dv = self.H, self.dk, self.dv
        sq, sk = self._view(q, "q", (B, H, N, dk)), self._view(k, "k", (B, H, N, dk))
        sv = self._view(v, "v", (B, H, N, dv))
        self._optional(B, lengths, state=state)
        with self._on(stream):
            if o is None:
                o = torch.empty_like(v)  # stored in the order of v's strides
            out = torch.empty((B, H, dk, dv), dtype=torch.float32, device=self.device) if final_state else None
            ws = self._workspace(0)
        a = _FWD.pack(_FWD.size, B, N, self.scale, q.data_ptr(), k.data_ptr(), v.data_ptr(), *sq, *sk, *sv,
                      _data(lengths), _data(state), o.data_ptr(), *self._view(o, "o", (B, H, N, dv)), _data(out))
        _check(self.lib.fftconv_linattn_fwd(self._handle, a, _data(ws), self._stream(stream)), "fftconv_linattn_fwd")
        return (o, out) if final_state else o

    def bwd(self, do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
            state: Optional[torch.Tensor] = None, dstate: Optional[torch.Tensor] = None,
            lengths: Optional[torch.Tensor] = None, stream=None) -> dict:
        """Gradients of fwd(q, k, v, state, lengths) for the gradient do of o and
        dstate of the final states (None: zero): dq, dk, dv of the plan's dtype and,
        where state is given, dstate (fp32, of the initial states; else None)."""
        B, N = self._tokens(q)
        H, dk, dv = self.H, self.dk, self.dv
        keys, values = (B, H, N, dk), (B, H, N, dv)
        strides = (*self._view(do, "do", values), *self._view(q, "q", keys), *self._view(k, "k", keys),
                   *self._view(v, "v", values))
        self._optional(B, lengths, state=state, dstate=dstate)
        with self._on(stream):
            gq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
            ds = torch.empty((B, H, dk, dv), dtype=torch.float32, device=self.device) if state is not None else None
            ws = self._workspace(1)
        a = _BWD.pack(_BWD.size, B, N, self.scale, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides,
                      _data(lengths), _data(state), _data(dstate), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
                      *self._view(gq, "dq", keys), *self._view(gk, "dk", keys), *self._view(gv, "dv", values),
                      _data(ds))
        _check(self.lib.fftconv_linattn_bwd(self._handle, a, _data(ws), self._stream(stream)), "fftconv_linattn_bwd")
        return {"dq": gq, "dk": gk, "dv": gv, "dstate": ds}

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, state: torch.Tensor,
             slots: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One token a row: o [B, H, dv] from q, k [B, H, dk], v [B, H, dv]; state
        [pool, H, dk, dv] fp32 is updated in place.  slots [B] int32: each row's
        state (None: row b has state b); a row whose slot is outside the pool is idle
        (zeros in o); rows with one slot are taken in row order."""
        if not isinstance(q, torch.Tensor) or q.dim() != 3 or not 1 <= q.shape[0] <= self.B:
            raise ValueError(f"q must be [B, H, dk] with at most {self.B} rows")
        B, H, dt = q.shape[0], self.H, self.torch_dtype
        self._need(q, "q", (B, H, self.dk), dt, False)
        self._need(k, "k", (B, H, self.dk), dt, False)
        self._need(v, "v", (B, H, self.dv), dt, False)
        if not isinstance(state, torch.Tensor) or state.dim() != 4:
            raise ValueError("state must be [pool, H, dk, dv]")
        self._need(state, "state", (state.shape[0], H, self.dk, self.dv), torch.float32)
        if slots is not None:
            self._need(slots, "slots", (B,), torch.int32)
        elif state.shape[0] < B:
            raise ValueError(f"{B} rows, but {state.shape[0]} states")
        if o is None:
            with self._on(stream):
                o = torch.empty((B, H, self.dv), dtype=dt, device=self.device)
        else:
            self._need(o, "o", (B, H, self.dv), dt, False)
        a = _STEP.pack(_STEP.size, B, state.shape[0], self.scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                       *_rows(q, "q"), *_rows(k, "k"), *_rows(v, "v"), _data(slots), state.data_ptr(), o.data_ptr(),
                       *_rows(o, "o"))
        _check(self.lib.fftconv_linattn_step(self._handle, a, self._stream(stream)), "fftconv_linattn_step")
        return o


def _rows(t: torch.Tensor, name: str):
    """Strides of a [B, H, d] view."""
    b, h, d = t.stride()
    if d != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return b, h, 0


class RotaryPlan(_Mixer):
    """Rotary positions on the first rot_dim of a head's dim elements (default: all).

    layout "half": pairs (i, i + rot_dim / 2); "interleaved": (2i, 2i + 1).
    scaling "none"; "linear" (positions divided by factor); "base" (the base grows
    with factor); "parts" (slow pairs interpolated, fast ones kept, values scaled by
    0.1 ln(factor) + 1; context: positions trained on)."""
    _destroy = "fftconv_rotary_plan_destroy"

    def __init__(self, dim: int, rot_dim: Optional[int] = None, layout: str = "half", dtype: str = "bf16",
                 base: float = 10000.0, scaling: str = "none", factor: float = 1.0, context: int = 4096):
        self.dim, self.rot_dim, self.layout, self.dtype = dim, dim if rot_dim is None else rot_dim, layout, dtype
        self.torch_dtype = TORCH_DTYPES[dtype]
        opts = _RotaryOptions(ctypes.sizeof(_RotaryOptions), dim, self.rot_dim, LAYOUTS[layout], SCALINGS[scaling],
                              float(base), float(factor), float(context))
        self._make("fftconv_rotary_plan_create", DTYPES[dtype], ctypes.byref(opts))

    def apply(self, x: torch.Tensor, x2: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
              inverse: bool = False, inplace: bool = False, stream=None):
        """x (and x2, e.g. keys, in the same launch) rotated: [B, H, N, dim] each, any
        number of heads, any strides.  positions int64 [B, N] or [N].  inverse: the
        rotation by the negated angle, which is the gradient of the rotation."""
        if not isinstance(x, torch.Tensor) or x.dim() != 4:
            raise ValueError("x must be [B, H, N, dim]")
        B, H, N, _ = x.shape
        dim = self.dim
        sx, sx2, H2 = self._view(x, "x", (B, H, N, dim)), (0, 0, 0), 0
        if x2 is not None:
            if not isinstance(x2, torch.Tensor) or x2.dim() != 4:
                raise ValueError("x2 must be [B, H, N, dim]")
            H2 = x2.shape[1]
            sx2 = self._view(x2, "x2", (B, H2, N, dim))
        if not isinstance(positions, torch.Tensor):
            raise ValueError("positions are needed")
        flat = positions.dim() == 1
        self._need(positions, "positions", (N,) if flat else (B, N), torch.int64)
        if inplace:
            y, y2, sy, sy2 = x, x2, sx, sx2
        else:
            with self._on(stream):
                y, y2 = torch.empty_like(x), None if x2 is None else torch.empty_like(x2)
            sy = self._view(y, "y", (B, H, N, dim))
            sy2 = sx2 if x2 is None else self._view(y2, "y2", (B, H2, N, dim))
        a = _ROTARY.pack(_ROTARY.size, B, N, H, H2, positions.data_ptr(), 0 if flat else N, int(inverse),
                         x.data_ptr(), _data(x2), y.data_ptr(), _data(y2), *sx, *sx2, *sy, *sy2)
        _check(self.lib.fftconv_rotary_apply(self._handle, a, self._stream(stream)), "fftconv_rotary_apply")
        return y if x2 is None else (y, y2)


class LayerNormPlan(_Mixer):
    """Layer norm over the last dimension of up to `rows` rows of C elements; row r
    uses weight row r mod groups (groups = heads: the norm behind each head)."""
    _destroy = "fftconv_norm_plan_destroy"

    def __init__(self, rows: int, C: int, dtype: str = "bf16", groups: int = 1, eps: float = 1e-5):
        self.rows, self.C, self.dtype, self.groups, self.eps = rows, C, dtype, groups, eps
        self.torch_dtype = TORCH_DTYPES[dtype]
        self._make("fftconv_norm_plan_create", rows, C, groups, DTYPES[dtype], ctypes.byref(ctypes.c_double(eps)))
        self._bytes = int(self.lib.fftconv_norm_bwd_workspace_bytes(self._handle))

    def _rows(self, x, name: str) -> int:
        if not isinstance(x, torch.Tensor) or x.dim() < 1 or x.shape[-1] != self.C:
            raise ValueError(f"{name} must be [..., {self.C}]")
        self._need(x, name, x.shape, self.torch_dtype)
        rows = x.numel() // self.C
        if not 1 <= rows <= self.rows or rows % self.groups:
            raise ValueError(f"{name} has {rows} rows: at most {self.rows}, a multiple of {self.groups}")
        return rows

    def _weights(self, **ts):
        for name, t in ts.items():
            shape = (self.C,) if self.groups == 1 and isinstance(t, torch.Tensor) and t.dim() == 1 else \
                (self.groups, self.C)
            self._need(t, name, shape, torch.float32)

    def fwd(self, x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor, statistics: bool = False,
            y: Optional[torch.Tensor] = None, stream=None):
        """y like x [..., C]; with statistics, (y, mean, rstd) for bwd.  weight, bias
        fp32 [groups, C] ([C] where groups is 1)."""
        rows = self._rows(x, "x")
        self._weights(weight=weight, bias=bias)
        if y is not None:
            self._need(y, "y", x.shape, self.torch_dtype)
        mean = rstd = None
        with self._on(stream):
            if y is None:
                y = torch.empty_like(x)
            if statistics:
                mean = torch.empty(rows, dtype=torch.float32, device=self.device)
                rstd = torch.empty_like(mean)
        _check(self.lib.fftconv_norm_fwd(self._handle, rows, x.data_ptr(), weight.data_ptr(), bias.data_ptr(),
                                         y.data_ptr(), _data(mean), _data(rstd), self._stream(stream)),
               "fftconv_norm_fwd")
        return (y, mean, rstd) if statistics else y

    def bwd(self, dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
            stream=None):
        """(dx, dweight, dbias) for the gradient dy of fwd's y; dweight and dbias fp32 [groups, C]."""
        rows = self._rows(x, "x")
        self._need(dy, "dy", x.shape, self.torch_dtype)
        self._weights(weight=weight)
        self._need(mean, "mean", (rows,), torch.float32)
        self._need(rstd, "rstd", (rows,), torch.float32)
        with self._on(stream):
            dx = torch.empty_like(x)
            dw = torch.empty((self.groups, self.C), dtype=torch.float32, device=self.device)
            db = torch.empty_like(dw)
            ws = torch.empty(self._bytes, dtype=torch.uint8, device=self.device)
        _check(self.lib.fftconv_norm_bwd(self._handle, rows, dy.data_ptr(), x.data_ptr(), weight.data_ptr(),
                                         mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(),
                                         db.data_ptr(), ws.data_ptr(), self._stream(stream)), "fftconv_norm_bwd")
        return dx, dw, db


class RetentionPlan:
    """The core of a retention layer: rotary positions on queries and keys, linear
    attention with a decay per head, a layer norm behind each head.

    rotary: keyword arguments of RotaryPlan beside dim and dtype.  log_decay
    defaults to log(1 - 2^(-5 - h)) for head h."""

    def __init__(self, B: int, H: int, N: int, dk: int, dv: int, log_decay=None, dtype: str = "bf16",
                 rotary: Optional[dict] = None, eps: float = 1e-5, scale: Optional[float] = None):
        if log_decay is None:
            log_decay = [math.log1p(-2.0 ** (-5.0 - h)) for h in range(H)]
        self.attention = LinearAttentionPlan(B, H, N, dk, dv, log_decay, dtype=dtype, scale=scale)
        self.rotary = RotaryPlan(dk, dtype=dtype, **(rotary or {}))
        self.norm = LayerNormPlan(B * H * N, dv, dtype=dtype, groups=H, eps=eps)
        self.H = H

    def fwd(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor,
            positions: torch.Tensor, state: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
            final_state: bool = False, save: bool = False, stream=None):
        """y [B, N, H, dv] = norm(attention(rotary(q), rotary(k), v)); weight, bias
        [H, dv].  Returns y, then the final states if asked for, then with `save` what
        bwd needs.  (The norm of a row behind a length is its bias.)"""
        with self.attention._on(stream):
            qr, kr = self.rotary.apply(q, k, positions=positions, stream=stream)
            # token by token: the order the norm's weights repeat in
            B, _, N, _ = qr.shape
            rows = torch.empty((B, N, self.H, self.attention.dv), dtype=self.attention.torch_dtype,
                               device=self.attention.device)
            got = self.attention.fwd(qr, kr, v, state=state, lengths=lengths, final_state=final_state,
                                     o=rows.transpose(1, 2), stream=stream)
            end = got[1] if final_state else None
            y, mean, rstd = self.norm.fwd(rows, weight, bias, statistics=True, stream=stream)
        out = [y] + ([end] if final_state else []) + ([(qr, kr, v, state, lengths, positions, rows, mean, rstd)]
                                                      if save else [])
        return out[0] if len(out) == 1 else tuple(out)

    def bwd(self, dy: torch.Tensor, saved, weight: torch.Tensor, dstate: Optional[torch.Tensor] = None,
            stream=None) -> dict:
        """Gradients for dy [B, N, H, dv]: dq, dk, dv, dweight, dbias and, where fwd had
        states, dstate."""
        qr, kr, v, state, lengths, positions, rows, mean, rstd = saved
        with self.attention._on(stream):
            do, dw, db = self.norm.bwd(dy, rows, weight, mean, rstd, stream=stream)
            g = self.attention.bwd(do.transpose(1, 2), qr, kr, v, state=state, dstate=dstate, lengths=lengths,
                                   stream=stream)
            dq, dk = self.rotary.apply(g["dq"], g["dk"], positions=positions, inverse=True, stream=stream)
        return {"dq": dq, "dk": dk, "dv": g["dv"], "dstate": g["dstate"], "dweight": dw, "dbias": db}

    def step(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor,
             positions: torch.Tensor, state: torch.Tensor, slots: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
        """One token a row: y [B, H, dv] from q, k [B, H, dk], v [B, H, dv] at positions [B] int64."""
        with self.attention._on(stream):
            qr, kr = self.rotary.apply(q.unsqueeze(2), k.unsqueeze(2), positions=positions.unsqueeze(1),
                                       stream=stream)
            o = self.attention.step(qr.squeeze(2), kr.squeeze(2), v, state, slots=slots, stream=stream)
            return self.norm.fwd(o, weight, bias, stream=stream)
