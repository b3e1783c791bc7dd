"""What a block around the recurrences needs (the C ABI of include/kla_block.h): the gated scan, a recurrence with a
gate and a state per channel (``gated_scan_fwd``, ``gated_scan_bwd``, ``gated_scan_step``); rotary positions of queries
and keys (``rotary_fwd``, ``rotary_bwd``, ``rotary_freqs``); the norms after and before a block with its gate and its
residual (``gated_norm_fwd``, ``gated_norm_bwd``, ``add_norm_fwd``, ``add_norm_bwd``); and the verification of drafted
tokens (``verify_draft``).

The binding checks and marshals; every operation runs in this package's CUDA kernels on the current stream of the
tensors' device, whether or not that device is the current one. Small calls are bound by the host, so the functions first
ask in one expression whether everything is as it should be, and only where it is not go through the arguments one by one
to name the one at fault or to take what strides they have.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _native
from .layer import _CODE, _F32, _MOST, _check, _code, _device, _norm_shape, _ptr, _refuse, _scratch, _size, _stream

_Strides4, _Strides6, _Strides12 = ctypes.c_int64 * 4, ctypes.c_int64 * 6, ctypes.c_int64 * 12
_MODES = {"sigmoid": _native.KLA_SCAN_SIGMOID, "log": _native.KLA_SCAN_LOG}
_LAYOUTS = {"half": _native.KLA_ROTARY_HALF, "interleaved": _native.KLA_ROTARY_INTERLEAVED}
_NORMS = {"rms": _native.KLA_NORM_RMS, "layer": _native.KLA_NORM_LAYER}
_ACTS = {"silu": _native.KLA_ACT_SILU, "sigmoid": _native.KLA_ACT_SIGMOID}
_POSITIONS = {torch.int32: 0, torch.int64: 1}
SCAN_SPAN = 128   # tokens between the states that gated_scan_fwd keeps for gated_scan_bwd


def _choice(name: str, table: dict, value) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, got {value!r}") from None


def _dense_last(*tensors) -> None:
    for t in tensors:
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("the last axis must be contiguous")


# ------------------------------------------------------------------------------------- gated scan


def _scan_shapes(x, gate, lengths):
    """Sizes of the call, and whether x and gate are contiguous."""
    try:
        shape, dtype, at = x.shape, x.dtype, x.get_device()
        dense = (at >= 0 and len(shape) == 3 and gate.shape == shape and gate.dtype is dtype and dtype in _CODE and
                 gate.get_device() == at and x.is_contiguous() and gate.is_contiguous())
    except AttributeError:
        dense = False
    if not dense:
        device = _device("x", x)
        _code("x", x)
        if x.dim() != 3:
            raise ValueError("x and gate must be [B, T, C]")
        _check("gate", gate, x.shape, x.dtype, device, False)
    device = x.device
    if lengths is not None:
        _check("lengths", lengths, shape[:1], torch.int32, device)
    return device, _CODE[dtype], shape, dense


def gated_scan_workspace_size(B: int, T: int, C: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Device scratch bytes ``gated_scan_fwd`` and ``gated_scan_bwd`` need for these sizes."""
    return _size("gated_scan", B, T, C, _CODE[dtype])


def gated_scan_fwd(x: torch.Tensor, gate: torch.Tensor, h0: Optional[torch.Tensor] = None, *, mode: str = "sigmoid",
                   lengths: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   final_state: bool = True, h_T: Optional[torch.Tensor] = None, states: bool = False,
                   workspace: Optional[torch.Tensor] = None):
    """A recurrence with one gate per channel over whole prompts: ``h_t = a_t h_{t-1} + (1 - a_t) x_t`` with
    ``a = sigmoid(gate)`` (mode "sigmoid"), or ``h_t = a_t h_{t-1} + x_t`` with ``a = exp(gate)`` (mode "log", gates of
    at most 0; where larger ones take the product of 256 neighbouring factors or fewer past fp32, ``device_status`` says so).

    x, gate: [B,T,C] (bf16 or fp32; any strides with a dense last axis, as the slices of a packed projection); h0: fp32
    [B,C] or None (zeros). ``lengths`` (int32 [B]) masks the tokens from lengths[b] on: they leave the state alone and
    their outputs are 0. A channel whose state is infinite or NaN stays one or the other. Returns (y = h [B,T,C] in x's dtype, h_T fp32 [B,C] or None, what ``gated_scan_bwd`` needs
    with ``states``, else None); ``h_T`` may be passed, and may be ``h0``.
    """
    device, code, (B, T, C), dense = _scan_shapes(x, gate, lengths)
    mode = _choice("mode", _MODES, mode)
    strides = None
    if not dense:
        _dense_last(x, gate)
        strides = _Strides4(*x.stride()[:2], *gate.stride()[:2])
    if h0 is not None:
        _check("h0", h0, (B, C), _F32, device)
    if out is None:
        out = torch.empty_like(x) if dense else torch.empty((B, T, C), dtype=x.dtype, device=device)
    else:
        _check("out", out, (B, T, C), x.dtype, device)
    if h_T is not None:
        _check("h_T", h_T, (B, C), _F32, device)
    elif final_state:
        h_T = torch.empty((B, C), dtype=_F32, device=device)
    kept = torch.empty((B, -(-T // SCAN_SPAN), C), dtype=_F32, device=device) if states else None
    workspace, size = _scratch(_size("gated_scan", B, T, C, code), workspace, device)
    st = _native.on(device).kla_gated_scan_fwd(
        x.data_ptr(), gate.data_ptr(), strides, _ptr(lengths), _ptr(h0), out.data_ptr(), _ptr(h_T), _ptr(kept), B, T,
        C, code, mode, _ptr(workspace), size, _stream(device))
    if st:
        _native.check(st, "kla_gated_scan_fwd")
    return out, h_T, kept


def gated_scan_bwd(x: torch.Tensor, gate: torch.Tensor, dy: torch.Tensor, states: torch.Tensor,
                   dh_T: Optional[torch.Tensor] = None, *, mode: str = "sigmoid",
                   lengths: Optional[torch.Tensor] = None, want_dh0: bool = True,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``gated_scan_fwd`` run with the same inputs, mode and lengths, given its ``states``, dy = dL/dy
    and dh_T = dL/dh_T. Returns dx and dgate [B,T,C] in x's dtype (zero at masked tokens) and dh0 fp32 [B,C] (None
    unless ``want_dh0``)."""
    device, code, (B, T, C), dense = _scan_shapes(x, gate, lengths)
    mode = _choice("mode", _MODES, mode)
    _check("dy", dy, x.shape, x.dtype, device, False)
    strides = None
    if not (dense and dy.is_contiguous()):
        _dense_last(x, gate, dy)
        strides = _Strides6(*x.stride()[:2], *gate.stride()[:2], *dy.stride()[:2])
    _check("states", states, (B, -(-T // SCAN_SPAN), C), _F32, device)
    if dh_T is not None:
        _check("dh_T", dh_T, (B, C), _F32, device)
    dx = torch.empty((B, T, C), dtype=x.dtype, device=device)
    dgate = torch.empty_like(dx)
    dh0 = torch.empty((B, C), dtype=_F32, device=device) if want_dh0 else None
    workspace, size = _scratch(_size("gated_scan", B, T, C, code), workspace, device)
    st = _native.on(device).kla_gated_scan_bwd(
        x.data_ptr(), gate.data_ptr(), dy.data_ptr(), strides, _ptr(lengths), states.data_ptr(), _ptr(dh_T),
        dx.data_ptr(), dgate.data_ptr(), _ptr(dh0), B, T, C, code, mode, _ptr(workspace), size, _stream(device))
    if st:
        _native.check(st, "kla_gated_scan_bwd")
    return {"dx": dx, "dgate": dgate, "dh0": dh0}


def gated_scan_step(x: torch.Tensor, gate: torch.Tensor, h: torch.Tensor, *, mode: str = "sigmoid",
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for B sequences of ``gated_scan_fwd``'s recurrence. x, gate: [B,C] (rows may be slices of a packed
    projection); h: fp32 [B,C], updated in place. Returns y [B,C]."""
    try:
        shape, dtype, at = x.shape, x.dtype, x.get_device()
        B, C = shape
        ok = (at >= 0 and gate.shape == shape and gate.dtype is dtype and gate.get_device() == at and dtype in _CODE and
              x.is_contiguous() and gate.is_contiguous() and h.shape == shape and h.dtype is _F32 and
              h.get_device() == at and h.is_contiguous() and 0 < B <= _MOST and 0 < C <= _MOST)
    except (AttributeError, ValueError):
        ok = False
    xs = gs = C if ok else 0
    if not ok:
        device = _device("x", x)
        _code("x", x)
        if x.dim() != 2:
            raise ValueError("x and gate must be [B, C]")
        if B > _MOST or C > _MOST:
            _refuse("kla_gated_scan_step", _native.KLA_ERR_UNSUPPORTED)
        _check("gate", gate, shape, dtype, device, False)
        _dense_last(x, gate)
        _check("h", h, (B, C), _F32, device)
        xs, gs = (x.stride(0), gate.stride(0)) if B > 1 else (C, C)   # one row may have any stride
    device = x.device
    if out is None:
        out = torch.empty_like(x) if ok else torch.empty((B, C), dtype=dtype, device=device)
    else:
        _check("out", out, (B, C), dtype, device)
    st = _native.on(device).kla_gated_scan_step(x.data_ptr(), xs, gate.data_ptr(), gs, h.data_ptr(), out.data_ptr(),
                                                B, C, _CODE[dtype], _choice("mode", _MODES, mode), _stream(device))
    if st:
        _native.check(st, "kla_gated_scan_step")
    return out


# ----------------------------------------------------------------------------------------- rotary


def rotary_freqs(rot: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                 original_length: Optional[int] = None, fast: float = 32.0, slow: float = 1.0,
                 device="cuda") -> Tuple[torch.Tensor, float]:
    """(freqs fp32 [rot / 2], scale) for ``rotary_fwd``: ``base ** (-2 i / rot)``, for contexts ``factor`` times as
    long as the trained ones scaled by

    - "linear": every frequency divided by ``factor``;
    - "ntk": the base grown so that the lowest frequency is divided by ``factor`` and the highest is kept;
    - "yarn": frequencies that turn more than ``fast`` times within ``original_length`` tokens kept, those that turn
      less than ``slow`` times divided by ``factor``, a ramp between them; ``scale`` is 0.1 ln(factor) + 1, else 1.
    """
    if rot < 0 or rot % 2:
        raise ValueError("rot must be even")
    if not (0 < base < math.inf and 0 < factor < math.inf):
        raise ValueError("base and factor must be positive and finite")
    n, scale = rot // 2, 1.0
    at = torch.arange(n, dtype=torch.float64)
    if scaling == "ntk" and n > 1:
        base = base * factor ** (n / (n - 1))
    freqs = base ** (-at / max(1, n))
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "yarn":
        if original_length is None or original_length < 1 or not fast > slow > 0 or base <= 1:
            raise ValueError('"yarn" needs original_length, fast > slow > 0 and a base above 1')
        # the place along the frequencies at which one turns `turns` times within original_length
        def place(turns):
            return n * math.log(original_length / (turns * 2 * math.pi)) / math.log(base)
        # the ramp may end beyond the last frequency, which is on it then
        low, high = max(0.0, math.floor(place(fast))), min(rot - 1.0, math.ceil(place(slow)))
        low = min(low, high - 1e-3)   # nothing turns `slow` times (or all do `fast` times): no ramp among the frequencies
        ramp = ((at - low) / (high - low)).clamp(0, 1)
        freqs = freqs * (1 - ramp) + freqs / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    return freqs.to(_F32).to(device), scale


def _rotary_shapes(entry, q, k, freqs, positions):
    """Sizes of the call, and whether q and k are contiguous."""
    try:
        shape, dtype, at = q.shape, q.dtype, q.get_device()
        B, T, H, d = shape
        dense = q.is_contiguous()
        ok = (at >= 0 and dtype in _CODE and (dense or q.stride(3) == 1) and freqs.dtype is _F32 and len(freqs.shape) == 1 and
              freqs.get_device() == at and freqs.is_contiguous() and 2 * freqs.shape[0] <= d and max(shape) <= _MOST and
              (positions is None or (positions.dtype in _POSITIONS and positions.shape == shape[:2] and
                                     positions.get_device() == at and positions.is_contiguous())))
        if k is not None:
            kshape = k.shape
            Hk = kshape[2]
            dense_k = k.is_contiguous()
            ok = (ok and k.dtype is dtype and kshape == (B, T, Hk, d) and k.get_device() == at and
                  (dense_k or k.stride(3) == 1) and Hk <= _MOST)
            dense = dense and dense_k
        else:
            Hk = 0
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        dense = False
        device = _device("q", q)
        _code("q", q)
        if q.dim() != 4 or (k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 4)):
            raise ValueError("q and k must be [B, T, H, d]")
        Hk = 0 if k is None else k.shape[2]
        if max(q.shape) > _MOST or Hk > _MOST:
            _refuse(entry, _native.KLA_ERR_UNSUPPORTED)
        _dense_last(q)
        if k is not None:
            _check("k", k, (B, T, Hk, d), dtype, device, False)
            _dense_last(k)
        if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
            raise ValueError("freqs must be [rot / 2]")
        _check("freqs", freqs, freqs.shape, _F32, device)
        if 2 * freqs.shape[0] > d:
            _refuse(entry, _native.KLA_ERR_INVALID_ARG)
        if positions is not None:
            if positions.dtype not in _POSITIONS:
                raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
            _check("positions", positions, (B, T), positions.dtype, device)
    return B, T, H, Hk, d, dense


def _rotary_out(name, x, out, dense):
    if out is None:
        return torch.empty_like(x) if dense else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _check(name, out, x.shape, x.dtype, x.device, False)
    return out


def _rotary(entry, q, k, freqs, positions, layout, scale, out_q, out_k, inverse):
    B, T, H, Hk, d, dense = _rotary_shapes(entry, q, k, freqs, positions)
    layout = _choice("layout", _LAYOUTS, layout)
    device = q.device
    given = out_q is not None or out_k is not None
    out_q = _rotary_out("out_q", q, out_q, dense)
    out_k = None if k is None else _rotary_out("out_k", k, out_k, dense)
    strides = None
    if not dense or given:
        if given:
            _dense_last(*(t for t in (out_q, out_k) if t is not None))
        a, b = q.stride(), out_q.stride()
        c, e = (b, b) if k is None else (k.stride(), out_k.stride())   # without keys: not looked at
        strides = _Strides12(a[0], a[1], a[2], c[0], c[1], c[2], b[0], b[1], b[2], e[0], e[1], e[2])
    st = _native.on(device).kla_rotary(
        q.data_ptr(), _ptr(k), out_q.data_ptr(), _ptr(out_k), strides, freqs.data_ptr(), _ptr(positions),
        0 if positions is None else _POSITIONS[positions.dtype], B, T, H, Hk, d, 2 * freqs.shape[0], layout,
        _CODE[q.dtype], scale, inverse, _stream(device))
    if st:
        _native.check(st, entry)
    return out_q, out_k


def rotary_fwd(q: torch.Tensor, k: Optional[torch.Tensor], freqs: torch.Tensor,
               positions: Optional[torch.Tensor] = None, *, layout: str = "half", scale: float = 1.0,
               out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """Queries and keys turned by their positions: pair i of the first ``2 len(freqs)`` values of every head by the
    angle ``position * freqs[i]``, times ``scale``; the values behind those are copied.

    q: [B,T,H,d], k: [B,T,K,d] or None (bf16 or fp32; any strides with a dense last axis, as the slices of a packed
    projection); freqs: fp32 [rot / 2] (``rotary_freqs``); positions: int64 or int32 [B,T], or None (token t has
    position t). ``layout``: "half" pairs values i and i + rot / 2, "interleaved" 2 i and 2 i + 1. Returns (q, k)
    turned, contiguous unless ``out_q`` and ``out_k`` are given, which may be q and k themselves, or slices of one tensor.
    """
    return _rotary("kla_rotary_fwd", q, k, freqs, positions, layout, scale, out_q, out_k, 0)


def rotary_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], freqs: torch.Tensor,
               positions: Optional[torch.Tensor] = None, *, layout: str = "half", scale: float = 1.0,
               out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """Gradients of ``rotary_fwd``'s inputs given those of its outputs: turned back, times ``scale``."""
    return _rotary("kla_rotary_bwd", dq, dk, freqs, positions, layout, scale, out_q, out_k, 1)


# ---------------------------------------------------------------------------------- a block's norms


def _heads(x, gate, weight):
    """(rows, groups, n, whether groups have weights of their own, gate's stride between rows, the weights' shape)."""
    rows, groups, n, shape = _norm_shape(x, weight, None)
    own = len(shape) == 2
    if gate.is_contiguous():
        return rows, groups, n, int(own), groups * n, shape
    # a slice of a packed projection: the last axis, or the last two, dense, and rows of those a constant stride apart
    tail = 2 if own or (x.dim() > 1 and gate.stride(-2) == n) else 1
    if tail == 2 and not own:
        groups = x.shape[-2]
        rows //= groups
    ok = gate.stride(-1) == 1 and (tail == 1 or groups == 1 or gate.stride(-2) == n)
    stride = apart = None
    for size, st in zip(reversed(gate.shape[:-tail]), reversed(gate.stride()[:-tail])):
        if size > 1:
            ok = ok and (apart is None or st == apart)
            stride, apart = st if stride is None else stride, st * size
    if not ok:
        raise ValueError("the rows of gate must be dense and a constant stride apart")
    return rows, groups, n, int(own), groups * n if stride is None else stride, shape


def _norm_inputs(entry, x, gate, weight):
    try:
        all_of, dtype, at = x.shape, x.dtype, x.get_device()
        ok = (at >= 0 and dtype in _CODE and gate.shape == all_of and gate.dtype is dtype and
              gate.get_device() == at and x.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        device = _device("x", x)
        _code("x", x)
        if not x.is_contiguous():
            raise ValueError("x must be contiguous")
        _check("gate", gate, x.shape, x.dtype, device, False)
    device = x.device
    rows, groups, n, own, stride, shape = _heads(x, gate, weight)
    if n > _MOST or groups > _MOST:
        _refuse(entry, _native.KLA_ERR_UNSUPPORTED)
    if weight is not None:
        _check("weight", weight, shape, _F32, device)
    return device, _CODE[dtype], rows, groups, n, own, stride, shape


def _stats(x, layer, wanted, device):
    rstd = torch.empty(x.shape[:-1], dtype=_F32, device=device) if wanted else None
    return torch.empty_like(rstd) if wanted and layer else None, rstd


def gated_norm_fwd(x: torch.Tensor, gate: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                   norm: str = "rms", act: str = "silu", out: Optional[torch.Tensor] = None, stats: bool = True):
    """The norm of a block's heads times the activation of its gate: ``y = norm(x) * weight * act(gate)`` over the
    last axis; ``norm`` is "rms" (no mean is taken) or "layer", ``act`` "silu" or "sigmoid".

    x: [..., n] bf16 or fp32, contiguous, 3 <= n <= 65536; gate: the same, or a slice of a packed projection (rows of
    the last axis or the last two dense and a constant stride apart); weight: fp32 [n], or [H, n] for x [..., H, n].
    Returns (y, mean, rstd fp32 [...] for the backward pass): mean is None with "rms", both without ``stats``.
    """
    norm, act = _choice("norm", _NORMS, norm), _choice("act", _ACTS, act)
    device, code, rows, groups, n, own, stride, _ = _norm_inputs("kla_gated_norm_fwd", x, gate, weight)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check("out", out, x.shape, x.dtype, device)
    mean, rstd = _stats(x, norm, stats, device)
    st = _native.on(device).kla_gated_norm_fwd(x.data_ptr(), gate.data_ptr(), stride, _ptr(weight), own,
                                               out.data_ptr(), _ptr(mean), _ptr(rstd), rows, groups, n, code, norm,
                                               act, eps, _stream(device))
    if st:
        _native.check(st, "kla_gated_norm_fwd")
    return out, mean, rstd


def gated_norm_bwd(dy: torch.Tensor, x: torch.Tensor, gate: torch.Tensor, weight: Optional[torch.Tensor],
                   mean: Optional[torch.Tensor], rstd: torch.Tensor, *, act: str = "silu",
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of ``gated_norm_fwd`` given its x, gate, weight, mean (None: "rms") and rstd: (dx, dgate in x's
    dtype, contiguous, dweight fp32 [n] or [H, n]). Equal calls give equal bits."""
    act = _choice("act", _ACTS, act)
    device, code, rows, groups, n, own, stride, shape = _norm_inputs("kla_gated_norm_bwd", x, gate, weight)
    _check("dy", dy, x.shape, x.dtype, device)
    if mean is not None:
        _check("mean", mean, x.shape[:-1], _F32, device)
    _check("rstd", rstd, x.shape[:-1], _F32, device)
    dx, dgate = torch.empty_like(x), torch.empty(x.shape, dtype=x.dtype, device=device)
    dw = torch.empty(shape, dtype=_F32, device=device)
    workspace, size = _scratch(_size("gated_norm_bwd", rows, groups, n, code, own), workspace, device)
    st = _native.on(device).kla_gated_norm_bwd(dy.data_ptr(), x.data_ptr(), gate.data_ptr(), stride, _ptr(weight),
                                               own, _ptr(mean), rstd.data_ptr(), dx.data_ptr(), dgate.data_ptr(),
                                               dw.data_ptr(), rows, groups, n, code, act, _ptr(workspace), size,
                                               _stream(device))
    if st:
        _native.check(st, "kla_gated_norm_bwd")
    return dx, dgate, dw


def _added_inputs(entry, x, residual, weight, scale):
    try:
        all_of, dtype, at = residual.shape, residual.dtype, residual.get_device()
        ok = (at >= 0 and dtype in _CODE and len(all_of) > 0 and residual.is_contiguous() and x.shape == all_of and
              x.dtype is dtype and x.get_device() == at and x.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        device = _device("residual", residual)
        _code("residual", residual)
        if residual.dim() < 1:
            raise ValueError("residual must have an axis to normalise")
        _check("residual", residual, residual.shape, residual.dtype, device)
        _check("x", x, residual.shape, residual.dtype, device)
    device, n = residual.device, all_of[-1]
    if n > _MOST:
        _refuse(entry, _native.KLA_ERR_UNSUPPORTED)
    if weight is not None:
        _check("weight", weight, (n,), _F32, device)
    if scale is not None:
        _check("scale", scale, (n,), _F32, device)
    return device, _CODE[dtype], residual.numel() // max(1, n), n


def add_norm_fwd(x: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor] = None,
                 scale: Optional[torch.Tensor] = None, eps: float = 1e-5, *, norm: str = "rms",
                 out: Optional[torch.Tensor] = None, out_residual: Optional[torch.Tensor] = None, stats: bool = True):
    """Between two blocks: ``residual + scale * x``, and its norm over the last axis times ``weight`` for the next.

    x, residual: [..., n] bf16 or fp32, contiguous, 3 <= n <= 65536; weight, scale: fp32 [n] or None (1). Returns (y,
    the sum, both in x's dtype, mean, rstd fp32 [...] for the backward pass): mean is None with norm "rms", both
    without ``stats``. The norm is taken of the sum before it is rounded. ``out_residual`` may be ``residual``
    where no ``add_norm_bwd`` follows.
    """
    norm = _choice("norm", _NORMS, norm)
    device, code, rows, n = _added_inputs("kla_add_norm_fwd", x, residual, weight, scale)
    if out is None:
        out = torch.empty_like(residual)
    else:
        _check("out", out, residual.shape, residual.dtype, device)
    if out_residual is None:
        out_residual = torch.empty_like(residual)
    else:
        _check("out_residual", out_residual, residual.shape, residual.dtype, device)
    mean, rstd = _stats(residual, norm, stats, device)
    st = _native.on(device).kla_add_norm_fwd(x.data_ptr(), residual.data_ptr(), _ptr(weight), _ptr(scale),
                                             out.data_ptr(), out_residual.data_ptr(), _ptr(mean), _ptr(rstd), rows, n,
                                             code, norm, eps, _stream(device))
    if st:
        _native.check(st, "kla_add_norm_fwd")
    return out, out_residual, mean, rstd


def add_norm_bwd(dy: torch.Tensor, dresidual: Optional[torch.Tensor], x: torch.Tensor, residual: torch.Tensor,
                 weight: Optional[torch.Tensor], scale: Optional[torch.Tensor],
                 mean: Optional[torch.Tensor], rstd: torch.Tensor, *, workspace: Optional[torch.Tensor] = None):
    """Gradients of ``add_norm_fwd`` given dy, dresidual (of the sum it returned; None: nothing reaches it), its x,
    residual, weight, scale, mean (None: "rms") and rstd. The sum is formed again from x and residual: a forward call
    that this one follows keeps its ``residual``.

    Returns (dx, the gradient of the residual, dweight, dscale): without a scale dx is the residual's gradient itself
    and dscale is None. Equal calls give equal bits.
    """
    device, code, rows, n = _added_inputs("kla_add_norm_bwd", x, residual, weight, scale)
    shape, dtype = residual.shape, residual.dtype
    _check("dy", dy, shape, dtype, device)
    if dresidual is not None:
        _check("dresidual", dresidual, shape, dtype, device)
    if mean is not None:
        _check("mean", mean, shape[:-1], _F32, device)
    _check("rstd", rstd, shape[:-1], _F32, device)
    dr = torch.empty_like(residual)
    dx = dscale = None
    if scale is not None:
        dx, dscale = torch.empty_like(dr), torch.empty((n,), dtype=_F32, device=device)
    dw = torch.empty((n,), dtype=_F32, device=device)
    workspace, size = _scratch(_size("add_norm_bwd", rows, n, code), workspace, device)
    st = _native.on(device).kla_add_norm_bwd(dy.data_ptr(), _ptr(dresidual), x.data_ptr(), residual.data_ptr(),
                                             _ptr(weight), _ptr(scale), _ptr(mean), rstd.data_ptr(), _ptr(dx),
                                             dr.data_ptr(), dw.data_ptr(), _ptr(dscale), rows, n, code,
                                             _ptr(workspace), size, _stream(device))
    if st:
        _native.check(st, "kla_add_norm_bwd")
    return (dr if dx is None else dx), dr, dw, dscale


# --------------------------------------------------------------------------------- drafted tokens


def verify_draft(draft: torch.Tensor, draft_probs: Optional[torch.Tensor], target_probs: torch.Tensor,
                 uniforms: torch.Tensor, *, lengths: Optional[torch.Tensor] = None):
    """Which drafted tokens the target accepts, and the token after them, by given random numbers.

    draft: int32 [B,K]; draft_probs: [B,K,V] that the tokens were drawn from, or None (a draft that was sure of its
    tokens); target_probs: [B,K+1,V] (bf16 or fp32, as draft_probs; any strides with a dense last axis); uniforms: fp32
    [B,K+1] in [0, 1): draft i is accepted if every one before it was and ``uniforms[b,i] * q(token) < p(token)``, and
    ``uniforms[b,K]`` draws the next token, from the target's row behind the last draft or, where draft i was refused,
    from ``max(p - q, 0)`` there. ``lengths`` (int32 [B]): how many drafts each sequence has.

    Returns (accepted int32 [B], tokens int32 [B,K+1]: the accepted drafts, the next token, then -1). A model with
    states runs on over ``accepted + 1`` tokens (the last one of before and the accepted drafts): ``linear_fwd`` and
    ``gated_scan_fwd`` take those as their ``lengths``.
    """
    try:
        shape, dtype, at = target_probs.shape, target_probs.dtype, target_probs.get_device()
        B, rows, V = shape
        K = rows - 1
        ok = (at >= 0 and dtype in _CODE and rows > 0 and target_probs.is_contiguous() and max(shape) <= _MOST and
              draft.shape == (B, K) and draft.dtype is torch.int32 and draft.get_device() == at and
              draft.is_contiguous() and uniforms.shape == (B, rows) and uniforms.dtype is _F32 and
              uniforms.get_device() == at and uniforms.is_contiguous() and
              (draft_probs is None or (draft_probs.shape == (B, K, V) and draft_probs.dtype is dtype and
                                       draft_probs.get_device() == at and draft_probs.is_contiguous())))
    except (AttributeError, ValueError):
        ok = False
    strides = None
    if not ok:
        device = _device("target_probs", target_probs)
        _code("target_probs", target_probs)
        if target_probs.dim() != 3 or target_probs.shape[1] < 1:
            raise ValueError("target_probs must be [B, K + 1, V]")
        if max(shape) > _MOST:
            _refuse("kla_verify_draft", _native.KLA_ERR_UNSUPPORTED)
        _check("draft", draft, (B, K), torch.int32, device)
        _check("uniforms", uniforms, (B, rows), _F32, device)
        _dense_last(target_probs)
        qs = (K * V, V)
        if draft_probs is not None:
            _check("draft_probs", draft_probs, (B, K, V), dtype, device, False)
            _dense_last(draft_probs)
            qs = draft_probs.stride()[:2]
        strides = _Strides4(*qs, *target_probs.stride()[:2])
    device = target_probs.device
    if lengths is not None:
        _check("lengths", lengths, (B,), torch.int32, device)
    accepted = torch.empty((B,), dtype=torch.int32, device=device)
    tokens = torch.empty((B, rows), dtype=torch.int32, device=device)
    st = _native.on(device).kla_verify_draft(
        draft.data_ptr(), _ptr(draft_probs), target_probs.data_ptr(), strides,
        uniforms.data_ptr(), _ptr(lengths), accepted.data_ptr(), tokens.data_ptr(), B, K, V, _CODE[dtype],
        _stream(device))
    if st:
        _native.check(st, "kla_verify_draft")
    return accepted, tokens
