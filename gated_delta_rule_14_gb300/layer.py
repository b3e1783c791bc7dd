"""What a layer and a decoding loop need next to the recurrence (the C ABI of include/kla_layer.h):
linear attention with one decay per head (``linear_fwd``, ``linear_step``, ``linear_bwd``), layer norm
with its gradients (``layer_norm_fwd``, ``layer_norm_bwd``) and beam search's selection with the states
following their beams (``beam_select``, ``reorder_states``).

The binding checks and marshals; every operation runs in this package's CUDA kernels on the current
stream of the tensors' device, whether or not that device is the current one. Small calls are bound by
the host, so linear attention's functions first ask in one expression whether everything is as it should
be, and only where it is not go through the arguments one by one to name the one at fault.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import _native

_F32, _BF16 = torch.float32, torch.bfloat16
_CODE = {_F32: _native.KLA_DTYPE_F32, _BF16: _native.KLA_DTYPE_BF16}
_Strides3, _Strides4 = ctypes.c_int64 * 9, ctypes.c_int64 * 12


def _code(name: str, t: torch.Tensor) -> int:
    try:
        return _CODE[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}") from None


def _check(name: str, t: torch.Tensor, shape, dtype, device, contiguous: bool = True) -> None:
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and (
                not contiguous or t.is_contiguous()):
            return
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    raise ValueError(f"{name} must be contiguous")


def _device(name: str, t: torch.Tensor) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    return t.device


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


_MOST = 2**31 - 1   # of a C int: ctypes would cut a larger number to its low 32 bits


def _refuse(entry: str, status: int):
    raise _native.KlaError(status, entry)


@functools.lru_cache(maxsize=256)
def _size(query: str, *sizes) -> int:
    """Scratch bytes of a call: they follow from its sizes alone."""
    if max(sizes) > _MOST:
        _refuse(f"kla_{query}", _native.KLA_ERR_UNSUPPORTED)
    return getattr(_native.lib(), f"kla_{query}_workspace_size")(*sizes)


def _scratch(need: int, given: Optional[torch.Tensor], device: torch.device) -> Tuple[Optional[torch.Tensor], int]:
    if given is None:
        return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)
    if given.device != device or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return given, given.numel() * given.element_size()


def _token_strides(kind, *tensors):
    """Batch, token and head strides of tensors whose last axis is dense."""
    out = []
    for t in tensors:
        st = t.stride()
        if st[3] != 1 and t.shape[3] > 1:
            raise ValueError("the last axis of q, k, v and dO must be contiguous")
        out += st[:3]
    return kind(*out)


# ------------------------------------------------------------------------------- linear attention


def _linear_shapes(q, k, v, decay, S0, lengths):
    """Sizes of the call, and whether q, k and v are contiguous and v is shaped like q."""
    try:
        shape, dtype, at = q.shape, q.dtype, q.get_device()
        alike = (at >= 0 and len(shape) == 4 and k.shape == shape and v.shape == shape and k.dtype is dtype and
                 v.dtype is dtype and k.get_device() == at and v.get_device() == at and q.is_contiguous() and
                 k.is_contiguous() and v.is_contiguous() and decay.dtype is _F32 and decay.shape == shape[2:3] and
                 decay.get_device() == at and decay.is_contiguous() and dtype in _CODE)
    except AttributeError:
        alike = False
    if not alike:
        device = _device("q", q)
        _code("q", q)
        if q.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
            raise ValueError("q and k must be [B, T, H, d_k] and v [B, T, H, d_v]")
        _check("k", k, q.shape, q.dtype, device, False)
        _check("v", v, (*q.shape[:3], v.shape[3]), q.dtype, device, False)
        _check("decay", decay, q.shape[2:3], _F32, device)
    device = q.device
    B, T, H, d_k = shape
    d_v = v.shape[3]
    if S0 is not None:
        _check("S0", S0, (B, H, d_k, d_v), _F32, device)
    if lengths is not None:
        _check("lengths", lengths, (B,), torch.int32, device)
    return device, _CODE[dtype], B, T, H, d_k, d_v, alike


def linear_workspace_size(B: int, T: int, H: int, d_k: int, d_v: int, dtype: torch.dtype = _BF16,
                          backward: bool = False) -> int:
    """Device scratch bytes ``linear_fwd`` (or ``linear_bwd``) needs for these sizes."""
    return _size("linear_bwd" if backward else "linear_fwd", B, T, H, d_k, d_v, _CODE[dtype])


def linear_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
               S0: Optional[torch.Tensor] = None, *, q_scale: float = 1.0, lengths: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, final_state: bool = True, S_T: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with one decay per head over whole prompts:
    ``S_t = decay S_{t-1} + k_t v_t^T``, ``o_t = S_t^T (q_scale q_t)``.

    q, k: [B,T,H,d_k], v: [B,T,H,d_v] (bf16 or fp32; any strides with a dense last axis, as the slices of a
    packed projection); decay: fp32 [H] in [0, 1]; S0: fp32 [B,H,d_k,d_v] or None (zeros). ``lengths``
    (int32 [B]) masks the tokens from lengths[b] on: they leave the state alone and their outputs are 0.
    Returns (o [B,T,H,d_v] in q's dtype, S_T fp32 or None); ``S_T`` may be passed, and may be ``S0``.
    """
    device, code, B, T, H, d_k, d_v, dense = _linear_shapes(q, k, v, decay, S0, lengths)
    if out is None:
        out = torch.empty_like(v) if dense else torch.empty((B, T, H, d_v), dtype=q.dtype, device=device)
    else:
        _check("out", out, (B, T, H, d_v), q.dtype, device)
    if S_T is not None:
        _check("S_T", S_T, (B, H, d_k, d_v), _F32, device)
    elif final_state:
        S_T = torch.empty((B, H, d_k, d_v), dtype=_F32, device=device)
    workspace, size = _scratch(_size("linear_fwd", B, T, H, d_k, d_v, code), workspace, device)
    st = _native.on(device).kla_linear_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), None if dense else _token_strides(_Strides3, q, k, v),
        decay.data_ptr(), _ptr(lengths), _ptr(S0), out.data_ptr(), _ptr(S_T), B, T, H, d_k, d_v, code, q_scale,
        _ptr(workspace), size, _stream(device))
    if st:
        _native.check(st, "kla_linear_fwd")
    return out, S_T


def linear_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor, dO: torch.Tensor,
               S0: Optional[torch.Tensor] = None, dS_T: Optional[torch.Tensor] = None, *, q_scale: float = 1.0,
               lengths: Optional[torch.Tensor] = None, want_dS0: bool = True,
               workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``linear_fwd`` run with the same inputs and options, given dO = dL/do and dS_T = dL/dS_T.

    Returns dq, dk [B,T,H,d_k] and dv [B,T,H,d_v] in q's dtype (zero at masked tokens) and dS0 fp32
    [B,H,d_k,d_v] (None unless ``want_dS0``). ``decay`` is a constant and gets no gradient.
    """
    device, code, B, T, H, d_k, d_v, dense = _linear_shapes(q, k, v, decay, S0, lengths)
    _check("dO", dO, (B, T, H, d_v), q.dtype, device, False)
    dense = dense and dO.is_contiguous()
    if dS_T is not None:
        _check("dS_T", dS_T, (B, H, d_k, d_v), _F32, device)
    dq = torch.empty((B, T, H, d_k), dtype=q.dtype, device=device)
    dk, dv = torch.empty_like(dq), torch.empty((B, T, H, d_v), dtype=q.dtype, device=device)
    dS0 = torch.empty((B, H, d_k, d_v), dtype=_F32, device=device) if want_dS0 else None
    workspace, size = _scratch(_size("linear_bwd", B, T, H, d_k, d_v, code), workspace, device)
    st = _native.on(device).kla_linear_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), dO.data_ptr(),
        None if dense else _token_strides(_Strides4, q, k, v, dO), decay.data_ptr(), _ptr(lengths), _ptr(S0),
        _ptr(dS_T), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(dS0), B, T, H, d_k, d_v, code, q_scale,
        _ptr(workspace), size, _stream(device))
    if st:
        _native.check(st, "kla_linear_bwd")
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS0}


def linear_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor, S: torch.Tensor, *,
                q_scale: float = 1.0, parent: Optional[torch.Tensor] = None, S_out: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for B sequences: ``S = decay S + k v^T``, ``o = S^T (q_scale q)``.

    q, k: [B,H,d_k]; v: [B,H,d_v]; S: fp32 [B,H,d_k,d_v], updated in place unless ``S_out`` is given.
    ``parent`` (int32 [B]): sequence b goes on from state ``S[parent[b]]`` (S may then hold any number of
    states; an index outside of them starts from zeros) and its new state goes to ``S_out[b]``, which is then
    required: a beam search's states follow their beams without a pass of their own. Returns o [B,H,d_v].
    """
    try:
        shape, dtype, at = q.shape, q.dtype, q.get_device()
        B, H, d_k = shape
        d_v = v.shape[2]
        ok = (at >= 0 and k.shape == shape and v.shape[:2] == shape[:2] and k.dtype is dtype and v.dtype is dtype and
              k.get_device() == at and v.get_device() == at and q.is_contiguous() and k.is_contiguous() and
              v.is_contiguous() and decay.dtype is _F32 and decay.shape == shape[1:2] and decay.get_device() == at and
              decay.is_contiguous() and dtype in _CODE)
    except (AttributeError, ValueError, IndexError):
        ok = False
    if not ok:
        device = _device("q", q)
        _code("q", q)
        if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
            raise ValueError("q and k must be [B, H, d_k] and v [B, H, d_v]")
        _check("q", q, q.shape, q.dtype, device)
        _check("k", k, q.shape, q.dtype, device)
        _check("v", v, (*q.shape[:2], v.shape[2]), q.dtype, device)
        _check("decay", decay, q.shape[1:2], _F32, device)
    device = q.device
    n = B
    if parent is not None:
        _check("parent", parent, (B,), torch.int32, device)
        if S_out is None:
            raise ValueError("parent needs S_out: a state may go on in several sequences")
        n = S.shape[0] if isinstance(S, torch.Tensor) and S.dim() == 4 else B
    _check("S", S, (n, H, d_k, d_v), _F32, device)
    if S_out is None:
        S_out = S
    else:
        _check("S_out", S_out, (B, H, d_k, d_v), _F32, device)
    if out is None:
        out = torch.empty_like(v)
    else:
        _check("out", out, v.shape, dtype, device)
    st = _native.on(device).kla_linear_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), _ptr(parent),
                                            S.data_ptr(), S_out.data_ptr(), out.data_ptr(), B, H, d_k, d_v, n,
                                            _CODE[dtype], q_scale, _stream(device))
    if st:
        _native.check(st, "kla_linear_step")
    return out


# ------------------------------------------------------------------------------------- layer norm


def _norm_shape(x: torch.Tensor, weight, bias):
    """(rows, groups, n): weights over the last axis, or over the last two (one set per head)."""
    if x.dim() < 1:
        raise ValueError("x must have an axis to normalise")
    param = weight if weight is not None else bias
    n = x.shape[-1]
    if param is not None and param.dim() == 2:
        if x.dim() < 2:
            raise ValueError("weights of two axes need an x of two axes or more")
        groups = x.shape[-2]
        return x.numel() // max(1, groups * n), groups, n, (groups, n)
    return x.numel() // max(1, n), 1, n, (n,)


def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, *, out: Optional[torch.Tensor] = None, stats: bool = True):
    """Layer norm over the last axis: ``y = (x - mean) / sqrt(var + eps) * weight + bias``.

    x: [..., n] bf16 or fp32, 3 <= n <= 65536; weight, bias: fp32 [n], or [H, n] for x [..., H, n] (every head's
    output with weights of its own). Returns (y in x's dtype, mean, rstd fp32 [...] for the backward pass, or
    None, None without ``stats``).
    """
    device = _device("x", x)
    code = _code("x", x)
    rows, groups, n, shape = _norm_shape(x, weight, bias)
    if n > _MOST or groups > _MOST:
        _refuse("kla_layer_norm_fwd", _native.KLA_ERR_UNSUPPORTED)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if weight is not None:
        _check("weight", weight, shape, _F32, device)
    if bias is not None:
        _check("bias", bias, shape, _F32, device)
    if out is None:
        out = torch.empty_like(x)
    else:
        _check("out", out, x.shape, x.dtype, device)
    mean = rstd = None
    if stats:
        mean = torch.empty(x.shape[:-1], dtype=_F32, device=device)
        rstd = torch.empty_like(mean)
    st = _native.on(device).kla_layer_norm_fwd(x.data_ptr(), _ptr(weight), _ptr(bias), out.data_ptr(), _ptr(mean),
                                               _ptr(rstd), rows, groups, n, code, eps, _stream(device))
    if st:
        _native.check(st, "kla_layer_norm_fwd")
    return out, mean, rstd


def layer_norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                   rstd: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of ``layer_norm_fwd`` given its x, weight, mean and rstd: (dx in x's dtype, dweight, dbias
    fp32, shaped like the parameters). ``bias``: the forward's, whose values are not read; it is needed where
    there is no weight and the bias is one of [H, n], as it alone says then that heads have gradients of their
    own (with neither, dweight and dbias are [n]). Equal calls give equal bits."""
    device = _device("x", x)
    code = _code("x", x)
    rows, groups, n, shape = _norm_shape(x, weight, bias)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _check("dy", dy, x.shape, x.dtype, device)
    if weight is not None:
        _check("weight", weight, shape, _F32, device)
    if bias is not None:
        _check("bias", bias, shape, _F32, device)
    _check("mean", mean, x.shape[:-1], _F32, device)
    _check("rstd", rstd, x.shape[:-1], _F32, device)
    dx = torch.empty_like(x)
    dw = torch.empty(shape, dtype=_F32, device=device)
    db = torch.empty_like(dw)
    workspace, size = _scratch(_size("layer_norm_bwd", rows, groups, n, code), workspace, device)
    st = _native.on(device).kla_layer_norm_bwd(dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(),
                                               rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(), db.data_ptr(), rows,
                                               groups, n, code, _ptr(workspace), size, _stream(device))
    if st:
        _native.check(st, "kla_layer_norm_bwd")
    return dx, dw, db


# ------------------------------------------------------------------------------------ beam search


def beam_select(logits: torch.Tensor, scores: torch.Tensor, finished: Optional[torch.Tensor] = None, *,
                eos: int = -1, workspace: Optional[torch.Tensor] = None):
    """One selection of W beams over W beams and V tokens, for B requests.

    logits: [B,W,V] bf16 or fp32 (dense last axis, rows a constant stride apart: a padded vocabulary may be
    sliced); scores: fp32 [B,W], the beams' log-probabilities (-inf: a dead beam); finished: bool [B,W] or
    None; eos: the token that finishes a beam (-1: none). A candidate scores ``scores[b,w] +
    log_softmax(logits[b,w])[token]``; a finished beam goes on with eos alone at no cost. Candidates of one
    beam rank by logit (equal: the lower token), beams merge by score (equal: the lower beam). Returns
    (scores [B,W] descending, parents int32, tokens int32, finished bool).
    """
    device = _device("logits", logits)
    code = _code("logits", logits)
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    B, W, V = logits.shape
    s0, stride, last = logits.stride()
    if W == 1:
        stride = s0 if B > 1 else V
    if (last != 1 and V > 1) or (B > 1 and s0 != W * stride):
        raise ValueError("the rows of logits must be dense and a constant stride apart")
    _check("scores", scores, (B, W), _F32, device)
    if finished is not None:
        _check("finished", finished, (B, W), torch.bool, device)
    if not -1 <= eos < V:
        _refuse("kla_beam_select", _native.KLA_ERR_INVALID_ARG)
    new_scores = torch.empty_like(scores)
    parents = torch.empty((B, W), dtype=torch.int32, device=device)
    tokens = torch.empty_like(parents)
    done = torch.empty((B, W), dtype=torch.bool, device=device)
    workspace, size = _scratch(_size("beam_select", B, W, V, code), workspace, device)
    st = _native.on(device).kla_beam_select(logits.data_ptr(), stride, scores.data_ptr(), _ptr(finished), eos,
                                            new_scores.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
                                            done.data_ptr(), B, W, V, code, _ptr(workspace), size, _stream(device))
    if st:
        _native.check(st, "kla_beam_select")
    return new_scores, parents, tokens, done


def reorder_states(S: torch.Tensor, parents: torch.Tensor, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``out[b, w] = S[b, parents[b, w]]``: S [B, W, ...] of any dtype whose states are a multiple of 16 bytes
    (the states of ``decode_step`` and ``linear_step`` alike), parents int32 [B, W]; a parent outside [0, W)
    gives a zero state. ``out`` must not overlap S."""
    device = _device("S", S)
    if S.dim() < 3:
        raise ValueError("S must be [B, W, ...]")
    if not S.is_contiguous():
        raise ValueError("S must be contiguous")
    shape = S.shape
    B, W = shape[:2]
    if B > _MOST or W > _MOST:
        _refuse("kla_reorder_states", _native.KLA_ERR_UNSUPPORTED)
    _check("parents", parents, (B, W), torch.int32, device)
    if out is None:
        out = torch.empty_like(S)
    else:
        _check("out", out, shape, S.dtype, device)
    # from the shape: an axis of one element may have any stride in a contiguous tensor
    st = _native.on(device).kla_reorder_states(S.data_ptr(), parents.data_ptr(), out.data_ptr(), B, W,
                                               math.prod(shape[2:]) * S.element_size(), _stream(device))
    if st:
        _native.check(st, "kla_reorder_states")
    return out
