"""ctypes handle on libkla_gb300.so (the C ABI of include/kla.h).

Argument marshalling only: no arithmetic of the recurrence happens in Python.
If the library has not been built, loading fails loudly; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

KLA_OK = 0
KLA_ERR_INVALID_ARG = 1
KLA_ERR_UNSUPPORTED = 2
KLA_ERR_CUDA = 3
KLA_ERR_TIMEOUT = 4

KLA_DTYPE_F32 = 0
KLA_DTYPE_BF16 = 1
KLA_GATE_SCALAR = 0
KLA_GATE_CHANNEL = 1
KLA_BETA_KACZMARZ = 0
KLA_BETA_RAW = 1
KLA_SCAN_SIGMOID = 0
KLA_SCAN_LOG = 1
KLA_ROTARY_HALF = 0
KLA_ROTARY_INTERLEAVED = 1
KLA_NORM_RMS = 0
KLA_NORM_LAYER = 1
KLA_ACT_SILU = 0
KLA_ACT_SIGMOID = 1

_lock = threading.Lock()
_lib = None


class KlaError(RuntimeError):
    """A KLA C-ABI call returned a status other than KLA_OK."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def library_path() -> str:
    return _build.LIB


def _declare(lib):
    vp, fp, i, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.kla_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, ctypes.c_float, fp, vp, fp,
                                  i, i, i, i, i, i, i, i, vp, sz, vp]
    lib.kla_chunk_fwd.restype = ctypes.c_int
    lib.kla_chunk_fwd_ex.argtypes = [vp, vp, vp, fp, fp, ctypes.c_float, fp, vp, fp,
                                     i, i, i, i, i, i, i, i, i, ctypes.c_float, vp, sz, vp]
    lib.kla_chunk_fwd_ex.restype = ctypes.c_int
    lib.kla_chunk_fwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
    lib.kla_chunk_fwd_workspace_size.restype = sz
    lib.kla_decode_step.argtypes = [vp, vp, vp, fp, fp, ctypes.c_float, fp, vp, i, i, i, i, i, i, vp]
    lib.kla_decode_step.restype = ctypes.c_int
    lib.kla_decode_step_ex.argtypes = [vp, vp, vp, fp, fp, ctypes.c_float, fp, vp, i, i, i, i, i, i, i,
                                       ctypes.c_float, vp]
    lib.kla_decode_step_ex.restype = ctypes.c_int
    lib.kla_chunk_fwd_host.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, vp, vp, vp, fp, fp, fp, vp, fp, ctypes.c_float,
                                       i, i, i, i, i, i, i, i, i, ctypes.c_float, i, vp]
    lib.kla_chunk_fwd_host.restype = ctypes.c_int
    lib.kla_chunk_bwd.argtypes = [vp, vp, vp, fp, fp, ctypes.c_float, fp, vp, fp, fp, fp, fp, fp, fp, fp,
                                  i, i, i, i, i, i, i, i, ctypes.c_float, vp, sz, vp]
    lib.kla_chunk_bwd.restype = ctypes.c_int
    lib.kla_chunk_bwd_workspace_size.argtypes = [i, i, i, i, i]
    lib.kla_chunk_bwd_workspace_size.restype = sz
    lib.kla_chunk_bwd_workspace_size_ex.argtypes = [i, i, i, i, i, i, i]
    lib.kla_chunk_bwd_workspace_size_ex.restype = sz
    i64, f = ctypes.c_int64, ctypes.c_float
    lib.kla_linear_fwd.argtypes = [vp, vp, vp, vp, fp, vp, fp, vp, fp, i, i, i, i, i, i, f, vp, sz, vp]
    lib.kla_linear_fwd_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.kla_linear_bwd.argtypes = [vp, vp, vp, vp, vp, fp, vp, fp, fp, vp, vp, vp, fp, i, i, i, i, i, i, f, vp, sz, vp]
    lib.kla_linear_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.kla_linear_step.argtypes = [vp, vp, vp, fp, vp, fp, fp, vp, i, i, i, i, i, i, f, vp]
    lib.kla_layer_norm_fwd.argtypes = [vp, fp, fp, vp, fp, fp, i64, i, i, i, f, vp]
    lib.kla_layer_norm_bwd.argtypes = [vp, vp, fp, fp, fp, vp, fp, fp, i64, i, i, i, vp, sz, vp]
    lib.kla_layer_norm_bwd_workspace_size.argtypes = [i64, i, i, i]
    lib.kla_beam_select.argtypes = [vp, i64, fp, vp, i, fp, vp, vp, vp, i, i, i, i, vp, sz, vp]
    lib.kla_beam_select_workspace_size.argtypes = [i, i, i, i]
    lib.kla_reorder_states.argtypes = [vp, vp, vp, i, i, sz, vp]
    lib.kla_gated_scan_fwd.argtypes = [vp, vp, vp, vp, fp, vp, fp, fp, i, i, i, i, i, vp, sz, vp]
    lib.kla_gated_scan_bwd.argtypes = [vp, vp, vp, vp, vp, fp, fp, vp, vp, fp, i, i, i, i, i, vp, sz, vp]
    lib.kla_gated_scan_step.argtypes = [vp, i64, vp, i64, fp, vp, i, i, i, i, vp]
    lib.kla_gated_scan_workspace_size.argtypes = [i, i, i, i]
    lib.kla_rotary.argtypes = [vp, vp, vp, vp, vp, fp, vp, i, i, i, i, i, i, i, i, i, f, i, vp]
    lib.kla_gated_norm_fwd.argtypes = [vp, vp, i64, fp, i, vp, fp, fp, i64, i, i, i, i, i, f, vp]
    lib.kla_gated_norm_bwd.argtypes = [vp, vp, vp, i64, fp, i, fp, fp, vp, vp, fp, i64, i, i, i, i, vp, sz, vp]
    lib.kla_gated_norm_bwd_workspace_size.argtypes = [i64, i, i, i, i]
    lib.kla_add_norm_fwd.argtypes = [vp, vp, fp, fp, vp, vp, fp, fp, i64, i, i, i, f, vp]
    lib.kla_add_norm_bwd.argtypes = [vp, vp, vp, vp, fp, fp, fp, fp, vp, vp, fp, fp, i64, i, i, vp, sz, vp]
    lib.kla_add_norm_bwd_workspace_size.argtypes = [i64, i, i]
    lib.kla_verify_draft.argtypes = [vp, vp, vp, vp, fp, vp, vp, vp, i, i, i, i, vp]
    for name in ("linear_fwd", "linear_bwd", "linear_step", "layer_norm_fwd", "layer_norm_bwd", "beam_select",
                 "reorder_states", "gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "rotary", "gated_norm_fwd",
                 "gated_norm_bwd", "add_norm_fwd", "add_norm_bwd", "verify_draft"):
        getattr(lib, "kla_" + name).restype = ctypes.c_int
    for name in ("linear_fwd", "linear_bwd", "layer_norm_bwd", "beam_select", "gated_scan", "gated_norm_bwd",
                 "add_norm_bwd"):
        getattr(lib, f"kla_{name}_workspace_size").restype = sz
    lib.kla_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
    lib.kla_selftest_wait_timeout.restype = ctypes.c_int
    lib.kla_selftest_team_timeout.argtypes = [ctypes.c_uint, vp, vp]
    lib.kla_selftest_team_timeout.restype = ctypes.c_int
    lib.kla_selftest_warp_timeout.argtypes = [ctypes.c_uint, vp, vp]
    lib.kla_selftest_warp_timeout.restype = ctypes.c_int
    lib.kla_selftest_scan_timeout.argtypes = [ctypes.c_uint, i, vp, fp, vp, vp, i, i, i, i, vp, sz, vp]
    lib.kla_selftest_scan_timeout.restype = ctypes.c_int
    lib.kla_device_status.argtypes = [vp]
    lib.kla_device_status.restype = ctypes.c_int
    lib.kla_status_string.argtypes = [ctypes.c_int]
    lib.kla_status_string.restype = ctypes.c_char_p
    lib.kla_abi_version.argtypes = []
    lib.kla_abi_version.restype = ctypes.c_int
    return lib


def lib():
    """Load libkla_gb300.so once; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"KLA CUDA library not found at {path}; build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
            _lib = _declare(ctypes.CDLL(path))
        return _lib


class _OnDevice:
    """The library's entry points with a device made current around each call."""

    def __init__(self, index: int):
        self._index = index

    def __getattr__(self, name):
        entry = getattr(lib(), name)

        def call(*args):
            with torch.cuda.device(self._index):
                return entry(*args)
        return call


def on(device: torch.device):
    """The library, for calls on tensors of ``device``: launches, kernel attributes and the error word go by the
    current device, whichever one the pointers and the stream belong to."""
    index = device.index
    if index is None or index == torch._C._cuda_getDevice():   # without an index: the current one
        return lib()
    return _OnDevice(index)


def status_string(status: int) -> str:
    return lib().kla_status_string(int(status)).decode()


def check(status: int, what: str) -> None:
    if status != KLA_OK:
        raise KlaError(status, what)
