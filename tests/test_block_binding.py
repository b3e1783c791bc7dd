"""What the Python binding of include/kla_block.h passes to the native library, on the CPU: a stand-in for the library
records every call, and host tensors stand for device ones."""
import contextlib

import pytest
import torch

import gated_delta_rule_14_gb300 as kla
from gated_delta_rule_14_gb300 import _native, block, layer


class Library:
    """Answers every entry point with success and keeps its arguments; workspaces are empty."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            if name.endswith("_workspace_size"):
                return 0
            if name == "kla_status_string":
                return b""
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(_native, "lib", lambda: lib)
    monkeypatch.setattr(block, "_device", lambda name, t: t.device)
    monkeypatch.setattr(block, "_check", lambda *a: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    layer._size.cache_clear()
    yield lib
    layer._size.cache_clear()


WIDE = 2**32 + 64   # 64 once cut to 32 bits


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, device="meta", dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: block.gated_scan_fwd(meta(1, WIDE, 1), meta(1, WIDE, 1)),
    lambda: block.gated_scan_fwd(meta(1, 1, WIDE), meta(1, 1, WIDE)),
    lambda: block.gated_scan_bwd(meta(WIDE, 1, 1), meta(WIDE, 1, 1), meta(WIDE, 1, 1), meta(WIDE, 1, 1)),
    lambda: block.gated_scan_step(meta(1, WIDE), meta(1, WIDE), meta(1, WIDE)),
    lambda: block.gated_scan_step(meta(WIDE, 1), meta(WIDE, 1), meta(WIDE, 1)),
    lambda: block.rotary_fwd(meta(1, WIDE, 1, 2), None, meta(1)),
    lambda: block.rotary_fwd(meta(1, 1, WIDE, 2), None, meta(1)),
    lambda: block.rotary_fwd(meta(1, 1, 1, 2), meta(1, 1, WIDE, 2), meta(1)),
    lambda: block.rotary_fwd(meta(1, 1, 1, WIDE), None, meta(WIDE // 2 + 1)),
    lambda: block.rotary_fwd(meta(1, 1, 1, 64), None, meta(2**31 + 4)),
    lambda: block.gated_norm_fwd(meta(3, WIDE), meta(3, WIDE)),
    lambda: block.gated_norm_fwd(meta(3, WIDE, 32), meta(3, WIDE, 32), meta(WIDE, 32)),
    lambda: block.gated_norm_bwd(meta(3, WIDE), meta(3, WIDE), meta(3, WIDE), None, None, meta(3)),
    lambda: block.add_norm_fwd(meta(3, WIDE), meta(3, WIDE)),
    lambda: block.add_norm_bwd(meta(3, WIDE), None, meta(3, WIDE), meta(3, WIDE), None, None, None, meta(3)),
    lambda: block.verify_draft(meta(1, 1), None, meta(1, 2, WIDE), meta(1, 2)),
    lambda: block.verify_draft(meta(1, WIDE), None, meta(1, WIDE, 10), meta(1, WIDE)),
    lambda: block.verify_draft(meta(WIDE, 1), None, meta(WIDE, 2, 10), meta(WIDE, 2)),
])
def test_numbers_past_32_bits_do_not_reach_the_library(library, call):
    """ctypes would cut them without a word, and the call would be one on other sizes."""
    with pytest.raises(_native.KlaError):
        call()
    assert not library.calls


def test_rows_are_64_bit(library):
    block.gated_norm_fwd(meta(2**31, 3, 4), meta(2**31, 3, 4), stats=False)   # the library's own limit refuses these
    block.add_norm_fwd(meta(2**31, 3, 4), meta(2**31, 3, 4), stats=False)
    assert library.calls[0][1][8:11] == (3 * 2**31, 1, 4) and library.calls[1][1][8:10] == (3 * 2**31, 4)


def gate_of(shape, kind):
    """(a gate of this shape, its rows' stride)"""
    n = shape[-1]
    if kind == "whole":
        return torch.zeros(shape)
    if kind == "slice":      # [..., H n] of a packed projection's [..., 3 H n]
        flat = torch.zeros(*shape[:-2], 3 * shape[-2] * n)
        return flat[..., shape[-2] * n:2 * shape[-2] * n].unflatten(-1, shape[-2:])
    return torch.zeros(*shape[:-1], 2 * n)[..., :n]


@pytest.mark.parametrize("shape,weight,kind,want", [
    ((4, 5, 6, 8), (8,), "whole", (120, 1, 8, 0, 8)),
    ((4, 5, 6, 8), (6, 8), "whole", (20, 6, 8, 1, 48)),
    ((4, 5, 6, 8), (8,), "slice", (20, 6, 8, 0, 144)),
    ((4, 5, 6, 8), (6, 8), "slice", (20, 6, 8, 1, 144)),
    ((4, 5, 6, 8), (8,), "rows", (120, 1, 8, 0, 16)),
    ((4, 5, 6, 8), None, "rows", (120, 1, 8, 0, 16)),
    ((1, 1, 6, 8), (6, 8), "slice", (1, 6, 8, 1, 48)),
    ((7, 8), (8,), "rows", (7, 1, 8, 0, 16)),
    ((4, 1, 8), (1, 8), "slice", (4, 1, 8, 1, 24)),
    ((4, 5, 1, 8), (8,), "slice", (20, 1, 8, 0, 24)),
])
def test_a_gate_of_a_packed_projection(library, shape, weight, kind, want):
    x, gate = torch.zeros(shape), gate_of(shape, kind)
    w = None if weight is None else torch.zeros(weight)
    block.gated_norm_fwd(x, gate, w)
    _, a = library.calls[-1]
    assert (a[8], a[9], a[10], a[4], a[2]) == want
    _, _, dw = block.gated_norm_bwd(x.clone(), x, gate, w, None, torch.zeros(shape[:-1]))
    _, b = library.calls[-1]
    assert (b[11], b[12], b[13], b[5], b[3]) == want and dw.shape == (weight or (8,))


@pytest.mark.parametrize("gate", [
    torch.zeros(5, 4, 6, 8).transpose(0, 1),
    torch.zeros(4, 5, 6, 16)[..., ::2],
    torch.zeros(4, 5, 12, 8)[:, :, ::2],
    torch.zeros(4, 10, 6, 8)[:, ::2][:, :, :, :].transpose(0, 1)[:4].transpose(0, 1)[:, :4].transpose(0, 1),
])
def test_a_gate_of_scattered_rows_is_refused(library, gate):
    with pytest.raises(ValueError, match="gate"):
        block.gated_norm_fwd(torch.zeros(gate.shape), gate, torch.zeros(6, 8))
    assert not library.calls


def test_one_row_may_have_any_stride(library):
    x = torch.zeros(8, 3).t()[:1, ::2]
    assert x.stride(1) != 1
    with pytest.raises(ValueError):
        block.gated_scan_step(x, x, torch.zeros(x.shape))
    one = torch.zeros(1, 5)[:, :4]
    block.gated_scan_step(one, one, torch.zeros(1, 4))
    assert library.calls[-1][1][1] == 4 and library.calls[-1][1][3] == 4


# ------------------------------------------------------------ whose device and stream a call runs on


class OnDevice1(torch.Tensor):
    device = property(lambda self: torch.device("cuda", 1))
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


def place(t):
    return t.as_subclass(OnDevice1)


@pytest.fixture
def calls(monkeypatch):
    """(entry point, current device, stream) of every call but the size queries."""
    current, seen, empty = [0], [], torch.empty

    class Native:
        def __getattr__(self, name):
            def entry(*args):
                if "_size" in name:
                    return 64
                seen.append((name, current[0], args[-1]))
                return 0
            return entry

    @contextlib.contextmanager
    def device(to):
        before, current[0] = current[0], to if isinstance(to, int) else to.index
        yield
        current[0] = before

    lib = Native()
    monkeypatch.setattr(_native, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: place(empty(*a, **k)))
    layer._size.cache_clear()
    yield seen
    layer._size.cache_clear()
    assert current == [0]


def test_calls_run_on_their_tensors_device(calls):
    x = place(torch.zeros(2, 4, 16))
    _, _, s = kla.gated_scan_fwd(x, x, states=True)
    kla.gated_scan_bwd(x, x, x, s)
    one = place(torch.zeros(2, 16))
    kla.gated_scan_step(one, one, place(torch.zeros(2, 16)))
    q, f = place(torch.zeros(2, 4, 3, 16)), place(torch.zeros(8))
    kla.rotary_fwd(q, q, f)
    kla.rotary_bwd(q, None, f)
    y, mean, rstd = kla.gated_norm_fwd(x, x)
    kla.gated_norm_bwd(x, x, x, None, mean, rstd)
    y, _, mean, rstd = kla.add_norm_fwd(x, x)
    kla.add_norm_bwd(x, None, x, x, None, None, mean, rstd)
    kla.verify_draft(place(torch.zeros(2, 3, dtype=torch.int32)), None, x, place(torch.zeros(2, 4)))
    assert calls == [(f"kla_{name}", 1, 101) for name in (
        "gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "rotary", "rotary", "gated_norm_fwd", "gated_norm_bwd",
        "add_norm_fwd", "add_norm_bwd", "verify_draft")]
