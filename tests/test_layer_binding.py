"""What the Python binding of include/kla_layer.h passes to the native library, on the CPU: a stand-in for the
library records every call, and host tensors stand for device ones."""
import pytest
import torch

from gated_delta_rule_14_gb300 import _native, layer


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
    monkeypatch.setattr(layer, "_device", lambda name, t: t.device)
    monkeypatch.setattr(layer, "_check", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    layer._size.cache_clear()
    yield lib
    layer._size.cache_clear()


@pytest.mark.parametrize("make", [
    lambda: torch.zeros(1, 3, 2, 16, 16).transpose(0, 1),   # three requests of one beam
    lambda: torch.zeros(1, 4, 2, 16, 16)[:, ::4],           # the first beam of one request
    lambda: torch.zeros(3, 1, 2, 16, 16),
    lambda: torch.zeros(2, 4, 2, 16, 16),
])
def test_a_state_has_the_bytes_of_its_shape(library, make):
    """An axis of one element may have any stride in a contiguous tensor, so a state's size is not a stride."""
    S = make()
    assert S.is_contiguous()
    layer.reorder_states(S, torch.zeros(S.shape[:2], dtype=torch.int32))
    (name, args), = library.calls
    assert name == "kla_reorder_states" and args[3:6] == (S.shape[0], S.shape[1], 2 * 16 * 16 * 4)


def test_bias_per_head_without_a_weight_has_its_gradient(library):
    """The forward takes heads apart by the bias' axes where there is no weight, and the backward has to do the same."""
    x, b = torch.randn(4, 6, 32), torch.zeros(6, 32)
    y, mean, rstd = layer.layer_norm_fwd(x, None, b)
    dx, dw, db = layer.layer_norm_bwd(x.clone(), x, None, mean, rstd, bias=b)
    (_, fwd), (_, bwd) = library.calls
    assert fwd[6:9] == bwd[8:11] == (4, 6, 32) and dw.shape == db.shape == (6, 32)
    _, dw, db = layer.layer_norm_bwd(x.clone(), x, None, mean, rstd)   # no parameters, or those of the last axis
    assert library.calls[-1][1][8:11] == (24, 1, 32) and dw.shape == db.shape == (32,)


WIDE = 2**32 + 64   # 64 once cut to 32 bits


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, device="meta", dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: layer.linear_fwd(*[meta(1, WIDE, 1, 16)] * 3, meta(1)),
    lambda: layer.linear_bwd(*[meta(1, WIDE, 1, 16)] * 3, meta(1), meta(1, WIDE, 1, 16)),
    lambda: layer.layer_norm_fwd(meta(3, WIDE)),
    lambda: layer.layer_norm_fwd(meta(3, WIDE, 32), meta(WIDE, 32)),
    lambda: layer.layer_norm_bwd(meta(3, WIDE), meta(3, WIDE), None, meta(3), meta(3)),
    lambda: layer.beam_select(meta(1, 1, WIDE), meta(1, 1)),
    lambda: layer.beam_select(meta(WIDE, 1, 10), meta(WIDE, 1)),
    lambda: layer.reorder_states(meta(WIDE, 1, 16), meta(WIDE, 1)),
    lambda: layer.reorder_states(meta(1, WIDE, 16), meta(1, WIDE)),
    lambda: layer.beam_select(meta(1, 1, 100), meta(1, 1), eos=2**32 + 5),
    lambda: layer.beam_select(meta(1, 1, 100), meta(1, 1), eos=-2**32 + 5),
])
def test_numbers_past_32_bits_do_not_reach_the_library(library, call):
    """ctypes would cut them without a word, and the call would be one on other sizes."""
    with pytest.raises(_native.KlaError):
        call()
    assert not library.calls


def test_rows_are_64_bit(library):
    layer.layer_norm_fwd(meta(2**31, 3, 4), stats=False)   # the library's own limit refuses these rows
    assert library.calls[0][1][6:9] == (3 * 2**31, 1, 4)
