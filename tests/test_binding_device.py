"""Every call of the binding runs with the tensors' device current and on its current stream, whatever device
is current outside. On the CPU: host tensors that say they are on cuda:1 while cuda:0 is current, and a stand-in
for the native library that notes which device is current when it is called. (On a GPU the wrong one would mean
launches on one device with pointers of another.)"""
import contextlib
import types

import pytest
import torch

import gated_delta_rule_14_gb300 as kla
from gated_delta_rule_14_gb300 import _native, layer


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

    class Library:
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

    monkeypatch.setattr(_native, "lib", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=100 + (
        current[0] if d is None or torch.device(d).index is None else torch.device(d).index)))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: place(empty(*a, **k)))
    lib = Library()
    layer._size.cache_clear()
    yield seen
    layer._size.cache_clear()
    assert current == [0]


def run_layer():
    q, g = place(torch.zeros(2, 4, 3, 16)), place(torch.zeros(3))
    kla.linear_fwd(q, q, q, g)
    kla.linear_bwd(q, q, q, g, q)
    one, S = place(torch.zeros(2, 3, 16)), place(torch.zeros(2, 3, 16, 16))
    kla.linear_step(one, one, one, g, S)
    _, mean, rstd = kla.layer_norm_fwd(one)
    kla.layer_norm_bwd(one, one, None, mean, rstd)
    _, parents, _, _ = kla.beam_select(place(torch.zeros(2, 3, 50)), place(torch.zeros(2, 3)))
    kla.reorder_states(S, parents)


def test_layer_operators(calls):
    run_layer()
    assert calls == [(f"kla_{name}", 1, 101) for name in (
        "linear_fwd", "linear_bwd", "linear_step", "layer_norm_fwd", "layer_norm_bwd", "beam_select",
        "reorder_states")]


def test_recurrence(calls):
    q, a = place(torch.zeros(2, 4, 3, 16)), place(torch.zeros(2, 4, 3))
    kla.chunk_fwd(q, q, q, a, a)
    kla.chunk_bwd(q, q, q, a, a, q)
    one, S = place(torch.zeros(2, 3, 16)), place(torch.zeros(2, 3, 16, 16))
    kla.decode_step(one, one, one, a[:, 0].contiguous(), a[:, 0].contiguous(), S)
    kla.device_status(torch.device("cuda", 1))
    assert calls == [(f"kla_{name}", 1, 101) for name in ("chunk_fwd_ex", "chunk_bwd", "decode_step_ex",
                                                          "device_status")]


def test_recurrence_of_host_tensors(calls):
    q, a = torch.zeros(2, 4, 3, 16), torch.zeros(2, 4, 3)
    buffers = {n: torch.zeros(1) for n in ("q", "k", "v", "alpha", "eta", "o", "S_T")}
    kla.chunk_fwd_host(q, q, q, a, a, device="cuda:1", buffers=buffers, out=torch.zeros(2, 4, 3, 16),
                       S_T=torch.zeros(2, 3, 16, 16))
    assert calls == [("kla_chunk_fwd_host", 1, 101)]


def test_status_of_the_current_device(calls):
    kla.device_status()
    assert calls == [("kla_device_status", 0, 100)]
