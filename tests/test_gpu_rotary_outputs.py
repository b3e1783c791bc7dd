"""Rotary positions into slices of one tensor: outputs that reach over each other, or over an input, and share no value."""
import ctypes

import pytest
import torch

from gpu_util import DEV

A = 1 << 40   # addresses that nothing is read from: refusals come before any launch


def call(q, k, oq, ok, st, H=4, K=2):
    from gated_delta_rule_14_gb300 import _native
    strides = (ctypes.c_int64 * 12)(*st)
    return _native.lib().kla_rotary(q, k, oq, ok, strides, ctypes.cast(A - (1 << 20), ctypes.POINTER(ctypes.c_float)), None, 0, 2, 3,
                                    H, K, 16, 16, 0, 1, 1.0, 0, None)


DENSE, PACKED = (3 * 4 * 16, 4 * 16, 16), (3 * 6 * 16, 6 * 16, 16)
DENSE_K = (3 * 2 * 16, 2 * 16, 16)


@pytest.mark.parametrize("ok", [A, A + 3 * 16 * 2, A + 4 * 16 * 2 - 2, A + 6 * 16 * 2])   # keys from the queries' heads, or a token's
def test_outputs_that_share_values_are_refused(ok):
    far = A + (1 << 30)
    assert call(far, far + (1 << 20), A, ok, (*DENSE, *DENSE_K, *PACKED, *PACKED)) == 1


def test_outputs_over_inputs_are_refused():
    far = A + (1 << 30)
    assert call(A, far, A + 32, far + (1 << 20), (*PACKED, *DENSE_K, *PACKED, *DENSE_K)) == 1   # a head further on
    assert call(A, far, far + (1 << 20), A + 3 * 32, (*PACKED, *DENSE_K, *DENSE, *PACKED)) == 1   # the keys over the queries' last
    assert call(A, far, A, A + 3 * 32, (*PACKED, *DENSE_K, *PACKED, *PACKED)) == 1   # the same, queries in place


@pytest.mark.gpu
@pytest.mark.parametrize("H,K,d,rot", [(4, 4, 64, 64), (4, 1, 128, 126), (2, 8, 16, 4), (1, 1, 7, 6)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_into_one_tensor(H, K, d, rot, layout, dtype):
    import gated_delta_rule_14_gb300 as kla
    B, T, gen = 3, 50, torch.Generator(device=DEV).manual_seed(d)
    freqs, _ = kla.rotary_freqs(rot, device=DEV)
    q, k = (torch.randn((B, T, h, d), generator=gen, device=DEV).to(dtype) for h in (H, K))
    want = kla.rotary_fwd(q, k, freqs, layout=layout)
    kv = torch.full((B, T, H + 2 * K, d), 7.0, dtype=dtype, device=DEV)
    oq, ok, rest = kv.split([H, K, K], 2)
    kla.rotary_fwd(q, k, freqs, layout=layout, out_q=oq, out_k=ok)   # both, beside what is left as it was
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]) and bool((rest == 7.0).all())
    kv.fill_(7.0)
    oq.copy_(q)
    kla.rotary_fwd(oq, k, freqs, layout=layout, out_q=oq, out_k=ok)   # queries in place, keys into the same tensor
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]) and bool((rest == 7.0).all())
    kv.fill_(7.0)
    rest.copy_(k)
    kla.rotary_fwd(q, rest, freqs, layout=layout, out_q=oq, out_k=ok)   # keys from one slice into another
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]) and torch.equal(rest, k)
    kla.device_status(DEV)


@pytest.mark.gpu
def test_frequencies_above_one_at_far_positions():
    """The angle's fraction of a turn by whole numbers, from 2 pi to 60 digits: off by 2^-24 of a turn at most, sine and
    cosine by 2^-22 more."""
    import math
    from decimal import Decimal, getcontext

    import gated_delta_rule_14_gb300 as kla
    getcontext().prec = 70
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194989")
    freqs = torch.tensor([4.0, 3.9375, 2.7182817459106445, 1.0, 0.3333333432674408], device=DEV)
    at = torch.tensor([[2**28, 2**28 - 1, 123456789, 5, -(2**28)]], device=DEV)
    x = torch.zeros(1, 5, 1, 10, device=DEV)
    x[..., :5] = 1.0
    y = kla.rotary_fwd(x, None, freqs, at)[0][0, :, 0].double().cpu()
    kla.device_status(DEV)
    tol = 2 * math.pi * 2.0**-24 + 2.0**-22
    for t, p in enumerate(at[0].tolist()):
        for i, f in enumerate(freqs.tolist()):
            turn = Decimal(f) * p / two_pi
            angle = float((turn - turn.to_integral_value()) * two_pi)
            assert abs(float(y[t, i]) - math.cos(angle)) <= tol and abs(float(y[t, 5 + i]) - math.sin(angle)) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot", [(40, 36), (48, 12), (48, 44), (56, 28), (56, 4), (64, 60)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_heads_on_either_side_of_4_byte_accesses(d, rot, layout, dtype):
    """A stored bf16 is off by 2^-8 of itself at most, and sine and cosine by 2^-20 of the pair; fp32 by 2^-21 in all."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(d + rot)
    freqs, _ = kla.rotary_freqs(rot, device=DEV)
    for B, T, H, K in ((2, 3, 5, 1), (3, 701, 9, 3)):
        q, k = (torch.randn((B, T, h, d), generator=gen, device=DEV).to(dtype) for h in (H, K))
        got = kla.rotary_fwd(q, k, freqs, layout=layout)
        t = (torch.arange(T, device=DEV).double()[:, None] * freqs.double())[:, None]
        for x, y in zip((q, k), got):
            z = x.double()[..., :rot]
            u, v = (z[..., :rot // 2], z[..., rot // 2:]) if layout == "half" else (z[..., ::2], z[..., 1::2])
            new = (u * t.cos() - v * t.sin(), v * t.cos() + u * t.sin())
            new = torch.cat(new, -1) if layout == "half" else torch.stack(new, -1).flatten(-2)
            size = (u.square() + v.square()).sqrt()
            size = torch.cat([size, size], -1) if layout == "half" else torch.stack([size, size], -1).flatten(-2)
            tol = new.abs() * 2.0**-8 + size * 2.0**-19 if dtype == torch.bfloat16 else size * 2.0**-21
            assert bool(((y.double()[..., :rot] - new).abs() <= tol).all()) and torch.equal(y[..., rot:], x[..., rot:])
    kla.device_status(DEV)
