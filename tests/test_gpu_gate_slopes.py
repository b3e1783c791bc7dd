"""The gradient of the gated norm's gate, value by value, where the activation is all but flat."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,shift", [(128, 0), (33, 0), (1001, 0), (128, 1), (9000, 0), (20001, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slopes_of_the_sigmoid(n, shift, dtype):
    """s (1 - s) between -60 and 60. fp32: the exponential's 2^-22, at most 8 roundings of 2^-24, the row's sum of n
    squares another sqrt(n) 2^-24 at most: (12 + sqrt(n)) 2^-24. bf16 besides half a step, 2^-8: the exponent of up to 87
    rounded by 2^-24, the hardware's exponential by 2^-22 and reciprocal by 2^-23: 1e-5."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(n)

    def place(t):
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
        flat[shift:] = t.reshape(-1)
        return flat[shift:].view(t.shape)
    x, dy = (place((torch.rand((5, n), generator=gen, device=DEV) + 0.5).to(dtype)) for _ in range(2))
    z = place((120 * torch.rand((5, n), generator=gen, device=DEV) - 60).to(dtype))
    y, _, rstd = kla.gated_norm_fwd(x, z, act="sigmoid")
    _, dz, _ = kla.gated_norm_bwd(dy, x, z, None, None, rstd, act="sigmoid")
    kla.device_status(DEV)
    z64 = z.double()
    xh = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-5).sqrt()
    want = dy.double() * xh * torch.sigmoid(z64) * torch.sigmoid(-z64)
    tol = (12 + n**0.5) * 2.0**-24 + (2.0**-8 + 1e-5 if dtype == torch.bfloat16 else 0.0)
    assert float((dz.double() / want - 1).abs().max()) <= tol
    want = xh * torch.sigmoid(z64)
    assert float((y.double() / want - 1).abs().max()) <= tol
