"""The gated norm with gates that are slices along the tokens: the rows between two sequences' strides are as many as there are
tokens."""
import pytest
import torch

from gpu_util import DEV


def test_more_tokens_than_a_grid_has_rows():
    """Groups without weights of their own are bounded by the count of rows alone; host logic."""
    from gated_delta_rule_14_gb300 import _native
    size = _native.lib().kla_gated_norm_bwd_workspace_size
    assert size(2, 70000, 32, 1, 0) == size(140000, 1, 32, 1, 0) > 0 and size(2, 70000, 32, 1, 1) == 0
    assert size(2, 2**30, 32, 1, 0) == 0   # rows past 2^31


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [32, 33, 100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("first", [0, 1])
def test_gates_sliced_along_the_tokens(n, dtype, first):
    """70000 tokens of each of 2 longer sequences. A stored bf16 is off by 2^-8 at most, 4e-3; fp32 rows of up to 100 values
    by 1e-5, sums over 140000 rows, of which each of 608 stretches is added up in turn, by 2^-24 sqrt(140000) = 2e-5."""
    import gated_delta_rule_14_gb300 as kla
    T, gen = 70000, torch.Generator(device=DEV).manual_seed(n)

    def rnd(*shape):
        return torch.randn(shape, generator=gen, device=DEV)
    x, dy, w = rnd(2, T, n).to(dtype), rnd(2, T, n).to(dtype), 1 + 0.3 * rnd(n)
    z = rnd(2, T + 1, n).to(dtype)[:, first:first + T]
    y, mean, rstd = kla.gated_norm_fwd(x, z, w)
    dx, dz, dw = kla.gated_norm_bwd(dy, x, z, w, mean, rstd)
    kla.device_status(DEV)
    leaves = [t.double().requires_grad_(True) for t in (x, z, w)]
    xh = leaves[0] / (leaves[0].square().mean(-1, keepdim=True) + 1e-5).sqrt()
    want = xh * leaves[2] * leaves[1] * torch.sigmoid(leaves[1])
    grads = torch.autograd.grad((want * dy.double()).sum(), leaves)
    tol = 4e-3 if dtype == torch.bfloat16 else 1e-5
    assert rel(y, want.detach()) <= tol and rel(dx, grads[0]) <= tol and rel(dz, grads[1]) <= tol
    assert rel(dw, grads[2]) <= 2e-5
