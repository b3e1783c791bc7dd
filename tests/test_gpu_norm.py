"""Layer norm and its gradients on the GPU against 64 bits.

Tolerances (relative L2): fp32 values are rounded a few times at 2^-24 after sums over the row: 1e-5; a
value stored in bf16 is rounded once, at most 2^-9 relative: 2e-3 and what fp32 adds: 4e-3. The sums over
the rows are fp32 sums of random signs: 1e-5.
"""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


def rel(a, b):
    a, b = a.double(), b.double()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def reference(x, w, b, eps, dy):
    x = x.double().requires_grad_(True)
    w = w.double().requires_grad_(True)
    b = b.double().requires_grad_(True)
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean) ** 2).mean(-1, keepdim=True).add(eps).rsqrt()
    y = (x - mean) * rstd * w + b
    return (y.detach(), mean.detach()[..., 0], rstd.detach()[..., 0],
            *torch.autograd.grad((y * dy.double()).sum(), (x, w, b)))


def check(shape, wshape, dtype, offset=0.5, scale=2.0, seed=0, view=0):
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=gen, device=DEV)

    def place(t):   # `view`: values past an allocation's start, which 16-byte accesses do not fit
        if not view:
            return t
        flat = torch.empty(t.numel() + view, dtype=t.dtype, device=DEV)
        flat[view:] = t.reshape(-1)
        return flat[view:].view(t.shape)
    x, dy = place((rnd(*shape) * scale + offset).to(dtype)), place(rnd(*shape).to(dtype))
    w, b = 1 + 0.3 * rnd(*wshape), rnd(*wshape)
    y, mean, rstd = kla.layer_norm_fwd(x, w, b, 1e-5)
    dx, dw, db = kla.layer_norm_bwd(dy, x, w, mean, rstd)
    kla.device_status(DEV)
    ref = reference(x, w, b, 1e-5, dy)
    tol = 4e-3 if dtype == torch.bfloat16 else 1e-5
    for name, got, want, t in zip(("y", "mean", "rstd", "dx", "dw", "db"), (y, mean, rstd, dx, dw, db), ref,
                                  (tol, 1e-5, 1e-5, tol, 1e-5, 1e-5)):
        assert got.shape == want.shape and rel(got, want) <= t, (name, rel(got, want))


# teams of 2 to 32 lanes, of several warps (513 to 8192 values) and CTAs that take longer rows by pieces, some at
# their borders, and widths that only pairs or single values fit
@pytest.mark.parametrize("n", [3, 16, 31, 127, 128, 255, 256, 257, 512, 513, 514, 1000, 2048, 4099, 16384,
                               16385, 20000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_lengths(n, dtype):
    check((7, n), (n,), dtype, seed=n)


@pytest.mark.parametrize("rows", [1, 2, 1000, 5003])
@pytest.mark.parametrize("n", [96, 400, 1536])
def test_row_counts(rows, n):
    check((rows, n), (n,), torch.bfloat16, seed=rows)


@pytest.mark.parametrize("G,n", [(16, 128), (3, 64), (5, 300), (2, 1024), (2, 17000), (40, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_heads_with_weights_of_their_own(G, n, dtype):
    check((3, 7, G, n), (G, n), dtype, seed=G)


@pytest.mark.parametrize("view", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_starts(view, dtype):
    check((5, 640), (640,), dtype, view=view)


def test_large_offset():
    """Values about 1000 with a spread of 1: the mean is subtracted before squares are summed. A value's fp32
    rounding is 1000 * 2^-24 = 6e-5 of the spread in the mean: 2e-4."""
    import gated_delta_rule_14_gb300 as kla
    x = torch.randn(33, 777, device=DEV) + 1000
    y, mean, rstd = kla.layer_norm_fwd(x)
    d = x.double()
    want = (d - d.mean(-1, keepdim=True)) / (d.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
    assert rel(y, want) <= 2e-4


def test_without_weights_and_stats_and_constant_rows():
    import gated_delta_rule_14_gb300 as kla
    x = torch.full((4, 96), 3.0, device=DEV)
    y, mean, rstd = kla.layer_norm_fwd(x, stats=False)
    assert mean is None and rstd is None and not y.any()
    y, mean, rstd = kla.layer_norm_fwd(x)
    dx, dw, db = kla.layer_norm_bwd(torch.ones_like(x), x, None, mean, rstd)
    assert not dx.any() and not dw.any() and torch.equal(db, torch.full((96,), 4.0, device=DEV))


def test_no_rows():
    import gated_delta_rule_14_gb300 as kla
    x = torch.empty(0, 32, device=DEV)
    w = torch.ones(32, device=DEV)
    y, mean, rstd = kla.layer_norm_fwd(x, w)
    dx, dw, db = kla.layer_norm_bwd(x, x, w, mean, rstd)
    assert y.shape == (0, 32) and not dw.any() and not db.any()


def test_gradient_against_differences():
    """Central differences of the 64-bit forward (error ~h^2) along a random direction; 1e-4 covers both."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, dy = (torch.randn((6, 50), generator=gen, device=DEV) for _ in range(2))
    w, b, e = (torch.randn(50, generator=gen, device=DEV) for _ in range(3))
    ex = torch.randn((6, 50), generator=gen, device=DEV)
    y, mean, rstd = kla.layer_norm_fwd(x, w, b)
    dx, dw, db = kla.layer_norm_bwd(dy, x, w, mean, rstd)

    def loss(h, hx, hw, hb):
        xx, ww, bb = x.double() + h * hx * ex.double(), w.double() + h * hw * e.double(), b.double() + h * hb * e.double()
        m = xx.mean(-1, keepdim=True)
        xh = (xx - m) / (((xx - m) ** 2).mean(-1, keepdim=True) + 1e-5).sqrt()
        return float(((xh * ww + bb) * dy.double()).sum())
    for on, got in (((1, 0, 0), (dx.double() * ex.double()).sum()), ((0, 1, 0), (dw.double() * e.double()).sum()),
                    ((0, 0, 1), (db.double() * e.double()).sum())):
        num = (loss(1e-4, *on) - loss(-1e-4, *on)) / 2e-4
        assert abs(num - float(got)) <= 1e-4 * max(1.0, abs(num))


def test_equal_calls_give_equal_bits():
    import gated_delta_rule_14_gb300 as kla
    x, dy = torch.randn(4001, 384, device=DEV), torch.randn(4001, 384, device=DEV)
    w = torch.ones(384, device=DEV)
    _, mean, rstd = kla.layer_norm_fwd(x, w)
    a, b = (kla.layer_norm_bwd(dy, x, w, mean, rstd) for _ in range(2))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals():
    import gated_delta_rule_14_gb300 as kla
    x = torch.randn(4, 6, 32, device=DEV)
    w = torch.ones(32, device=DEV)
    with pytest.raises(ValueError):
        kla.layer_norm_fwd(x.transpose(1, 2), w)
    with pytest.raises(ValueError):
        kla.layer_norm_fwd(x, w[:31])
    with pytest.raises(ValueError):
        kla.layer_norm_fwd(x, torch.ones(5, 32, device=DEV))
    with pytest.raises(TypeError):
        kla.layer_norm_fwd(x, w.double())
    with pytest.raises(TypeError):
        kla.layer_norm_fwd(x.double(), w)
    with pytest.raises(kla.KlaError):
        kla.layer_norm_fwd(x, w, eps=-1.0)
    with pytest.raises(kla.KlaError):
        kla.layer_norm_fwd(x, w, out=x)
    for n in (1, 2, 70000):
        with pytest.raises(kla.KlaError):
            kla.layer_norm_fwd(torch.randn(1, n, device=DEV))
    _, mean, rstd = kla.layer_norm_fwd(x, w)
    with pytest.raises(ValueError):
        kla.layer_norm_bwd(x[:2], x, w, mean, rstd)
    with pytest.raises(kla.KlaError):
        kla.layer_norm_bwd(x.clone(), x, w, mean, rstd, workspace=torch.empty(8, device=DEV))


# rows longer than a CTA holds: few and many rows, whose sums of dw and db come from several CTAs
@pytest.mark.parametrize("rows", [1, 5, 1300])
@pytest.mark.parametrize("n,dtype", [(8200, torch.bfloat16), (8202, torch.bfloat16), (8193, torch.float32)])
def test_many_long_rows(rows, n, dtype):
    check((rows, n), (n,), dtype, seed=rows)


def test_long_rows_whose_weights_fit_no_wide_access():
    """The weights start 4 bytes past a 16-byte boundary; the same values on one give the same gradients to
    the sums' order (fp32, 1e-5) and y to one bf16 rounding (4e-3)."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(9)
    n = 8208
    x, dy = (torch.randn((37, n), generator=gen, device=DEV).bfloat16() for _ in range(2))
    flat = torch.randn(2 * n + 1, generator=gen, device=DEV)
    w, b = flat[1:n + 1], flat[n + 1:]
    y, mean, rstd = kla.layer_norm_fwd(x, w, b)
    dx, dw, db = kla.layer_norm_bwd(dy, x, w, mean, rstd)
    ref = reference(x, w, b, 1e-5, dy)
    for got, want, t in zip((y, mean, rstd, dx, dw, db), ref, (4e-3, 1e-5, 1e-5, 4e-3, 1e-5, 1e-5)):
        assert rel(got, want) <= t


def test_long_rows_without_weights_and_with_a_large_offset():
    """As test_large_offset: the offset of 1000 costs 6e-5 of the spread through the mean's rounding, 2e-4."""
    import gated_delta_rule_14_gb300 as kla
    x = torch.randn(33, 9001, device=DEV) + 1000
    y, mean, rstd = kla.layer_norm_fwd(x)
    d = x.double()
    want = (d - d.mean(-1, keepdim=True)) / (d.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
    assert rel(y, want) <= 2e-4
    c = torch.full((4, 8201), 3.0, device=DEV)
    y, mean, rstd = kla.layer_norm_fwd(c)
    dx, dw, db = kla.layer_norm_bwd(torch.ones_like(c), c, None, mean, rstd)
    assert not y.any() and not dx.any() and not dw.any() and torch.equal(db, torch.full((8201,), 4.0, device=DEV))


@pytest.mark.parametrize("shape", [(7, 5, 64), (3, 4, 2, 640), (2, 3, 8200)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bias_per_head_without_a_weight(shape, dtype):
    """The bias' axes say how the forward took x apart; its gradient, and the unit weight's, are per head too."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(shape[-1])
    x, dy = (torch.randn(shape, generator=gen, device=DEV).to(dtype) for _ in range(2))
    b = torch.randn(shape[-2:], generator=gen, device=DEV)
    y, mean, rstd = kla.layer_norm_fwd(x, None, b)
    dx, dw, db = kla.layer_norm_bwd(dy, x, None, mean, rstd, bias=b)
    ref = reference(x, torch.ones_like(b), b, 1e-5, dy)
    tol = 4e-3 if dtype == torch.bfloat16 else 1e-5
    for got, want, t in zip((y, mean, rstd, dx, dw, db), ref, (tol, 1e-5, 1e-5, tol, 1e-5, 1e-5)):
        assert got.shape == want.shape and rel(got, want) <= t


def test_backward_checks_the_bias():
    import gated_delta_rule_14_gb300 as kla
    x = torch.randn(4, 6, 32, device=DEV)
    _, mean, rstd = kla.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        kla.layer_norm_bwd(x, x.clone(), None, mean, rstd, bias=torch.ones(5, 32, device=DEV))
    with pytest.raises(ValueError):
        kla.layer_norm_bwd(x, x.clone(), torch.ones(32, device=DEV), mean, rstd, bias=torch.ones(6, 32, device=DEV))


# Rows of 513 to 8192 values go through shared memory, several at a time for every team of threads: enough rows here
# that each team walks four or more, so that stages are filled again, their phases flip and the two output
# buffers alternate, in fp32 with one to four stages, and off the 16-byte grid, where a row's first and last
# values go by themselves between rows of other teams.
@pytest.mark.parametrize("rows,n,dtype", [
    (10007, 1024, torch.float32), (10007, 1023, torch.float32), (5003, 2048, torch.float32),
    (2600, 4095, torch.float32), (1300, 8192, torch.float32), (1300, 8192, torch.bfloat16),
    (5003, 1537, torch.bfloat16), (2600, 2050, torch.bfloat16)])
def test_many_rows_through_shared_memory(rows, n, dtype):
    check((rows, n), (n,), dtype, seed=n)


@pytest.mark.parametrize("view", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_rows_from_unaligned_starts(view, dtype):
    check((10007, 640), (640,), dtype, view=view)


@pytest.mark.parametrize("G,n", [(3, 700), (2, 2049)])
def test_many_heads_through_shared_memory(G, n):
    check((4001, G, n), (G, n), torch.float32, seed=G)


@pytest.mark.parametrize("n", [128, 1001, 8200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensors_with_different_starts(n, dtype):
    """x, dy and the output each start at another place against 16 bytes; what lies around the output stays."""
    import gated_delta_rule_14_gb300 as kla
    rows = 3000 if n < 8192 else 40
    gen = torch.Generator(device=DEV).manual_seed(n)

    def at(k, fill=None):
        flat = torch.randn(rows * n + 8, generator=gen, device=DEV).to(dtype)
        if fill is not None:
            flat.fill_(fill)
        return flat, flat[k:k + rows * n].view(rows, n)
    (_, x), (_, dy), (around, out) = at(1), at(2), at(3, 7.0)
    w, b = (torch.randn(n, generator=gen, device=DEV) for _ in range(2))
    y, mean, rstd = kla.layer_norm_fwd(x, w, b, out=out)
    dx, dw, db = kla.layer_norm_bwd(dy, x, w, mean, rstd)
    assert y is out and bool((around[:3] == 7).all()) and bool((around[3 + rows * n:] == 7).all())
    tol = 4e-3 if dtype == torch.bfloat16 else 1e-5
    for got, want, t in zip((y, mean, rstd, dx, dw, db), reference(x, w, b, 1e-5, dy), (tol, 1e-5, 1e-5, tol, 1e-5, 1e-5)):
        assert rel(got, want) <= t
