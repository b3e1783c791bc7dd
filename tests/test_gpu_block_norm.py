"""A block's norms and their gradients on the GPU against 64 bits.

Tolerances (relative L2): fp32 values are rounded a few times at 2^-24 after sums over the row: 1e-5; a value stored in
bf16 is rounded once, by 2^-8 of it at most, and what fp32 adds: 4e-3. The sums over the rows are fp32 sums of random
signs: 1e-5.
"""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def rel(a, b):
    a, b = a.double(), b.double()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def normed(x, w, eps, norm):
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    return w * x / ((x * x).mean(-1, keepdim=True) + eps).sqrt()


def active(z, act):
    return torch.sigmoid(z) * (z if act == "silu" else 1.0)


def rnd(seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s: torch.randn(s, generator=gen, device=DEV)


def place(t, shift):
    """Values past an allocation's start, which wide accesses do not fit."""
    if not shift:
        return t
    flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
    flat[shift:] = t.reshape(-1)
    return flat[shift:].view(t.shape)


def gated(shape, wshape, dtype, norm="rms", act="silu", seed=0, shift=0, slices=0):
    import gated_delta_rule_14_gb300 as kla
    r = rnd(seed)
    x, dy, z = (place(t.to(dtype), shift) for t in (r(*shape) * 2 + 0.5, r(*shape), r(*shape) * 2))
    if slices:   # the gate as a slice of a packed projection
        flat = z.reshape(*shape[:-2], -1) if slices == 2 else z
        wide = torch.cat([flat, flat + 1, flat], -1)
        z = wide[..., flat.shape[-1]:2 * flat.shape[-1]].unflatten(-1, shape[-2:] if slices == 2 else shape[-1:])
        assert not z.is_contiguous() or z.numel() == flat.shape[-1]
    w = 1 + 0.3 * r(*wshape)
    y, mean, rstd = kla.gated_norm_fwd(x, z, w, 1e-5, norm=norm, act=act)
    dx, dz, dw = kla.gated_norm_bwd(dy, x, z, w, mean, rstd, act=act)
    assert (mean is None) == (norm == "rms")
    kla.device_status(DEV)
    leaves = [t.double().requires_grad_(True) for t in (x, z, w)]
    want = normed(leaves[0], leaves[2], 1e-5, norm) * active(leaves[1], act)
    grads = torch.autograd.grad((want * dy.double()).sum(), leaves)
    tol = 4e-3 if dtype == BF else 1e-5
    for name, a, b, t in (("y", y, want.detach(), tol), ("dx", dx, grads[0], tol), ("dgate", dz, grads[1], tol),
                          ("dw", dw, grads[2], 1e-5)):
        assert a.shape == b.shape and rel(a, b) <= t, (name, rel(a, b))
    assert dz.is_contiguous()
    y2, none, none2 = kla.gated_norm_fwd(x, z, w, 1e-5, norm=norm, act=act, stats=False)
    assert none is None and none2 is None and torch.equal(y, y2)


def added(shape, dtype, norm="rms", scaled=True, given=True, seed=0, shift=0):
    import gated_delta_rule_14_gb300 as kla
    r = rnd(seed)
    x, res, dy, ds = (place(t.to(dtype), shift) for t in (r(*shape), r(*shape) + 0.25, r(*shape), r(*shape)))
    w, scale = 1 + 0.3 * r(shape[-1]), (0.3 + 0.1 * r(shape[-1]) if scaled else None)
    y, total, mean, rstd = kla.add_norm_fwd(x, res, w, scale, 1e-5, norm=norm)
    dx, dr, dw, dl = kla.add_norm_bwd(dy, ds if given else None, x, res, w, scale, mean, rstd)
    assert (mean is None) == (norm == "rms")
    kla.device_status(DEV)
    leaves = [t.double().requires_grad_(True) for t in (x, res, w)] + (
        [scale.double().requires_grad_(True)] if scaled else [])
    s64 = leaves[1] + (leaves[3] if scaled else 1.0) * leaves[0]
    want = normed(s64, leaves[2], 1e-5, norm)
    loss = (want * dy.double()).sum() + ((s64 * ds.double()).sum() if given else 0)
    grads = torch.autograd.grad(loss, leaves)
    tol = 4e-3 if dtype == BF else 1e-5
    checks = [("y", y, want.detach(), tol), ("sum", total, s64.detach(), tol), ("dx", dx, grads[0], tol),
              ("dres", dr, grads[1], tol), ("dw", dw, grads[2], 1e-5)]
    if scaled:
        checks.append(("dscale", dl, grads[3], 1e-5))
    else:
        assert dl is None and dx is dr
    for name, a, b, t in checks:
        assert a.shape == b.shape and rel(a, b) <= t, (name, rel(a, b))


# parts of a warp, whole warps, teams of warps, and rows of more than a team holds; widths that only single values fit
LENGTHS = [3, 16, 31, 64, 100, 127, 128, 255, 256, 257, 512, 513, 1000, 1024, 1536, 2048, 4096, 4099, 8192, 8200, 20000]


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_gated_row_lengths(n, dtype, norm):
    gated((7, n), (n,), dtype, norm, "silu" if n % 2 else "sigmoid", seed=n)


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_added_row_lengths(n, dtype, norm):
    added((7, n), dtype, norm, scaled=n % 3 > 0, given=n % 4 > 0, seed=n)


@pytest.mark.parametrize("rows", [1, 2, 3, 17, 300, 1000, 5003])
@pytest.mark.parametrize("n", [128, 400, 1536, 2048])
def test_row_counts(rows, n):
    gated((rows, n), (n,), BF, seed=rows)
    added((rows, n), BF, seed=rows)


@pytest.mark.parametrize("G,n", [(16, 128), (3, 64), (5, 300), (2, 1024), (40, 16), (1, 128), (7, 100), (12, 256)])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("slices", [0, 2])
@pytest.mark.parametrize("dtype", [BF, F])
def test_heads(G, n, own, slices, dtype):
    """Weights shared by the heads or of their own; the gate whole, or a slice of a packed projection."""
    gated((3, 70, G, n), (G, n) if own else (n,), dtype, seed=G, slices=slices)


def test_sliced_gate_of_plain_rows():
    gated((3, 50, 96), (96,), BF, slices=1)
    gated((1, 50, 96), (96,), F, "layer", slices=1)


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("n", [128, 640, 4096])
@pytest.mark.parametrize("dtype", [BF, F])
def test_unaligned_starts(shift, n, dtype):
    gated((5, n), (n,), dtype, shift=shift)
    added((5, n), dtype, shift=shift)


@pytest.mark.parametrize("rows,G,n", [(1, 1, 3), (2, 1, 5), (3, 1, 1001), (301, 1, 33), (300, 3, 65), (7, 5, 101),
                                      (1, 3, 127), (64, 2, 63), (9, 4, 2049), (2000, 1, 511), (5, 1, 8191), (4, 1, 8193)])
@pytest.mark.parametrize("own,norm", [(False, "rms"), (True, "layer")])
@pytest.mark.parametrize("slices,shift", [(0, 0), (2, 0), (0, 1)])
def test_rows_of_odd_length(rows, G, n, own, norm, slices, shift):
    """Of bf16 every second one starts in the middle of 4 bytes."""
    gated((rows, G, n), (G, n) if own else (n,), BF, norm, seed=n, slices=slices, shift=shift)
    added((rows * G, n), BF, norm, seed=n, given=own, shift=shift)


@pytest.mark.parametrize("rows,G,n", [(50, 4, 100), (60, 8, 33), (30, 8, 1001), (2, 8, 5), (700, 1, 60), (33, 6, 20),
                                      (1, 1, 6), (3, 7, 129), (40, 16, 9), (5, 1, 4090), (2, 200, 11)])
@pytest.mark.parametrize("own,norm", [(False, "layer"), (True, "rms")])
@pytest.mark.parametrize("dtype,slices", [(BF, 0), (BF, 2), (F, 0), (F, 2)])
def test_rows_that_start_in_the_middle_of_16_bytes(rows, G, n, own, norm, dtype, slices):
    """At two, four or eight places, with the gate's rows alike or not."""
    gated((rows, G, n), (G, n) if own else (n,), dtype, norm, seed=n, slices=slices)
    added((rows * G, n), dtype, norm, seed=n, scaled=own)


@pytest.mark.parametrize("n", [3, 65, 1001, 2047])
@pytest.mark.parametrize("rows", [1, 2, 41])
def test_rows_of_odd_length_keep_to_themselves(rows, n):
    """NaN in a row reach no other, and nothing is written behind the last row."""
    import gated_delta_rule_14_gb300 as kla
    r = rnd(n + rows)
    x, z, dy, ds = (r(rows, n).to(BF) for _ in range(4))
    w, scale = r(n), r(n)
    want = kla.gated_norm_fwd(x, z, w), kla.add_norm_fwd(x, z, w, scale)
    bad = torch.arange(rows, device=DEV) % 2 == 1
    others = [t.masked_fill(bad[:, None], float("nan")) for t in (x, z)]
    # bits are compared, and tensors that start elsewhere may be added up in another order: both on 16 bytes, as the others
    back = torch.full((2, (rows * n + 15) // 8 * 8), 7.0, dtype=BF, device=DEV)
    out = [b[:rows * n].view(rows, n) for b in back]
    got = kla.gated_norm_fwd(*others, w, out=out[0]), kla.add_norm_fwd(*others, w, scale, out=out[0], out_residual=out[1])
    y = kla.gated_norm_fwd(*others, w)[0]
    assert torch.equal(y[~bad], want[0][0][~bad]) and bool(y[bad].isnan().all())
    assert torch.equal(out[0][~bad], want[1][0][~bad]) and torch.equal(out[1][~bad], want[1][1][~bad])
    assert bool(out[0][bad].isnan().all()) and bool((back[:, rows * n:] == 7).all())
    clean = kla.gated_norm_bwd(dy, x, z, w, None, want[0][2]), kla.add_norm_bwd(dy, ds, x, z, w, scale, None, want[1][3])
    with_nan = (kla.gated_norm_bwd(dy, *others, w, None, got[0][2]),
                kla.add_norm_bwd(dy, ds, *others, w, scale, None, got[1][3]))
    for a, b in zip(clean, with_nan):
        for i in (0, 1):
            assert torch.equal(a[i][~bad], b[i][~bad]) and bool(b[i][bad].isnan().all())


def test_large_offset():
    """Values about 1000 with a spread of 1: the mean is subtracted before squares are summed. A value's fp32 rounding
    is 1000 * 2^-24 = 6e-5 of the spread in the mean: 2e-4."""
    import gated_delta_rule_14_gb300 as kla
    x = rnd(1)(33, 777) + 1000
    z = torch.full_like(x, 0.5)
    y, _, _ = kla.gated_norm_fwd(x, z, norm="layer", act="sigmoid")
    assert rel(y, normed(x.double(), 1.0, 1e-5, "layer") * torch.sigmoid(z.double())) <= 2e-4
    y, total, _, _ = kla.add_norm_fwd(x, x, norm="layer")
    assert rel(y, normed(2 * x.double(), 1.0, 1e-5, "layer")) <= 2e-4


def test_extreme_gates_and_zero_rows():
    """silu(z) goes to z and to 0, sigmoid to 1 and 0, with their slopes; rows of zeros have gradients 1 / sqrt(eps)
    times dy and no NaN."""
    import gated_delta_rule_14_gb300 as kla
    x = rnd(2)(4, 64)
    z = torch.tensor([100.0, -100.0, 3e4, -3e4], device=DEV)[:, None].expand(4, 64).contiguous()
    for act, want in (("sigmoid", [1.0, 0.0, 1.0, 0.0]), ("silu", [100.0, 0.0, 3e4, 0.0])):
        y, _, rstd = kla.gated_norm_fwd(x, z, act=act)
        assert rel(y, normed(x.double(), 1.0, 1e-5, "rms") * torch.tensor(want, device=DEV)[:, None]) <= 1e-5
        dx, dz, dw = kla.gated_norm_bwd(torch.ones_like(x), x, z, None, None, rstd, act=act)
        assert all(t.isfinite().all() for t in (dx, dz, dw))
    zero = torch.zeros(3, 96, device=DEV)
    y, _, rstd = kla.gated_norm_fwd(zero, zero + 1, norm="rms")
    dx, dz, dw = kla.gated_norm_bwd(zero + 2, zero, zero + 1, None, None, rstd)
    assert not y.any() and not dz.any() and not dw.any()
    assert rel(dx, torch.full_like(dx, 2 * 0.7310585786300049 / 1e-5 ** 0.5)) <= 1e-5


def test_rows_near_32_bits():
    """65535 heads of three values in 32768 rows: the row behind the last one's team is past 2^31."""
    import gated_delta_rule_14_gb300 as kla
    rows, G = 32768, 65535
    x, z = torch.zeros(rows, G, 3, dtype=BF, device=DEV), torch.zeros(rows, G, 3, dtype=BF, device=DEV)
    r = rnd(21)
    x[-1], z[-1], w = r(G, 3).to(BF), r(G, 3).to(BF), r(G, 3)
    y, _, rstd = kla.gated_norm_fwd(x, z, w)
    kla.device_status(DEV)
    want = normed(x[-1].double(), w.double(), 1e-5, "rms") * active(z[-1].double(), "silu")
    assert rel(y[-1], want) <= 4e-3 and not y[:-1].any()


def test_no_rows():
    import gated_delta_rule_14_gb300 as kla
    x, w = torch.empty(0, 32, device=DEV), torch.ones(32, device=DEV)
    y, mean, rstd = kla.gated_norm_fwd(x, x.clone(), w)
    dx, dz, dw = kla.gated_norm_bwd(x, x, x, w, mean, rstd)
    assert y.shape == dx.shape == dz.shape == (0, 32) and not dw.any()
    y, s, mean, rstd = kla.add_norm_fwd(x, x.clone(), w, w)
    dx, dr, dw, dl = kla.add_norm_bwd(x, None, x, x, w, w, mean, rstd)
    assert not dw.any() and not dl.any()


def test_in_place_residual():
    import gated_delta_rule_14_gb300 as kla
    for n in (96, 2048, 9000):
        r = rnd(n)
        x, res = r(50, n).to(BF), r(50, n).to(BF)
        y, s, _, _ = kla.add_norm_fwd(x, res)
        keep = res.clone()
        y2, same, _, _ = kla.add_norm_fwd(x, keep, out_residual=keep)
        assert same is keep and torch.equal(s, keep) and torch.equal(y, y2)


@pytest.mark.parametrize("n", [3, 33, 100, 1001, 2047])
@pytest.mark.parametrize("dtype", [BF, F])
def test_in_place_rows_off_16_bytes(n, dtype):
    """Two rows may share 16 bytes, of which each writes its own."""
    import gated_delta_rule_14_gb300 as kla
    r = rnd(n)
    x, res, w, scale = r(5003, n).to(dtype), r(5003, n).to(dtype), r(n), r(n)
    y, s, _, rstd = kla.add_norm_fwd(x, res, w, scale)
    keep = res.clone()
    y2, same, _, rstd2 = kla.add_norm_fwd(x, keep, w, scale, out_residual=keep)
    assert same is keep and torch.equal(s, keep) and torch.equal(y, y2) and torch.equal(rstd, rstd2)
    want = res.double() + scale.double() * x.double()
    assert rel(s, want) <= (4e-3 if dtype == BF else 1e-5)


def test_equal_calls_give_equal_bits():
    import gated_delta_rule_14_gb300 as kla
    r = rnd(7)
    x, z, dy = (r(4000, 4, 128).to(BF) for _ in range(3))
    w = r(128)
    _, _, rstd = kla.gated_norm_fwd(x, z, w)
    first = kla.gated_norm_bwd(dy, x, z, w, None, rstd)
    flat = [t.view(4000, 512) for t in (dy, x, z)]
    l2 = r(512)
    _, _, _, rs = kla.add_norm_fwd(flat[0], flat[1], None, l2)
    second = kla.add_norm_bwd(flat[2], flat[0], flat[0], flat[1], None, l2, None, rs)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, kla.gated_norm_bwd(dy, x, z, w, None, rstd)))
        again = kla.add_norm_bwd(flat[2], flat[0], flat[0], flat[1], None, l2, None, rs)
        assert all(torch.equal(a, b) for a, b in zip(second, again))


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_gradients_against_differences(norm):
    """Central differences with steps of 1e-2 along the gradient's signs: off by their squares, 1e-4, times a curvature
    of order ten."""
    import gated_delta_rule_14_gb300 as kla
    r = rnd(13)
    x, z, dy, ds = (r(6, 40) for _ in range(4))
    w, l2 = 1 + 0.3 * r(40), 0.5 + 0.1 * r(40)

    def one(x, z, w):
        return float((kla.gated_norm_fwd(x, z, w, norm=norm)[0].double() * dy.double()).sum())

    def two(x, z, w, l2):
        y, s, _, _ = kla.add_norm_fwd(x, z, w, l2, norm=norm)
        return float((y.double() * dy.double()).sum() + (s.double() * ds.double()).sum())
    _, mean, rstd = kla.gated_norm_fwd(x, z, w, norm=norm)
    g1 = kla.gated_norm_bwd(dy, x, z, w, mean, rstd)
    _, s, mean, rstd = kla.add_norm_fwd(x, z, w, l2, norm=norm)
    g2 = kla.add_norm_bwd(dy, ds, x, z, w, l2, mean, rstd)
    for f, at, grads in ((one, [x, z, w], g1), (two, [x, z, w, l2], g2)):
        for i, g in enumerate(grads):
            d = g.sign() * 1e-2
            up, down = list(at), list(at)
            up[i], down[i] = at[i] + d, at[i] - d
            want, got = (f(*up) - f(*down)) / 2, float((g.double() * d.double()).sum())
            assert abs(got - want) <= 1e-3 * abs(want), (f.__name__, i, got, want)


def test_refusals():
    import gated_delta_rule_14_gb300 as kla
    x = rnd(3)(4, 6, 32)
    z, w = x.clone(), torch.ones(32, device=DEV)
    with pytest.raises(ValueError, match="norm"):
        kla.gated_norm_fwd(x, z, w, norm="batch")
    with pytest.raises(ValueError, match="act"):
        kla.gated_norm_fwd(x, z, w, act="relu")
    with pytest.raises(TypeError):
        kla.gated_norm_fwd(x, z.to(BF), w)
    with pytest.raises(TypeError):
        kla.gated_norm_fwd(x, z, w.to(BF))
    with pytest.raises(ValueError):
        kla.gated_norm_fwd(x, z, torch.ones(5, 32, device=DEV))
    with pytest.raises(ValueError):
        kla.gated_norm_fwd(x.transpose(0, 1), z, w)
    with pytest.raises(ValueError, match="gate"):
        kla.gated_norm_fwd(x, z.transpose(0, 1).contiguous().transpose(0, 1), torch.ones(6, 32, device=DEV))
    with pytest.raises(kla.KlaError):
        kla.gated_norm_fwd(x[..., :2].contiguous(), z[..., :2].contiguous())
    with pytest.raises(kla.KlaError):
        kla.gated_norm_fwd(x, z, w, -1.0)
    with pytest.raises(kla.KlaError):
        kla.gated_norm_fwd(x, z, w, out=x)
    with pytest.raises(kla.KlaError):
        kla.gated_norm_fwd(x, x[:1].expand(4, 6, 32), w)   # rows of the gate in one place
    _, _, rstd = kla.gated_norm_fwd(x, z, w)
    with pytest.raises(ValueError):
        kla.gated_norm_bwd(x, x, z, w, None, rstd[:3])
    with pytest.raises(ValueError):
        kla.add_norm_fwd(x, z[:3], w)
    with pytest.raises(ValueError):
        kla.add_norm_fwd(x, z, w, torch.ones(6, 32, device=DEV))
    with pytest.raises(kla.KlaError):
        kla.add_norm_fwd(x, z, w, out=z)
    y, s, mean, rstd = kla.add_norm_fwd(x, z, w, w)
    with pytest.raises(TypeError):
        kla.add_norm_bwd(x, None, None, z, w, w, mean, rstd)
    with pytest.raises(ValueError):
        kla.add_norm_bwd(x, None, x[:3], z, w, w, mean, rstd)
