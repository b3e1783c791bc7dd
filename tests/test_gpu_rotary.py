"""Rotary positions on the GPU against 64 bits.

Tolerances (relative L2): an angle is off by 2^-24 of a turn (4e-7 of the pair's length), its sine and cosine by 2^-23,
the two products and their sum by 2^-24 each: 1e-6 in fp32, and one rounding of 2^-8 at most in bf16: 4e-3.
"""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 1e-6, torch.bfloat16: 4e-3}


def rel(a, b):
    a, b = a.double(), b.double()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def reference(x, freqs, positions, layout, scale):
    n = freqs.shape[0]
    x = x.double()
    t = positions.double()[..., None] * freqs.double()
    c, s = scale * torch.cos(t)[:, :, None], scale * torch.sin(t)[:, :, None]
    y = x.clone()
    i = torch.arange(n, device=x.device)
    u, v = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., v] * c + x[..., u] * s
    return y


def check(B, T, H, K, d, rot, layout, dtype, positions=None, scale=1.0, seed=0, packed=False):
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if packed:
        q, k, _ = torch.randn(B, T, H + 2 * K, d, generator=gen, device=DEV).to(dtype).split([H, K, K], 2)
    else:
        q = torch.randn(B, T, H, d, generator=gen, device=DEV).to(dtype)
        k = torch.randn(B, T, K, d, generator=gen, device=DEV).to(dtype)
    freqs, _ = kla.rotary_freqs(rot, device=DEV)
    at = torch.arange(T, device=DEV).expand(B, T) if positions is None else positions
    oq, ok = kla.rotary_fwd(q, k, freqs, positions, layout=layout, scale=scale)
    for x, y in ((q, oq), (k, ok)):
        want = reference(x, freqs, at, layout, scale)
        assert y.shape == x.shape and y.is_contiguous()
        assert rel(y, want) <= TOL[dtype], rel(y, want)
        assert torch.equal(y[..., rot:], x[..., rot:])
    bq, bk = kla.rotary_bwd(oq, ok, freqs, positions, layout=layout, scale=scale)
    assert rel(bq, reference(oq, freqs, -at, layout, scale)) <= TOL[dtype]
    if k.numel():
        assert rel(bk, reference(ok, freqs, -at, layout, scale)) <= TOL[dtype]


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 64), (64, 30), (16, 16), (80, 20), (256, 254), (2, 2),
                                   (1, 0), (96, 0), (7, 6), (40, 32), (1024, 1024), (200, 200)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_heads(d, rot, layout, dtype):
    check(2, 5, 6, 2, d, rot, layout, dtype, seed=d)


@pytest.mark.parametrize("B,T,H,K", [(1, 1, 1, 1), (1, 1, 32, 8), (64, 1, 16, 4), (3, 33, 5, 1), (2, 1000, 12, 12),
                                     (2, 700, 3, 3), (1, 9, 40, 0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("packed", [False, True])
def test_sizes_and_packed_projections(B, T, H, K, layout, packed):
    check(B, T, H, K, 128, 128, layout, torch.bfloat16, seed=T, packed=packed)


@pytest.mark.parametrize("H,K,d,rot", [(1, 1, 128, 128), (1, 0, 128, 128), (3, 1, 64, 64), (2, 1, 64, 30), (1, 1, 32, 8),
                                       (2, 1, 7, 6), (1, 0, 96, 0), (1, 1, 40, 20)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_tokens_of_few_heads(H, K, d, rot, layout, dtype):
    """A warp's lanes hold all heads of several tokens then, the last of them in part."""
    check(3, 6007, H, K, d, rot, layout, dtype, seed=H, packed=True)


@pytest.mark.parametrize("H,K,d,rot", [(16, 16, 128, 126), (5, 1, 80, 20), (3, 3, 64, 62), (40, 8, 256, 130),
                                       (2, 0, 1024, 1022), (9, 2, 32, 30), (33, 11, 16, 14), (6, 2, 104, 104), (4, 4, 128, 2)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pairs_that_fit_no_wide_accesses(H, K, d, rot, layout, dtype):
    """Heads through shared memory, whole tokens and parts of them, few tokens and many."""
    check(2, 3, H, K, d, rot, layout, dtype, seed=d, packed=True)
    check(3, 701, H, K, d, rot, layout, dtype, seed=d + 1)


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_positions(kind):
    """Given positions, far ones and negative ones among them: whole turns cost no bits. At 2^31 the frequency's own
    53 bits leave 2^-24 of a turn more."""
    p = torch.tensor([[0, 1, 2**31 - 1, 2**20 + 3], [-5, 4095, 10**9 + 7, 131071]], device=DEV).to(kind)
    for layout in ("half", "interleaved"):
        check(2, 4, 3, 3, 128, 128, layout, torch.float32, positions=p, scale=1.2)


def test_positions_past_32_bits():
    """A product with the frequency's 64-bit fraction, of which 53 are known: 2^40 positions leave 2^-14 of a turn."""
    import gated_delta_rule_14_gb300 as kla
    p = torch.tensor([[2**40 + 12345]], device=DEV)
    freqs, _ = kla.rotary_freqs(64, device=DEV)
    q = torch.randn(1, 1, 4, 64, device=DEV)
    oq, _ = kla.rotary_fwd(q, None, freqs, p)
    assert rel(oq, reference(q, freqs, p, "half", 1.0)) <= 4e-4


def test_in_place_and_given_outputs():
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(6)
    freqs, _ = kla.rotary_freqs(128, device=DEV)
    qkv = torch.randn(2, 50, 3, 4, 128, generator=gen, device=DEV).bfloat16()
    keep = qkv.clone()
    q, k, v = qkv.unbind(2)
    want = kla.rotary_fwd(q, k, freqs)
    got = kla.rotary_fwd(q, k, freqs, out_q=q, out_k=k)
    assert got[0] is q and all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(v, keep[:, :, 2])
    out = [torch.zeros(2, 50, 4, 128, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    given = kla.rotary_fwd(keep[:, :, 0], keep[:, :, 1], freqs, out_q=out[0], out_k=out[1])
    assert given[0] is out[0] and all(torch.equal(a, b) for a, b in zip(given, want))
    single, none = kla.rotary_fwd(keep[:, :, 0], None, freqs)
    assert none is None and torch.equal(single, want[0])


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 1, 3), (1, 0, 2, 3)])
@pytest.mark.parametrize("B,T,H,K", [(2, 50, 4, 4), (3, 7, 6, 2), (1, 9, 3, 1), (4, 1, 1, 1), (2, 16, 2, 8)])
def test_slices_of_one_tensor_in_place(order, B, T, H, K):
    """Queries, keys and values of any number of heads beside each other, batch, tokens and heads in any order."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(16)
    freqs, _ = kla.rotary_freqs(64, device=DEV)
    sizes = (B, T, H + 2 * K, 64)
    packed = torch.randn([sizes[a] for a in order], generator=gen, device=DEV).bfloat16()
    keep = packed.clone()

    def views(x):
        x = x.permute([order.index(a) for a in range(4)])
        return x[:, :, :H], x[:, :, H:H + K], x[:, :, H + K:]
    (q, k, v), old = views(packed), views(keep)
    want = kla.rotary_fwd(old[0].contiguous(), old[1].contiguous(), freqs)
    kla.rotary_fwd(q, k, freqs, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, old[2])
    only, beside = views(keep.clone())[:2]
    _, turned = kla.rotary_fwd(only, beside, freqs, out_q=only, out_k=torch.empty_like(want[1]))
    assert torch.equal(only, want[0]) and torch.equal(turned, want[1])


def test_no_tokens():
    import gated_delta_rule_14_gb300 as kla
    freqs, _ = kla.rotary_freqs(16, device=DEV)
    for shape in ((0, 4, 2, 16), (2, 0, 2, 16)):
        q, k = kla.rotary_fwd(torch.empty(shape, device=DEV), torch.empty(shape, device=DEV), freqs)
        assert q.shape == k.shape == shape


def test_unaligned_and_broadcast_inputs():
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(8)
    freqs, _ = kla.rotary_freqs(64, device=DEV)
    x = torch.randn(2, 6, 5, 64, generator=gen, device=DEV).bfloat16()
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)
    flat[1:] = x.reshape(-1)
    wide = torch.randn(1, 1, 5, 64, generator=gen, device=DEV).bfloat16().expand(2, 6, 5, 64)
    for layout in ("half", "interleaved"):
        a, _ = kla.rotary_fwd(x, None, freqs, layout=layout)
        b, _ = kla.rotary_fwd(flat[1:].view(x.shape), None, freqs, layout=layout)
        assert torch.equal(a, b)
        c, _ = kla.rotary_fwd(wide, None, freqs, layout=layout)
        d, _ = kla.rotary_fwd(wide.contiguous(), None, freqs, layout=layout)
        assert torch.equal(c, d)


def test_gradient_against_the_formula_and_differences():
    """The map is linear: differences are exact but for rounding (1e-6 of the sums' terms)."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(9)
    freqs, scale = kla.rotary_freqs(48, scaling="yarn", factor=8.0, original_length=4096, device=DEV)
    q, k, dq, dk = (torch.randn(2, 30, h, 64, generator=gen, device=DEV) for h in (4, 2, 4, 2))
    gq, gk = kla.rotary_bwd(dq, dk, freqs, layout="interleaved", scale=scale)
    x = q.double().requires_grad_(True)
    at = torch.arange(30, device=DEV).expand(2, 30)
    t = at.double()[..., None] * freqs.double()
    z = torch.view_as_complex(x[..., :48].unflatten(-1, (24, 2)).contiguous()) * torch.polar(
        torch.full_like(t, scale), t)[:, :, None]
    y = torch.cat([torch.view_as_real(z).flatten(-2), x[..., 48:]], -1)
    want, = torch.autograd.grad((y * dq.double()).sum(), x)
    assert rel(gq, want) <= 1e-6
    oq, ok = kla.rotary_fwd(q, k, freqs, layout="interleaved", scale=scale)
    for a, b, c, d in ((oq, dq, q, gq), (ok, dk, k, gk)):
        left, right = (a.double() * b.double()).sum(), (c.double() * d.double()).sum()
        assert abs(float(left - right)) <= 1e-5 * float(a.norm() * b.norm())


def test_frequencies():
    import gated_delta_rule_14_gb300 as kla
    plain, one = kla.rotary_freqs(64, device=DEV)
    i = torch.arange(32, device=DEV, dtype=torch.float64)
    assert one == 1.0 and rel(plain, 10000.0 ** (-i / 32)) <= 1e-7
    linear, _ = kla.rotary_freqs(64, scaling="linear", factor=4.0, device=DEV)
    assert rel(linear, plain / 4) <= 1e-7
    ntk, _ = kla.rotary_freqs(64, scaling="ntk", factor=4.0, device=DEV)
    assert float(ntk[0]) == 1.0 and abs(float(ntk[-1] / plain[-1]) - 0.25) <= 1e-6
    yarn, scale = kla.rotary_freqs(64, scaling="yarn", factor=4.0, original_length=4096, device=DEV)
    turns = 4096 * plain.double() / (2 * torch.pi)
    assert abs(scale - 1.1386294) <= 1e-6
    assert torch.equal(yarn[turns > 50], plain[turns > 50]) and rel(yarn[turns < 0.8], plain[turns < 0.8] / 4) <= 1e-7
    assert ((yarn <= plain) & (yarn >= plain / 4 * 0.999999)).all()
    for bad in (dict(rot=3), dict(rot=8, scaling="cubic"), dict(rot=8, scaling="yarn"), dict(rot=8, factor=0.0),
                dict(rot=8, base=-1.0)):
        with pytest.raises(ValueError):
            kla.rotary_freqs(**bad)


def test_refusals():
    import gated_delta_rule_14_gb300 as kla
    freqs, _ = kla.rotary_freqs(16, device=DEV)
    q = torch.randn(2, 3, 4, 16, device=DEV)
    with pytest.raises(ValueError):
        kla.rotary_fwd(q, q[:, :2], freqs)
    with pytest.raises(ValueError):
        kla.rotary_fwd(q, q, freqs, layout="quarter")
    with pytest.raises(TypeError):
        kla.rotary_fwd(q, q, freqs.double())
    with pytest.raises(TypeError):
        kla.rotary_fwd(q, q, freqs, torch.zeros(2, 3, device=DEV))
    with pytest.raises(ValueError):
        kla.rotary_fwd(q, q, freqs, torch.zeros(3, 2, dtype=torch.int64, device=DEV))
    with pytest.raises(kla.KlaError):
        kla.rotary_fwd(q[..., :8].contiguous(), None, freqs)          # more values turned than there are
    with pytest.raises(kla.KlaError):
        kla.rotary_fwd(q, None, freqs, scale=float("inf"))
    with pytest.raises(kla.KlaError):
        kla.rotary_fwd(q, q.clone(), freqs, out_q=q, out_k=q)
    with pytest.raises(ValueError):
        kla.rotary_fwd(q.transpose(2, 3), None, freqs[:2])
    with pytest.raises(ValueError):
        kla.rotary_fwd(q.cpu(), None, freqs)
