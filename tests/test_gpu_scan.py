"""The gated scan, its gradients and its single tokens on the GPU against 64 bits.

Tolerances (relative L2): an fp32 step rounds at most five times at 2^-24 of what meets there (the gate's exponential
and quotient, a difference, a product, a sum), and what it leaves decays with the state: 5 2^-24 / (1 - a), 3e-5 at the
gates used here (a of 0.95 in the mean, 0.99 at most). A value stored in bf16 is rounded once, by 2^-8 of it at most, and
3e-5 more: 4e-3.
"""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 3e-5, torch.bfloat16: 4e-3}


def rel(a, b):
    a, b = a.double(), b.double()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def factors(gate, mode):
    return (torch.exp(gate), torch.ones_like(gate)) if mode == "log" else (torch.sigmoid(gate), torch.sigmoid(-gate))


def reference(x, gate, h0, mode, lengths):
    """(y, h_T) in 64 bits, token by token, by operations that autograd follows."""
    B, T, C = x.shape
    h = h0 if h0 is not None else torch.zeros(B, C, device=x.device, dtype=torch.float64)
    ys = []
    for t in range(T):
        live = (t < lengths)[:, None]
        a, w = factors(gate[:, t].masked_fill(~live, 0.0), mode)
        h = torch.where(live, a * h + w * x[:, t].masked_fill(~live, 0.0), h)
        ys.append(torch.where(live, h, 0.0))
    return (torch.stack(ys, 1) if ys else x.new_zeros(B, 0, C)), h


def make(B, T, C, dtype, mode, seed, lengths=None, packed=False):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*s):
        return torch.randn(s, generator=gen, device=DEV)
    x, gate = rnd(B, T, C).to(dtype), rnd(B, T, C)
    gate = (gate + 3).to(dtype) if mode == "sigmoid" else (-torch.nn.functional.softplus(gate - 3)).to(dtype)
    dy = rnd(B, T, C).to(dtype)
    if packed:
        x, gate, dy = torch.cat([x, gate, dy], -1).split(C, -1)
    n = torch.full((B,), T) if lengths is None else torch.tensor(lengths)
    n = n.to(torch.int32).to(DEV)
    for t in (x, gate, dy):   # what masked tokens hold counts for nothing
        t.masked_fill_((torch.arange(T, device=DEV) >= n[:, None])[..., None], float("nan"))
    return x, gate, dy, rnd(B, C), rnd(B, C), (None if lengths is None else n), n


def check(B, T, C, dtype, mode, seed=0, lengths=None, packed=False, state=True):
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, given, n = make(B, T, C, dtype, mode, seed, lengths, packed)
    if not state:
        h0 = dh = None
    y, h_T, states = kla.gated_scan_fwd(x, gate, h0, mode=mode, lengths=given, states=True)
    got = kla.gated_scan_bwd(x, gate, dy, states, dh, mode=mode, lengths=given)
    plain = kla.gated_scan_fwd(x, gate, h0, mode=mode, lengths=given)
    kla.device_status(DEV)
    assert torch.equal(plain[0], y) and torch.equal(plain[1], h_T) and plain[2] is None
    leaves = [t.double().nan_to_num(0.0).requires_grad_(True) for t in (x, gate)]
    h64 = torch.zeros(B, C, device=DEV, dtype=torch.float64) if h0 is None else h0.double()
    leaves.append(h64.requires_grad_(True))
    wy, wh = reference(leaves[0], leaves[1], leaves[2], mode, n)
    loss = (wy * dy.double().nan_to_num(0.0)).sum() + (0 if dh is None else (wh * dh.double()).sum())
    grads = torch.autograd.grad(loss, leaves, allow_unused=True)
    grads = [torch.zeros_like(a) if g is None else g for a, g in zip(leaves, grads)]
    for name, a, b, tol in (("y", y, wy, TOL[dtype]), ("h_T", h_T, wh, 3e-5), ("dx", got["dx"], grads[0], TOL[dtype]),
                            ("dgate", got["dgate"], grads[1], TOL[dtype]), ("dh0", got["dh0"], grads[2], 3e-5)):
        assert a.shape == b.shape and rel(a, b.detach()) <= tol, (name, rel(a, b.detach()))


# around the borders of a thread's, a warp's and a CTA's tokens
@pytest.mark.parametrize("T", [0, 1, 2, 7, 8, 9, 16, 17, 63, 64, 65, 127, 128, 129, 256, 300, 700])
@pytest.mark.parametrize("mode", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lengths(T, mode, dtype):
    check(2, T, 96, dtype, mode, seed=T)


# channels that pairs and quads of values fit, or do not; blocks of 32 to 128 of them in part
@pytest.mark.parametrize("C", [1, 2, 3, 31, 32, 34, 64, 65, 127, 130, 260])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("packed", [False, True])
def test_channels(C, dtype, packed):
    check(3, 150, C, dtype, "sigmoid", seed=C, packed=packed)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", ["sigmoid", "log"])
def test_ragged_batches(dtype, mode):
    check(7, 400, 66, dtype, mode, lengths=[400, 0, 1, 128, 129, 399, 257])
    check(2, 5, 8, dtype, mode, lengths=[9, -3])   # taken into [0, T]


@pytest.mark.parametrize("C,dtype", [(2056, torch.bfloat16), (1992, torch.bfloat16), (1036, torch.float32)])
@pytest.mark.parametrize("mode,packed", [("sigmoid", False), ("log", True)])
def test_tiles_by_tensor_maps(C, dtype, mode, packed):
    """More tiles than the SMs take at once, of rows that fit 16 bytes: the last channels' and the last tokens' are there in
    part, sequences end within a tile, at its border and before any."""
    check(4, 700, C, dtype, mode, seed=C, lengths=[700, 513, 0, 256], packed=packed)


def test_without_states():
    check(2, 200, 40, torch.float32, "sigmoid", state=False)
    check(2, 200, 40, torch.bfloat16, "log", state=False)


@pytest.mark.parametrize("mode", ["sigmoid", "log"])
def test_many_spans(mode):
    """One sequence of hundreds of spans, whose states meet only through one another."""
    check(1, 20000, 34, torch.float32, mode, seed=5)


@pytest.mark.parametrize("B,T,C,dtype", [(1, 9001, 64, torch.bfloat16), (2, 5000, 33, torch.float32),
                                         (1, 6000, 513, torch.float32), (3, 7000, 101, torch.bfloat16)])
@pytest.mark.parametrize("mode", ["sigmoid", "log"])
def test_long_prompts_of_few_channels(B, T, C, dtype, mode):
    """Many tiles of few chains at once; equal calls give equal bits, whichever tile was heard first."""
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, n, _ = make(B, T, C, dtype, mode, C, [T, 1, 4097][:B])
    first = None
    for _ in range(5):
        y, h_T, states = kla.gated_scan_fwd(x, gate, h0, mode=mode, lengths=n, states=True)
        grads = kla.gated_scan_bwd(x, gate, dy, states, dh, mode=mode, lengths=n)
        got = [y, h_T, *grads.values()]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    kla.device_status(DEV)
    clean = [t.double().nan_to_num(0.0) for t in (x, gate)]
    wy, wh = reference(clean[0], clean[1], h0.double(), mode, n)
    assert rel(first[0], wy) <= TOL[dtype] and rel(first[1], wh) <= 3e-5


def test_more_tiles_than_fit_at_once():
    """Equal calls give equal bits, whatever order the tiles finish in, and the state that enters a late token is that
    of the whole prompt: against the same prompt cut in two."""
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, _, _ = make(3, 9000, 1000, torch.bfloat16, "sigmoid", 9)
    y, h_T, s = kla.gated_scan_fwd(x, gate, h0, states=True)
    g = kla.gated_scan_bwd(x, gate, dy, s, dh)
    cut = 5003
    y1, h1, _ = kla.gated_scan_fwd(x[:, :cut], gate[:, :cut], h0)
    y2, h2, _ = kla.gated_scan_fwd(x[:, cut:], gate[:, cut:], h1)
    assert rel(torch.cat([y1, y2], 1), y) <= 4e-3 and rel(h2, h_T) <= 3e-5
    for _ in range(3):
        y3, h3, s3 = kla.gated_scan_fwd(x, gate, h0, states=True)
        g3 = kla.gated_scan_bwd(x, gate, dy, s3, dh)
        assert rel(h3, h_T) <= 3e-5 and rel(y3, y) <= 4e-3 and rel(g3["dgate"], g["dgate"]) <= 4e-3
    kla.device_status(DEV)


def test_gates_that_keep_and_forget():
    """Gates of +-inf and near them: a state is kept or dropped at once, and no NaN comes of it."""
    import gated_delta_rule_14_gb300 as kla
    inf = float("inf")
    for mode, keep, drop, dtype, C in (("sigmoid", inf, -inf, torch.float32, 33), ("log", 0.0, -inf, torch.float32, 33),
                                       ("sigmoid", 200.0, -200.0, torch.float32, 33),
                                       ("sigmoid", inf, -inf, torch.bfloat16, 34),
                                       ("sigmoid", 200.0, -200.0, torch.bfloat16, 33),
                                       ("log", 0.0, -inf, torch.bfloat16, 34)):
        T = 300
        x = torch.randn(1, T, C, device=DEV).to(dtype)
        gate = torch.full((1, T, C), keep, device=DEV, dtype=dtype)
        gate[:, 150] = drop
        xs = torch.zeros_like(x) if mode == "log" else x
        xs = xs.clone()
        xs[:, 150] = x[:, 150]
        h0 = torch.randn(1, C, device=DEV).to(dtype).float()
        y, h_T, s = kla.gated_scan_fwd(xs, gate, h0, mode=mode, states=True)
        g = kla.gated_scan_bwd(xs, gate, torch.ones_like(x), s, None, mode=mode)
        assert torch.equal(y[:, :150].float(), h0[:, None].expand(1, 150, C)), mode
        assert torch.equal(y[:, 150:], x[:, 150:151].expand(1, 150, C)), mode
        assert all(t.isfinite().all() for t in g.values()), mode


def test_long_memory():
    """Gates that keep the state for thousands of tokens: 1 - a is taken by itself, not as what is left of a rounded a.
    The state's rounding of 2^-24 a step adds up over 1 / (1 - a) = 3000 steps as a random walk does: sqrt(3000) 2^-24
    = 3e-6 of the state that is there, which is about 1/40 of x; 40 times that: 1.3e-4."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, gate = torch.randn(1, 6000, 64, generator=gen, device=DEV), torch.full((1, 6000, 64), 8.0, device=DEV)
    y, h_T, _ = kla.gated_scan_fwd(x, gate)
    wy, wh = reference(x.double(), gate.double(), None, "sigmoid", torch.tensor([6000], device=DEV))
    assert rel(y, wy) <= 1.3e-4 and rel(h_T, wh) <= 1.3e-4


@pytest.mark.parametrize("mode", ["sigmoid", "log"])
def test_gradients_against_differences(mode):
    """Directional derivatives of sum(y dy) + sum(h_T dh) by central differences with steps of 1e-2: off by their
    squares, 1e-4, times a curvature of order one."""
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, _, _ = make(2, 160, 40, torch.float32, mode, 11)

    def loss(x, gate, h0):
        y, h_T, _ = kla.gated_scan_fwd(x, gate, h0, mode=mode)
        return float((y.double() * dy.double()).sum() + (h_T.double() * dh.double()).sum())
    _, _, s = kla.gated_scan_fwd(x, gate, h0, mode=mode, states=True)
    g = kla.gated_scan_bwd(x, gate, dy, s, dh, mode=mode)
    gen = torch.Generator(device=DEV).manual_seed(12)
    for i, name in enumerate(("dx", "dgate", "dh0")):
        at = [x, gate, h0]
        # along the gradient's signs, so that no cancellation is left
        d = g[name].sign() * torch.rand(at[i].shape, generator=gen, device=DEV) * 1e-2
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + d, at[i] - d
        want = (loss(*up) - loss(*down)) / 2
        got = float((g[name].double() * d.double()).sum())
        assert abs(got - want) <= 1e-3 * abs(want), (name, got, want)


def test_shared_and_broadcast_inputs():
    """Strides of zero: one gate for all tokens, one for all sequences, dy of a sum."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(3, 140, 50, generator=gen, device=DEV)
    g1 = torch.randn(1, 1, 50, generator=gen, device=DEV).expand(3, 140, 50)
    g2 = torch.randn(1, 140, 50, generator=gen, device=DEV).expand(3, 140, 50)
    dy = torch.ones(1, 1, 50, device=DEV).expand(3, 140, 50)
    for g in (g1, g2):
        a = kla.gated_scan_fwd(x, g, states=True)
        b = kla.gated_scan_fwd(x, g.contiguous(), states=True)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
        da, db = kla.gated_scan_bwd(x, g, dy, a[2]), kla.gated_scan_bwd(x, g.contiguous(), dy.contiguous(), b[2])
        assert all(torch.equal(da[n], db[n]) for n in da)


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_starts(shift, dtype):
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, _, _ = make(2, 140, 64, dtype, "sigmoid", shift)

    def place(t):
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
        flat[shift:] = t.reshape(-1)
        return flat[shift:].view(t.shape)
    a = kla.gated_scan_fwd(x, gate, h0, states=True)
    b = kla.gated_scan_fwd(place(x), place(gate), place(h0), states=True, out=place(torch.zeros_like(x)))
    assert all(rel(u, v) <= 1e-6 for u, v in zip(a, b))
    ga, gb = kla.gated_scan_bwd(x, gate, dy, a[2], dh), kla.gated_scan_bwd(place(x), place(gate), place(dy), b[2], dh)
    # values on a border of bf16 may go either way where sums are joined in another order
    assert all(rel(gb[n], ga[n]) <= TOL[dtype] for n in ga)


@pytest.mark.parametrize("C,pad,T", [(64, 1, 300), (65, 0, 600), (130, 3, 260), (127, 2, 1000), (1, 0, 700), (129, 0, 129)])
@pytest.mark.parametrize("mode", ["sigmoid", "log"])
def test_rows_that_start_in_the_middle_of_4_bytes(C, pad, T, mode):
    """bf16 rows an odd number of values apart, or of odd length, in tensors that start on 4 bytes; past the last channel lie
    NaN that nothing may take up, and past the outputs' last value one that nothing may overwrite."""
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, _, _ = make(2, T, C, torch.bfloat16, mode, C)

    def place(t):
        wide = torch.full((2 * T * (C + pad) + 2,), float("nan"), dtype=t.dtype, device=DEV)
        view = wide.as_strided((2, T, C), (T * (C + pad), C + pad, 1))
        view.copy_(t)
        return view
    a = kla.gated_scan_fwd(x, gate, h0, mode=mode, states=True)
    room = torch.full((2 * T * C + 1,), 7.0, dtype=torch.bfloat16, device=DEV)
    b = kla.gated_scan_fwd(place(x), place(gate), h0, mode=mode, states=True, out=room[:-1].view(2, T, C))
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and float(room[-1]) == 7.0
    ga, gb = kla.gated_scan_bwd(x, gate, dy, a[2], dh, mode=mode), kla.gated_scan_bwd(place(x), place(gate), place(dy),
                                                                                      b[2], dh, mode=mode)
    assert all(torch.equal(ga[n], gb[n]) for n in ga)
    want, wh = reference(x.double(), gate.double(), h0.double(), mode, torch.full((2,), T, device=DEV))
    assert rel(b[0], want) <= 4e-3 and rel(b[1], wh) <= 3e-5


def test_offsets_past_32_bits():
    """Sequences 2^31 + 64 values apart."""
    import gated_delta_rule_14_gb300 as kla
    far, T, C = 2**31 + 64, 130, 64
    base = torch.empty(far + T * 2 * C, dtype=torch.bfloat16, device=DEV)
    x = base.as_strided((2, T, C), (far, 2 * C, 1), 0)
    gate = base.as_strided((2, T, C), (far, 2 * C, 1), C)
    gen = torch.Generator(device=DEV).manual_seed(2)
    x.copy_(torch.randn(2, T, C, generator=gen, device=DEV))
    gate.copy_(torch.randn(2, T, C, generator=gen, device=DEV))
    a = kla.gated_scan_fwd(x, gate, states=True)
    b = kla.gated_scan_fwd(x.contiguous(), gate.contiguous(), states=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    da, db = kla.gated_scan_bwd(x, gate, x, a[2]), kla.gated_scan_bwd(x.contiguous(), gate.contiguous(), x, b[2])
    assert all(torch.equal(da[n], db[n]) for n in da)


def test_state_in_place_and_no_state():
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, _, _ = make(2, 300, 70, torch.bfloat16, "sigmoid", 4)
    y, h_T, _ = kla.gated_scan_fwd(x, gate, h0)
    h = h0.clone()
    y2, same, _ = kla.gated_scan_fwd(x, gate, h, h_T=h)
    assert same is h and torch.equal(h, h_T) and torch.equal(y, y2)
    y3, none, _ = kla.gated_scan_fwd(x, gate, h0, final_state=False)
    assert none is None and torch.equal(y, y3)
    _, _, s = kla.gated_scan_fwd(x, gate, h0, states=True)
    assert kla.gated_scan_bwd(x, gate, dy, s, dh, want_dh0=False)["dh0"] is None


@pytest.mark.parametrize("C", [1, 7, 32, 2048, 5000])
@pytest.mark.parametrize("mode", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_equal_a_prompt(C, mode, dtype):
    import gated_delta_rule_14_gb300 as kla
    x, gate, _, h0, _, _, _ = make(3, 40, C, dtype, mode, C, packed=True)
    y, h_T, _ = kla.gated_scan_fwd(x, gate, h0, mode=mode)
    h = h0.clone()
    ys = [kla.gated_scan_step(x[:, t], gate[:, t], h, mode=mode) for t in range(40)]
    assert rel(h, h_T) <= 3e-5 and rel(torch.stack(ys, 1), y) <= TOL[dtype]


def test_refusals():
    import gated_delta_rule_14_gb300 as kla
    x = torch.randn(2, 10, 8, device=DEV)
    s = torch.zeros(2, 1, 8, device=DEV)
    with pytest.raises(ValueError, match="mode"):
        kla.gated_scan_fwd(x, x, mode="tanh")
    with pytest.raises(TypeError):
        kla.gated_scan_fwd(x.half(), x.half())
    with pytest.raises(TypeError):
        kla.gated_scan_fwd(x, x.bfloat16())
    with pytest.raises(ValueError):
        kla.gated_scan_fwd(x, x[:, :9])
    with pytest.raises(ValueError):
        kla.gated_scan_fwd(x.transpose(1, 2), x.transpose(1, 2))   # the last axis is not dense
    with pytest.raises(ValueError):
        kla.gated_scan_fwd(x, x, torch.zeros(2, 9, device=DEV))
    with pytest.raises(TypeError):
        kla.gated_scan_fwd(x, x, lengths=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        kla.gated_scan_fwd(x.cpu(), x.cpu())
    with pytest.raises(ValueError):
        kla.gated_scan_bwd(x, x, x, s[:, :0])
    with pytest.raises(kla.KlaError):
        kla.gated_scan_fwd(x, x.clone(), out=x)
    with pytest.raises(ValueError):
        kla.gated_scan_step(x[:, 0], x[:, 0], torch.zeros(2, 8))
    with pytest.raises(kla.KlaError):
        kla.gated_scan_step(x[:1, 0].expand(2, 8), x[:, 0], torch.zeros(2, 8, device=DEV))
