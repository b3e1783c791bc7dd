"""The gated scan where its gates are far from the ordinary, value by value against 64 bits: states and gradients that such
a gate leaves are small, and a norm over a whole tensor does not see them."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}   # of a stored value: half a step

# how rows reach the kernels: 16-byte and 4-byte copies, rows off 4 bytes, tensors that start off 4 bytes, tensor maps
LAYOUTS = [(2, 64, 0), (2, 34, 0), (2, 65, 0), (2, 64, 1), (8, 1024, 0)]


def scan(x, gate, h0, mode, dy=None, dh=None):
    """y, h_T and, with dy, the gradients (dx, dgate, dh0) from the definition in 64 bits, token by token."""
    x, gate, h0 = x.double(), gate.double(), h0.double()
    a = torch.exp(gate) if mode == "log" else torch.sigmoid(gate)
    w = torch.ones_like(a) if mode == "log" else torch.sigmoid(-gate)
    before = torch.empty_like(x)
    y = torch.empty_like(x)
    h = h0
    for t in range(x.shape[1]):
        before[:, t] = h
        h = a[:, t] * h + w[:, t] * x[:, t]
        y[:, t] = h
    if dy is None:
        return y, h
    dx, dg, e = torch.empty_like(x), torch.empty_like(x), dh.double()
    for t in range(x.shape[1] - 1, -1, -1):
        full = dy[:, t].double() + e
        e = a[:, t] * full
        dx[:, t] = w[:, t] * full
        dg[:, t] = before[:, t] * e if mode == "log" else w[:, t] * (before[:, t] - x[:, t]) * e
    return y, h, dx, dg, e


def place(t, shift):
    """The same values `shift` of them behind a 16-byte border."""
    flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
    flat[shift:] = t.reshape(-1)
    return flat[shift:].view(t.shape)


def run(x, gate, h0, mode, dy, dh):
    import gated_delta_rule_14_gb300 as kla
    y, h_T, s = kla.gated_scan_fwd(x, gate, h0, mode=mode, states=True)
    g = kla.gated_scan_bwd(x, gate, dy, s, dh, mode=mode)
    kla.device_status(DEV)
    return y, h_T, g["dx"], g["dgate"], g["dh0"]


def close(got, want, tol):
    """Every value within `tol` of itself, and of what is stored in few bits half a step more."""
    for name, a, b in zip(("y", "h_T", "dx", "dgate", "dh0"), got, want):
        off = ((a.double() - b).abs() / b.abs().clamp(min=1e-30)).max()
        assert float(off) <= tol + (HALF[a.dtype] if name in ("y", "dx", "dgate") else 0.0), (name, float(off))


@pytest.mark.parametrize("B,C,shift", LAYOUTS)
def test_gates_that_forget(B, C, shift):
    """bf16, sigmoid: three tokens with gates of -3 to -20 among such as keep, x of zero, so that all that there is of
    a state and of dgate is what these leave. 600 steps of the state at 2^-24 for each product and its factor, 7e-5; at a
    forgetting token the exponent's rounding, 29 x 2^-24, the exponential's 2^-22 and the reciprocal's 2^-23, or where a is
    still 1 - w 2^-23 / sigmoid(-6) = 4.8e-5: 6e-5 for three, or 1.5e-4 where all three are just above -6. dgate has a state
    and a gradient, which three such tokens and the 600 steps are shared out between, and its own factor, one more: 2.6e-4."""
    import gated_delta_rule_14_gb300 as kla
    T, gen = 600, torch.Generator(device=DEV).manual_seed(C)

    def some(*shape):
        return torch.rand(shape, generator=gen, device=DEV) + 0.5
    gate = torch.full((B, T, C), 6.0, device=DEV)
    gate[:, [7, 70, 431]] = -3 - 17 * torch.arange(C, device=DEV) / (C - 1)
    gate, x, dy = gate.bfloat16(), torch.zeros(B, T, C, device=DEV).bfloat16(), some(B, T, C).bfloat16()
    h0, dh = 1e4 * some(B, C), some(B, C)
    want = scan(x, gate, h0, "sigmoid", dy, dh)
    assert float(want[1].min()) > 1e-25
    close(run(place(x, shift), place(gate, shift), h0, "sigmoid", place(dy, shift), dh), want, 2.6e-4)
    h = h0.clone()   # token by token
    for t in range(T):
        kla.gated_scan_step(x[:, t], gate[:, t], h)
    assert float((h / want[1] - 1).abs().max()) <= 2.6e-4


TYPED = [(*at, dtype) for dtype in (torch.bfloat16, torch.float32) for at in LAYOUTS if dtype == torch.bfloat16 or at[1] != 34]


@pytest.mark.parametrize("B,C,shift,dtype", TYPED)
def test_gates_that_grow(B, C, shift, dtype):
    """Logarithms above 0: factors whose products fp32 holds (e^30 here) give what the definition does. Of 600 factors each
    is off by 2^-22 and its products by 2^-24, with nothing that cancels: 600 x 1.25 x 2^-22 = 1.8e-4, twice that for
    dgate, which has a state and a gradient. Masked tokens' gates count for nothing."""
    import gated_delta_rule_14_gb300 as kla
    T, gen = 600, torch.Generator(device=DEV).manual_seed(C)

    def some(*shape):
        return torch.rand(shape, generator=gen, device=DEV) + 0.5
    gate = torch.where(torch.arange(T, device=DEV) % 300 < 150, 0.2, -0.2)[None, :, None] * some(1, 1, C)
    gate = gate.expand(B, T, C).to(dtype)
    x, dy, h0, dh = some(B, T, C).to(dtype), some(B, T, C).to(dtype), some(B, C), some(B, C)
    want = scan(x, gate, h0, "log", dy, dh)
    close(run(place(x, shift), place(gate, shift), h0, "log", place(dy, shift), dh), want, 3.6e-4)
    n = torch.full((B,), T - 170, dtype=torch.int32, device=DEV)
    far = gate.clone()
    far[:, T - 170:] = 90.0
    y, h_T, _ = kla.gated_scan_fwd(place(x, shift), place(far, shift), h0, mode="log", lengths=n)
    kla.device_status(DEV)
    assert float(((h_T / want[0][:, T - 171]) - 1).abs().max()) <= 1.8e-4 and float(y[:, T - 170:].abs().max()) == 0.0


@pytest.mark.parametrize("B,C,shift,dtype", TYPED)
def test_products_past_fp32_are_reported(B, C, shift, dtype):
    """128 factors of e, times a state of zero: the product of a stretch is infinite, and a NaN may come of it. The call says
    so, forward and backward, and the next one is as good as any."""
    import gated_delta_rule_14_gb300 as kla
    T = 600
    x = torch.zeros(B, T, C, dtype=dtype, device=DEV)
    x, grow, calm = place(x, shift), place(torch.full_like(x, 1.0), shift), place(torch.full_like(x, -1.0), shift)
    kla.device_status(DEV)
    kla.gated_scan_fwd(x, grow, mode="log")
    with pytest.raises(kla.KlaError):
        kla.device_status(DEV)
    states = torch.zeros(B, -(-T // 128), C, device=DEV)
    kla.gated_scan_bwd(x, grow, x, states, mode="log")
    with pytest.raises(kla.KlaError):
        kla.device_status(DEV)
    y, h_T, s = kla.gated_scan_fwd(x, calm, mode="log", states=True)
    g = kla.gated_scan_bwd(x, calm, x, s, mode="log")
    kla.device_status(DEV)
    assert all(float(t.abs().max()) == 0.0 for t in (y, h_T, *g.values()))


# losses of 1e-5 to 1e-3 a token, one for every channel
def slow_gates(C, dtype, mode):
    rate = 10.0 ** (-5 + 2 * torch.arange(C, device=DEV, dtype=torch.float64) / (C - 1))
    return (-rate if mode == "log" else torch.log((1 - rate) / rate)).to(dtype)


@pytest.mark.parametrize("mode", ["log", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,C,shift", [(1, 100000, 64, 0), (1, 100000, 65, 0), (1, 100000, 34, 1), (2, 50000, 512, 0)])
def test_memory_of_100000_tokens(B, T, C, shift, dtype, mode):
    """Constant gates, whose errors all go to one side, and x, dy above zero, so that nothing cancels. What is told of 128
    tokens or more has 8 stretches' products, 7 of those and a state, each rounded by 2^-25: of the decay per token r that
    is 2^-28 / r, 3.7e-4 at 1e-5. Within a stretch of at most 32 tokens a factor's 2^-22 make 8e-6 and sums 32 x 2^-24 as
    much: 3e-5 more."""
    gen = torch.Generator(device=DEV).manual_seed(C)

    def some(*shape):
        return torch.rand(shape, generator=gen, device=DEV) + 0.5
    one = slow_gates(C, dtype, mode)
    x, dy, dh = some(B, T, C).to(dtype), some(B, T, C).to(dtype), some(B, C)
    gate = place(one.expand(B, T, C).contiguous(), shift)
    y, h_T, dx, dg, dh0 = run(place(x, shift), gate, torch.zeros(B, C, device=DEV), mode, place(dy, shift), dh)
    g = one.double()
    log_a, w = (g, torch.ones_like(g)) if mode == "log" else (torch.nn.functional.logsigmoid(g), torch.sigmoid(-g))
    past = torch.exp(torch.arange(T, device=DEV)[:, None] * log_a)
    state = (x.double() * past.flip(0)).sum(1) * w
    reach = torch.exp(log_a) * (dh.double() * past[-1] + (dy.double() * past).sum(1))
    tol = 2.0**-28 / (1 - torch.exp(log_a)) + 3e-5
    for name, a, b in (("h_T", h_T, state), ("dh0", dh0, reach)):
        off = (a.double() / b - 1).abs() / tol
        assert float(off.max()) <= 1, (name, float(off.max()))


@pytest.mark.parametrize("mode", ["log", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_with_long_memory(dtype, mode):
    """4096 single tokens with the same gates: every step rounds the state by 2^-24, in the mean of a random walk 4e-6;
    ten times that."""
    import gated_delta_rule_14_gb300 as kla
    C, T, gen = 64, 4096, torch.Generator(device=DEV).manual_seed(7)
    one = slow_gates(C, dtype, mode)
    x = (torch.rand((T, 1, C), generator=gen, device=DEV) + 0.5).to(dtype)
    h, gate = torch.zeros(1, C, device=DEV), one[None].contiguous()
    for t in range(T):
        kla.gated_scan_step(x[t], gate, h, mode=mode)
    g = one.double()
    log_a, w = (g, torch.ones_like(g)) if mode == "log" else (torch.nn.functional.logsigmoid(g), torch.sigmoid(-g))
    want = (x[:, 0].double() * torch.exp(torch.arange(T, device=DEV).flip(0)[:, None] * log_a)).sum(0) * w
    assert float((h[0].double() / want - 1).abs().max()) <= 4e-5


@pytest.mark.parametrize("mode", ["log", "sigmoid"])
@pytest.mark.parametrize("B,C,shift,dtype", TYPED)
def test_states_that_are_not_finite(B, C, shift, dtype, mode):
    """A state that begins as infinity, one that an infinite input makes so, one that a NaN does: from there on nothing
    finite comes of these channels, whether their gates keep or forget, and the others keep their bits, gradients too."""
    import gated_delta_rule_14_gb300 as kla
    T, gen = 600, torch.Generator(device=DEV).manual_seed(C)
    x, dy = (torch.randn((B, T, C), generator=gen, device=DEV).to(dtype) for _ in range(2))
    gate = torch.randn((B, T, C), generator=gen, device=DEV)
    gate = (-torch.nn.functional.softplus(gate) if mode == "log" else gate).to(dtype)
    gate[:, 400, 5:9] = -float("inf")
    h0, dh = torch.randn((B, C), generator=gen, device=DEV), torch.zeros(B, C, device=DEV)
    clean = run(place(x, shift), place(gate, shift), h0, mode, place(dy, shift), dh)
    x, h0 = x.clone(), h0.clone()
    h0[:, 5] = float("inf")
    x[:, 270, 6] = -float("inf")
    x[:, 0, 7] = float("nan")
    got = run(place(x, shift), place(gate, shift), h0, mode, place(dy, shift), dh)
    y, h_T = got[0].float(), got[1]
    assert not y[:, :, 5].isfinite().any() and not y[:, 270:, 6].isfinite().any() and not y[:, :, 7].isfinite().any()
    assert not h_T[:, 5:8].isfinite().any() and torch.equal(y[:, :270, 6], clean[0][:, :270, 6].float())
    rest = [c for c in range(C) if c not in (5, 6, 7)]
    assert all(torch.equal(a[..., rest], b[..., rest]) for a, b in zip(got, clean))


@pytest.mark.parametrize("B,C,shift,dtype", TYPED)
def test_products_that_a_gate_of_minus_infinity_follows_are_reported(B, C, shift, dtype):
    """An infinite product times zero is a NaN, not a state forgotten. In one stretch of tokens (e^180) it is there whatever
    the stretches are. Across them, e^110 of tokens 10 to 119, it depends on them: with 32 tokens a stretch the products up
    to token 95 are e^86, which fp32 holds, and that of the next one is zero, as the -inf is in it; so either the call is
    reported, or all is as the definition has it, zero."""
    import gated_delta_rule_14_gb300 as kla
    T = 600
    x = place(torch.zeros(B, T, C, dtype=dtype, device=DEV), shift)
    states = torch.zeros(B, -(-T // 128), C, device=DEV)
    for grow, drop in ((slice(0, 2), 3), (slice(10, 120), 125)):   # e^180 in one stretch, e^110 over several
        gate = torch.full((B, T, C), -0.5, device=DEV)
        gate[:, grow] = 90.0 if drop == 3 else 1.0
        gate[:, drop] = -float("inf")
        gate = place(gate.to(dtype), shift)
        kla.device_status(DEV)
        for call in (lambda: kla.gated_scan_fwd(x, gate, mode="log")[:2],
                     lambda: kla.gated_scan_bwd(x, gate, x, states, mode="log").values()):
            out = list(call())
            try:
                kla.device_status(DEV)
                assert drop != 3 and all(float(t.abs().max()) == 0.0 for t in out)
            except kla.KlaError:
                pass
    n = torch.zeros(B, dtype=torch.int32, device=DEV)   # masked, they are nobody's
    kla.gated_scan_fwd(x, gate, mode="log", lengths=n)
    kla.gated_scan_bwd(x, gate, x, states, mode="log", lengths=n)
    kla.device_status(DEV)
