"""Linear attention with one decay per head (prompts, gradients, single tokens) on the GPU against
the recurrence in 64 bits, token by token.

Tolerances (relative L2), from the arithmetic: fp32 calls round at 2^-24 over sums of a few hundred
terms, 1e-5 as for every fp32 path of the library. bf16 calls round the score tile, the state as an
operand and the output to 8 bits, each at most 2^-9 relative: 3 * 2^-9 = 6e-3. Their fp32 states come
from products of bf16 values with decays kept to two bf16 terms (2^-17): 1e-5.
"""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 1e-5, torch.bfloat16: 6e-3}


def rel(a, b):
    a, b = a.double(), b.double()
    n = b.norm()
    return float((a - b).norm() / n) if n > 0 else float((a - b).norm())


def recurrence(q, k, v, g, s, S, n):
    """Token by token in 64 bits; differentiable. n: valid tokens of each sequence."""
    B, T = q.shape[:2]
    n = torch.as_tensor(n, device=q.device).view(B, 1, 1, 1)
    outs = []
    for t in range(T):
        live = t < n
        S = torch.where(live, g.view(1, -1, 1, 1) * S + k[:, t, :, :, None] * v[:, t, :, None, :], S)
        o = s * torch.einsum("bhd,bhde->bhe", q[:, t], S)
        outs.append(torch.where(live[..., 0], o, 0.0))
    o = torch.stack(outs, 1) if outs else v[:, :0]
    return o, S


def make(B, T, H, dk, dv, dtype, seed=0, s0=True, lengths=None, g=None):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *sh, dt=dtype: torch.randn(sh, generator=gen, device=DEV).to(dt)   # noqa: E731
    d = {"q": r(B, T, H, dk), "k": r(B, T, H, dk), "v": r(B, T, H, dv), "dO": r(B, T, H, dv),
         "S0": r(B, H, dk, dv, dt=torch.float32) if s0 else None,
         "dS_T": r(B, H, dk, dv, dt=torch.float32) if s0 else None,
         "g": torch.tensor(g, device=DEV) if g is not None else 1 - torch.rand(H, generator=gen, device=DEV) * 0.1}
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    d["n"] = [T] * B if lengths is None else [min(max(x, 0), T) for x in lengths]
    d["s"] = dk ** -0.5
    return d


def reference(d, grads=False):
    n = torch.tensor(d["n"], device=DEV)
    live = (torch.arange(d["q"].shape[1], device=DEV) < n[:, None])[:, :, None, None]
    leaf = [torch.where(live, d[x].double(), 0.0).requires_grad_(grads) for x in "qkv"]
    B, _, H, dk = d["q"].shape
    S0 = d["S0"].double() if d["S0"] is not None else torch.zeros(B, H, dk, d["v"].shape[3], device=DEV).double()
    S0.requires_grad_(grads)
    o, S = recurrence(*leaf, d["g"].double(), d["s"], S0, d["n"])
    if not grads:
        return o, S
    dO = torch.where(live, d["dO"].double(), 0.0)
    loss = (o * dO).sum() + ((S * d["dS_T"].double()).sum() if d["dS_T"] is not None else 0.0)
    return dict(zip(("dq", "dk", "dv", "dS0"), torch.autograd.grad(loss, leaf + [S0])))


def run_fwd(d, **kw):
    import gated_delta_rule_14_gb300 as kla
    o, S = kla.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["S0"], q_scale=d["s"], lengths=d["lengths"], **kw)
    kla.device_status(DEV)
    return o, S


def run_bwd(d):
    import gated_delta_rule_14_gb300 as kla
    r = kla.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], d["S0"], d["dS_T"], q_scale=d["s"],
                       lengths=d["lengths"])
    kla.device_status(DEV)
    return r


def check(d):
    tol = TOL[d["q"].dtype]
    o, S = run_fwd(d)
    o_ref, S_ref = reference(d)
    assert rel(o, o_ref) <= tol and rel(S, S_ref) <= 1e-5, (rel(o, o_ref), rel(S, S_ref))
    got, want = run_bwd(d), reference(d, True)
    for x in ("dq", "dk", "dv", "dS0"):
        assert rel(got[x], want[x]) <= (1e-5 if x == "dS0" else tol), (x, rel(got[x], want[x]))


# one token, inside the fp32 scan's chunk of 64 tokens, below / at / above the tensor cores' 128, several chunks,
# odd tails
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 127, 128, 129, 256, 385])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lengths_of_one_chunk_and_more(T, dtype):
    check(make(2, T, 3, 128, 128, dtype, seed=T))


@pytest.mark.parametrize("dk,dv", [(16, 16), (16, 128), (32, 64), (64, 32), (128, 16), (64, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_head_sizes(dk, dv, dtype):
    check(make(1, 75, 2, dk, dv, dtype, seed=dk + dv))


@pytest.mark.parametrize("dtype,T", [(torch.bfloat16, 2500), (torch.float32, 1300)])
@pytest.mark.parametrize("lengths", [None, [0, 1], [1111, 700]])
def test_few_heads_long_sequences(dtype, T, lengths):
    """Enough tokens a chain for the sequence to be cut into segments; lengths that end inside one."""
    check(make(2, T, 2, 128, 128, dtype, seed=5, lengths=lengths))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [70, 300])
def test_masked_tokens_hold_anything(dtype, T):
    d = make(5, T, 2, 128, 128, dtype, seed=9, lengths=[0, T, 1, T // 2, -3])
    for b, n in enumerate(d["n"]):
        for i, x in enumerate(("q", "k", "v", "dO")):
            d[x][b, n:] = (float("nan"), float("inf"), float("-inf"), float("nan"))[i]
    o, S = run_fwd(d)
    o_ref, S_ref = reference(d)
    assert rel(o, o_ref) <= TOL[dtype] and rel(S, S_ref) <= 1e-5
    assert torch.equal(S[0], d["S0"][0]) and torch.equal(S[4], d["S0"][4])   # nothing valid: the state stays
    got, want = run_bwd(d), reference(d, True)
    for x in ("dq", "dk", "dv", "dS0"):
        assert rel(got[x], want[x]) <= (1e-5 if x == "dS0" else TOL[dtype]), x
    for b, n in enumerate(d["n"]):
        assert not o[b, n:].any() and not got["dq"][b, n:].any() and not got["dv"][b, n:].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decays_from_zero_to_one(dtype):
    """0 (every token for itself), one near the smallest power that fp32 holds over a chunk, 1 (no decay)."""
    check(make(1, 300, 5, 128, 128, dtype, seed=2, g=[0.0, 1e-3, 0.3, 0.9999, 1.0]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_initial_state(dtype):
    check(make(1, 200, 2, 128, 128, dtype, seed=3, s0=False))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_strided_inputs_equal_contiguous_ones(dtype, pad):
    """Slices of a packed projection; `pad` = 1 leaves rows that no 16-byte access fits."""
    B, T, H, d = 2, 150, 3, 128
    gen = torch.Generator(device=DEV).manual_seed(1)
    wide = torch.randn((B, T, 4, H, d + pad), generator=gen, device=DEV).to(dtype)
    view = {x: wide[:, :, i, :, pad:] for i, x in enumerate(("q", "k", "v", "dO"))}
    base = make(B, T, H, d, d, dtype, seed=4, lengths=[T, 97])
    dense = {**base, **{x: t.contiguous() for x, t in view.items()}}
    check(dense)
    strided = {**base, **view}
    a, b = run_fwd(dense), run_fwd(strided)
    assert rel(b[0], a[0]) <= TOL[dtype] and rel(b[1], a[1]) <= 1e-5
    ga, gb = run_bwd(dense), run_bwd(strided)
    for x in ga:
        assert rel(gb[x], ga[x]) <= (1e-5 if x == "dS0" else TOL[dtype]), x


def test_state_in_place_and_continuation():
    import gated_delta_rule_14_gb300 as kla
    d = make(2, 333, 2, 128, 128, torch.bfloat16, seed=8)
    o, S = run_fwd(d)
    cut = 131
    S2 = d["S0"].clone()
    parts = []
    for sl in (slice(0, cut), slice(cut, None)):
        p, _ = kla.linear_fwd(d["q"][:, sl], d["k"][:, sl], d["v"][:, sl], d["g"], S2, q_scale=d["s"], S_T=S2)
        parts.append(p)
    assert rel(torch.cat(parts, 1), o) <= 6e-3 and rel(S2, S) <= 1e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_state_in_place_over_segments(dtype):
    import gated_delta_rule_14_gb300 as kla
    d = make(1, 3000, 2, 128, 128, dtype, seed=12)
    o, S = run_fwd(d)
    S2 = d["S0"].clone()
    o2, _ = kla.linear_fwd(d["q"], d["k"], d["v"], d["g"], S2, q_scale=d["s"], S_T=S2)
    assert torch.equal(o, o2) and torch.equal(S, S2)


def test_no_tokens():
    import gated_delta_rule_14_gb300 as kla
    d = make(2, 0, 2, 64, 32, torch.float32, seed=8)
    o, S = run_fwd(d)
    assert o.shape == (2, 0, 2, 32) and torch.equal(S, d["S0"])
    assert torch.equal(run_bwd(d)["dS0"], d["dS_T"])
    _, S = kla.linear_fwd(d["q"], d["k"], d["v"], d["g"])
    assert not S.any()


def test_gradient_against_differences():
    """fp32 gradients along a random direction against central differences of the 64-bit recurrence: the
    difference's own error is ~h^2 = 1e-8 of the loss's third derivative (zero in each input alone, small
    jointly) plus 1e-16 / h; 1e-4 leaves room for both and for fp32."""
    d = make(2, 45, 2, 16, 32, torch.float32, seed=6, lengths=[45, 17])
    got = run_bwd(d)
    gen = torch.Generator(device=DEV).manual_seed(77)
    for x, gx in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("S0", "dS0")):
        e = torch.randn(d[x].shape, generator=gen, device=DEV, dtype=torch.float64)

        def loss(h):
            m = dict(d)
            m[x] = d[x].double() + h * e
            o, S = reference(m)
            return float((o * d["dO"].double()).sum() + (S * d["dS_T"].double()).sum())
        h = 1e-4
        num = (loss(h) - loss(-h)) / (2 * h)
        ana = float((got[gx].double() * e).sum())
        assert abs(num - ana) <= 1e-4 * max(1.0, abs(num)), (x, num, ana)


def test_equal_calls_give_equal_bits():
    d = make(1, 2000, 2, 128, 128, torch.bfloat16, seed=10)
    a, b = run_fwd(d), run_fwd(d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = run_bwd(d), run_bwd(d)
    assert all(torch.equal(ga[x], gb[x]) for x in ga)


def test_on_another_stream():
    d = make(1, 500, 2, 128, 128, torch.bfloat16, seed=11)
    a = run_fwd(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run_fwd(d)
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dk,dv", [(128, 128), (16, 16), (32, 128), (64, 16)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_step(dk, dv, dtype):
    import gated_delta_rule_14_gb300 as kla
    d = make(3, 5, 2, dk, dv, dtype, seed=dk)
    S, outs = d["S0"].clone(), []
    for t in range(5):
        outs.append(kla.linear_step(d["q"][:, t].contiguous(), d["k"][:, t].contiguous(), d["v"][:, t].contiguous(),
                                    d["g"], S, q_scale=d["s"]))
    o_ref, S_ref = reference(d)
    tol = 1e-5 if dtype == torch.float32 else 4e-3   # one rounding of the output to bf16: 2^-9
    assert rel(torch.stack(outs, 1), o_ref) <= tol and rel(S, S_ref) <= 1e-6


def test_step_follows_parents():
    import gated_delta_rule_14_gb300 as kla
    d = make(6, 1, 2, 128, 128, torch.float32, seed=21)
    parent = torch.tensor([0, 0, 5, -1, 9, 3], dtype=torch.int32, device=DEV)   # -1, 9: from zeros
    start = torch.zeros_like(d["S0"])
    for b, p in enumerate(parent.tolist()):
        if 0 <= p < 6:
            start[b] = d["S0"][p]
    before = d["S0"].clone()
    S_out = torch.empty_like(d["S0"])
    o = kla.linear_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"], d["S0"], q_scale=d["s"], parent=parent,
                        S_out=S_out)
    o_ref, S_ref = reference({**d, "S0": start})
    assert rel(o, o_ref[:, 0]) <= 1e-5 and rel(S_out, S_ref) <= 1e-6
    assert torch.equal(before, d["S0"])


def test_step_from_a_larger_pool():
    import gated_delta_rule_14_gb300 as kla
    d = make(2, 1, 2, 64, 64, torch.float32, seed=22)
    pool = torch.randn(7, 2, 64, 64, device=DEV)
    parent = torch.tensor([6, 2], dtype=torch.int32, device=DEV)
    S_out = torch.empty_like(d["S0"])
    kla.linear_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"], pool, parent=parent, S_out=S_out)
    _, S_ref = reference({**d, "S0": pool[parent.long()]})
    assert rel(S_out, S_ref) <= 1e-6


def test_refusals():
    import gated_delta_rule_14_gb300 as kla
    d = make(1, 4, 2, 16, 16, torch.float32)
    a = (d["q"], d["k"], d["v"], d["g"])
    with pytest.raises(TypeError):
        kla.linear_fwd(d["q"].half(), *a[1:])
    with pytest.raises(TypeError):
        kla.linear_fwd(d["q"], d["k"].bfloat16(), d["v"], d["g"])
    with pytest.raises(ValueError):
        kla.linear_fwd(d["q"], d["k"][:, :3], d["v"], d["g"])
    with pytest.raises(ValueError):
        kla.linear_fwd(d["q"].cpu(), *a[1:])
    with pytest.raises(ValueError):
        kla.linear_fwd(*a[:3], d["g"].cpu())
    with pytest.raises(ValueError):
        kla.linear_fwd(*a[:3], d["g"][:1])
    with pytest.raises(ValueError):
        kla.linear_fwd(d["q"].transpose(2, 3).contiguous().transpose(2, 3), *a[1:])   # last axis not dense
    with pytest.raises(TypeError):
        kla.linear_fwd(*a, lengths=torch.tensor([4], device=DEV))                      # int64
    with pytest.raises(kla.KlaError):
        kla.linear_fwd(*a, q_scale=float("nan"))
    with pytest.raises(kla.KlaError):
        kla.linear_fwd(d["q"][..., :8].contiguous(), d["k"][..., :8].contiguous(), d["v"], d["g"])
    with pytest.raises(kla.KlaError):
        kla.linear_fwd(*a, out=d["v"])                                                # output over an input
    with pytest.raises(ValueError):
        kla.linear_bwd(*a, d["dO"][:, :2])
    st = (d["q"][:, 0].contiguous(), d["k"][:, 0].contiguous(), d["v"][:, 0].contiguous(), d["g"])
    with pytest.raises(ValueError):
        kla.linear_step(*st, d["S0"], parent=torch.zeros(1, dtype=torch.int32, device=DEV))
    with pytest.raises(kla.KlaError):
        kla.linear_step(*st, d["S0"], parent=torch.zeros(1, dtype=torch.int32, device=DEV), S_out=d["S0"])


# around the fp32 scan's chunk of 64 tokens
@pytest.mark.parametrize("T", [63, 64, 65])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lengths_around_the_fp32_chunk(T, dtype):
    check(make(2, T, 3, 64, 64, dtype, seed=T))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 32)])
def test_uneven_heads_over_segments(dk, dv, dtype):
    """Long sequences of few heads whose lengths end inside segments; dv's state is the transpose of the others'."""
    check(make(3, 1300, 2, dk, dv, dtype, seed=dk, lengths=[1111, 0, 700]))
