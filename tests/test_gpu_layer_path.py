"""The layer operators together, as a layer trains and decodes (examples/decay_layer.py)."""
import importlib.util
import os

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decay_layer", os.path.join(ROOT, "examples", "decay_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_gradients_of_the_layer_against_64_bits(example):
    """Every activation is rounded to bf16 once or twice on its way (2^-9 each) through six products: 3e-2."""
    layer = example.DecayLayer(vocab=64, heads=2, seed=3)
    tokens = torch.randint(0, 64, (2, 150), device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    loss, got = layer.gradients(tokens)

    p = {n: (t.bfloat16() if n in ("embed", "qkv", "out") else t).double().requires_grad_(True)
         for n, t in layer.params.items()}
    h = p["embed"][tokens[:, :-1]]
    q, k, v = (h @ p["qkv"]).view(2, 149, 3, 2, 128).unbind(2)
    t = torch.arange(149, device=DEV)
    w = torch.tril(layer.decay.double()[:, None, None] ** (t[:, None] - t).clamp(min=0))
    o = layer.scale * torch.einsum("bihd,bjhd,hij,bjhe->bihe", q, k, w, v)
    xh = (o - o.mean(-1, keepdim=True)) / (o.var(-1, correction=0, keepdim=True) + 1e-5).sqrt()
    z = (xh * p["norm_w"] + p["norm_b"]).flatten(-2) @ p["out"] + h
    want = -torch.log_softmax(z @ p["embed"].t(), -1).gather(-1, tokens[:, 1:, None]).mean()
    grads = torch.autograd.grad(want, list(p.values()))
    assert abs(float(loss) - float(want.detach())) <= 3e-2 * float(want.detach())
    for name, g in zip(p, grads):
        assert rel(got[name], g) <= 3e-2, (name, rel(got[name], g))


def test_the_example_learns_and_decodes(example):
    losses, right = example.main()
    assert losses[-1] < 0.5 * losses[0] and right > 0.5


def test_prompt_then_steps_equals_one_prompt():
    """States and outputs of 40 single-token steps after a prompt against the whole sequence as one prompt (its
    outputs round the scores and the state to 8 bits: 6e-3; its state keeps 17: 1e-5)."""
    import gated_delta_rule_14_gb300 as kla
    q, k, v = (torch.randn(3, 200, 2, 128, device=DEV).bfloat16() for _ in range(3))
    g = torch.tensor([0.97, 0.999], device=DEV)
    o, S = kla.linear_fwd(q, k, v, g, q_scale=0.1)
    _, S2 = kla.linear_fwd(q[:, :160], k[:, :160], v[:, :160], g, q_scale=0.1)
    outs = [kla.linear_step(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(), g, S2, q_scale=0.1)
            for t in range(160, 200)]
    kla.device_status(DEV)
    assert rel(torch.stack(outs, 1), o[:, 160:]) <= 6e-3 and rel(S2, S) <= 1e-5


def test_states_follow_beams_either_way():
    """linear_step with parents equals reorder_states and then linear_step, bit for bit."""
    import gated_delta_rule_14_gb300 as kla
    B, W, H = 3, 4, 2
    S = torch.randn(B, W, H, 128, 128, device=DEV)
    q, k, v = (torch.randn(B * W, H, 128, device=DEV).bfloat16() for _ in range(3))
    g = torch.tensor([0.97, 0.999], device=DEV)
    logits, scores = torch.randn(B, W, 700, device=DEV), -torch.rand(B, W, device=DEV)
    _, parents, _, _ = kla.beam_select(logits, scores)
    moved = kla.reorder_states(S, parents).view(B * W, H, 128, 128)
    a = kla.linear_step(q, k, v, g, moved)
    first = (torch.arange(B, device=DEV, dtype=torch.int32) * W)[:, None]
    out = torch.empty_like(moved)
    b = kla.linear_step(q, k, v, g, S.view(B * W, H, 128, 128), parent=(parents + first).view(-1), S_out=out)
    assert torch.equal(a, b) and torch.equal(moved, out)


def test_operators_in_a_graph():
    """A decode step captured as one CUDA graph gives the eager step's results."""
    import gated_delta_rule_14_gb300 as kla
    B, H = 4, 2
    q, k, v = (torch.randn(B, H, 128, device=DEV).bfloat16() for _ in range(3))
    g = torch.tensor([0.97, 0.999], device=DEV)
    w = torch.randn(H, 128, device=DEV)
    S0 = torch.randn(B, H, 128, 128, device=DEV)
    S = S0.clone()
    head = torch.randn(H * 128, 900, device=DEV).bfloat16()

    def step():
        o = kla.linear_step(q, k, v, g, S)
        y, _, _ = kla.layer_norm_fwd(o, w, stats=False)
        return kla.beam_select((y.flatten(1) @ head).view(1, B, 900), torch.zeros(1, B, device=DEV))
    eager = step()
    state = S.clone()
    S.copy_(S0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    S.copy_(S0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    S.copy_(S0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(S, state) and all(torch.equal(x, y) for x, y in zip(out, eager))


def test_calls_of_several_launches_in_a_graph():
    """A training step whose calls launch kernels that depend on one another (sequences cut into segments, partial
    sums of the norm's gradients), captured as one CUDA graph, gives the eager step's results."""
    import gated_delta_rule_14_gb300 as kla
    gen = torch.Generator(device=DEV).manual_seed(31)
    q, k, v, dy = (torch.randn(1, 3000, 2, 128, generator=gen, device=DEV).bfloat16() for _ in range(4))
    g, w = torch.tensor([0.97, 0.999], device=DEV), torch.randn(2, 128, generator=gen, device=DEV)

    def step():
        o, S = kla.linear_fwd(q, k, v, g, q_scale=0.1)
        y, mean, rstd = kla.layer_norm_fwd(o, w)
        do, dw, db = kla.layer_norm_bwd(dy, o, w, mean, rstd)
        d = kla.linear_bwd(q, k, v, g, do, q_scale=0.1)
        return o, S, y, do, dw, db, *d.values()
    eager = step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        graph.replay()
    kla.device_status(DEV)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
