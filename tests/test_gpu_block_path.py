"""The block operators together, as a block trains, decodes and verifies drafts with them, in graphs and on streams."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
B, T, H, D = 2, 300, 2, 128


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def rnd(seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return lambda *s, scale=1.0: torch.randn(s, generator=gen, device=DEV) * scale


def params():
    r = rnd(1)
    N = H * D
    return {"qkvz": r(N, 4 * N, scale=N ** -0.5), "heads": 1 + 0.1 * r(H, D), "out": r(N, N, scale=N ** -0.5),
            "scale": 0.5 + 0.1 * r(N), "norm": 1 + 0.1 * r(N), "xg": r(N, 2 * N, scale=N ** -0.5),
            "decay": torch.tensor([0.97, 0.999], device=DEV)}


def block(p, h, freqs, scale, lengths=None):
    """One block: rotary positions, decayed linear attention, the heads' gated norm, a projection, the residual's norm, a
    gated scan. Everything that its gradients take."""
    import gated_delta_rule_14_gb300 as kla
    N = H * D
    c = {"h": h}
    proj = h @ p["qkvz"].bfloat16()
    q, k, v, z = (t.unflatten(-1, (H, D)) for t in proj.split(N, -1))
    c["v"], c["z"] = v, z
    c["q"], c["k"] = kla.rotary_fwd(q, k, freqs, scale=scale)
    c["o"], c["S"] = kla.linear_fwd(c["q"], c["k"], v, p["decay"], q_scale=D ** -0.5, lengths=lengths)
    c["a"], _, c["rstd1"] = kla.gated_norm_fwd(c["o"], z, p["heads"])
    c["x"] = c["a"].flatten(-2) @ p["out"].bfloat16()
    c["y"], c["r"], _, c["rstd2"] = kla.add_norm_fwd(c["x"], h, p["norm"], p["scale"])
    c["xs"], c["gs"] = (c["y"] @ p["xg"].bfloat16()).split(N, -1)
    c["out"], c["h_T"], c["states"] = kla.gated_scan_fwd(c["xs"], c["gs"], lengths=lengths, states=True)
    return c


def gradients(p, c, d_out, d_res, freqs, scale):
    """Gradients of sum(out d_out) + sum(residual d_res) of every parameter and of h."""
    import gated_delta_rule_14_gb300 as kla
    flat = lambda t: t.reshape(-1, t.shape[-1]).float()   # noqa: E731
    g = {}
    s = kla.gated_scan_bwd(c["xs"], c["gs"], d_out, c["states"], want_dh0=False)
    dxg = torch.cat([s["dx"], s["dgate"]], -1)
    g["xg"] = flat(c["y"]).t() @ flat(dxg)
    dy = dxg @ p["xg"].bfloat16().t()
    dx, dres, g["norm"], g["scale"] = kla.add_norm_bwd(dy, d_res, c["x"], c["h"], p["norm"], p["scale"], None, c["rstd2"])
    g["out"] = flat(c["a"].flatten(-2)).t() @ flat(dx)
    da = (dx @ p["out"].bfloat16().t()).unflatten(-1, (H, D))
    do, dz, g["heads"] = kla.gated_norm_bwd(da, c["o"], c["z"], p["heads"], None, c["rstd1"])
    d = kla.linear_bwd(c["q"], c["k"], c["v"], p["decay"], do, q_scale=D ** -0.5, want_dS0=False)
    dq, dk = kla.rotary_bwd(d["dq"], d["dk"], freqs, scale=scale, out_q=d["dq"], out_k=d["dk"])
    dproj = torch.cat([t.flatten(-2) for t in (dq, dk, d["dv"], dz)], -1)
    g["qkvz"] = flat(c["h"]).t() @ flat(dproj)
    g["h"] = dproj @ p["qkvz"].bfloat16().t() + dres
    return g


def reference(p, h, freqs, scale):
    """The block in 64 bits, by operations that autograd follows."""
    N, n = H * D, freqs.shape[0]
    q, k, v, z = (t.unflatten(-1, (H, D)) for t in (h @ p["qkvz"]).split(N, -1))
    t = torch.arange(T, device=DEV)
    turn = torch.polar(torch.full((T, n), scale, device=DEV, dtype=torch.float64), t[:, None].double() * freqs.double())

    def rotary(x):
        w = torch.complex(x[..., :n], x[..., n:]) * turn[:, None]
        return torch.cat([w.real, w.imag], -1)
    w = torch.tril(p["decay"].double()[:, None, None] ** (t[:, None] - t).clamp(min=0))
    o = D ** -0.5 * torch.einsum("bihd,bjhd,hij,bjhe->bihe", rotary(q), rotary(k), w, v)
    rms = lambda x: x / ((x * x).mean(-1, keepdim=True) + 1e-5).sqrt()   # noqa: E731
    a = rms(o) * p["heads"] * torch.nn.functional.silu(z)
    r = h + p["scale"] * (a.flatten(-2) @ p["out"])
    xs, gs = (rms(r) * p["norm"] @ p["xg"]).split(N, -1)
    state, out = torch.zeros_like(xs[:, 0]), []
    for i in range(T):
        f = torch.sigmoid(gs[:, i])
        state = f * state + (1 - f) * xs[:, i]
        out.append(state)
    return torch.stack(out, 1), r


def test_a_block_and_its_gradients_against_64_bits():
    """Every activation is rounded to bf16 once or twice on its way (2^-8 at most each) through seven products and two
    recurrences: 3e-2."""
    import gated_delta_rule_14_gb300 as kla
    p, r = params(), rnd(2)
    freqs, scale = kla.rotary_freqs(D, scaling="yarn", factor=4.0, original_length=128, device=DEV)
    h, d_out, d_res = (r(B, T, H * D).bfloat16() for _ in range(3))
    c = block(p, h, freqs, scale)
    got = gradients(p, c, d_out, d_res, freqs, scale)
    kla.device_status(DEV)
    leaves = {n: (t.bfloat16() if n in ("qkvz", "out", "xg") else t).double().requires_grad_(True)
              for n, t in p.items() if n != "decay"}
    leaves["h"] = h.double().requires_grad_(True)
    want, res = reference({**leaves, "decay": p["decay"]}, leaves["h"], freqs, scale)
    grads = torch.autograd.grad((want * d_out.double()).sum() + (res * d_res.double()).sum(), list(leaves.values()))
    assert rel(c["out"], want.detach()) <= 3e-2 and rel(c["r"], res.detach()) <= 3e-2
    for name, g in zip(leaves, grads):
        assert rel(got[name], g) <= 3e-2, (name, rel(got[name], g))


def test_prompt_then_steps():
    """A prompt and 20 single tokens give the states and outputs of the whole: rotary positions by their numbers, the
    attention's and the scan's states carried on."""
    import gated_delta_rule_14_gb300 as kla
    p, N = params(), H * D
    freqs, scale = kla.rotary_freqs(D, device=DEV)
    h = rnd(3)(B, T, N).bfloat16()
    whole = block(p, h, freqs, scale)
    c = block(p, h[:, :280].contiguous(), freqs, scale)
    S, state, outs = c["S"], c["h_T"], []
    for t in range(280, T):
        proj = h[:, t] @ p["qkvz"].bfloat16()
        q, k, v, z = (x.unflatten(-1, (H, D)) for x in proj.split(N, -1))
        at = torch.full((B, 1), t, dtype=torch.int32, device=DEV)
        q, k = kla.rotary_fwd(q[:, None], k[:, None], freqs, at, scale=scale)
        o = kla.linear_step(q[:, 0], k[:, 0], v.contiguous(), p["decay"], S, q_scale=D ** -0.5)
        a, _, _ = kla.gated_norm_fwd(o, z, p["heads"], stats=False)
        y, _, _, _ = kla.add_norm_fwd(a.flatten(-2) @ p["out"].bfloat16(), h[:, t].contiguous(), p["norm"], p["scale"],
                                      stats=False)
        xs, gs = (y @ p["xg"].bfloat16()).split(N, -1)
        outs.append(kla.gated_scan_step(xs, gs, state))
    kla.device_status(DEV)
    # the prompt's tensor cores round the attention's scores to 8 bits, a step does not, and products follow: 1e-2
    assert rel(torch.stack(outs, 1), whole["out"][:, 280:]) <= 1e-2
    assert rel(S, whole["S"]) <= 1e-2 and rel(state, whole["h_T"]) <= 1e-2


def test_accepted_drafts_advance_the_states():
    """A draft verified, and the states of both recurrences run on over the last token and the accepted drafts: the same
    as those tokens by themselves."""
    import gated_delta_rule_14_gb300 as kla
    r, K, V = rnd(4), 5, 700
    gen = torch.Generator(device=DEV).manual_seed(5)
    p = torch.softmax(3 * r(4, K + 1, V), -1)
    q = torch.softmax(torch.log(p[:, :K]) + 0.5 * r(4, K, V), -1)
    draft = torch.multinomial(q.reshape(-1, V), 1, generator=gen).view(4, K).int()
    accepted, tokens = kla.verify_draft(draft, q, p, torch.rand(4, K + 1, generator=gen, device=DEV))
    n = accepted + 1
    qq, k, v = (r(4, K + 1, H, D).bfloat16() for _ in range(3))
    S0, h0 = r(4, H, D, D), r(4, H * D)
    g = torch.tensor([0.97, 0.999], device=DEV)
    _, S = kla.linear_fwd(qq, k, v, g, S0, lengths=n)
    _, h, _ = kla.gated_scan_fwd(qq.flatten(-2), k.flatten(-2), h0, lengths=n)
    kla.device_status(DEV)
    for b in range(4):
        m = int(n[b])
        assert (tokens[b, :m] >= 0).all() and (tokens[b, m:] == -1).all()
        one = slice(b, b + 1)
        _, want = kla.linear_fwd(qq[one, :m], k[one, :m], v[one, :m], g, S0[one])
        _, state, _ = kla.gated_scan_fwd(qq[one, :m].flatten(-2), k[one, :m].flatten(-2), h0[one])
        assert rel(S[one], want) <= 1e-5 and rel(h[one], state) <= 1e-6


def training_step(seed=6):
    import gated_delta_rule_14_gb300 as kla
    p, r = params(), rnd(seed)
    freqs, scale = kla.rotary_freqs(D, device=DEV)
    h, d_out, d_res = (r(B, T, H * D).bfloat16() for _ in range(3))

    def step():
        c = block(p, h, freqs, scale)
        return c["out"], c["h_T"], *gradients(p, c, d_out, d_res, freqs, scale).values()
    return step


def test_a_training_step_in_a_graph():
    """A captured forward and backward pass gives the eager one's bits, replayed again and again over the same
    workspaces."""
    import gated_delta_rule_14_gb300 as kla
    step = training_step()
    eager = step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
    kla.device_status(DEV)


def test_two_graphs_over_one_workspace():
    """Calls that share a workspace, replayed in turn: each lays it out anew."""
    import gated_delta_rule_14_gb300 as kla
    r = rnd(7)
    sizes = ((2, 2000, 66), (1, 5000, 130))
    ws = torch.empty(max(kla.gated_scan_workspace_size(*s) for s in sizes), dtype=torch.uint8, device=DEV)
    graphs = []
    for b, t, c in sizes:
        x, g, dy = (r(b, t, c).bfloat16() for _ in range(3))

        def call(x=x, g=g, dy=dy):
            y, h, s = kla.gated_scan_fwd(x, g, states=True, workspace=ws)
            return y, h, *kla.gated_scan_bwd(x, g, dy, s, workspace=ws).values()
        eager = [t.clone() for t in call()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        graphs.append((graph, out, eager, (x, g, dy)))   # the inputs have to live as long as the graph
    for _ in range(3):
        for graph, out, eager, _ in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, eager))
    kla.device_status(DEV)


def test_two_streams_at_once():
    """Scans of many tiles on two streams, whose CTAs share the SMs: each ends, with its own bits."""
    import gated_delta_rule_14_gb300 as kla
    r = rnd(8)
    data = [[r(2, 6000, 514).bfloat16() for _ in range(3)] for _ in range(2)]

    def call(x, g, dy):
        y, h, s = kla.gated_scan_fwd(x, g, states=True)
        return y, h, *kla.gated_scan_bwd(x, g, dy, s).values()
    alone = [call(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(4):
        got = []
        for s, d in zip(streams, data):
            with torch.cuda.stream(s):
                got.append(call(*d))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    kla.device_status(DEV)


def test_a_decoding_step_in_a_graph():
    """Rotary, norms, the scan's single token and a verification captured as one graph."""
    import gated_delta_rule_14_gb300 as kla
    r = rnd(9)
    freqs, _ = kla.rotary_freqs(64, device=DEV)
    q, k = r(4, 1, 6, 128).bfloat16(), r(4, 1, 2, 128).bfloat16()
    at = torch.full((4, 1), 100, dtype=torch.int64, device=DEV)
    z, res, w = r(4, 1, 6, 128).bfloat16(), r(4, 768).bfloat16(), r(768)
    gate, h0 = r(4, 768).bfloat16(), r(4, 768)
    state = h0.clone()
    p, u = torch.softmax(3 * r(4, 3, 500), -1), torch.rand(4, 3, device=DEV)
    draft = torch.randint(0, 500, (4, 2), device=DEV, dtype=torch.int32)

    def step():
        a, b = kla.rotary_fwd(q, k, freqs, at, layout="interleaved")
        y, _, _ = kla.gated_norm_fwd(a, z, stats=False)
        n, s, _, _ = kla.add_norm_fwd(y.view(4, 768), res, w, stats=False)
        return a, b, n, s, kla.gated_scan_step(n, gate, state), *kla.verify_draft(draft, None, p, u)
    eager, after = step(), state.clone()
    state.copy_(h0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    state.copy_(h0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, after) and all(torch.equal(a, b) for a, b in zip(out, eager))
