"""Work for the decayed linear attention, layer norm and beam search operators: cases, inputs, plain forms, exact values.

Every case names a ``kind``:

- ``fwd``    linear attention with one decay per head over whole prompts
- ``train``  the same and its backward pass
- ``step``   one token for every sequence, the states updated (``beams``: each state read at its beam's parent)
- ``norm``   layer norm forward, with ``train`` the backward pass and the weight's gradient too
- ``beam``   selection over beams and vocabulary, the states following their beams
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a chat turn of a few words on a small model: latency is all that counts
        {"name": "prompt_short", "kind": "fwd", "B": 1, "T": 77, "H": 4, "d": 128, "dtype": "bf16", "ragged": False,
         "packed": False, "s0": False},
        # the repository's 4K prefill shape
        {"name": "prompt_4k", "kind": "fwd", "B": 8, "T": 4096, "H": 16, "d": 128, "dtype": "bf16", "ragged": False,
         "packed": False, "s0": False},
        # the repository's long context: one sequence, few chains, the largest call
        {"name": "prompt_131k", "kind": "fwd", "B": 1, "T": 131072, "H": 16, "d": 128, "dtype": "bf16",
         "ragged": False, "packed": False, "s0": False},
        # a served batch of prompts of unequal length (one slot empty), q/k/v as one projection wrote them, going on
        # from earlier states
        {"name": "prompt_ragged", "kind": "fwd", "B": 7, "T": 1531, "H": 12, "d": 128, "dtype": "bf16",
         "ragged": True, "packed": True, "s0": True},
        # a small model trained in 32 bits
        {"name": "train_f32", "kind": "train", "B": 2, "T": 1000, "H": 4, "d": 64, "dtype": "f32", "ragged": False,
         "packed": False, "s0": True},
        # a training step's layer at the 4K shape
        {"name": "train_4k", "kind": "train", "B": 8, "T": 4096, "H": 16, "d": 128, "dtype": "bf16",
         "ragged": False, "packed": False, "s0": False},
        # one user, one token
        {"name": "step_1", "kind": "step", "B": 1, "H": 16, "d": 128, "dtype": "bf16", "beams": 1},
        # the repository's decode batch, as 16 requests of four beams whose states have just been reselected
        {"name": "step_beams", "kind": "step", "B": 64, "H": 16, "d": 128, "dtype": "bf16", "beams": 4},
        # the heads' norm within a decode step
        {"name": "norm_heads", "kind": "norm", "rows": 64, "G": 16, "N": 128, "dtype": "bf16", "train": False},
        # a training step's norm over a whole row, an odd count of rows
        {"name": "norm_train", "kind": "norm", "rows": 16397, "G": 1, "N": 2048, "dtype": "bf16", "train": True},
        # one request with four beams on a small vocabulary
        {"name": "beam_1", "kind": "beam", "B": 1, "W": 4, "V": 32000, "H": 4, "d": 64, "dtype": "bf16"},
        # eight requests with eight beams on a large odd vocabulary, logits in 32 bits
        {"name": "beam_batch", "kind": "beam", "B": 8, "W": 8, "V": 100003, "H": 16, "d": 128, "dtype": "f32"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "train", "step", "norm", "norm", "beam"])
    if kind in ("fwd", "train"):
        f32 = rng.random() < 0.25
        B, H = _spread(rng, 1, 16), _spread(rng, 1, 24)
        most = (40_000 if f32 else 500_000 if kind == "train" else 1_500_000) // (B * H)
        return {"kind": kind, "B": B, "T": _spread(rng, 1, max(2, min(65536, most))), "H": H,
                "d": rng.choice([16, 32, 64, 128]) if f32 else 128, "dtype": "f32" if f32 else "bf16",
                "ragged": rng.random() < 0.4, "packed": rng.random() < 0.4, "s0": rng.random() < 0.5}
    if kind == "step":
        W = rng.choice([1, 1, 2, 4, 5])
        return {"kind": "step", "B": W * _spread(rng, 1, 128 // W), "H": _spread(rng, 1, 24), "d": 128,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "beams": W}
    if kind == "norm":
        heads = rng.random() < 0.4
        N = rng.choice([16, 32, 64, 128]) if heads else _spread(rng, 16, 8192)
        G = _spread(rng, 2, 32) if heads else 1
        return {"kind": "norm", "rows": _spread(rng, 1, 30_000_000 // (N * G)), "G": G, "N": N,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "train": rng.random() < 0.6}
    W = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    return {"kind": "beam", "B": _spread(rng, 1, max(2, 64 // W)), "W": W, "V": _spread(rng, 500, 150_000),
            "H": _spread(rng, 1, 16), "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "f32"])}


# ------------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)


def _decays(H):
    """Decays from 1 - 2^-5 to 1 - 2^-10 over the heads; one head alone has the first."""
    e = torch.arange(H, device=DEV, dtype=torch.float32) * (5.0 / max(1, H - 1))
    return 1.0 - torch.exp2(-5.0 - e)


def prepare(case, seed):
    g = _gen(seed)
    dt = TYPES[case["dtype"]]
    kind = case["kind"]

    def rnd(*shape, scale=1.0, dtype=dt):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)

    if kind in ("fwd", "train"):
        B, T, H, d = case["B"], case["T"], case["H"], case["d"]
        if case["packed"]:   # as one projection writes them: [B, T, 3, H, d]
            qkv = rnd(B, T, 3, H, d)
            q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
        else:
            q, k, v = rnd(B, T, H, d), rnd(B, T, H, d), rnd(B, T, H, d)
        s = {"case": case, "q": q, "k": k, "v": v, "decay": _decays(H), "scale": d ** -0.5, "S0": None,
             "lengths": None}
        if case["s0"]:
            s["S0"] = rnd(B, H, d, d, scale=2.0, dtype=torch.float32)
        if case["ragged"]:
            n = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
            n[0] = T
            if B > 1:
                n[1] = 0
            s["lengths"] = n
        if kind == "train":
            s["dO"] = rnd(B, T, H, d)
            s["dS_T"] = rnd(B, H, d, d, dtype=torch.float32) if case["s0"] else None
        return s
    if kind == "step":
        B, H, d, W = case["B"], case["H"], case["d"], case["beams"]
        s = {"case": case, "q": rnd(B, H, d), "k": rnd(B, H, d), "v": rnd(B, H, d), "decay": _decays(H),
             "scale": d ** -0.5, "S": rnd(B, H, d, d, scale=4.0, dtype=torch.float32), "parent": None}
        if W > 1:
            first = torch.arange(B, device=DEV) // W * W
            s["parent"] = (first + torch.randint(0, W, (B,), generator=g, device=DEV)).to(torch.int32)
            s["S_next"] = torch.empty_like(s["S"])
        return s
    if kind == "norm":
        shape = (case["rows"], case["N"]) if case["G"] == 1 else (case["rows"], case["G"], case["N"])
        x = (rnd(*shape, scale=3.0, dtype=torch.float32) + 0.5).to(dt)
        s = {"case": case, "x": x, "w": 1.0 + rnd(*shape[1:], scale=0.2, dtype=torch.float32),
             "b": rnd(*shape[1:], scale=0.1, dtype=torch.float32), "eps": 1e-5}
        if case["train"]:
            s["dy"] = rnd(*shape)
        return s
    B, W, V, H, d = case["B"], case["W"], case["V"], case["H"], case["d"]
    logits = rnd(B, W, V, scale=3.0)
    scores = -torch.rand((B, W), generator=g, device=DEV) * 6.0 - 4.0
    finished = torch.rand((B, W), generator=g, device=DEV) < 0.15
    if W > 1:
        finished[:, 0] = False
        scores[0, W - 1] = -math.inf   # a beam that has died
    S = rnd(B, W, H, d, d, dtype=torch.float32)
    return {"case": case, "logits": logits, "scores": scores, "finished": finished, "eos": 2, "S": S,
            "S_next": torch.empty_like(S)}


# ------------------------------------------------------------------------------------------------ plain forms


def _scan(q, k, v, g):
    """sum_{j<=i} g^(i-j) (q_i.k_j) v_j for [B, H, T, d] in 32 bits, by chunks: the chunks' own states, each chunk's
    entering state as a weighted sum of the earlier ones, and the products within a chunk."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    C = 256 if T > 256 else T
    n = -(-T // C)
    pad = n * C - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).reshape(B, H, n, C, -1) for x in (q, k, v))
    at = torch.arange(C, device=q.device)
    g = g.view(1, H, 1, 1, 1)
    diff = (at[:, None] - at[None, :]).float()
    o = (q @ k.transpose(-1, -2) * torch.where(diff >= 0, g ** diff.clamp(min=0), 0.0)) @ v
    if n > 1:
        Z = (k * g ** (C - 1 - at).float()[:, None]).transpose(-1, -2) @ v
        step = torch.arange(n, device=q.device)
        back = (step[:, None] - 1 - step[None, :]).float()
        L = torch.where(back >= 0, g.view(H, 1, 1) ** (back.clamp(min=0) * C), 0.0)
        S = (L @ Z.reshape(B, H, n, dk * dv)).reshape(B, H, n, dk, dv)
        o = o + (q * g ** (at + 1).float()[:, None]) @ S
    return o.reshape(B, H, n * C, dv)[:, :, :T]


def _heads_first(s, *names):
    """[B, H, T, d] in 32 bits with the tokens past each sequence's length set to zero, and the lengths."""
    T, B = s["q"].shape[1], s["q"].shape[0]
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=DEV)
    live = (torch.arange(T, device=DEV) < n[:, None])[:, None, :, None]
    return [torch.where(live, s[m].float().transpose(1, 2), 0.0) for m in names], n, live


def _plain_fwd(s):
    (q, k, v), n, live = _heads_first(s, "q", "k", "v")
    T, g = q.shape[2], s["decay"].view(1, -1, 1, 1)
    t = torch.arange(T, device=DEV)
    o = _scan(q, k, v, s["decay"])
    if s["S0"] is not None:
        o = o + (q * g ** (t + 1).float()[:, None]) @ s["S0"]
    left = (n[:, None] - 1 - t).clamp(min=0).float()[:, None, :, None]
    S_T = (k * g ** left).transpose(-1, -2) @ v
    if s["S0"] is not None:
        S_T = S_T + g ** n.float().view(-1, 1, 1, 1) * s["S0"]
    return {"o": (o * s["scale"]).transpose(1, 2).to(s["q"].dtype), "S_T": S_T}


def _plain_bwd(s):
    (q, k, v, dO), n, live = _heads_first(s, "q", "k", "v", "dO")
    T, g, dt = q.shape[2], s["decay"].view(1, -1, 1, 1), s["q"].dtype
    t = torch.arange(T, device=DEV)
    q = q * s["scale"]
    dq = _scan(dO * s["scale"], v, k, s["decay"])
    dk = _scan(v.flip(2), dO.flip(2), q.flip(2), s["decay"]).flip(2)
    dv = _scan(k.flip(2), q.flip(2), dO.flip(2), s["decay"]).flip(2)
    enter = g ** (t + 1).float()[:, None]
    dS0 = (q * enter).transpose(-1, -2) @ dO
    if s["S0"] is not None:
        dq = dq + (dO * (enter * s["scale"])) @ s["S0"].transpose(-1, -2)
    if s["dS_T"] is not None:
        left = g ** (n[:, None] - 1 - t).clamp(min=0).float()[:, None, :, None] * live
        dk = dk + (v * left) @ s["dS_T"].transpose(-1, -2)
        dv = dv + (k * left) @ s["dS_T"]
        dS0 = dS0 + g ** n.float().view(-1, 1, 1, 1) * s["dS_T"]
    return {"dq": dq.transpose(1, 2).to(dt), "dk": dk.transpose(1, 2).to(dt), "dv": dv.transpose(1, 2).to(dt),
            "dS0": dS0}


def _plain_step(s):
    S = s["S"] if s["parent"] is None else s["S"][s["parent"].long()]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    S = S * s["decay"].view(1, -1, 1, 1) + k[..., :, None] * v[..., None, :]
    o = (q[..., None, :] @ S)[..., 0, :] * s["scale"]
    s["S"] = S
    return {"o": o.to(s["q"].dtype), "S": S}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + s["eps"])
    xh = (x - mean) * rstd
    r = {"y": (xh * s["w"] + s["b"]).to(s["x"].dtype), "mean": mean[..., 0], "rstd": rstd[..., 0]}
    if s["case"]["train"]:
        dy = s["dy"].float()
        wdy = dy * s["w"]
        dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
        r |= {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    return r


def _plain_beam(s):
    c = s["case"]
    B, W, V = c["B"], c["W"], c["V"]
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x).clamp(max=torch.finfo(torch.float32).max)
    only = torch.where(torch.arange(V, device=DEV) == s["eos"], 0.0, -math.inf)
    x = torch.where(s["finished"][..., None], only, x)
    top = x.amax(-1, keepdim=True)
    total = torch.exp(x - top).sum(-1, keepdim=True)
    best, token = torch.sort(x, dim=-1, descending=True, stable=True)   # each beam's own list
    n = min(W, V)
    key = ((best[..., :n] - top) - torch.log(total)) + s["scores"][..., None]
    key = torch.where(key.isnan(), -math.inf, key).reshape(B, W * n)
    key, place = torch.sort(key, dim=-1, descending=True, stable=True)
    key, place = key[:, :W], place[:, :W]
    parent = place // n
    token = torch.gather(token[..., :n].reshape(B, W * n), 1, place)
    finished = torch.gather(s["finished"], 1, parent) | (token == s["eos"])
    S = torch.gather(s["S"], 1, parent.view(B, W, 1, 1, 1).expand_as(s["S"]))
    return {"scores": key, "parents": parent.int(), "tokens": token.int(), "finished": finished, "S": S}


# ------------------------------------------------------------------------------------------------ calls


def _own(s):
    import gated_delta_rule_14_gb300 as kla
    kind = s["case"]["kind"]
    if kind in ("fwd", "train"):
        o, S_T = kla.linear_fwd(s["q"], s["k"], s["v"], s["decay"], s["S0"], q_scale=s["scale"],
                                lengths=s["lengths"])
        r = {"o": o, "S_T": S_T}
        if kind == "train":
            r |= kla.linear_bwd(s["q"], s["k"], s["v"], s["decay"], s["dO"], s["S0"], s["dS_T"],
                                q_scale=s["scale"], lengths=s["lengths"])
        return r
    if kind == "step":
        if s["parent"] is None:
            o = kla.linear_step(s["q"], s["k"], s["v"], s["decay"], s["S"], q_scale=s["scale"])
        else:
            o = kla.linear_step(s["q"], s["k"], s["v"], s["decay"], s["S"], q_scale=s["scale"],
                                parent=s["parent"], S_out=s["S_next"])
            s["S"], s["S_next"] = s["S_next"], s["S"]
        return {"o": o, "S": s["S"]}
    if kind == "norm":
        y, mean, rstd = kla.layer_norm_fwd(s["x"], s["w"], s["b"], s["eps"])
        r = {"y": y, "mean": mean, "rstd": rstd}
        if s["case"]["train"]:
            dx, dw, db = kla.layer_norm_bwd(s["dy"], s["x"], s["w"], mean, rstd)
            r |= {"dx": dx, "dw": dw, "db": db}
        return r
    scores, parents, tokens, finished = kla.beam_select(s["logits"], s["scores"], s["finished"], eos=s["eos"])
    S = kla.reorder_states(s["S"], parents, out=s["S_next"])
    return {"scores": scores, "parents": parents, "tokens": tokens, "finished": finished, "S": S}


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "fwd":
        return _plain_fwd(state)
    if kind == "train":
        return _plain_fwd(state) | _plain_bwd(state)
    return {"step": _plain_step, "norm": _plain_norm, "beam": _plain_beam}[kind](state)


def work(case):
    kind, e = case["kind"], 2 if case["dtype"] == "bf16" else 4
    if kind in ("fwd", "train"):
        B, T, H, d = case["B"], case["T"], case["H"], case["d"]
        # lengths drawn from 0 to T: about half of the tokens of all sequences but the full and the empty one
        n = H * ((T + max(0, B - 2) * T // 2) if case["ragged"] else B * T)
        state = B * H * d * d * 4
        move, ops = n * d * 4 * e + state * (2 if case["s0"] else 1), n * 4 * d * d   # write and read of the state
        if kind == "train":
            move += n * d * 7 * e + state * (3 if case["s0"] else 1)
            ops += n * 8 * d * d
        return {"bytes": move, "flops": ops}
    if kind == "step":
        n, d = case["B"] * case["H"], case["d"]
        return {"bytes": n * (2 * d * d * 4 + 4 * d * e), "flops": n * 5 * d * d}
    if kind == "norm":
        n, r, p = case["rows"] * case["G"] * case["N"], case["rows"] * case["G"], case["G"] * case["N"] * 4
        if case["train"]:
            return {"bytes": 5 * n * e + 16 * r + 4 * p, "flops": 20 * n}
        return {"bytes": 2 * n * e + 8 * r + 2 * p, "flops": 8 * n}
    n, one = case["B"] * case["W"], case["H"] * case["d"] ** 2 * 4
    return {"bytes": n * case["V"] * e + 2 * n * one, "flops": 4 * n * case["V"]}


# ------------------------------------------------------------------------------------------------ exact values


def _recurrence(q, k, v, g, scale, S, n):
    """The recurrence in 64 bits, 32 tokens at a time, every sequence for itself; differentiable."""
    outs, states = [], []
    for b in range(q.shape[0]):
        Sb, parts, nb = S[b], [], int(n[b])
        for t0 in range(0, nb, 32):
            qc, kc, vc = (x[b, t0:min(nb, t0 + 32)].transpose(0, 1) for x in (q, k, v))   # [H, m, d]
            m = qc.shape[1]
            i = torch.arange(m, device=DEV, dtype=torch.float64)
            w = torch.tril(g[:, None, None] ** (i[:, None] - i).clamp(min=0))
            one = torch.einsum("hid,hjd,hij,hje->hie", qc, kc, w, vc)
            one = one + g[:, None, None] ** (i[:, None] + 1) * torch.einsum("hid,hde->hie", qc, Sb)
            Sb = g[:, None, None] ** m * Sb + torch.einsum("hjd,hj,hje->hde", kc, g[:, None] ** (m - 1 - i), vc)
            parts.append(scale * one.transpose(0, 1))
        parts.append(torch.zeros((q.shape[1] - nb, q.shape[2], v.shape[3]), device=DEV, dtype=torch.float64))
        outs.append(torch.cat(parts))
        states.append(Sb)
    return torch.stack(outs), torch.stack(states)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("fwd", "train"):
        B, T = case["B"], case["T"]
        if B * T > 200_000:
            return None
        n = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
        q, k, v = (s[x].double() for x in "qkv")
        S0 = s["S0"].double() if s["S0"] is not None else torch.zeros((B, case["H"], case["d"], case["d"]),
                                                                      device=DEV, dtype=torch.float64)
        leaf = [x.requires_grad_(kind == "train") for x in (q, k, v, S0)]
        o, S_T = _recurrence(*leaf[:3], s["decay"].double(), s["scale"], leaf[3], n)
        r = {"o": o.detach(), "S_T": S_T.detach()}
        if kind == "train":
            loss = (o * s["dO"].double()).sum()
            if s["dS_T"] is not None:
                loss = loss + (S_T * s["dS_T"].double()).sum()
            r |= dict(zip(("dq", "dk", "dv", "dS0"), torch.autograd.grad(loss, leaf)))
        return r
    if kind == "step":
        H, d = case["H"], case["d"]
        S = s["S"].double()
        if s["parent"] is not None:
            S = torch.index_select(S, 0, s["parent"].long())
        S = torch.einsum("h,bhij->bhij", s["decay"].double(), S)
        S = S + torch.einsum("bhi,bhj->bhij", s["k"].double(), s["v"].double())
        return {"o": torch.einsum("bhi,bhij->bhj", s["q"].double(), S) * s["scale"], "S": S}
    if kind == "norm":
        x = s["x"].double().requires_grad_(True)
        w, b = s["w"].double().requires_grad_(True), s["b"].double().requires_grad_(True)
        var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
        rstd = torch.rsqrt(var + s["eps"])
        y = (x - mean) * rstd * w + b
        r = {"y": y.detach(), "mean": mean.detach()[..., 0], "rstd": rstd.detach()[..., 0]}
        if case["train"]:
            r |= dict(zip(("dx", "dw", "db"), torch.autograd.grad((y * s["dy"].double()).sum(), (x, w, b))))
        return r
    B, W, V = case["B"], case["W"], case["V"]
    keys, parents = [], []
    for b in range(B):
        rows = torch.log_softmax(s["logits"][b].double(), -1)
        for w in range(W):
            if bool(s["finished"][b, w]):
                rows[w] = -math.inf
                rows[w, s["eos"]] = 0.0
        rows = rows + s["scores"][b].double()[:, None]
        key, at = torch.topk(rows.reshape(-1), W)
        keys.append(key)
        parents.append(at // V)
    S = torch.stack([s["S"][b, parents[b]] for b in range(B)]).double()
    return {"scores": torch.stack(keys), "parents": None, "tokens": None, "finished": None, "S": S}
