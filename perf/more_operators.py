"""Work for the operators around the recurrence: cases, inputs, plain forms, exact values.

Every case names a ``kind``:

- ``scan``    the gated scan (a recurrence with one gate per channel) over whole prompts, ``train``: and its gradients
- ``hop``     one token of it for every sequence, the states updated
- ``rotary``  queries and keys turned by their positions
- ``gated``   the norm of a block's heads times the activation of its gate, ``train``: and its gradients
- ``added``   a block's output added to the residual and normalised for the next block, ``train``: and its gradients
- ``verify``  drafted tokens accepted or not against the target's probabilities, and the token after them
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a chat turn of a few words on a small model: latency is all that counts
        {"name": "scan_short", "kind": "scan", "B": 1, "T": 77, "C": 512, "dtype": "bf16", "mode": "sigmoid",
         "ragged": False, "packed": False, "h0": False, "train": False},
        # the repository's long context, 16 heads of 128 as channels: one sequence, the largest call
        {"name": "scan_131k", "kind": "scan", "B": 1, "T": 131072, "C": 2048, "dtype": "bf16", "mode": "sigmoid",
         "ragged": False, "packed": False, "h0": False, "train": False},
        # a training step's layer at the repository's 4K shape, x and gate as one projection wrote them
        {"name": "scan_train", "kind": "scan", "B": 8, "T": 4096, "C": 2048, "dtype": "bf16", "mode": "sigmoid",
         "ragged": False, "packed": True, "h0": False, "train": True},
        # a batch of sequences of unequal length trained in 32 bits from earlier states, an odd count of channels
        {"name": "scan_ragged", "kind": "scan", "B": 7, "T": 1531, "C": 1001, "dtype": "f32", "mode": "log",
         "ragged": True, "packed": False, "h0": True, "train": True},
        # a decode batch's token
        {"name": "hop_64", "kind": "hop", "B": 64, "C": 2048, "dtype": "bf16", "mode": "sigmoid"},
        # a prompt at the repository's 4K shape, whole heads in halves
        {"name": "rotary_4k", "kind": "rotary", "B": 8, "T": 4096, "H": 16, "K": 16, "d": 128, "rot": 128,
         "layout": "half", "dtype": "bf16", "packed": True, "far": 4096},
        # a decode batch's token at far positions, part of the head in pairs, fewer heads of keys
        {"name": "rotary_step", "kind": "rotary", "B": 64, "T": 1, "H": 16, "K": 4, "d": 128, "rot": 64,
         "layout": "interleaved", "dtype": "bf16", "packed": False, "far": 1_000_000},
        # the heads' norm and gate within a decode step
        {"name": "gated_step", "kind": "gated", "rows": 64, "G": 16, "N": 128, "dtype": "bf16", "norm": "rms",
         "act": "silu", "train": False},
        # the same in a training step at the 4K shape
        {"name": "gated_train", "kind": "gated", "rows": 32768, "G": 16, "N": 128, "dtype": "bf16", "norm": "rms",
         "act": "silu", "train": True},
        # a training step's residual, an odd count of rows, the block's output scaled by channel
        {"name": "added_train", "kind": "added", "rows": 16397, "N": 2048, "dtype": "bf16", "norm": "rms",
         "scaled": True, "train": True},
        # one request, four drafted tokens, a small vocabulary
        {"name": "verify_1", "kind": "verify", "B": 1, "K": 4, "V": 32000, "dtype": "f32", "ragged": False,
         "sure": False},
        # the repository's decode batch, eight drafted tokens at most, a large odd vocabulary
        {"name": "verify_64", "kind": "verify", "B": 64, "K": 8, "V": 100003, "dtype": "f32", "ragged": True,
         "sure": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "scan", "hop", "rotary", "rotary", "gated", "added", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "scan":
        B, C, train = _spread(rng, 1, 16), _spread(rng, 1, 4096), rng.random() < 0.5
        most = (30_000_000 if train else 100_000_000) // (B * C)
        return {"kind": kind, "B": B, "T": _spread(rng, 1, max(2, min(131072, most))), "C": C, "dtype": dtype,
                "mode": rng.choice(["sigmoid", "log"]), "ragged": rng.random() < 0.4, "packed": rng.random() < 0.4,
                "h0": rng.random() < 0.5, "train": train}
    if kind == "hop":
        return {"kind": kind, "B": _spread(rng, 1, 256), "C": _spread(rng, 1, 8192), "dtype": dtype,
                "mode": rng.choice(["sigmoid", "log"])}
    if kind == "rotary":
        H, d = _spread(rng, 1, 32), rng.choice([16, 32, 64, 80, 128, 128, 256])
        K = rng.choice([k for k in range(1, H + 1) if H % k == 0])
        B = _spread(rng, 1, 64)
        return {"kind": kind, "B": B, "T": _spread(rng, 1, max(2, min(131072, 60_000_000 // (B * (H + K) * d)))),
                "H": H, "K": K, "d": d, "rot": rng.choice([d, d, d // 2, d // 4, d - 2]),
                "layout": rng.choice(["half", "interleaved"]), "dtype": dtype, "packed": rng.random() < 0.5,
                "far": rng.choice([4096, 131072, 1_000_000, 2_000_000_000])}
    if kind == "gated":
        heads = rng.random() < 0.7
        N = rng.choice([16, 32, 64, 100, 128, 128, 256]) if heads else _spread(rng, 16, 8192)
        G = _spread(rng, 2, 32) if heads else 1
        return {"kind": kind, "rows": _spread(rng, 1, 30_000_000 // (N * G)), "G": G, "N": N, "dtype": dtype,
                "norm": rng.choice(["rms", "layer"]), "act": rng.choice(["silu", "sigmoid"]),
                "train": rng.random() < 0.6}
    if kind == "added":
        N = _spread(rng, 16, 8192)
        return {"kind": kind, "rows": _spread(rng, 1, 30_000_000 // N), "N": N, "dtype": dtype,
                "norm": rng.choice(["rms", "layer"]), "scaled": rng.random() < 0.6, "train": rng.random() < 0.6}
    return {"kind": kind, "B": _spread(rng, 1, 64), "K": rng.choice([1, 2, 3, 4, 5, 7, 8]),
            "V": _spread(rng, 50, 150_000), "dtype": rng.choice(["f32", "f32", "bf16"]), "ragged": rng.random() < 0.5,
            "sure": rng.random() < 0.3}


# ------------------------------------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)
    dt = TYPES[case["dtype"]]
    kind = case["kind"]

    def rnd(*shape, scale=1.0, shift=0.0, dtype=dt):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).add_(shift).to(dtype)

    def lengths(B, T):
        n = torch.randint(0, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        n[0] = T
        if B > 1:
            n[1] = 0
        return n

    if kind in ("scan", "hop"):
        B, C, mode = case["B"], case["C"], case["mode"]
        shape = (B, C) if kind == "hop" else (B, case["T"], C)
        # the gates of the repository's workloads: sigmoid(N(3, 1)), or a logarithm of -softplus(N(-4, 1))
        x, gate = rnd(*shape), rnd(*shape, shift=3.0 if mode == "sigmoid" else -4.0)
        if mode == "log":
            gate = (-torch.log1p(torch.exp(gate.float()))).to(dt)
        if kind == "hop":
            return {"case": case, "x": x, "gate": gate, "h": rnd(B, C, dtype=torch.float32)}
        if case["packed"]:
            x, gate = torch.cat([x, gate], -1).split(C, -1)
        s = {"case": case, "x": x, "gate": gate, "h0": rnd(B, C, dtype=torch.float32) if case["h0"] else None,
             "lengths": lengths(B, case["T"]) if case["ragged"] else None}
        if case["train"]:
            s["dy"] = rnd(*shape)
            s["dh_T"] = rnd(B, C, dtype=torch.float32) if case["h0"] else None
        return s
    if kind == "rotary":
        B, T, H, K, d = (case[n] for n in ("B", "T", "H", "K", "d"))
        if case["packed"]:   # queries, keys and values as one projection writes them
            q, k, _ = rnd(B, T, H + 2 * K, d).split([H, K, K], 2)
        else:
            q, k = rnd(B, T, H, d), rnd(B, T, K, d)
        # every sequence goes on from a position of its own
        start = torch.randint(0, max(1, case["far"] - T + 1), (B, 1), generator=g, device=DEV)
        n = case["rot"] // 2
        freqs = (10000.0 ** (-torch.arange(n, device=DEV, dtype=torch.float64) / n)).float()
        return {"case": case, "q": q, "k": k, "freqs": freqs,
                "positions": (start + torch.arange(T, device=DEV)).contiguous(),
                "scale": 1.0 if case["far"] <= 131072 else 0.1 * math.log(8.0) + 1.0}
    if kind == "gated":
        shape = (case["rows"], case["N"]) if case["G"] == 1 else (case["rows"], case["G"], case["N"])
        s = {"case": case, "x": rnd(*shape, scale=3.0, shift=0.5), "gate": rnd(*shape, scale=2.0),
             "w": rnd(*shape[1:], scale=0.2, shift=1.0, dtype=torch.float32), "eps": 1e-5}
        if case["train"]:
            s["dy"] = rnd(*shape)
        return s
    if kind == "added":
        rows, N = case["rows"], case["N"]
        s = {"case": case, "x": rnd(rows, N), "res": rnd(rows, N, scale=3.0, shift=0.5),
             "w": rnd(N, scale=0.2, shift=1.0, dtype=torch.float32), "eps": 1e-5,
             "scale": rnd(N, scale=0.1, shift=0.3, dtype=torch.float32) if case["scaled"] else None}
        if case["train"]:
            s["dy"], s["dres"] = rnd(rows, N), rnd(rows, N)
        return s
    B, K, V = case["B"], case["K"], case["V"]
    # the target as a softmax, the draft as the softmax of logits near the target's
    z = rnd(B, K + 1, V, scale=3.0, dtype=torch.float32)
    p = torch.softmax(z, -1).to(dt)
    q = torch.softmax(z[:, :K] + rnd(B, K, V, scale=0.7, dtype=torch.float32), -1)
    token = torch.multinomial(q.reshape(B * K, V), 1, generator=g).view(B, K)
    return {"case": case, "token": token.int(), "p": p, "q": None if case["sure"] else q.to(dt),
            "u": torch.rand((B, K + 1), generator=g, device=DEV), "lengths": lengths(B, K) if case["ragged"] else None}


# ------------------------------------------------------------------------------------------------ plain forms


def _scanned(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0 along axis 1, by doubling."""
    T, step = a.shape[1], 1
    while step < T:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _gate_of(gate, mode):
    """The factor of the state and the factor of the input."""
    if mode == "log":
        return torch.exp(gate), None
    return 1.0 / (1.0 + torch.exp(-gate)), 1.0 / (1.0 + torch.exp(gate))


def _plain_scan(s):
    c = s["case"]
    B, T, C, mode = c["B"], c["T"], c["C"], c["mode"]
    dt = s["x"].dtype
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(T, device=DEV) < s["lengths"][:, None])[..., None]
    x, gate = s["x"].float(), s["gate"].float()
    a, w = _gate_of(gate, mode)
    b = x if w is None else w * x
    if live is not None:
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros((B, C), device=DEV)
    h = _scanned(a, torch.cat([(b[:, 0] + a[:, 0] * h0)[:, None], b[:, 1:]], 1))
    r = {"y": (h if live is None else torch.where(live, h, 0.0)).to(dt), "h_T": h[:, -1].clone()}
    if c["train"]:
        dy = s["dy"].float()
        if live is not None:
            dy = torch.where(live, dy, 0.0)
        if s["dh_T"] is not None:
            dy = torch.cat([dy[:, :-1], (dy[:, -1] + s["dh_T"])[:, None]], 1)
        after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
        dh = _scanned(after.flip(1), dy.flip(1)).flip(1)
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        dx = dh if w is None else w * dh
        dg = a * dh * before if w is None else a * w * (before - x) * dh
        if live is not None:
            dx, dg = torch.where(live, dx, 0.0), torch.where(live, dg, 0.0)
        r |= {"dx": dx.to(dt), "dgate": dg.to(dt), "dh0": a[:, 0] * dh[:, 0]}
    return r


def _plain_hop(s):
    x = s["x"].float()
    a, w = _gate_of(s["gate"].float(), s["case"]["mode"])
    s["h"] = a * s["h"] + (x if w is None else w * x)
    return {"y": s["h"].to(s["x"].dtype), "h": s["h"]}


def _plain_rotary(s):
    c = s["case"]
    n = c["rot"] // 2
    angle = s["positions"].double()[..., None] * s["freqs"].double()   # far positions: whole turns cost the bits
    cos, sin = ((f(angle) * s["scale"]).float()[:, :, None] for f in (torch.cos, torch.sin))

    def turned(t):
        x = t.float()
        u, v = (x[..., :n], x[..., n:2 * n]) if c["layout"] == "half" else (x[..., 0:2 * n:2], x[..., 1:2 * n:2])
        new = (u * cos - v * sin, v * cos + u * sin)
        new = torch.cat(new, -1) if c["layout"] == "half" else torch.stack(new, -1).flatten(-2)
        return torch.cat([new, x[..., 2 * n:]], -1).to(t.dtype)
    return {"q": turned(s["q"]), "k": turned(s["k"])}


def _normed(x, norm, eps):
    """The normalised values, the mean (None without) and the reciprocal of the deviation."""
    mean = x.mean(-1, keepdim=True) if norm == "layer" else None
    if mean is not None:
        x = x - mean
    rstd = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * rstd, mean, rstd


def _norm_grad(xh, rstd, u, norm):
    g = u - xh * (u * xh).mean(-1, keepdim=True)
    if norm == "layer":
        g = g - u.mean(-1, keepdim=True)
    return rstd * g


def _plain_gated(s):
    c, dt = s["case"], s["x"].dtype
    x, z = s["x"].float(), s["gate"].float()
    xh, mean, rstd = _normed(x, c["norm"], s["eps"])
    sig = 1.0 / (1.0 + torch.exp(-z))
    act = z * sig if c["act"] == "silu" else sig
    r = {"y": (xh * s["w"] * act).to(dt)}
    if c["train"]:
        dy = s["dy"].float()
        slope = sig * (1.0 + z * (1.0 - sig)) if c["act"] == "silu" else sig * (1.0 - sig)
        r |= {"dx": _norm_grad(xh, rstd, dy * act * s["w"], c["norm"]).to(dt),
              "dgate": (dy * xh * s["w"] * slope).to(dt), "dw": (dy * act * xh).sum(0)}
    return r


def _plain_added(s):
    c, dt = s["case"], s["x"].dtype
    x = s["x"].float()
    r = s["res"].float() + (x if s["scale"] is None else x * s["scale"])
    xh, mean, rstd = _normed(r, c["norm"], s["eps"])
    out = {"y": (xh * s["w"]).to(dt), "res": r.to(dt)}
    if c["train"]:
        dy = s["dy"].float()
        dr = s["dres"].float() + _norm_grad(xh, rstd, dy * s["w"], c["norm"])
        out |= {"dres": dr.to(dt), "dw": (dy * xh).sum(0)}
        if s["scale"] is not None:
            out |= {"dx": (dr * s["scale"]).to(dt), "dscale": (dr * x).sum(0)}
    return out


def _plain_verify(s):
    c = s["case"]
    B, K, V = c["B"], c["K"], c["V"]
    token, u = s["token"].long(), s["u"].double()   # borders between tokens: products and sums in 64 bits
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), K, device=DEV)
    at = torch.arange(K, device=DEV)
    pt = torch.gather(s["p"][:, :K], 2, token[..., None])[..., 0].double()
    qt = torch.ones_like(pt) if s["q"] is None else torch.gather(s["q"], 2, token[..., None])[..., 0].double()
    took = (u[:, :K] * qt < pt) & (at < n[:, None])
    accepted = torch.cumprod(took.long(), 1).sum(1)
    b = torch.arange(B, device=DEV)
    p = s["p"][b, accepted].double()
    refused = accepted < n
    slot = accepted.clamp(max=K - 1)
    if s["q"] is None:
        q = torch.where(torch.arange(V, device=DEV) == token[b, slot][:, None], math.inf, 0.0)
    else:
        q = s["q"][b, slot].double()
    rest = torch.where(refused[:, None], (p - q).clamp(min=0.0), p)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p)
    cum = rest.cumsum(1)
    mark = u[:, K] * cum[:, -1]
    new = (cum > mark[:, None]).long().argmax(1)
    out = torch.cat([token, torch.zeros_like(token[:, :1])], 1)
    at = torch.arange(K + 1, device=DEV)
    out = torch.where(at < accepted[:, None], out, torch.where(at == accepted[:, None], new[:, None], -1))
    return {"accepted": accepted.int(), "tokens": out.int()}


# ------------------------------------------------------------------------------------------------ calls


def _own(s):
    import gated_delta_rule_14_gb300 as kla
    c = s["case"]
    kind, train = c["kind"], c.get("train", False)
    if kind == "scan":
        y, h_T, states = kla.gated_scan_fwd(s["x"], s["gate"], s["h0"], mode=c["mode"], lengths=s["lengths"],
                                            states=train)
        r = {"y": y, "h_T": h_T}
        if train:
            r |= kla.gated_scan_bwd(s["x"], s["gate"], s["dy"], states, s["dh_T"], mode=c["mode"],
                                    lengths=s["lengths"])
        return r
    if kind == "hop":
        return {"y": kla.gated_scan_step(s["x"], s["gate"], s["h"], mode=c["mode"]), "h": s["h"]}
    if kind == "rotary":
        q, k = kla.rotary_fwd(s["q"], s["k"], s["freqs"], s["positions"], layout=c["layout"], scale=s["scale"])
        return {"q": q, "k": k}
    if kind == "gated":
        y, mean, rstd = kla.gated_norm_fwd(s["x"], s["gate"], s["w"], s["eps"], norm=c["norm"], act=c["act"],
                                           stats=train)
        r = {"y": y}
        if train:
            dx, dgate, dw = kla.gated_norm_bwd(s["dy"], s["x"], s["gate"], s["w"], mean, rstd, act=c["act"])
            r |= {"dx": dx, "dgate": dgate, "dw": dw}
        return r
    if kind == "added":
        y, res, mean, rstd = kla.add_norm_fwd(s["x"], s["res"], s["w"], s["scale"], s["eps"], norm=c["norm"],
                                              stats=train)
        r = {"y": y, "res": res}
        if train:
            dx, dres, dw, dscale = kla.add_norm_bwd(s["dy"], s["dres"], s["x"], s["res"], s["w"], s["scale"], mean,
                                                   rstd)
            r |= {"dres": dres, "dw": dw}
            if s["scale"] is not None:
                r |= {"dx": dx, "dscale": dscale}
        return r
    accepted, tokens = kla.verify_draft(s["token"], s["q"], s["p"], s["u"], lengths=s["lengths"])
    return {"accepted": accepted, "tokens": tokens}


def run(state):
    if own:
        return _own(state)
    return {"scan": _plain_scan, "hop": _plain_hop, "rotary": _plain_rotary, "gated": _plain_gated,
            "added": _plain_added, "verify": _plain_verify}[state["case"]["kind"]](state)


# ------------------------------------------------------------------------------------------------ floors


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    kind, train = case["kind"], case.get("train", False)
    if kind == "scan":
        n, states = case["B"] * case["T"] * case["C"], case["B"] * case["C"] * 4
        # x, gate -> y; with gradients dy -> dx, dgate too; a gate is an exponential, a quotient and two sums
        moved = (6 if train else 3) * n * size + states * (1 + case["h0"]) * (2 if train else 1)
        return {"bytes": moved, "flops": n * (20 if train else 7)}
    if kind == "hop":
        n = case["B"] * case["C"]
        return {"bytes": n * (3 * size + 8), "flops": 7 * n}
    if kind == "rotary":
        tokens, heads = case["B"] * case["T"], case["H"] + case["K"]
        return {"bytes": 2 * tokens * heads * case["d"] * size + 8 * tokens + 2 * case["rot"],
                "flops": 3 * tokens * heads * case["rot"]}
    if kind == "gated":
        n, w = case["rows"] * case["G"] * case["N"], case["G"] * case["N"] * 4
        return {"bytes": (6 if train else 3) * n * size + w * (2 if train else 1), "flops": n * (30 if train else 11)}
    if kind == "added":
        n, w = case["rows"] * case["N"], case["N"] * 4 * (1 + case["scaled"])
        # x, residual -> y, sum; with gradients dy, dsum -> the residual's and, where it is scaled, the block's
        return {"bytes": (4 + (3 + case["scaled"] if train else 0)) * n * size + w * (2 if train else 1),
                "flops": n * (22 if train else 7)}
    # one row of the target and one of the draft for every sequence, and the drafted tokens' own probabilities
    B, K = case["B"], case["K"]
    return {"bytes": B * (case["V"] * size * (1 if case["sure"] else 2) + K * (4 + 2 * size) + (K + 1) * 8),
            "flops": 3 * B * case["V"]}


# ------------------------------------------------------------------------------------------------ exact values


def _walk(a, b, h):
    """h_t = a_t h + b_t in place of b, [B, T, C] in 64 bits: pieces of 128 tokens side by side, each from zero and
    with the product of its gates; then the state that enters each piece; then what that adds."""
    B, T, C = a.shape
    n = -(-T // 128)
    pad = n * 128 - T
    a = torch.nn.functional.pad(a, (0, 0, 0, pad), value=1.0).view(B, n, 128, C)
    b = torch.nn.functional.pad(b, (0, 0, 0, pad)).view(B, n, 128, C)
    carry = a.clone()
    for t in range(1, 128):
        b[:, :, t].addcmul_(a[:, :, t], b[:, :, t - 1])
        carry[:, :, t].mul_(carry[:, :, t - 1])
    for i in range(n):
        b[:, i].addcmul_(carry[:, i], h[:, None])
        h = b[:, i, -1]
    return b.view(B, n * 128, C)[:, :T]


def _exact_scan(c, s):
    B, T, C = c["B"], c["T"], c["C"]
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=DEV)
    out = (torch.arange(T, device=DEV) >= n[:, None])[..., None]
    x, z = s["x"].double().masked_fill(out, 0.0), s["gate"].double()
    if c["mode"] == "log":
        a, w = torch.exp(z), torch.ones((), device=DEV, dtype=torch.float64)
    else:
        a, w = torch.sigmoid(z), torch.sigmoid(-z)
    a = a.masked_fill(out, 1.0)
    h0 = torch.zeros((B, C), device=DEV, dtype=torch.float64) if s["h0"] is None else s["h0"].double()
    h = _walk(a, (w * x).masked_fill(out, 0.0), h0)
    r = {"y": h.masked_fill(out, 0.0), "h_T": h[:, -1].clone()}
    if c["train"]:
        # against time: e_t = a_t dh_t is what reaches the state before token t
        end = torch.zeros((B, C), device=DEV, dtype=torch.float64) if s["dh_T"] is None else s["dh_T"].double()
        dy = s["dy"].double().masked_fill(out, 0.0)
        e = _walk(a.flip(1), (a * dy).flip(1), end).flip(1)
        dh = dy + torch.cat([e[:, 1:], end[:, None]], 1)
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        slope = a if c["mode"] == "log" else a * w
        lead = before if c["mode"] == "log" else before - x
        r |= {"dx": (w * dh).masked_fill(out, 0.0), "dgate": (slope * lead * dh).masked_fill(out, 0.0),
              "dh0": e[:, 0].clone()}
    return r


def _exact_hop(c, s):
    x, z = s["x"].double(), s["gate"].double()
    if c["mode"] == "log":
        h = torch.exp(z) * s["h"].double() + x
    else:
        h = x + torch.sigmoid(z) * (s["h"].double() - x)
    return {"y": h, "h": h}


def _exact_rotary(c, s):
    n = c["rot"] // 2
    turn = torch.polar(torch.full((), s["scale"], device=DEV, dtype=torch.float64),
                       s["positions"].double()[:, :, None, None] * s["freqs"].double())

    def one(t):
        t = t.double()
        part = t[..., :2 * n]
        pairs = part.unflatten(-1, (2, n)).transpose(-1, -2) if c["layout"] == "half" else part.unflatten(-1, (n, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2) if c["layout"] == "half" else z
        return torch.cat([z.flatten(-2), t[..., 2 * n:]], -1)
    return {"q": one(s["q"]), "k": one(s["k"])}


def _exact_rows(x, w, eps, norm):
    """w (x - mean) / sqrt(var + eps) by autograd's elementary operations; x needs a gradient."""
    if norm == "layer":
        x = x - x.sum(-1, keepdim=True) / x.shape[-1]
    return w * x * ((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps).rsqrt()


def _exact_gated(c, s):
    x, z, w = (s[n].double().requires_grad_(c["train"]) for n in ("x", "gate", "w"))
    y = _exact_rows(x, w, s["eps"], c["norm"]) * (z if c["act"] == "silu" else 1.0) * torch.sigmoid(z)
    r = {"y": y.detach()}
    if c["train"]:
        r["dx"], r["dgate"], r["dw"] = torch.autograd.grad(y, (x, z, w), s["dy"].double())
    return r


def _exact_added(c, s):
    x, res, w = (s[n].double().requires_grad_(c["train"]) for n in ("x", "res", "w"))
    scale = None if s["scale"] is None else s["scale"].double().requires_grad_(c["train"])
    total = res + (x if scale is None else scale * x)
    y = _exact_rows(total, w, s["eps"], c["norm"])
    r = {"y": y.detach(), "res": total.detach()}
    if c["train"]:
        wanted = (res, w) if scale is None else (res, w, x, scale)
        r |= dict(zip(("dres", "dw", "dx", "dscale"),
                      torch.autograd.grad((y, total), wanted, (s["dy"].double(), s["dres"].double()))))
    return r


def _exact_verify(c, s):
    import numpy as np
    K = c["K"]

    def host(t):
        return None if t is None else t.double().cpu().numpy()
    p, q, u = host(s["p"]), host(s["q"]), host(s["u"])
    token = s["token"].cpu().numpy()
    n = np.full(c["B"], K) if s["lengths"] is None else s["lengths"].cpu().numpy()
    accepted = np.zeros(c["B"], np.int32)
    tokens = np.full((c["B"], K + 1), -1, np.int32)
    for b in range(c["B"]):
        i = 0
        while i < n[b] and u[b, i] * (1.0 if q is None else q[b, i, token[b, i]]) < p[b, i, token[b, i]]:
            tokens[b, i] = token[b, i]
            i += 1
        rest = p[b, i]
        if i < n[b]:
            if q is None:
                rest = rest.copy()
                rest[token[b, i]] = 0.0
            else:
                rest = np.maximum(rest - q[b, i], 0.0)
            if not rest.any():
                rest = p[b, i]
        total = np.cumsum(rest)
        accepted[b] = i
        tokens[b, i] = np.searchsorted(total, u[b, K] * total[-1], side="right")
    return {"accepted": torch.from_numpy(accepted).to(DEV), "tokens": torch.from_numpy(tokens).to(DEV)}


def exact(case, seed):
    """What run returns for these inputs, from the definitions in 64 bits."""
    s = prepare(case, seed)
    with torch.enable_grad():
        return {"scan": _exact_scan, "hop": _exact_hop, "rotary": _exact_rotary, "gated": _exact_gated,
                "added": _exact_added, "verify": _exact_verify}[case["kind"]](case, s)
