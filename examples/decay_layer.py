"""One layer of linear attention with decaying states, trained for a few steps and decoded with beams.

    python examples/decay_layer.py

Projections are torch matmuls; the attention, the heads' norm, their gradients, the single-token steps and
the beam search run in this package's kernels: ``linear_fwd`` -> ``layer_norm_fwd`` -> ``layer_norm_bwd`` ->
``linear_bwd`` in training, ``linear_fwd`` for the prompt and then ``linear_step`` (which takes each beam's
state from its parent) -> ``layer_norm_fwd`` -> ``beam_select`` for every token.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_14_gb300 as kla  # noqa: E402


class DecayLayer:
    """Token embedding, one attention layer with a norm per head, and the embedding again as output."""

    def __init__(self, vocab: int, heads: int, d: int = 128, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale
        D = heads * d
        self.heads, self.d, self.scale = heads, d, d ** -0.5
        self.decay = 1 - torch.exp2(-5 - torch.arange(heads, device=device) * (5.0 / max(1, heads - 1)))
        self.params = {"embed": w(vocab, D, scale=0.1), "qkv": w(D, 3 * D, scale=D ** -0.5),
                       "out": w(D, D, scale=D ** -0.5), "norm_w": torch.ones(heads, d, device=device),
                       "norm_b": torch.zeros(heads, d, device=device)}

    def _qkv(self, h):   # [..., D] -> three [..., heads, d] slices of one tensor
        qkv = (h @ self.params["qkv"].bfloat16()).view(*h.shape[:-1], 3, self.heads, self.d)
        return qkv.unbind(-3)

    def _logits(self, o, h):
        y, mean, rstd = kla.layer_norm_fwd(o, self.params["norm_w"], self.params["norm_b"])
        z = y.flatten(-2) @ self.params["out"].bfloat16() + h
        return z @ self.params["embed"].bfloat16().t(), (y, mean, rstd, z)

    def gradients(self, tokens):
        """Mean cross-entropy of the next token, and the gradients of every parameter."""
        p = self.params
        B, T = tokens.shape[0], tokens.shape[1] - 1
        h = p["embed"].bfloat16()[tokens[:, :-1]]
        q, k, v = self._qkv(h)
        o, _ = kla.linear_fwd(q, k, v, self.decay, q_scale=self.scale, final_state=False)
        logits, (y, mean, rstd, z) = self._logits(o, h)
        logp = torch.log_softmax(logits.float(), -1)
        target = tokens[:, 1:]
        loss = -logp.gather(-1, target[..., None]).mean()

        dl = logp.exp()
        dl.scatter_add_(-1, target[..., None], torch.full_like(target, -1, dtype=dl.dtype)[..., None])
        dl = (dl / (B * T)).bfloat16()
        flat = lambda t: t.reshape(B * T, -1)   # noqa: E731
        dz = dl @ p["embed"].bfloat16()
        g = {"embed": flat(dl).t().float() @ flat(z).float(), "out": flat(y).t().float() @ flat(dz).float()}
        dy = (dz @ p["out"].bfloat16().t()).view(B, T, self.heads, self.d)
        do, g["norm_w"], g["norm_b"] = kla.layer_norm_bwd(dy, o, p["norm_w"], mean, rstd)
        d = kla.linear_bwd(q, k, v, self.decay, do, q_scale=self.scale, want_dS0=False)
        dqkv = torch.stack([d["dq"], d["dk"], d["dv"]], -3).flatten(-3)
        g["qkv"] = flat(h).t().float() @ flat(dqkv).float()
        dh = dqkv @ p["qkv"].bfloat16().t() + dz
        g["embed"].index_add_(0, tokens[:, :-1].reshape(-1), flat(dh).float())
        return loss, g

    def train(self, tokens, steps, rate=3e-3):
        opt = torch.optim.Adam(list(self.params.values()), lr=rate)
        losses = []
        for _ in range(steps):
            loss, g = self.gradients(tokens)
            for name, p in self.params.items():
                p.grad = g[name]
            opt.step()
            losses.append(float(loss))
        return losses

    def beams(self, prompt, width, steps, eos=-1):
        """[B, T] prompts -> (tokens [B, width, steps], scores [B, width])."""
        B, V = prompt.shape[0], self.params["embed"].shape[0]
        h = self.params["embed"].bfloat16()[prompt]
        o, S = kla.linear_fwd(*self._qkv(h), self.decay, q_scale=self.scale)
        logits, _ = self._logits(o[:, -1:].contiguous(), h[:, -1:])
        S = S.repeat_interleave(width, 0)                      # every beam starts from the prompt's state
        logits = logits.expand(B, width, V).contiguous()
        scores = torch.full((B, width), -torch.inf, device=prompt.device)
        scores[:, 0] = 0.0                                     # and only one of them is alive
        first = (torch.arange(B, device=prompt.device, dtype=torch.int32) * width)[:, None]
        finished = torch.zeros((B, width), dtype=torch.bool, device=prompt.device) if eos >= 0 else None
        S_next, history = torch.empty_like(S), None
        for _ in range(steps):
            scores, parents, tokens, done = kla.beam_select(logits, scores, finished, eos=eos)
            if eos >= 0:
                finished = done
            if history is not None:
                history = torch.gather(history, 1, parents.long()[..., None].expand_as(history))
            history = tokens[..., None] if history is None else torch.cat([history, tokens[..., None]], -1)
            h = self.params["embed"].bfloat16()[tokens.view(-1).long()]
            q, k, v = (t.contiguous() for t in self._qkv(h))
            o = kla.linear_step(q, k, v, self.decay, S, q_scale=self.scale, parent=(parents + first).view(-1),
                                S_out=S_next)
            S, S_next = S_next, S
            logits = self._logits(o, h)[0].view(B, width, V)
        return history, scores


def main():
    layer = DecayLayer(vocab=256, heads=2)
    period = torch.randint(0, 256, (1, 17), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    tokens = period.repeat(4, 12)[:, :200]                     # a repeating text
    losses = layer.train(tokens, 100)
    out, scores = layer.beams(tokens[:2, :100], width=4, steps=17)
    right = (out[:, 0] == tokens[:2, 100:117]).float().mean()
    kla.device_status()
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}; best beam's score {float(scores[0, 0]):.3f}, "
          f"{100 * float(right):.0f} % of its tokens continue the text")
    return losses, float(right)


if __name__ == "__main__":
    main()
