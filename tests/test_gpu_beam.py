"""Beam search's selection and the states' reordering on the GPU against a plain selection in 64 bits.

Parents and tokens have to be equal, ties and dead beams included. The inputs keep scores of different
beams apart by far more than fp32 rounding, or make them equal exactly. Scores: log-probabilities of
magnitude ~20 round at 2^-20, sums over the vocabulary add a few 2^-24: 1e-5 absolute of 20 is 1e-4.
"""
import math

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


def reference(logits, scores, finished, eos):
    B, W, V = logits.shape
    out = []
    for b in range(B):
        cand = []
        for w in range(W):
            x = logits[b, w].double().cpu()
            x = torch.where(x.isnan(), -math.inf, x).clamp(max=torch.finfo(torch.float32).max)
            if finished is not None and bool(finished[b, w]):
                x = torch.full((V,), -math.inf, dtype=torch.float64)
                x[eos] = 0.0
            key = torch.log_softmax(x, 0) + scores[b, w].double().cpu()
            key = torch.where(key.isnan(), -math.inf, key)
            best, tok = torch.sort(x, descending=True, stable=True)
            cand += [(-float(key[t]), w, i, int(t)) for i, t in enumerate(tok[:W].tolist())]
        cand.sort(key=lambda c: c[:3])
        out.append([(-k, w, t, (finished is not None and bool(finished[b, w])) or t == eos)
                    for k, w, _, t in cand[:W]])
    return out


def check(logits, scores, finished=None, eos=-1):
    import gated_delta_rule_14_gb300 as kla
    s, p, t, f = kla.beam_select(logits, scores, finished, eos=eos)
    kla.device_status(DEV)
    want = reference(logits, scores, finished, eos)
    for b, rows in enumerate(want):
        got = list(zip(s[b].tolist(), p[b].tolist(), t[b].tolist(), f[b].tolist()))
        for (gs, gp, gt, gf), (ws, wp, wt, wf) in zip(got, rows):
            assert (gp, gt, gf) == (wp, wt, wf), (b, got, rows)
            assert gs == ws or abs(gs - ws) <= 1e-4, (b, got, rows)


def draw(B, W, V, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    logits = (torch.randn((B, W, V), generator=gen, device=DEV) * 3).to(dtype)
    scores = -torch.rand((B, W), generator=gen, device=DEV) * 5
    return logits, scores


# vocabularies below, at and above one CTA's piece (4096 tokens), down to one token
@pytest.mark.parametrize("V", [1, 2, 5, 255, 4095, 4096, 4097, 33333])
@pytest.mark.parametrize("W", [1, 2, 5, 16])
def test_sizes(V, W):
    check(*draw(3, W, V, torch.float32, V + W))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_requests(dtype):
    check(*draw(40, 4, 5000, dtype, 1))


def test_equal_logits_take_the_lowest_token():
    logits = torch.zeros(1, 3, 9000, device=DEV)
    logits[0, 1, 4095:4099] = 2.0   # equal values on both sides of a piece's border
    check(logits, torch.tensor([[-1.0, -1.5, -9.0]], device=DEV))


def test_equal_beams_take_the_lowest_beam():
    row = torch.randn(700, device=DEV)
    logits = row.expand(2, 4, 700).contiguous()
    check(logits, torch.full((2, 4), -2.0, device=DEV))


def test_negative_zero_equals_zero():
    logits = torch.full((1, 2, 64), -5.0, device=DEV)
    logits[0, :, 10] = 0.0
    logits[0, :, 7] = -0.0
    check(logits, torch.tensor([[-1.0, -3.0]], device=DEV))


def test_masked_vocabulary():
    logits, scores = draw(4, 4, 6000, torch.float32, 3)
    logits[0, 0] = -math.inf                     # a beam with no candidate
    logits[1, :, 5:] = -math.inf                 # five tokens left
    logits[2, :, 3:] = torch.finfo(torch.float32).min
    logits[3, 1, ::2] = math.nan                 # NaN counts as masked
    check(logits, scores)


def test_first_step_and_dead_beams():
    logits, scores = draw(3, 4, 6000, torch.float32, 4)
    scores[0, 1:] = -math.inf                    # the first step: one live beam
    scores[1] = -math.inf                        # none at all
    scores[2, 2] = math.nan
    check(logits, scores)


def test_infinite_logits():
    logits, scores = draw(2, 2, 100, torch.float32, 5)
    logits[0, 0, 17] = math.inf
    logits[1] = -math.inf
    check(logits, scores)


@pytest.mark.parametrize("eos", [0, 2, 4999])
def test_finished_beams(eos):
    logits, scores = draw(4, 5, 5000, torch.bfloat16, 6)
    finished = torch.rand(4, 5, device=DEV) < 0.5
    finished[0] = True                            # all of them: each goes on with eos
    check(logits, scores, finished, eos)


def test_padded_vocabulary():
    wide, scores = draw(3, 4, 5008, torch.bfloat16, 7)
    wide[:, :, 5000:] = 100.0                     # past the slice: never read as candidates
    check(wide[:, :, :5000], scores)


@pytest.mark.parametrize("shape", [(2, 3, 4), (1, 4, 16, 128, 128), (5, 1, 2, 16, 16)])
def test_reorder_states(shape):
    import gated_delta_rule_14_gb300 as kla
    S = torch.randn(shape, device=DEV)
    B, W = shape[:2]
    parents = torch.randint(0, W, (B, W), dtype=torch.int32, device=DEV)
    parents[0, W - 1] = W                          # outside: zeros
    out = kla.reorder_states(S, parents)
    for b in range(B):
        for w in range(W):
            p = int(parents[b, w])
            assert torch.equal(out[b, w], S[b, p] if p < W else torch.zeros_like(S[b, 0]))


def test_refusals():
    import gated_delta_rule_14_gb300 as kla
    logits, scores = draw(2, 4, 50, torch.float32, 1)
    fin = torch.zeros(2, 4, dtype=torch.bool, device=DEV)
    with pytest.raises(kla.KlaError):
        kla.beam_select(logits, scores, fin)                      # finished beams without eos
    with pytest.raises(kla.KlaError):
        kla.beam_select(logits, scores, fin, eos=50)
    with pytest.raises(TypeError):
        kla.beam_select(logits, scores, fin.int(), eos=1)
    with pytest.raises(ValueError):
        kla.beam_select(logits, scores[:, :3])
    with pytest.raises(ValueError):
        kla.beam_select(logits.transpose(1, 2).contiguous().transpose(1, 2), scores)
    with pytest.raises(TypeError):
        kla.beam_select(logits.double(), scores)
    with pytest.raises(kla.KlaError):
        kla.beam_select(*draw(1, 17, 50, torch.float32, 1))
    with pytest.raises(kla.KlaError):
        kla.reorder_states(torch.zeros(1, 2, 3, device=DEV), torch.zeros(1, 2, dtype=torch.int32, device=DEV))
    S = torch.zeros(1, 2, 4, device=DEV)
    with pytest.raises(kla.KlaError):
        kla.reorder_states(S, torch.zeros(1, 2, dtype=torch.int32, device=DEV), out=S)


@pytest.mark.parametrize("score", [-1.0, -math.inf])
def test_more_equal_candidates_than_are_ranked_at_once(score):
    """Every logit and every score equal: 2560 list entries reach the merge's threshold, which ranks 256 at once,
    and beam 0's lowest tokens are taken one after the other."""
    check(torch.zeros(1, 16, 40000, device=DEV), torch.full((1, 16), score, device=DEV))


def test_more_entries_than_a_merge_starts_with():
    """35 pieces of 16 beams leave 8960 entries; 8192 are on their way from the start."""
    check(*draw(1, 16, 140001, torch.float32, 8))


def test_long_runs_of_equal_values_in_many_pieces():
    gen = torch.Generator(device=DEV).manual_seed(9)
    row = torch.randint(0, 3, (140001,), generator=gen, device=DEV).float()
    logits = row.expand(1, 16, 140001).contiguous()
    check(logits, torch.zeros(1, 16, device=DEV))                              # equal beams
    check(logits, -0.5 * torch.arange(16., device=DEV).flip(0)[None])          # the last beam is the best
