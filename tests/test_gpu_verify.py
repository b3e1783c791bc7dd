"""Verification of drafted tokens on the GPU: whole numbers, equal to a plain walk over the rows in 64 bits. Inputs are
drawn so that no running sum lies within 1e-12 of its mark, where the order of 64-bit sums could tell."""
import numpy as np
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def walk(draft, q, p, u, n):
    """Plain: (accepted, tokens) of one sequence."""
    K = len(draft)
    big = np.finfo(np.float32).max
    weight = lambda v: np.where(v > 0, np.minimum(v, big), 0.0)   # noqa: E731
    p = weight(p)
    q = None if q is None else weight(q)
    out = np.full(K + 1, -1)
    i = 0
    while i < n:
        t = draft[i]
        if not (0 <= t < p.shape[1]) or not u[i] * (1.0 if q is None else q[i, t]) < p[i, t]:
            break
        out[i] = t
        i += 1
    rest = p[i]
    if i < n:
        if q is None:
            rest = rest.copy()
            if 0 <= draft[i] < p.shape[1]:
                rest[draft[i]] = 0
        else:
            rest = np.maximum(rest - q[i], 0.0)
        if not rest.any():
            rest = p[i]
    if rest.any():
        run = np.cumsum(rest)
        mark = u[K] * run[-1]
        assert np.abs(run - mark).min() > 1e-12 * run[-1] or u[K] == 0.0
        out[i] = np.searchsorted(run, mark, side="right")
    return i, out


def check(draft, q, p, u, n=None):
    import gated_delta_rule_14_gb300 as kla
    accepted, tokens = kla.verify_draft(draft, q, p, u, lengths=n)
    kla.device_status(DEV)
    B, K = draft.shape
    assert accepted.dtype == tokens.dtype == torch.int32 and tokens.shape == (B, K + 1)
    host = lambda t: t.double().cpu().numpy()   # noqa: E731
    lens = np.full(B, K) if n is None else np.clip(n.cpu().numpy(), 0, K)
    for b in range(B):
        want, row = walk(draft[b].cpu().numpy(), None if q is None else host(q[b]), host(p[b]), host(u[b]), lens[b])
        assert int(accepted[b]) == want and np.array_equal(tokens[b].cpu().numpy(), row), b
    return accepted


def make(B, K, V, dtype=F, seed=0, near=0.7):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = 3 * torch.randn(B, K + 1, V, generator=g, device=DEV)
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :K] + near * torch.randn(B, K, V, generator=g, device=DEV), -1)
    draft = torch.multinomial(q.reshape(B * K, V), 1, generator=g).view(B, K).int() if K else torch.empty(
        B, 0, dtype=torch.int32, device=DEV)
    return draft, q.to(dtype), p.to(dtype), torch.rand(B, K + 1, generator=g, device=DEV)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 100, 1000, 1024, 4097, 32000, 100003])
@pytest.mark.parametrize("dtype", [F, BF])
def test_vocabularies(V, dtype):
    draft, q, p, u = make(5, 4, V, dtype, seed=V)
    check(draft, q, p, u)
    check(draft, None, p, u)


@pytest.mark.parametrize("B,K", [(1, 0), (1, 1), (3, 0), (200, 1), (64, 8), (2, 33), (1, 70)])
def test_batches_and_drafts(B, K):
    draft, q, p, u = make(B, K, 777, seed=B + K, near=0.2)
    check(draft, q, p, u)
    n = torch.randint(0, K + 1, (B,), generator=torch.Generator(DEV).manual_seed(1), device=DEV, dtype=torch.int32)
    check(draft, q, p, u, n)


def test_lengths_outside_the_draft():
    draft, q, p, u = make(3, 4, 500, seed=3)
    check(draft, q, p, u, torch.tensor([9, -2, 4], dtype=torch.int32, device=DEV))


def test_all_accepted_and_none():
    draft, q, p, u = make(6, 5, 3000, seed=4, near=0.0)
    u[:, :5] *= 0.999
    assert (check(draft, p[:, :5].contiguous(), p, u) == 5).all()
    other = (draft + 1) % 3000
    zero = p.clone()
    zero[:, :5].scatter_(2, other[..., None].long(), 0.0)
    assert (check(other, q, zero, u) == 0).all()


def test_tokens_outside_the_vocabulary():
    draft, q, p, u = make(4, 3, 60, seed=5)
    draft[0, 0], draft[1, 1], draft[2, 2], draft[3, 0] = 60, -1, 2**31 - 1, -2**31
    check(draft, q, p, u)
    check(draft, None, p, u)


def test_rows_that_leave_nothing():
    """A draft equal to the target, refused by a random number of one: the target's own row; a target row of zeros has
    no token."""
    import gated_delta_rule_14_gb300 as kla
    draft, q, p, u = make(3, 2, 400, seed=6)
    q = p[:, :2].contiguous()
    u[:, 0] = 1.0
    assert (check(draft, q, p, u) == 0).all()
    p = torch.zeros_like(p)
    accepted, tokens = kla.verify_draft(draft, q, p, u)
    assert (accepted == 0).all() and (tokens == -1).all()


def test_values_that_are_no_probabilities():
    """NaN, infinities, negative values and subnormals, in rows and at drafted tokens."""
    draft, q, p, u = make(4, 2, 300, seed=7)
    p[0, 0, ::7] = float("nan")
    q[0, 0, ::5] = float("nan")
    p[1, 0, draft[1, 0]] = float("nan")
    q[1, 0, 3] = float("inf")
    p[2, 0, 11] = float("inf")
    p[2, 0, draft[2, 0]] = 0.0
    p[3] = -p[3]
    p[3, :, 250] = 1e-40
    check(draft, q, p, u)
    check(draft, None, p, u)


def test_first_and_last_tokens():
    """Random numbers of 0 and of 1 - 2^-24 draw the first and the last token with any weight."""
    draft, q, p, u = make(2, 0, 5000, seed=8)
    p[:, :, :17] = 0
    p[:, :, 4900:] = 0
    u[0, 0], u[1, 0] = 0.0, 1.0 - 2.0 ** -24
    p[1] = 0
    p[1, 0, [40, 4899]] = 0.5
    check(draft, None, p, u)


def test_strided_rows():
    draft, q, p, u = make(3, 4, 1001, seed=9)
    wide_q, wide_p = torch.empty(3, 7, 1100, device=DEV), torch.empty(3, 9, 1100, device=DEV)
    wide_q[:, 1:5, :1001], wide_p[:, 2:7, :1001] = q, p
    check(draft, wide_q[:, 1:5, :1001], wide_p[:, 2:7, :1001], u)
    one = p[:, :1].expand(3, 5, 1001)
    check(draft, one[:, :4], one, u)


def test_distribution():
    """20000 draws from one pair of rows: every token's count within six deviations of the target's probability."""
    import gated_delta_rule_14_gb300 as kla
    g = torch.Generator(device=DEV).manual_seed(10)
    B, V = 20000, 12
    p, q = (torch.softmax(torch.randn(V, generator=g, device=DEV), -1) for _ in range(2))
    draft = torch.multinomial(q, B, replacement=True, generator=g)[:, None].int()
    u = torch.rand(B, 2, generator=g, device=DEV)
    _, tokens = kla.verify_draft(draft, q.expand(B, 1, V), p.expand(B, 2, V), u)
    counts = torch.bincount(tokens[:, 0].long(), minlength=V).double()
    assert ((counts - B * p.double()).abs() <= 6 * (B * p.double()).sqrt()).all()


def test_refusals():
    import gated_delta_rule_14_gb300 as kla
    draft, q, p, u = make(2, 3, 50)
    with pytest.raises(TypeError):
        kla.verify_draft(draft.long(), q, p, u)
    with pytest.raises(TypeError):
        kla.verify_draft(draft, q.to(BF), p, u)
    with pytest.raises(TypeError):
        kla.verify_draft(draft, q.half(), p.half(), u)
    with pytest.raises(ValueError):
        kla.verify_draft(draft, q, p[:, :3], u)
    with pytest.raises(ValueError):
        kla.verify_draft(draft, q, p, u[:, :3])
    with pytest.raises(ValueError):
        kla.verify_draft(draft, q, p.transpose(1, 2).contiguous().transpose(1, 2), u)
    with pytest.raises(ValueError):
        kla.verify_draft(draft, q, p[0], u)
    with pytest.raises(ValueError):
        kla.verify_draft(draft.cpu(), q, p, u)


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("V", [2048, 2049])
def test_one_large_weight_and_many_small_ones(V, dtype):
    """A token of nearly all the weight and 2^-25 to 2^-24 of it for each of the others, the sums' worst case: running sums
    are off by 2^-39 of the whole at most, and marks that lie 2^-38 or more from a border find their token. Once from the
    row itself, once from what a draft leaves of it."""
    import gated_delta_rule_14_gb300 as kla
    g = torch.Generator().manual_seed(V)
    small = (2.0**-25 * (1 + torch.rand(V, generator=g))).to(dtype)
    row = small.clone()
    at = [0, 5, 700, V - 1]
    rows = []
    for i in at:
        r = row.clone()
        r[i] = 1.0
        rows.append(r)
    B = 256
    target = torch.stack([rows[b % 4] for b in range(B)])
    u = 1 - torch.randint(1, 2**11, (B,), generator=g).float() * 2.0**-24
    run = target.double().cumsum(1)
    mark = u.double()[:, None] * run[:, -1:]
    clear = ((run - mark).abs() > 2.0**-38 * run[:, -1:]).all(1)
    assert int(clear.sum()) >= 200
    want = (run > mark).int().argmax(1)
    empty = torch.empty(B, 0, dtype=torch.int32, device=DEV)
    _, tokens = kla.verify_draft(empty, None, target[:, None].contiguous().to(DEV), u[:, None].to(DEV))
    assert torch.equal(tokens[:, 0].cpu()[clear].long(), want[clear])
    # a draft refused whose row covers a quarter of every weight: exact in either type
    draft, us = torch.full((B, 1), 1, dtype=torch.int32, device=DEV), torch.stack([torch.full((B,), 1 - 2.0**-24), u], 1)
    two = target[:, None].expand(B, 2, V).contiguous()
    q = target[:, None] * 0.25
    q[:, 0, 1] = 1.0   # above the target's: refused, and nothing left of token 1
    rest = (target.double() - q[:, 0].double()).clamp(min=0)
    run = rest.cumsum(1)
    mark = u.double()[:, None] * run[:, -1:]
    clear = ((run - mark).abs() > 2.0**-38 * run[:, -1:]).all(1)
    assert int(clear.sum()) >= 200
    took, tokens = kla.verify_draft(draft, q.to(DEV), two.to(DEV), us.to(DEV))
    kla.device_status(DEV)
    assert int(took.sum()) == 0
    assert torch.equal(tokens[:, 0].cpu()[clear].long(), (run > mark).int().argmax(1)[clear])
