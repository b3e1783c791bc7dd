"""The frequencies of rotary positions for long contexts, on the CPU, one by one against their formula."""
import math

import pytest
import torch

from gated_delta_rule_14_gb300 import rotary_freqs

# Python's numbers hold 2^-53 of the formula; the result is rounded once, by 2^-24
TOL = 2**-24 + 2**-40


def yarn(rot, base, factor, length, fast=32.0, slow=1.0):
    """Frequency i turns length f_i / (2 pi) times within the trained length. The ramp goes from the index at which that is
    `fast`, rounded down, to the one at which it is `slow`, rounded up, whether or not there is a frequency of that index."""
    def index(turns):
        return rot / 2 * math.log(length / (2 * math.pi * turns)) / math.log(base)
    low, high = max(0, math.floor(index(fast))), min(rot - 1, math.ceil(index(slow)))
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        r = 0.0 if i <= low else min(1.0, (i - low) / (high - low))   # before the ramp: kept
        out.append((1 - r) * f + r * f / factor)
    return out


# on either side of the length, 2 pi base, from which on the lowest frequency turns more than `slow` times
@pytest.mark.parametrize("length", [2048, 4096, 32768, 60000, 65536, 131072, 1048576])
@pytest.mark.parametrize("rot,base,factor", [(128, 10000.0, 4.0), (64, 10000.0, 32.0), (128, 1000000.0, 8.0), (4, 100.0, 2.0)])
def test_yarn_frequencies(rot, base, factor, length):
    got, scale = rotary_freqs(rot, base, scaling="yarn", factor=factor, original_length=length, device="cpu")
    assert abs(scale - (0.1 * math.log(factor) + 1)) <= 1e-15
    for i, (a, b) in enumerate(zip(got.tolist(), yarn(rot, base, factor, length))):
        assert abs(a - b) <= TOL * b, i


def test_yarn_keeps_most_of_a_frequency_that_still_turns():
    """131072 trained tokens: the lowest of 64 frequencies turns 2.4 times and stands on the ramp, not behind it."""
    plain, _ = rotary_freqs(128, device="cpu")
    got, _ = rotary_freqs(128, scaling="yarn", factor=4.0, original_length=131072, device="cpu")
    assert 2.4 <= 131072 * float(plain[-1]) / (2 * math.pi) <= 2.5 and 0.45 <= float(got[-1] / plain[-1]) <= 0.47


def test_yarn_of_contexts_in_which_nothing_turns():
    """Trained on fewer tokens than the highest frequency needs for `slow` turns: every one is divided."""
    plain, _ = rotary_freqs(16, device="cpu")
    for length, slow in ((6, 1.0), (2, 1.0), (40, 10.0)):
        got, _ = rotary_freqs(16, scaling="yarn", factor=4.0, original_length=length, slow=slow, device="cpu")
        assert length / (2 * math.pi) < slow and torch.equal(got, plain / 4), (length, slow)


@pytest.mark.parametrize("bad", [dict(base=1.0, scaling="yarn", original_length=4096),
                                 dict(base=0.5, scaling="yarn", original_length=4096), dict(base=math.inf),
                                 dict(factor=math.inf), dict(base=math.nan), dict(factor=math.nan)])
def test_frequencies_that_have_no_meaning_are_refused(bad):
    with pytest.raises(ValueError):
        rotary_freqs(8, device="cpu", **bad)
