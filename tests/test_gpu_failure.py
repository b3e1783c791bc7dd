"""Failure detection without a GPU fault: a bounded wait that gives up is reported by
kla_device_status as KLA_ERR_TIMEOUT, the flag is cleared by that read, and the context keeps
working (a prefill right after matches the oracle)."""
import pytest

import oracle
import synth
from gpu_util import DEV, oracle_chains, run_prefill

pytestmark = pytest.mark.gpu


def test_bounded_wait_timeout_is_reported_and_recovered():
    import torch

    import gated_delta_rule_14_gb300 as kla
    lib = kla._native.lib()
    stream = torch.cuda.current_stream(DEV).cuda_stream
    kla.device_status(DEV)                                        # start from a clear flag
    assert lib.kla_selftest_wait_timeout(200, stream) == 0        # gives up after <= 4 ms
    assert lib.kla_device_status(stream) == kla._native.KLA_ERR_TIMEOUT
    assert lib.kla_device_status(stream) == kla._native.KLA_OK    # cleared by the read
    inp = synth.make_prefill("gdn4k", seed=12, B=1, T=130, H=2, s0_sigma=0.05)
    o, S = run_prefill(inp)
    o_ref, s_ref = oracle_chains(inp)
    assert oracle.rel_l2(o[0].transpose(1, 0, 2), o_ref) <= 1e-2
    assert oracle.rel_l2(S[0], s_ref) <= 1e-2


@pytest.mark.parametrize("limit", [20, 50, 100])   # the time-out falls on different turns of the other teams
def test_a_team_that_gives_up_leaves_as_one(limit):
    """Four teams of one CTA with barriers of their own: the first gives up in its second turn, and every one
    of its threads leaves there; the other teams finish their turns, and the time-out is reported once."""
    import torch

    import gated_delta_rule_14_gb300 as kla
    lib = kla._native.lib()
    stream = torch.cuda.current_stream(DEV).cuda_stream
    kla.device_status(DEV)
    for _ in range(20):
        turns = torch.full((256,), -1, dtype=torch.int32, device=DEV)
        assert lib.kla_selftest_team_timeout(limit, turns.data_ptr(), stream) == 0
        assert lib.kla_device_status(stream) == kla._native.KLA_ERR_TIMEOUT
        assert turns.tolist() == [1] * 64 + [20000] * 192
    assert lib.kla_device_status(stream) == kla._native.KLA_OK


def test_a_warp_that_gives_up_calls_the_others_out():
    """Eight warps of one CTA wait on barriers of their own: the first gives up, and every warp leaves its wait
    as one, long before the 2 s that the others would wait by themselves."""
    import torch

    import gated_delta_rule_14_gb300 as kla
    lib = kla._native.lib()
    stream = torch.cuda.current_stream(DEV).cuda_stream
    kla.device_status(DEV)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(20):
        turns = torch.full((256,), -1, dtype=torch.int32, device=DEV)
        start.record()
        assert lib.kla_selftest_warp_timeout(200, turns.data_ptr(), stream) == 0   # 4 ms
        end.record()
        assert lib.kla_device_status(stream) == kla._native.KLA_ERR_TIMEOUT
        assert turns.tolist() == [1] * 32 + [100] * 224 and start.elapsed_time(end) < 1000
    assert lib.kla_device_status(stream) == kla._native.KLA_OK
