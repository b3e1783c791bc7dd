"""The gated scan's bounded waits made to run out: a tile is left out, those that wait for its state give up after a few
polls, the whole call ends, the time-out is reported once, and the next call is as good as any."""
import pytest
import torch

from gpu_util import DEV

A = 1 << 40


def test_arguments_are_refused_on_the_host():
    from gated_delta_rule_14_gb300 import _native
    f = _native.lib().kla_selftest_scan_timeout

    def call(limit=10, T=600, C=64, x=A, ws=A + (1 << 30), size=1 << 24):
        return f(limit, 0, x, None, A + (1 << 28), None, 1, T, C, 1, ws, size, None)
    assert call(limit=0) == 1 and call(limit=2**21 + 1) == 1 and call(T=256) == 1 and call(C=0) == 1
    assert call(x=None) == 1 and call(ws=None) == 1 and call(size=8) == 1


# by tensor maps, by 16-byte, 4-byte and row-by-row copies, without copies, and in fp32; more tiles than CTAs, and fewer
@pytest.mark.gpu
@pytest.mark.parametrize("B,T,C,shift,dtype", [(8, 4096, 1024, 0, torch.bfloat16), (2, 3000, 64, 0, torch.bfloat16),
                                               (2, 3000, 70, 0, torch.bfloat16), (2, 3000, 65, 0, torch.bfloat16),
                                               (2, 3000, 64, 1, torch.bfloat16), (8, 2048, 1024, 0, torch.float32),
                                               (1, 9000, 33, 0, torch.float32)])
@pytest.mark.parametrize("backward", [False, True])
def test_waits_that_give_up(B, T, C, shift, dtype, backward):
    import gated_delta_rule_14_gb300 as kla
    lib, stream = kla._native.lib(), torch.cuda.current_stream(DEV).cuda_stream
    gen = torch.Generator(device=DEV).manual_seed(C)
    x, out, out2 = (torch.randn(B * T * C + shift, generator=gen, device=DEV).to(dtype)[shift:].view(B, T, C)
                    for _ in range(3))
    states = torch.zeros(B, -(-T // 128), C, device=DEV)
    size = kla.gated_scan_workspace_size(B, T, C, dtype)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    y, h_T, s = kla.gated_scan_fwd(x, x, states=True)
    g = kla.gated_scan_bwd(x, x, x, s)
    kla.device_status(DEV)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for limit in (1, 64, 3000):
        start.record()
        assert lib.kla_selftest_scan_timeout(limit, backward, x.data_ptr(), states.data_ptr(), out.data_ptr(),
                                             out2.data_ptr(), B, T, C, 0 if dtype == torch.float32 else 1, ws.data_ptr(),
                                             size, stream) == 0
        end.record()
        assert lib.kla_device_status(stream) == kla._native.KLA_ERR_TIMEOUT
        assert lib.kla_device_status(stream) == kla._native.KLA_OK
        assert start.elapsed_time(end) < 1000
        y2, h2, s2 = kla.gated_scan_fwd(x, x, states=True, workspace=ws)
        g2 = kla.gated_scan_bwd(x, x, x, s2, workspace=ws)
        kla.device_status(DEV)
        assert torch.equal(y, y2) and torch.equal(h_T, h2) and all(torch.equal(g[n], g2[n]) for n in g)
