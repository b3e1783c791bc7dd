"""Equal calls of the gated scan give equal bits, whichever tile is heard first: by tensor maps, by 16-byte and by 4-byte
copies and without any, with gates of all kinds, beside other work and in a graph."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


def inputs(B, T, C, dtype, mode, shift):
    gen = torch.Generator(device=DEV).manual_seed(C)
    flat = [torch.randn(B * T * C + shift, generator=gen, device=DEV) for _ in range(3)]
    if mode == "log":
        flat[1] = -torch.nn.functional.softplus(2 * flat[1] - 4)
    else:   # gates that forget and such as keep among them
        flat[1] = flat[1] * 4
    x, gate, dy = (t.to(dtype)[shift:].view(B, T, C) for t in flat)
    n = torch.tensor([T - 100 * b for b in range(B)], dtype=torch.int32, device=DEV)
    return x, gate, dy, torch.randn(B, C, generator=gen, device=DEV), torch.randn(B, C, generator=gen, device=DEV), n


@pytest.mark.parametrize("B,T,C,shift", [(4, 3000, 2048, 0), (1, 20001, 1032, 0), (2, 5000, 1034, 0), (3, 4000, 1001, 0),
                                         (2, 4000, 514, 1)])
@pytest.mark.parametrize("mode", ["sigmoid", "log"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_calls(B, T, C, shift, dtype, mode):
    import gated_delta_rule_14_gb300 as kla
    x, gate, dy, h0, dh, n = inputs(B, T, C, dtype, mode, shift)
    other, noise = torch.cuda.Stream(DEV), torch.randn(4096, 4096, device=DEV)

    def call():
        y, h_T, s = kla.gated_scan_fwd(x, gate, h0, mode=mode, lengths=n, states=True)
        g = kla.gated_scan_bwd(x, gate, dy, s, dh, mode=mode, lengths=n)
        return [y, h_T, *g.values()]
    first = call()
    for i in range(6):
        if i % 2:
            other.wait_stream(torch.cuda.current_stream(DEV))
            with torch.cuda.stream(other):   # fewer SMs for the tiles, which then finish in another order
                for _ in range(4):
                    noise @ noise
        assert all(torch.equal(a, b) for a, b in zip(first, call())), i
    torch.cuda.synchronize(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    kla.device_status(DEV)
