"""The norm where kernels meet: its weights when another kernel has just written them."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim", [(64, 77), (3000, 2047), (3000, 2048), (40, 5001), (20, 9001)])
def test_weights_written_by_the_kernel_in_front(dtype, rows, dim):
    """Each call takes the weights as the kernel before it on the stream left them, forwards and backwards, called and
    replayed from a graph."""
    dev, steps = device(), 24
    g = torch.Generator().manual_seed(dim)
    draw = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, dy = draw(rows, dim).to(dtype).to(dev), draw(rows, dim).to(dtype).to(dev)
    every = [v.clone() for v in draw(steps, dim).to(dev)]  # (each on a boundary of its own)
    w = torch.empty(dim, device=dev)

    def outputs():
        return [torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)]

    def step(weight, o):
        ss.add_rmsnorm_backward(o[1], None, o[2], dy, None, x, weight, 1e-5)

    want = [outputs() for _ in range(steps)]
    for k in range(steps):  # with weights that nothing is writing
        ss.add_rmsnorm(want[k][0], x, every[k], 1e-5)
        step(every[k], want[k])
        torch.cuda.synchronize()
    got = [outputs() for _ in range(steps)]
    for k in range(steps):
        w.copy_(every[k])
        step(w, got[k])
        w.fill_(float("nan"))
        w.copy_(every[k])
        ss.add_rmsnorm(got[k][0], x, w, 1e-5)
    torch.cuda.synchronize()
    for k in range(steps):
        for a, b in zip(got[k], want[k]):
            assert_bits_equal(a, b, f"call {k}")
    source, o = torch.empty(dim, device=dev), outputs()
    step(every[0], o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.copy_(source)
        step(w, o)
        ss.add_rmsnorm(o[0], x, w, 1e-5)
    for k in range(steps):
        source.copy_(every[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(o, want[k]):
            assert_bits_equal(a, b, f"replay {k}")
