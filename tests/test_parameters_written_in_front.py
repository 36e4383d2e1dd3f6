"""The gated norm's weight when the kernel before the call on its stream has just written it: the norm is launched as
that kernel's dependent, and may read nothing before it has finished."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu
STEPS = 16


def both(fn, params, dev):
    """fn(parameters) with parameters that nothing is writing, and with ones that the kernels in front have written,
    called and replayed from a graph: the outputs agree bit for bit."""
    g = torch.Generator().manual_seed(9)
    every = [[(p.float() * (0.5 + torch.rand(p.shape, generator=g))).to(p.dtype).to(dev) for p in params] for _ in range(STEPS)]
    want = []
    for e in every:
        torch.cuda.synchronize()
        want.append([t.clone() for t in fn(e)])
    mine = [torch.empty_like(p) for p in every[0]]

    def written(e):
        for m, p in zip(mine, e):
            m.copy_(p)
            m.add_(0)  # (a kernel, where the copy may be none)
        return fn(mine)

    got = [[t.clone() for t in written(e)] for e in every]
    torch.cuda.synchronize()
    for k in range(STEPS):
        for a, b in zip(got[k], want[k]):
            assert_bits_equal(a, b, f"call {k}")
    source = [p.clone() for p in every[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = written(source)
    for k in range(STEPS):
        for s, p in zip(source, every[k]):
            s.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[k]):
            assert_bits_equal(a, b, f"replay {k}")


@pytest.mark.parametrize("rows,dim,groups", [(4, 256, 1), (300, 1536, 1), (64, 1024, 4), (8, 16384, 1)])
def test_gated_norm(rows, dim, groups):
    dev = device()
    g = torch.Generator().manual_seed(dim)
    y, z = (torch.randn((rows, dim), generator=g).bfloat16().to(dev) for _ in range(2))

    def norm(p):
        out = torch.empty_like(y)
        ss.gated_rmsnorm(out, y, z, p[0], groups, 1e-5)
        return [out]

    both(norm, [torch.randn(dim, generator=g)], dev)
