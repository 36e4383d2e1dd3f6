"""The norm's and the decode step's parameters when the kernel before the call on its stream has just written them:
both are launched as that kernel's dependents, and may read nothing before it has finished."""
import pytest
import torch

import selective_scan_gb300 as ss
import workloads as W
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


@pytest.mark.parametrize("n,dims", [(1, W.DIMS_130M), (5, W.DIMS_TINY)])
def test_decode_step(n, dims):
    dev = device()
    wl = W.decode_batch(seed=11, num_seqs=n, steps=1, num_slots=n + 2, dims=dims)
    p, b = wl.params, wl.batch
    x, z, dt = (t[0].contiguous().to(dev) for t in (wl.dec_xBC, wl.dec_z, wl.dec_dt))
    conv0, ssm0 = wl.conv_state.to(dev), wl.ssm_state.to(dev)
    conv, ssm = torch.empty_like(conv0), torch.empty_like(ssm0)

    def step(q):
        conv.copy_(conv0)
        ssm.copy_(ssm0)
        q[-1].add_(0)
        out = torch.empty((n, wl.dims.d_inner), dtype=x.dtype, device=dev)
        ss.decode_step(out, x, z, dt, *q, p.norm_groups, p.eps, conv, ssm, wl.dims, b.slots, b.fresh)
        return [out, conv, ssm]

    both(step, [p.conv_w, p.conv_b, p.A_log, p.dt_bias, p.D, p.norm_w], dev)
