"""The norm's weights when another kernel has just written them, and its 8-bit output bit for bit."""
import numpy as np
import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


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


def eight_bits(y):
    """(q, scale) of fp32 rows: scale = max |y| / 448 rounded to nearest, up where that is not a normal number; q = y /
    scale in e4m3."""
    top = y.abs().amax(1)
    scale = top / 448
    for r in range(len(scale)):
        if 0 < float(top[r]) and float(scale[r]) < 2.0 ** -126:
            exact = float(top[r]) / 448
            s = np.float32(exact)
            scale[r] = float(s if float(s) >= exact else np.nextafter(s, np.float32(np.inf)))
    scale[top == 0] = 1
    return (y / scale[:, None]).to(E4M3), scale


# widths: units on the rows' boundaries and on the matrix's, several rows to a CTA and one, and more than a CTA holds
WIDTHS = [(7, 33), (400, 1536), (300, 2047), (3, 9001), (2, 20000), (2, 20001)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim", WIDTHS)
def test_8_bit_output_is_the_quotient(dtype, rows, dim):
    """The same rows with an f32 output give y before it is divided."""
    dev = device()
    g = torch.Generator().manual_seed(dim)
    x = torch.randn((rows, dim), generator=g).to(dtype).to(dev)
    w = (torch.randn(dim, generator=g) * 0.3 + 1).to(dev)
    y, q, scale = torch.empty((rows, dim), device=dev), torch.empty((rows, dim), dtype=E4M3, device=dev), torch.empty(rows, device=dev)
    ss.add_rmsnorm(y, x.float(), w, 1e-5)
    ss.add_rmsnorm(q, x, w, 1e-5, scale=scale)
    qref, sref = eight_bits(y.cpu())
    assert_bits_equal(scale, sref, "scale")
    assert_bits_equal(q.view(torch.uint8), qref.view(torch.uint8), "q")


@pytest.mark.parametrize("size", [1e-35, 1e-37, 1e-40, 3e-42, 1e-44])
@pytest.mark.parametrize("rows,dim", WIDTHS)
def test_8_bit_output_of_tiny_rows(rows, dim, size):
    """Scales below the normal numbers: finite values, zeros stay zeros, and q scale is y to half a step of both."""
    dev = device()
    g = torch.Generator().manual_seed(dim)
    x = torch.randn((rows, dim), generator=g)
    x[:, ::5] = 0
    w = torch.full((dim,), size)
    y, q, scale = torch.empty((rows, dim), device=dev), torch.empty((rows, dim), dtype=E4M3, device=dev), torch.empty(rows, device=dev)
    ss.add_rmsnorm(y, x.to(dev), w.to(dev), 1e-5)
    ss.add_rmsnorm(q, x.to(dev), w.to(dev), 1e-5, scale=scale)
    y, q, scale = y.cpu(), q.cpu(), scale.cpu()
    qref, sref = eight_bits(y)
    assert_bits_equal(scale, sref, "scale")
    assert_bits_equal(q.view(torch.uint8), qref.view(torch.uint8), "q")
    v, s = q.float().double(), scale.double()[:, None]
    assert torch.isfinite(v).all() and (v[:, ::5] == 0).all()
    assert ((v * s - y.double()).abs() <= torch.maximum(y.double().abs() * 2.0 ** -4, 2.0 ** -10 * s) * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("rows,dim", WIDTHS)
def test_8_bit_output_of_rows_that_overflow(rows, dim):
    """y is infinite in places: the scale too, the finite values are zeros beside it and the infinite ones NaN."""
    dev = device()
    x = torch.randn((rows, dim), generator=torch.Generator().manual_seed(dim))
    w = torch.full((dim,), 2e38)
    y, q, scale = torch.empty((rows, dim), device=dev), torch.empty((rows, dim), dtype=E4M3, device=dev), torch.empty(rows, device=dev)
    ss.add_rmsnorm(y, x.to(dev), w.to(dev), 1e-5)
    ss.add_rmsnorm(q, x.to(dev), w.to(dev), 1e-5, scale=scale)
    y, q, scale = y.cpu(), q.cpu().float(), scale.cpu()
    inf = torch.isinf(y)
    assert torch.equal(torch.isinf(scale), inf.any(1)) and inf.any() and not torch.isnan(scale).any()
    assert torch.equal(torch.isnan(q), inf)
    over = inf.any(1)[:, None] & ~inf
    assert (q[over] == 0).all()
