"""linear's activations where they go wrong most easily: values that are not finite, and GELU far below zero, by the
kernel of few rows, whole blocks of pairs' tiles and their edges and unaligned rows."""
import math

import pytest
import torch

import selective_scan_gb300 as ss
from tests import block_ref as R
from tests.gpu_util import device

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN, INF = float("nan"), float("inf")
ACTIVATIONS = ["none", "relu", "silu", "gelu"]
# few rows; pairs of CTAs with whole blocks and an edge; with rows of no alignment
SHAPES = [(5, 200), (2000, 1300), (2000, 1301)]


def same_kind(got, want, what):
    """NaN where `want` is NaN and the same infinities; the mask of what is finite."""
    g = got.detach().cpu().double()
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what + ": NaN"
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(g), inf) and torch.equal(g[inf], want[inf]), what + ": infinities"
    return torch.isfinite(want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("activation", ACTIVATIONS)
def test_what_is_not_finite_stays_so(activation, rows, n, out_type, fp8):
    """A NaN or an infinity among the inputs reaches the outputs that depend on it, and no others."""
    dev, k = device(), 32
    g = torch.Generator().manual_seed(n)
    x, w, bias = torch.randn((rows, k), generator=g), torch.randn((n, k), generator=g) * k ** -0.5, torch.randn(n, generator=g)
    bias[3], bias[n - 1], bias[7], bias[8] = NAN, NAN, INF, -INF
    xs = ws = None
    if fp8:
        xs, ws = x.abs().amax(1) / 448, w.abs().amax(1) / 448
        x, w = (x / xs[:, None]).to(E4M3), (w / ws[:, None]).to(E4M3)
        xs[1] = NAN
        x[rows - 1, 2] = NAN
    else:
        x, w = x.to(BF16), w.to(BF16)
        x[1, 5], x[rows - 1, k - 1] = NAN, NAN
        x[2, 4], x[3, 4] = INF, -INF
    (p, pslack), (want, slack) = R.linear(x.float(), w.float(), xs, ws, bias, None, activation)
    assert torch.isnan(want[1]).all() and torch.isnan(want[:, 3]).all()
    put = lambda t: t.to(dev) if t is not None else None  # noqa: E731
    out, pre = torch.empty((rows, n), dtype=out_type, device=dev), torch.empty((rows, n), dtype=BF16, device=dev)
    ss.linear(out, x.to(dev), w.to(dev), x_scale=put(xs), w_scale=put(ws), bias=bias.to(dev), activation=activation, pre=pre)
    fin = same_kind(out, want, "out")
    R.check(out.cpu()[fin], (want[fin], slack[fin]), "out")
    fin = same_kind(pre, p, "pre")
    R.check(pre.cpu()[fin], (p[fin], pslack[fin]), "pre")


@pytest.mark.parametrize("n", [64, 77])
@pytest.mark.parametrize("activation", ACTIVATIONS[1:])
def test_a_pre_activation_that_is_nan_reaches_its_gradients(activation, n):
    dev, rows, k = device(), 300, 72
    g = torch.Generator().manual_seed(n)
    draw = lambda *s: torch.randn(s, generator=g).to(BF16)  # noqa: E731
    x, w, dy, pre = draw(rows, k), draw(n, k), draw(rows, n), draw(rows, n)
    want = R.linear_backward(dy, pre, x, w, activation)
    pre[17, 5], pre[rows - 1, n - 1] = NAN, NAN
    dx, dw, db = torch.empty((rows, k), dtype=BF16, device=dev), torch.empty((n, k), dtype=BF16, device=dev), torch.empty(n, device=dev)
    ss.linear_backward(dx, dw, db, dy.to(dev), x.to(dev), w.to(dev), activation=activation, pre=pre.to(dev))
    for name, got, hit in (("dx", dx, [17, rows - 1]), ("dw", dw, [5, n - 1]), ("dbias", db, [5, n - 1])):
        got = got.cpu()
        keep = torch.tensor([i for i in range(got.shape[0]) if i not in hit])
        assert torch.isnan(got[hit]).all(), name
        R.check(got[keep], tuple(v[keep] for v in want[name]), name)


def gelu_slack(p):
    """Relative error of the tail 1 - Phi(|p|) in 32 bits: 2 roundings of p^2 / 2 and one of its factor, which the
    exponential turns into 3 |p^2 / 2| 2^-24 (2 p^2 is taken, as the exponential rounds its argument too), and 64
    roundings for the rest (eight terms of a polynomial without cancellation, a reciprocal, an exponential and four
    products)."""
    return (64 + 2 * p * p) * R.U


@pytest.mark.parametrize("rows,n", SHAPES)
def test_gelu_keeps_its_digits_below_zero(rows, n):
    """x = 0, so that the bias is the pre-activation: p Phi(p) to a relative error, however small it is."""
    dev, k = device(), 16
    p = torch.linspace(-12.5, 3.0, n)
    zero = lambda *s: torch.zeros(s, dtype=BF16, device=dev)  # noqa: E731
    v = p.double()
    want = 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    for t in (F32, BF16):
        out = torch.empty((rows, n), dtype=t, device=dev)
        ss.linear(out, zero(rows, k), zero(n, k), bias=p.to(dev), activation="gelu")
        R.check(out, (want.expand(rows, n), (gelu_slack(v) * want.abs()).expand(rows, n)), "gelu")


def test_gelu_slope_keeps_its_digits_below_zero():
    """One row, so that dbias is dy gelu'(pre) unrounded."""
    dev, n, k = device(), 400, 16
    pre = torch.linspace(-12.5, 3.0, n).to(BF16)
    dy = torch.randn((1, n), generator=torch.Generator().manual_seed(2)).to(BF16)
    v = pre.double()
    phi = torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    tail = 0.5 * torch.erfc(-v * math.sqrt(0.5))
    db = torch.empty(n, device=dev)
    ss.linear_backward(None, None, db, dy.to(dev), torch.zeros((1, k), dtype=BF16, device=dev),
                       torch.zeros((n, k), dtype=BF16, device=dev), activation="gelu", pre=pre[None].to(dev))
    d = dy[0].double()
    R.check(db, (d * (tail + v * phi), d.abs() * gelu_slack(v) * (tail + v.abs() * phi)), "dbias")
