"""The recurrent block's operators in 64 bits on the CPU, element by element with a bound on how far an
implementation that computes in 32 bits may be off (no method arithmetic is shared with the CUDA path).

Each reference returns (value, slack): |got - value| <= slack + half a step of got's type at value. The slack
counts roundings of U = 2^-24 relative to the magnitudes that enter, carried through the same recurrences:
DELTA covers one gate and one step of the recurrence (the exponential's argument, itself, the reciprocal, two
products and an addition, and the products of gates that a split over time forms)."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
DELTA = 64 * U


def gates(gate, lower):
    g = gate.double()
    lo = torch.zeros(g.shape[1], dtype=torch.float64) if lower is None else lower.double()
    up, down = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    return lo + (1 - lo) * up, (1 - lo) * down, up, down, lo


def recurrence(x, gate, lower, pool, cu, slots, fresh):
    """y, pool and their slacks, and per token the state before it with its magnitude and slack."""
    f, k, _, _, _ = gates(gate, lower)
    x = x.double()
    y, prev, mag, err = (torch.zeros_like(x) for _ in range(4))
    yerr = torch.zeros_like(x)
    pool = pool.double().clone()
    perr = torch.zeros_like(pool)
    for i, s in enumerate(slots):
        h = torch.zeros_like(pool[s]) if fresh[i] else pool[s].clone()
        m, e = h.abs(), torch.zeros_like(h)
        for t in range(cu[i], cu[i + 1]):
            prev[t], mag[t], err[t] = h, m, e
            h = f[t] * h + k[t] * x[t]
            m = f[t] * m + k[t] * x[t].abs()
            e = f[t] * e + DELTA * m
            y[t], yerr[t] = h, e
        pool[s], perr[s] = h, e
    return dict(y=(y, yerr), pool=(pool, perr), prev=(prev, mag, err))


def recurrence_backward(x, gate, lower, fwd, cu, dy, dstate_end):
    f, k, up, down, lo = gates(gate, lower)
    x, dy = x.double(), dy.double()
    prev, mag, err = fwd["prev"]
    n = len(cu) - 1
    G, GM, GE = (torch.zeros_like(x) for _ in range(3))
    d0, e0 = torch.zeros((n, x.shape[1]), dtype=torch.float64), torch.zeros((n, x.shape[1]), dtype=torch.float64)
    for i in range(n):
        g = torch.zeros(x.shape[1], dtype=torch.float64) if dstate_end is None else dstate_end[i].double()
        m, e = g.abs(), torch.zeros_like(g)
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            g, m = g + dy[t], m + dy[t].abs()
            e = e + DELTA * m
            G[t], GM[t], GE[t] = g, m, e
            g, m, e = f[t] * g, f[t] * m, f[t] * (e + DELTA * m)
        d0[i], e0[i] = g, e
    df = G * (prev - x)
    diff = mag + x.abs()
    dfe = GE * diff + GM * (err + 2 * DELTA * diff)
    c = (1 - lo) * up * down
    terms, terr = df * down, (dfe + DELTA * GM * diff) * down
    total = x.shape[0]
    return dict(dx=(k * G, k * (GE + 2 * DELTA * GM)), dgate=(df * c, (dfe + DELTA * GM * diff) * c),
                dlower=(terms.sum(0), terr.sum(0) + (total + 16) * U * (GM * diff * down).sum(0)), dstate=(d0, e0))


def add_rmsnorm(x, residual, weight, eps):
    s = x.double() + (residual.double() if residual is not None else 0)
    dim = s.shape[1]
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * weight.double()
    # the sum of squares in 32 bits: at most dim / 64 terms one after another in a thread, then a tree
    rel = (dim / 64 + 32) * U
    return (s, U * s.abs()), (y, rel * y.abs()), rel


def add_rmsnorm_backward(s, weight, eps, dy, dsum):
    s, w, dy = s.double(), weight.double(), dy.double()
    rows, dim = s.shape
    inv = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    wd = w * dy
    d = inv * (wd - s * inv ** 2 * (wd * s).mean(1, keepdim=True))
    size = inv * (wd.abs() + s.abs() * inv ** 2 * (wd * s).abs().mean(1, keepdim=True))
    rel = (dim / 64 + 64) * U
    slack = 3 * rel * size
    if dsum is not None:
        d = d + dsum.double()
        slack = slack + U * (dsum.double().abs() + size)
    terms = dy * s * inv
    return (d, slack), (terms.sum(0), (rel + (rows + 16) * U) * terms.abs().sum(0))


def act(name, v):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    return v


def slope(name, v):
    if name == "relu":
        return (v > 0).double()
    if name == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p + v * p * (1 - p)
    if name == "gelu":
        return 0.5 * torch.erfc(-v * math.sqrt(0.5)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(v)


def linear(x, w, x_scale, w_scale, bias, residual, activation):
    x, w = x.double(), w.double()
    if x_scale is not None:
        x, w = x * x_scale.double()[:, None], w * w_scale.double()[:, None]
    p = x @ w.T
    # products are exact in 32 bits; each addition may cut (not round) at 2^-23
    slack = 2 * (x.shape[1] + 16) * U * (x.abs() @ w.abs().T)
    if bias is not None:
        p = p + bias.double()
    slack = slack + 4 * U * p.abs()
    out = act(activation, p)
    # |act'| <= 1.13; the activation itself: 32 roundings of its value, and of p where erf cancels
    oslack = 1.13 * slack + 32 * U * (out.abs() + (p.abs() if activation == "gelu" else 0))
    if residual is not None:
        out = out + residual.double()
        oslack = oslack + U * out.abs()
    return (p, slack), (out, oslack)


def linear_backward(dy, pre, x, w, activation):
    dy, x, w = dy.double(), x.double(), w.double()
    d = slope(activation, pre.double()) if activation != "none" else torch.ones_like(dy)
    dp = dy * d
    dpe = 64 * U * dy.abs() * (d.abs() + 1)   # the derivative in 32 bits
    half = torch.finfo(torch.bfloat16).eps / 2  # dp enters the products as bf16 (exactly dy without an activation)
    r = dpe + (half * dp.abs() if activation != "none" else 0)
    rows, n = dy.shape
    return dict(dx=(dp @ w, r @ w.abs() + 2 * (n + 16) * U * (dp.abs() @ w.abs())),
                dw=(dp.T @ x, r.T @ x.abs() + 2 * (rows + 16) * U * (dp.abs().T @ x.abs())),
                dbias=(dp.sum(0), dpe.sum(0) + (rows + 16) * U * dp.abs().sum(0)))


def check(got, ref, what):
    value, slack = ref
    g = got.detach().cpu()
    half = torch.finfo(g.dtype).eps / 2
    g = g.double()
    assert g.shape == value.shape, (what, g.shape, value.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    # a value off by the slack may round up to half a step of its own further
    bound = slack * (1 + half) + half * value.abs() + 2.0 ** -126
    bad = (g - value).abs() > bound
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {at}: got {g[at].item()}, "
                             f"expected {value[at].item()} within {bound[at].item()}")
