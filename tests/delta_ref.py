"""The gated delta rule and beam search in 64 bits on the CPU, token by token (no method is shared with the CUDA path),
with bounds on how far an implementation may be off.

One token maps a row of the state by a (I - beta k k^T), whose 2-norm is at most a <= 1 where 0 <= beta |k|^2 <= 2. So an
error in a row does not grow in its 2-norm, and the bounds are norms: a row's magnitude m (what its terms' norms add up
to), its error e. LOCAL32 counts what one token adds in 32 bits, in units of 2^-24 of the magnitudes (dot products of at
most 16 terms a lane and a tree of four, exponential, length, update). On the tensor cores (bf16 inputs) an operand of the
state's own products is split into two bf16 numbers, off by at most 2^-16 of it, and at most four such operands stand one
behind another in a chunk: LOCAL16. Operands of products that end in a bf16 output are rounded to one bf16 number, off by
2^-8 at most (half a step)."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
LOCAL32 = 64 * U
LOCAL16 = 4 * 2.0 ** -16
HALF16 = 2.0 ** -8


def unit(x, eps):
    """x divided by its length, and the length (1 where it stays as it is)."""
    x = x.double()
    if eps is None:
        return x, torch.ones(x.shape[:-1], dtype=torch.float64)
    n = torch.sqrt((x * x).sum(-1) + eps)
    return x / n[..., None], n


def forward(q, k, v, g, beta, pool, cu, slots, fresh, scale, eps, local):
    """y, pool, what each token's backward needs, the states before every 64th token of a run."""
    rows, H, P = v.shape
    per = H // q.shape[1]
    (qu, qn), (ku, kn) = unit(q, eps), unit(k, eps)
    qh, kh = (qu * scale).repeat_interleave(per, 1), ku.repeat_interleave(per, 1)
    v = v.double()
    a = torch.ones((rows, H), dtype=torch.float64) if g is None else torch.exp(g.double())
    b = torch.ones((rows, H), dtype=torch.float64) if beta is None else beta.double()
    pool = pool.double().clone()
    perr = torch.zeros(pool.shape[:3], dtype=torch.float64)
    y, ymag, yerr = (torch.zeros((rows, H, P), dtype=torch.float64) for _ in range(3))
    before, us, err, mags, kept, kerr = [], [], [], [], [], []
    for i, s in enumerate(slots):
        S = torch.zeros_like(pool[s]) if fresh[i] else pool[s].clone()
        m = S.norm(dim=-1)
        e = torch.zeros_like(m)
        for t in range(cu[i], cu[i + 1]):
            if (t - cu[i]) % 64 == 0:
                kept.append(S)
                kerr.append(e)
            before.append(S)
            mags.append(m)
            at, kt, qt = a[t][:, None], kh[t], qh[t]
            dec = at[..., None] * S
            r = v[t] - (dec * kt[:, None, :]).sum(-1)
            u = b[t][:, None] * r
            us.append(u)
            err.append(r)
            S = dec + u[..., None] * kt[:, None, :]
            kl, ql = kt.norm(dim=-1)[:, None], qt.norm(dim=-1)[:, None]
            size = at * m * (1 + b[t][:, None] * kl ** 2) + b[t][:, None] * v[t].abs() * kl
            m = at * m + u.abs() * kl
            e = at * e + local * (size + m)
            y[t] = (S * qt[:, None, :]).sum(-1)
            ymag[t], yerr[t] = ql * m, ql * e + LOCAL32 * ql * m
        pool[s], perr[s] = S, e
    keep = dict(qu=qu, qn=qn, ku=ku, kn=kn, qh=qh, kh=kh, a=a, b=b, before=before, us=us, err=err, mags=mags)
    return dict(y=y, ymag=ymag, yerr=yerr, pool=pool, perr=perr, keep=keep,
                kept=torch.stack(kept) if kept else torch.zeros((0, H, P, q.shape[2]), dtype=torch.float64),
                kerr=torch.stack(kerr) if kept else torch.zeros((0, H, P), dtype=torch.float64))


def backward(keep, cu, dy, dstate_end, scale, groups):
    """Gradients by name, and for each a bound on its magnitude (the norm of a vector, for q and k); for those of g and
    beta, which are single sums over a state and may cancel, the 2-norm of their terms too."""
    qh, kh, a, b = keep["qh"], keep["kh"], keep["a"], keep["b"]
    rows, H, P = dy.shape
    n = len(cu) - 1
    dy = dy.double()
    dqh, dkh, dv = torch.zeros_like(qh), torch.zeros_like(kh), torch.zeros_like(dy)
    dg, db = torch.zeros_like(a), torch.zeros_like(b)
    mq, mk, mg, mb, tg, tb = (torch.zeros_like(a) for _ in range(6))
    mv = torch.zeros_like(dy)
    N = qh.shape[2]
    d0, e0 = torch.zeros((n, H, P, N), dtype=torch.float64), torch.zeros((n, H, P), dtype=torch.float64)
    for i in range(n):
        D = torch.zeros((H, P, N), dtype=torch.float64) if dstate_end is None else dstate_end[i].double().clone()
        m = D.norm(dim=-1)
        e = torch.zeros_like(m)
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            S, u, r, ms = keep["before"][t], keep["us"][t], keep["err"][t], keep["mags"][t]
            at, bt, kt, qt = a[t][:, None], b[t][:, None], kh[t], qh[t]
            kl, ql = kt.norm(dim=-1)[:, None], qt.norm(dim=-1)[:, None]
            dec = at[..., None] * S
            D = D + dy[t][..., None] * qt[:, None, :]
            m = m + dy[t].abs() * ql
            dqh[t] = (dy[t][..., None] * (dec + u[..., None] * kt[:, None, :])).sum(1)
            after = at * ms + u.abs() * kl
            mq[t] = (dy[t].abs() * after).sum(-1)
            du = (D * kt[:, None, :]).sum(-1)
            dkh[t] = (u[..., None] * D).sum(1)
            db[t] = (du * r).sum(-1)
            mb[t] = (m * kl * r.abs()).sum(-1)
            tb[t] = (D * kt[:, None, :] * r[..., None]).norm(dim=(-1, -2))
            dv[t] = bt * du
            mv[t] = bt * m * kl
            dkh[t] -= (dv[t][..., None] * dec).sum(1)
            mk[t] = (u.abs() * m + mv[t] * at * ms).sum(-1)
            D = D - dv[t][..., None] * kt[:, None, :]
            e = e + LOCAL16 * (m + mv[t] * kl)
            m = m + mv[t] * kl
            dg[t] = (D * dec).sum((-1, -2))
            mg[t] = (m * at * ms).sum(-1)
            tg[t] = (D * dec).norm(dim=(-1, -2))
            D, m, e = at[..., None] * D, at * m, at * e
        d0[i], e0[i] = D, e
    per = H // groups

    def gather(d, mag, unit_, length, by):
        d, mag = d.unflatten(1, (groups, per)).sum(2) * by, mag.unflatten(1, (groups, per)).sum(2) * abs(by)
        return (d - unit_ * (d * unit_).sum(-1, keepdim=True)) / length[..., None], 2 * mag / length

    plain = bool((keep["qn"] == 1).all()) and bool((keep["kn"] == 1).all())
    if plain:
        dq, dk = dqh.unflatten(1, (groups, per)).sum(2) * scale, dkh.unflatten(1, (groups, per)).sum(2)
        mq, mk = mq.unflatten(1, (groups, per)).sum(2) * abs(scale), mk.unflatten(1, (groups, per)).sum(2)
    else:
        dq, mq = gather(dqh, mq, keep["qu"], keep["qn"], scale)
        dk, mk = gather(dkh, mk, keep["ku"], keep["kn"], 1.0)
    return dict(dq=(dq, mq[..., None]), dk=(dk, mk[..., None]), dv=(dv, mv), dg=(dg, mg), dbeta=(db, mb),
                dstate=(d0, e0[..., None]), terms=dict(dg=tg, dbeta=tb))


def within(got, value, slack, what):
    """Every element within the slack and the rounding of its own type."""
    g = got.detach().cpu()
    half = torch.finfo(g.dtype).eps / 2
    g = g.double()
    assert g.shape == value.shape, (what, g.shape, value.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    bound = slack * (1 + half) + half * value.abs() + 2.0 ** -126
    bad = (g - value).abs() > bound
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {at}: got {g[at].item()}, "
                             f"expected {value[at].item()} within {bound.expand(value.shape)[at].item()}")


def near(got, value, most, what, terms=None):
    """The 2-norm of the difference, relative to the values' own (with the terms' of values that are sums)."""
    g, n = got.detach().cpu().double(), float(value.norm())
    if terms is not None:
        n = math.hypot(n, float(terms.norm()))
    off = float((g - value).norm())
    assert off <= most * n, f"{what}: off by {off / n if n else off:.3g} of its norm, at most {most:.3g}"


def beam(logits, scores, finished, eos, out):
    """Every candidate sorted by value, beam, token."""
    B, b = scores.shape
    V = logits.shape[1]
    x = logits.double().view(B, b, V)
    value = scores.double()[:, :, None] + (x - torch.logsumexp(x, -1, keepdim=True))
    value = torch.where(torch.isnan(value), -float("inf"), value)
    if finished is not None:
        for i in range(B):
            for j in range(b):
                if finished[i, j]:
                    value[i, j] = -float("inf")
                    value[i, j, eos] = scores[i, j].double()
    flat = value.view(B, b * V)
    picked = [sorted(range(b * V), key=lambda c: (-flat[i, c].item(), c))[:out] for i in range(B)]
    at = torch.tensor(picked)
    return torch.gather(flat, 1, at), (at // V).int(), (at % V).int()
