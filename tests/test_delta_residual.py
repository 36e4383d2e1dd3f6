"""Gradients where the state predicts the values well, as it does once it has learnt them: v is what the state gives for
the key plus a residual of a small part of its size. u and the gradients of beta and of the keys are proportional to that
residual, a difference of two numbers many times its size, so it has to come from operands of more digits than bf16's."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests import delta_ref as R
from tests.gpu_util import device
from tests.test_delta_gpu import BF16, EPS, cu_of, inputs, randn

pytestmark = pytest.mark.gpu


def predicted(q, k, v, g, beta, pool, cu, slots, residual, repeat):
    """v_t = a_t S_{t-1} k_t plus `residual` of its size; with `repeat`, the keys of a run are 16 in turn, and its values
    those that go with them (so that it is the run itself that teaches them)."""
    k = k.clone()
    per = v.shape[1] // k.shape[1]
    if repeat:
        for i in range(len(slots)):
            for t in range(cu[i] + 16, cu[i + 1]):
                k[t] = k[t - 16]
    kh = R.unit(k, EPS)[0].repeat_interleave(per, 1)
    noise, v = randn(99, *v.shape).double(), v.clone()
    for i, s in enumerate(slots):
        S = pool[s].double()
        for t in range(cu[i], cu[i + 1]):
            S = torch.exp(g[t].double())[:, None, None] * S
            p = (S * kh[t][:, None, :]).sum(-1)
            if not repeat:
                v[t] = (p + residual * noise[t] * p.norm(dim=-1, keepdim=True) * p.shape[-1] ** -0.5).to(BF16)
            elif t >= cu[i] + 16:
                was = v[t - 16].double()
                v[t] = (was + residual * noise[t] * was.norm(dim=-1, keepdim=True) * was.shape[-1] ** -0.5).to(BF16)
            S = S + (beta[t].double()[:, None] * (v[t].double() - p))[..., None] * kh[t][:, None, :]
    return k, v


@pytest.mark.parametrize("groups,heads,d_state,headdim", [(1, 2, 128, 128), (2, 2, 64, 64), (1, 3, 72, 104), (2, 4, 40, 128)])
@pytest.mark.parametrize("residual,repeat", [(0.1, False), (0.03, False), (0.01, False), (0.003, False), (0.01, True)])
def test_gradients(groups, heads, d_state, headdim, residual, repeat):
    dev, lengths, N = device(), [150, 64, 5], d_state
    cu, rows, n = cu_of(lengths), sum(lengths), len(lengths)
    q, k, v, g, beta, pool, slots, _ = inputs(17, lengths, groups, heads, d_state, headdim, BF16, True)
    g = g * 0.02
    if repeat:
        beta = 1.0 - 0.05 * beta  # (a key's value is all but learnt the first time)
    k, v = predicted(q, k, v, g, beta, pool, cu, slots, residual, repeat)
    ref = R.forward(q, k, v, g, beta, pool, cu, slots, [0] * n, N ** -0.5, EPS, R.LOCAL16)
    dy, ends = randn(18, rows, heads, headdim).to(BF16), randn(19, n, heads, headdim, d_state, std=0.3)
    want = R.backward(ref["keep"], cu, dy, ends, N ** -0.5, groups)
    gin = [t.to(dev) for t in (q, k, v, g, beta)]
    kept = torch.empty((ss.gated_delta_rule_checkpoints(cu),) + pool.shape[1:], device=dev)
    ss.gated_delta_rule(torch.empty_like(gin[2]), *gin, pool.to(dev), cu, slots, [0] * n, l2_eps=EPS, checkpoints=kept)
    out = [torch.empty_like(t) for t in gin[:3]] + [torch.empty((rows, heads), dtype=BF16, device=dev) for _ in range(2)]
    ss.gated_delta_rule_backward(*out, None, dy.to(dev), ends.to(dev), *gin, kept, cu, l2_eps=EPS)
    torch.cuda.synchronize()
    off = {}
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta"), out):
        value, terms = want[name][0], want["terms"].get(name)
        if name == "dbeta" and repeat:  # (of the tokens whose key the run has taught: the others' r is as large as v)
            at = torch.tensor([j for i in range(n) for j in range(cu[i] + 16, cu[i + 1])])
            t, value, terms = t[at.to(dev)], value[at], terms[at]
        norm = float(value.norm()) if terms is None else (float(value.norm()) ** 2 + float(terms.norm()) ** 2) ** 0.5
        off[name] = float((t.cpu().double() - value).norm()) / norm
    # 1.7e-3 a bf16 rounding (rms), eight of them and the output's own, all relative to r; r itself comes from checkpoints
    # that are 2e-6 of the state off (1e-5 at most, above), which is 3.3e-3 of a residual of 0.003 at most
    assert all(v <= 5.1e-3 + (1e-5 / residual if name == "dbeta" else 0) for name, v in off.items()), off
