"""The gradient of a decay that leaves nothing of the state is 0: no term of it remains, whatever the chunk's others are
(dg_t is made of what comes before t and is read behind it, and of that alone)."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests import delta_ref as R
from tests.gpu_util import device
from tests.test_delta_gpu import BF16, EPS, cu_of, inputs, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,heads,d_state,headdim", [(1, 2, 128, 128), (2, 2, 64, 64), (1, 3, 72, 104)])
@pytest.mark.parametrize("every,first", [(7, 0), (16, 0), (16, 15), (29, 3), (2, 1)])
def test_forgetting_tokens(groups, heads, d_state, headdim, every, first):
    dev, lengths = device(), [150, 64, 5]
    cu, rows, n = cu_of(lengths), sum(lengths), len(lengths)
    q, k, v, g, beta, pool, slots, _ = inputs(23, lengths, groups, heads, d_state, headdim, BF16, True)
    g = g * 0.05
    g[first::every] = -30000.0
    v = (v.float() * 100).to(BF16)
    fwd = R.forward(q, k, v, g, beta, pool, cu, slots, [0] * n, d_state ** -0.5, EPS, R.LOCAL16)
    dy, ends = randn(24, rows, heads, headdim).to(BF16), randn(25, n, heads, headdim, d_state, std=0.3)
    want, size = R.backward(fwd["keep"], cu, dy, ends, d_state ** -0.5, groups)["dg"]
    gin = [t.to(dev) for t in (q, k, v, g, beta)]
    kept = torch.empty((ss.gated_delta_rule_checkpoints(cu),) + pool.shape[1:], device=dev)
    ss.gated_delta_rule(torch.empty_like(gin[2]), *gin, pool.to(dev), cu, slots, [0] * n, l2_eps=EPS, checkpoints=kept)
    out = [torch.empty_like(t) for t in gin[:3]] + [torch.empty((rows, heads), dtype=BF16, device=dev) for _ in range(2)]
    ss.gated_delta_rule_backward(*out, None, dy.to(dev), ends.to(dev), *gin, kept, cu, l2_eps=EPS)
    torch.cuda.synchronize()
    dg = out[3].cpu()
    assert (want[first::every] == 0).all()
    assert (dg[first::every] == 0).all(), dg[first::every].abs().max()
    # eight operands one behind another in bf16, of what this token's own terms add up to: nothing of the chunk's others
    R.within(dg, want, 8 * R.HALF16 * size, "dg")
