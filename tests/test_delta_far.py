"""The delta rule and the reordering where offsets pass 32 bits: rows a megaelement apart, and slots at the end of a pool of
more than 2^31 elements. The results are, bit for bit, those of the same values close together."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HEADS, GROUPS, DK, DV = 2, 1, 64, 48
CU = [0, 70, 70, 2150]  # rows of 2^20 + 8 elements: the last begin past 2^31


def inputs(dev, rows, dtype):
    g = torch.Generator().manual_seed(rows)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k, v = r(rows, GROUPS, DK).to(dev, dtype), r(rows, GROUPS, DK).to(dev, dtype), r(rows, HEADS, DV).to(dev, dtype)
    return q, k, v, (-torch.rand((rows, HEADS), generator=g) * 0.3).to(dev), torch.rand((rows, HEADS), generator=g).to(dev)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_far_apart(dtype):
    dev, rows = device(), CU[-1]
    q, k, v, g, beta = inputs(dev, rows, dtype)
    far = torch.empty((rows, (1 << 20) + 8), dtype=dtype, device=dev)
    out = torch.empty_like(far)
    cut = lambda t, at, like: t[:, at:at + like.shape[1] * like.shape[2]].unflatten(1, like.shape[1:])  # noqa: E731
    columns = (512, 100000, (1 << 20) - 400)
    wide, results = [cut(far, at, t) for at, t in zip(columns, (q, k, v))], []
    for t, w in zip((q, k, v), wide):
        w.copy_(t)
    near_out = [torch.empty_like(t) for t in (v, q, k, v)]
    far_out = [cut(out, at, t) for at, t in zip((0, 1024, 90000, (1 << 20) - 256), near_out)]
    for (a, b, c), (y, dq, dk, dv) in (((q, k, v), near_out), (wide, far_out)):
        pool = torch.zeros((3, HEADS, DV, DK), device=dev)
        kept = torch.empty((ss.gated_delta_rule_checkpoints(CU), HEADS, DV, DK), device=dev)
        ss.gated_delta_rule(y, a, b, c, g, beta, pool, CU, [0, 1, 2], [1, 1, 1], l2_eps=1e-6, checkpoints=kept)
        results.append([y.contiguous(), pool, kept])
        if dtype == BF16:
            dg, dbeta = (torch.empty((rows, HEADS), dtype=dtype, device=dev) for _ in range(2))
            ss.gated_delta_rule_backward(dq, dk, dv, dg, dbeta, None, c, None, a, b, c, g, beta, kept, CU, l2_eps=1e-6)
            results[-1] += [t.contiguous() for t in (dq, dk, dv)] + [dg, dbeta]
    torch.cuda.synchronize()
    for near, there in zip(*results):
        assert torch.isfinite(near.float()).all()
        assert_bits_equal(near.cpu(), there.cpu(), "far apart")


def test_slots_far_apart():
    dev, slots = device(), (1 << 31) // (HEADS * DV * DK) + 7
    q, k, v, g, beta = inputs(dev, 4, F32)
    pool, near = torch.empty((slots, HEADS, DV, DK), device=dev), torch.empty((4, HEADS, DV, DK), device=dev)
    there = [slots - 1, slots - 3, slots - 4, 0]
    start = torch.randn(near.shape, generator=torch.Generator().manual_seed(1)).to(dev)
    i32 = lambda *s: torch.tensor(s, dtype=torch.int32, device=dev)  # noqa: E731
    n, status, results = i32(4), i32(0), []
    for p, at in ((near, [0, 1, 2, 3]), (pool, there)):
        p[at] = start
        ys = [torch.empty_like(v) for _ in range(3)]
        ss.gated_delta_rule_step(ys[0], q, k, v, g, beta, p, at, [0] * 4)
        ss.gated_delta_rule_step_device(ys[1], q, k, v, g, beta, p, i32(*at), None, n, status)
        ss.gated_delta_rule(ys[2], q, k, v, g, beta, p, [0, 1, 2, 3, 4], at, [0] * 4)
        ss.reorder_states([p], i32(*at).view(2, 2), i32(1, 0, 1, 1).view(2, 2), status)
        results.append(ys + [p[at]])
    torch.cuda.synchronize()
    assert status.item() == ss.OK
    for a, b in zip(*results):
        assert torch.isfinite(a).all()
        assert_bits_equal(a.cpu(), b.cpu(), "slots far apart")
