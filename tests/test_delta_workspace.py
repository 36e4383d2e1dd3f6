"""What a workspace holds before a call does not matter: the results with one of ones in every bit (NaN in every type) are,
bit for bit, those with zeros; shapes that fill no tile, runs that fill no chunk."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("groups,heads,d_state,headdim", [(1, 2, 8, 8), (2, 2, 40, 24), (1, 1, 72, 104), (3, 3, 128, 40), (1, 20, 64, 128),
                                                          (2, 80, 24, 128), (1, 3, 120, 56)])
@pytest.mark.parametrize("lengths", [(1,), (63, 0, 66), (130, 7, 64, 1)], ids=str)
def test_delta_rule(groups, heads, d_state, headdim, lengths):
    dev, n = device(), len(lengths)
    cu = [sum(lengths[:i]) for i in range(n + 1)]
    rows, gen = cu[-1], torch.Generator().manual_seed(heads + d_state)
    r = lambda *s: torch.randn(s, generator=gen).to(dev)  # noqa: E731
    q, k, v, dy = r(rows, groups, d_state).to(BF16), r(rows, groups, d_state).to(BF16), r(rows, heads, headdim).to(BF16), r(rows, heads, headdim).to(BF16)
    g, beta, ends = -r(rows, heads).abs() * 0.2, torch.sigmoid(r(rows, heads)), r(n, heads, headdim, d_state)
    start, results = r(n, heads, headdim, d_state), []
    for fill in (0, 0xff):
        ws = [torch.full((max(1, ss.gated_delta_rule_workspace_bytes(cu, heads, headdim, d_state, groups, BF16, backward=b)),), fill,
                         dtype=torch.uint8, device=dev) for b in (False, True)]
        y, pool = torch.empty_like(v), start.clone()
        kept = torch.empty((ss.gated_delta_rule_checkpoints(cu), heads, headdim, d_state), device=dev)
        ss.gated_delta_rule(y, q, k, v, g, beta, pool, cu, list(range(n)), [0] * n, l2_eps=1e-6, checkpoints=kept, workspace=ws[0])
        out = [torch.empty_like(t) for t in (q, k, v)] + [torch.empty((rows, heads), dtype=BF16, device=dev) for _ in range(2)] + [torch.empty_like(start)]
        ss.gated_delta_rule_backward(*out, dy, ends, q, k, v, g, beta, kept, cu, l2_eps=1e-6, workspace=ws[1])
        results.append([y, pool, kept] + out)
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert torch.isfinite(a.float()).all()
        assert_bits_equal(a, b, "a workspace's content")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,beams,out,vocab", [(1, 1, 1, 3), (2, 3, 7, 40001), (40, 8, 8, 9001), (1, 32, 32, 300000)])
def test_beam_selection(dtype, batch, beams, out, vocab):
    dev, gen = device(), torch.Generator().manual_seed(vocab)
    logits, scores = torch.randn((batch * beams, vocab), generator=gen).to(dev, dtype), -torch.rand((batch, beams), generator=gen).to(dev)
    finished = (torch.rand((batch, beams), generator=gen) < 0.3).to(dev, torch.uint8)
    results = []
    for fill in (0, 0xff):
        need = int(ss.library().mamba2_beam_select_workspace_bytes(batch, beams, out, vocab))
        got = [torch.empty((batch, out), dtype=t, device=dev) for t in (F32, torch.int32, torch.int32, torch.uint8)]
        ss.beam_select(*got[:3], logits, scores, finished=finished, finished_out=got[3], eos=2,
                       workspace=torch.full((need,), fill, dtype=torch.uint8, device=dev))
        results.append(got)
    torch.cuda.synchronize()
    for a, b in zip(*results):
        assert_bits_equal(a, b, "a workspace's content")
