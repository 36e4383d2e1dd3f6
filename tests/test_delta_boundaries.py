"""A batch's cu_seqlens may have more boundaries than the batch has runs (an array of a fixed size, say): those behind are
not looked at, by the workspace and the checkpoints neither."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests.gpu_util import device
from tests.test_delta_gpu import BF16, EPS, inputs
from tests.util import assert_bits_equal

EXACT = [0, 70, 70, 135]


class Library:
    """The library, but for the forward call."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def mamba2_gated_delta_rule(self, *args):
        return ss.OK


@pytest.mark.parametrize("behind", [[0, 0], [500], [7, 1 << 30, 3]], ids=str)
def test_workspace_and_checkpoints_are_the_runs(product_lib, monkeypatch, behind):
    lib, sizes = Library(product_lib), []
    monkeypatch.setattr(ss, "_lib", lambda: lib)
    monkeypatch.setattr(ss, "_workspace", lambda need, *_: (sizes.append(need) or 256, need, None))
    q, k, v, g, beta, pool, slots, fresh = inputs(3, [70, 0, 65], 1, 2, 64, 48, BF16, True)
    kept = torch.empty((4,) + pool.shape[1:])
    for cu in (EXACT, EXACT + behind):
        ss.gated_delta_rule(torch.empty_like(v), q, k, v, g, beta, pool, cu, slots, fresh, checkpoints=kept, stream=0)
        with pytest.raises(ValueError):
            ss.gated_delta_rule(torch.empty_like(v), q, k, v, g, beta, pool, cu, slots, fresh, checkpoints=kept[:3], stream=0)
    assert sizes[0] > 0 and sizes[0] == sizes[1]


@pytest.mark.gpu
def test_more_boundaries_than_runs():
    dev = device()
    q, k, v, g, beta, pool, slots, fresh = inputs(3, [70, 0, 65], 1, 2, 64, 48, BF16, True)
    args, results = [t.to(dev) for t in (q, k, v, g, beta)], []
    for cu in (EXACT, EXACT + [0, 0], EXACT + [1 << 30]):
        y, st, kept = torch.empty_like(args[2]), pool.to(dev), torch.empty((4,) + pool.shape[1:], device=dev)
        ss.gated_delta_rule(y, *args, st, cu, slots, fresh, l2_eps=EPS, checkpoints=kept)
        results.append([y, st, kept])
    torch.cuda.synchronize()
    for r in results[1:]:
        for a, b in zip(r, results[0]):
            assert_bits_equal(a.cpu(), b.cpu(), "the same runs")
