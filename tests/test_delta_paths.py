"""The gated delta rule's bf16 kernels where batches are large enough for every form of them: more blocks of 16 state rows
than the SMs take with two warps each (one warp to 16 rows, four of them to a chunk's tiles, forwards and backwards), some
more than the SMs (two blocks a CTA), chunks and key groups that a CTA takes one after another (whole and partial ones in
turn, one and three heads a group), heads of a group that are made from one product of keys and queries. Outputs, end
states, checkpoints and every gradient against the 64-bit token loop. Most runs are short, so that it stays quick."""
import random

import pytest
import torch

import selective_scan_gb300 as ss
from tests import delta_ref as R
from tests.gpu_util import device
from tests.test_delta_gpu import BF16, EPS, NAN, cu_of, in_rows, inputs, poison, randn

pytestmark = pytest.mark.gpu


def short_runs(seed, n, longer, every=9):
    """n runs, most of a few tokens, every so-manieth of them one of `longer`."""
    rng = random.Random(seed)
    return [rng.choice((0, 1, 1, 1, 2, 2, 3, 5)) if i % every else rng.choice(longer) for i in range(n)]


def blocks(lengths, heads, headdim):
    return len(lengths) * heads * ((headdim + 15) // 16)


def chunks(lengths):
    return sum((n + 63) // 64 for n in lengths)


def check(seed, lengths, groups, heads, d_state, headdim, l2, pad=None):
    dev = device()
    q, k, v, g, beta, pool, slots, fresh = inputs(seed, lengths, groups, heads, d_state, headdim, BF16, l2)
    cu, rows, n, eps, by = cu_of(lengths), sum(lengths), len(lengths), EPS if l2 else None, d_state ** -0.5
    ref = R.forward(q, k, v, g, beta, pool, cu, slots, fresh, by, eps, R.LOCAL16)
    dy, ends = randn(seed + 8, rows, heads, headdim).to(BF16), randn(seed + 9, n, heads, headdim, d_state, std=0.3)
    want = R.backward(ref["keep"], cu, dy, ends, by, groups)
    gq, gk, gv, gdy, y, dq, dk, dv = in_rows([q, k, v, dy, torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k),
                                              torch.zeros_like(v)], dev, pad)
    gg, gb, st = g.to(dev), beta.to(dev), poison(pool, slots, fresh).to(dev)
    kept = torch.full((ss.gated_delta_rule_checkpoints(cu),) + pool.shape[1:], NAN, device=dev)
    at = torch.tensor(slots)
    others = torch.tensor([s for s in range(pool.shape[0]) if s not in slots])
    for checkpoints in (None, kept):  # (serving, then training)
        y.fill_(NAN)
        st.copy_(poison(pool, slots, fresh))
        ss.gated_delta_rule(y, gq, gk, gv, gg, gb, st, cu, slots, fresh, l2_eps=eps, checkpoints=checkpoints)
        torch.cuda.synchronize()
        # the state, the scores and the corrections may each be rounded to bf16 in what ends in y
        R.within(y, ref["y"], ref["yerr"] + 3 * R.HALF16 * ref["ymag"], "y")
        R.near(y, ref["y"], 4e-3, "y")
        R.within(st[at.to(dev)], ref["pool"][at], ref["perr"][at][..., None], "state")
        R.near(st[at.to(dev)], ref["pool"][at], 1e-5, "state")
        assert torch.isnan(st.cpu()[others]).all(), "a slot outside the batch was written"
    R.within(kept, ref["kept"], ref["kerr"][..., None], "checkpoints")
    dg, db = (torch.full((rows, heads), NAN, dtype=BF16, device=dev) for _ in range(2))
    ds = torch.full((n,) + pool.shape[1:], NAN, device=dev)
    ss.gated_delta_rule_backward(dq, dk, dv, dg, db, ds, gdy, ends.to(dev), gq, gk, gv, gg, gb, kept, cu, l2_eps=eps)
    torch.cuda.synchronize()
    R.within(ds, *want["dstate"], "dstate")
    R.near(ds, want["dstate"][0], 1e-5, "dstate")
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv), ("dg", dg), ("dbeta", db)):
        value, size = want[name]
        # at most eight operands one behind another are rounded to bf16; sums over a chunk in 32 bits (192 additions)
        R.within(t, value, 8 * R.HALF16 * size + (192 * R.U * size.amax() if name == "dg" else 0), name)
        R.near(t, value, 5.1e-3, name, want["terms"].get(name))


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("groups,heads,d_state,headdim", [(2, 8, 128, 128), (3, 9, 72, 104), (8, 8, 64, 128)])
def test_more_blocks_than_sms(groups, heads, d_state, headdim):
    device()
    lengths = [200, 64, 65]
    assert sms() < blocks(lengths, heads, headdim) <= 3 * sms()
    check(1, lengths, groups, heads, d_state, headdim, True)


@pytest.mark.parametrize("groups,heads,d_state,headdim,runs", [(2, 8, 128, 128, 10), (2, 6, 72, 104, 15), (4, 20, 64, 128, 5), (1, 5, 128, 40, 42)])
@pytest.mark.parametrize("l2", [True, False])
def test_blocks_enough_for_one_warp_each(groups, heads, d_state, headdim, runs, l2):
    device()
    lengths = ([130, 64, 1, 70, 3, 128, 65, 200, 0, 2] * 5)[:runs] if runs <= 15 else short_runs(3, runs, (64, 65, 130))
    assert blocks(lengths, heads, headdim) >= 4 * sms()
    check(2, lengths, groups, heads, d_state, headdim, l2)


@pytest.mark.parametrize("groups,heads,d_state,headdim", [(6, 6, 128, 40), (4, 12, 80, 72), (16, 16, 64, 16)])
def test_chunks_that_a_cta_takes_one_after_another(groups, heads, d_state, headdim):
    device()
    lengths = [64, 1, 130, 5, 65, 128, 2, 64] * 4 + short_runs(4, 70, (64, 66, 128))
    assert chunks(lengths) * groups > 2 * sms()
    check(5, lengths, groups, heads, d_state, headdim, True, pad=8)


@pytest.mark.parametrize("groups,heads,d_state,headdim,several", [(1, 8, 128, 16, 8), (2, 6, 64, 24, 3), (2, 4, 120, 16, 2), (1, 5, 40, 8, 5)])
def test_heads_of_a_group_from_one_product(groups, heads, d_state, headdim, several):
    device()
    lengths = short_runs(6, 560, (64, 65, 128), every=60) + [64] * 8
    fits = [d for d in range(1, 9) if heads // groups % d == 0 and chunks(lengths) * (heads // d) >= 3 * sms()]
    assert max(fits) == several
    check(7, lengths, groups, heads, d_state, headdim, True)
