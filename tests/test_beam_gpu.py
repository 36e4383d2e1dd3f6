"""Beam search's selection against a sort of every candidate in 64 bits, and the reordering of state pools: ties, masked
tokens and rows, dead and finished beams, infinities and NaN, one beam and the most, vocabularies of one token and of
sizes that fill no vector, unaligned rows; permutations, one parent for all, slots of odd sizes, several pools at once."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests import delta_ref as R
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def select(dev, logits, scores, finished, eos, out, ld=None, off=0):
    """On the GPU, with the logits as a column range where ld is given."""
    B = scores.shape[0]
    x = logits.to(dev)
    if ld is not None:
        wide = torch.full((logits.shape[0], ld), INF, dtype=logits.dtype, device=dev)
        wide[:, off:off + logits.shape[1]] = x
        x = wide[:, off:off + logits.shape[1]]
    got = [torch.full((B, out), -7, dtype=t, device=dev) for t in (F32, torch.int32, torch.int32, torch.uint8)]
    ss.beam_select(*got[:3], x, scores.to(dev), finished=finished.to(dev) if finished is not None else None,
                   finished_out=got[3] if eos is not None else None, eos=eos)
    torch.cuda.synchronize()
    return [t.cpu() for t in got]


def check(dev, logits, scores, finished, eos, out, **kw):
    got = select(dev, logits, scores, finished, eos, out, **kw)
    value, parents, tokens = R.beam(logits, scores, finished, eos, out)
    assert torch.equal(got[1], parents) and torch.equal(got[2], tokens)
    # an fp32 sum of exponentials (relative 2^-24 for each of its roundings, 64 at most one behind another, and the
    # exponents' own), and the output's rounding
    live = torch.isfinite(value)
    assert torch.equal(torch.isfinite(got[0]), live)
    assert ((got[0].double() - value)[live].abs() <= 256 * R.U + R.U * value[live].abs()).all()
    if eos is not None:
        was = torch.gather(finished, 1, parents.long()) if finished is not None else torch.zeros_like(got[3])
        assert torch.equal(got[3], ((was != 0) | (tokens == eos)).to(torch.uint8))


def draw(seed, B, beams, vocab, dtype, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((B * beams, vocab), generator=g) * 2.5
    logits[torch.rand((B * beams, vocab), generator=g) < masked] = -INF
    return logits.to(dtype), -torch.rand((B, beams), generator=g) * 5


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,beams,out,vocab", [(1, 1, 1, 1), (1, 1, 1, 1000), (2, 4, 4, 777), (1, 3, 6, 5000), (3, 32, 32, 130), (2, 2, 32, 31),
                                               (1, 2, 2, 40001), (70, 5, 5, 64)])
def test_selection(dtype, B, beams, out, vocab):
    dev = device()
    logits, scores = draw(vocab + B, B, beams, vocab, dtype)
    check(dev, logits, scores, None, None, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ld,off", [(1003, 0), (1011, 1), (1012, 3), (1016, 8), (1020, 6)])
def test_rows_of_any_alignment(dtype, ld, off):
    dev = device()
    logits, scores = draw(ld, 2, 3, 1003, dtype)
    check(dev, logits, scores, None, None, 3, ld=ld, off=off)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ties(dtype):
    """Equal logits in a row go by token; rows and scores alike go by beam."""
    dev = device()
    logits = torch.zeros((6, 5000))
    logits[:, 4000::3] = 1.0
    logits[3] = 2.0
    check(dev, logits.to(dtype), torch.zeros((2, 3)), None, None, 8)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("out", [3, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("order", ["falling", "rising", "one lane", "few", "none but one vector's"])
def test_logits_in_order(dtype, out, order):
    """A bound that is taken from groups of threads: the largest all in a few of them, or most of them without any."""
    dev, vocab = device(), 20000
    base = torch.linspace(4, -4, vocab).to(dtype).float()  # (bf16: hundreds alike)
    if order == "rising":
        base = base.flip(0)
    elif order == "one lane":
        base[torch.arange(vocab) // 8 % 32 == 5] += 20.0
    elif order == "few":
        base[torch.arange(vocab) % 700 != 3] = -INF
    elif order == "none but one vector's":
        base[16:] = -INF
    logits = base.expand(4, vocab).clone()
    logits[1] = logits[1].roll(4321)
    check(dev, logits.to(dtype), torch.tensor([[0.0, -1.0], [-0.5, -0.5]]), None, None, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masks_dead_beams_and_values_that_are_no_numbers(dtype):
    dev = device()
    logits, scores = draw(5, 5, 4, 300, dtype, masked=0.3)
    logits[0] = -INF                              # nothing may follow
    logits[4:8, 7:] = -INF                        # fewer tokens than are asked for
    scores[2, 1:] = -INF                          # beams that are not yet in being
    scores[3] = -INF                              # no candidate at all
    logits[16, 100], logits[17, 5], logits[18, 0] = NAN, INF, torch.finfo(dtype).min
    check(dev, logits, scores, None, None, 16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_finished_beams(dtype):
    dev = device()
    logits, scores = draw(6, 4, 5, 900, dtype, masked=0.05)
    logits[3] = NAN
    finished = torch.zeros((4, 5), dtype=torch.uint8)
    finished[0, 3], finished[1], finished[2, 0] = 1, 1, 1
    for eos in (0, 3, 899):
        check(dev, logits, scores, finished, eos, 10)
    check(dev, logits, scores, None, 17, 5)


def test_selection_of_no_sequence():
    dev = device()
    got = [torch.empty((0, 2), dtype=t, device=dev) for t in (F32, torch.int32, torch.int32)]
    ss.beam_select(*got, torch.empty((0, 9), device=dev), torch.empty((0, 3), device=dev))
    torch.cuda.synchronize()


def reorder(dev, pools, slots, parents):
    got = [p.to(dev) for p in pools]
    status = torch.full((1,), -1, dtype=torch.int32, device=dev)
    ss.reorder_states(got, slots.to(dev), parents.to(dev), status)
    torch.cuda.synchronize()
    return [p.cpu() for p in got], int(status)


def expected(pools, slots, parents):
    out = [p.clone() for p in pools]
    for old, new in zip(pools, out):
        for row, up in zip(slots.tolist(), parents.tolist()):
            for s, p in zip(row, up):
                new[s] = old[row[p]]
    return out


@pytest.mark.parametrize("B,beams", [(1, 1), (1, 2), (3, 4), (2, 7), (40, 8), (5, 16), (32, 32)])
@pytest.mark.parametrize("shapes", [[((4, 16), F32)], [((3, 24), BF16), ((2, 8, 8), F32), ((5,), torch.uint8), ((1100, 5), BF16)], [((3, 1), F32), ((0,), F32)]],
                         ids=["one", "mixed", "words"])
def test_reordering(B, beams, shapes):
    dev = device()
    g = torch.Generator().manual_seed(B * beams)
    n = B * beams + 5
    pools = [torch.randint(0, 200, (n,) + s, generator=g).to(t) for s, t in shapes]
    slots = torch.randperm(n, generator=g)[:B * beams].view(B, beams).int()
    for parents in (torch.randint(0, beams, (B, beams), generator=g), torch.arange(beams).flip(0).expand(B, beams),
                    torch.arange(beams).roll(1).expand(B, beams), torch.full((B, beams), beams - 1),
                    torch.arange(beams).expand(B, beams)):
        parents = parents.int().contiguous()
        got, status = reorder(dev, pools, slots, parents)
        assert status == ss.OK
        for a, b in zip(got, expected(pools, slots, parents)):
            assert torch.equal(a, b)


def test_reordering_of_pools_that_start_anywhere():
    dev = device()
    g = torch.Generator().manual_seed(8)
    base = torch.randint(0, 250, (4096,), generator=g).to(torch.uint8)
    slots, parents = torch.tensor([[2, 0, 3]]).int(), torch.tensor([[1, 2, 2]]).int()
    for off, size in ((1, 48), (4, 52), (16, 64), (2, 33)):
        buf = base.to(dev)
        pool = buf[off:off + 5 * size].view(5, size)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        ss.reorder_states([pool], slots.to(dev), parents.to(dev), status)
        torch.cuda.synchronize()
        want = base.clone()
        want[off:off + 5 * size] = expected([base[off:off + 5 * size].view(5, size)], slots, parents)[0].flatten()
        assert int(status) == ss.OK and torch.equal(buf.cpu(), want)


@pytest.mark.parametrize("B", [2, 100])
def test_bad_orders_are_reported_and_touch_nothing(B):
    dev = device()
    beams = 4
    n = B * beams
    pool = torch.arange(n * 8, dtype=F32).view(n, 8)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(1)).view(B, beams).int()
    parents = torch.arange(beams).flip(0).expand(B, beams).int().contiguous()

    def with_(t, value):
        t = t.clone()
        t[B - 1, 2] = value
        return t

    for s, p, want in ((with_(slots, -1), parents, ss.ERR_SLOT_OUT_OF_RANGE), (with_(slots, n), parents, ss.ERR_SLOT_OUT_OF_RANGE),
                       (with_(slots, int(slots[0, 0])), parents, ss.ERR_SLOT_SHARED), (slots, with_(parents, -1), ss.ERR_INVALID_ARGUMENT),
                       (slots, with_(parents, beams), ss.ERR_INVALID_ARGUMENT)):
        got, status = reorder(dev, [pool], s, p)
        assert status == want
        assert_bits_equal(got[0], pool, "pool")


def test_reordering_of_nothing():
    dev = device()
    status = torch.full((1,), -1, dtype=torch.int32, device=dev)
    ss.reorder_states([torch.ones((3, 4), device=dev)], torch.empty((0, 2), dtype=torch.int32, device=dev),
                      torch.empty((0, 2), dtype=torch.int32, device=dev), status)
    assert int(status) == ss.OK
    status.fill_(-1)
    ss.reorder_states([], torch.zeros((0, 1), dtype=torch.int32, device=dev), torch.zeros((0, 1), dtype=torch.int32, device=dev), status)
    assert int(status) == ss.OK
