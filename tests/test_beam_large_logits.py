"""Beam selection where the logits' own size must not matter: rows offset by thousands, each by another amount; masks of
the type's lowest value and of -1e9, over whole parts of a row and over all of it; the largest numbers there are.

The bound: a term's exponent is off by the roundings of x - m, of its product with log2(e) and of that constant, 3 U of
|x - m| at most, which is about 5 for the terms that carry the sum here (15 U, 64 U where one term of 1e4 draws stands
alone); the exponential by 4 U; the sum by at most 32 additions in a thread, 5 across its warp, 8 across the warps and
5 across the parts (50 U). So the log-sum-exp is off by less than 128 U, and the output is rounded once."""
import pytest
import torch

from tests import delta_ref as R
from tests.gpu_util import device
from tests.test_beam_gpu import BF16, F32, INF, draw, select

pytestmark = pytest.mark.gpu


def check(logits, scores, out, finished=None, eos=None):
    got = select(device(), logits, scores, finished, eos, out)
    value, parents, tokens = R.beam(logits, scores, finished, eos, out)
    assert torch.equal(got[1], parents) and torch.equal(got[2], tokens)
    live = torch.isfinite(value)
    assert torch.equal(torch.isfinite(got[0]), live)
    assert ((got[0].double() - value)[live].abs() <= 128 * R.U + R.U * value[live].abs()).all()
    return got[0]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e8])
def test_rows_that_are_offset(dtype, size):
    """Every row by another amount of about +-size. (The logits lie on the type's grid there; the reference takes them as
    they are.)"""
    logits, scores = draw(7, 2, 4, 5000, F32)
    by = torch.tensor([1.0, -0.93, 0.71, -1.13, 0.57, 1.21, -0.67, -1.0]) * size
    step = torch.finfo(dtype).eps * size  # (spread over the grid's steps, so that no row is ties alone)
    check(((logits * max(1.0, step)) + by[:, None]).to(dtype), scores, 4)


def test_a_certain_token():
    """One token far above the others: its log-probability is 0, from logits of any size. (The others are 1 770 below it
    and more: exp(-1770) is nothing in 64 bits.)"""
    for size in (1e3, 1e6, 1e9):
        logits = torch.full((2, 9000), -size)
        logits[0, 77], logits[1, 8500] = size * 1.37, size * 0.77
        got = check(logits, torch.tensor([[0.0, -0.5]]), 2)
        assert got.tolist() == [[0.0, -0.5]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mask", ["lowest", -1e9, -1e30])
def test_masks_of_a_finite_value(dtype, mask):
    """Tokens that are masked by the type's lowest number, or by a large negative one: everything behind the first tokens
    (whole parts of a row), everything before the last, and a row of them alone."""
    value = torch.finfo(dtype).min if mask == "lowest" else mask
    logits, scores = draw(9, 2, 3, 40000, dtype)
    logits[0, 50:] = value
    logits[1, :-50] = value
    logits[2] = value
    logits[3, ::2] = value
    logits[4, :17000] = value
    logits[5, 16000:] = value
    check(logits, scores, 6)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_largest_numbers(dtype):
    top = torch.finfo(dtype).max
    logits, scores = draw(11, 1, 4, 20000, dtype)
    logits[0, 19000] = top
    logits[1], logits[1, 3], logits[1, 18000] = -top, top, top
    logits[2, 5], logits[2, 6] = top, -top
    logits[3, 7] = -INF
    check(logits, scores, 4)
