"""Beam search over more pools than one call of the library reorders (a convolution and a state pool of each of many
layers): all of them move, and what cannot be moved is refused before anything has been."""
import re
from pathlib import Path

import pytest
import torch

import selective_scan_gb300 as ss
from selective_scan_gb300.beams import Beams
from tests import delta_ref as R
from tests.gpu_util import device

F32 = torch.float32


class Recorder:
    """The library, but for the reordering, which is recorded."""

    def __init__(self, lib, fail_at=None):
        self.lib, self.calls, self.fail_at = lib, [], fail_at

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def mamba2_reorder_states(self, pools, sizes, n, num_slots, slots, parents, batch, beams, status, stream):
        self.calls.append((list(pools)[:n], list(sizes)[:n], num_slots, batch, beams, status))
        return ss.ERR_CUDA if len(self.calls) - 1 == self.fail_at else ss.OK


def orders(batch=2, beams=3):
    order = torch.arange(batch * beams, dtype=torch.int32).view(batch, beams)
    return order, torch.zeros_like(order), torch.zeros(1, dtype=torch.int32)


def test_the_constant_is_the_headers():
    text = (Path(ss.__file__).resolve().parent.parent / "include" / "beam.h").read_text()
    assert int(re.search(r"#define MAMBA2_MAX_POOLS (\d+)", text).group(1)) == ss.MAX_POOLS


@pytest.mark.parametrize("n", [0, 1, 64, 65, 128, 200])
def test_pools_are_split_over_calls(product_lib, monkeypatch, n):
    lib = Recorder(product_lib)
    monkeypatch.setattr(ss, "_lib", lambda: lib)
    pools = [torch.zeros((9, 1 + i % 5)) for i in range(n)]
    slots, parents, status = orders()
    assert ss.reorder_states(pools, slots, parents, status, stream=0) == ss.OK
    assert [len(c[0]) for c in lib.calls] == ([64] * (n // 64) + ([n % 64] if n % 64 else []) or [0])
    assert [p for c in lib.calls for p in c[0]] == [t.data_ptr() for t in pools]
    assert [s for c in lib.calls for s in c[1]] == [t.nbytes // 9 for t in pools]
    assert all(c[3:] == (2, 3, status.data_ptr()) for c in lib.calls)


def test_a_call_that_fails_ends_them(product_lib, monkeypatch):
    lib = Recorder(product_lib, fail_at=1)
    monkeypatch.setattr(ss, "_lib", lambda: lib)
    slots, parents, status = orders()
    assert ss.reorder_states([torch.zeros((9, 4)) for _ in range(200)], slots, parents, status, stream=0, check=False) == ss.ERR_CUDA
    assert len(lib.calls) == 2


@pytest.mark.parametrize("at", [(0, 64), (3, 150), (100, 101)])
def test_pools_of_different_calls_that_overlap(product_lib, monkeypatch, at):
    """One pool twice, or two that share bytes, would be moved twice, whichever calls they are in."""
    lib = Recorder(product_lib)
    monkeypatch.setattr(ss, "_lib", lambda: lib)
    slots, parents, status = orders()
    room = torch.zeros(13 * 4)
    for second in (room[:36].view(9, 4), room[16:].view(9, 4)):
        pools = [torch.zeros((9, 4)) for _ in range(200)]
        pools[at[0]], pools[at[1]] = room[:36].view(9, 4), second
        with pytest.raises(ss.Mamba2Error):
            ss.reorder_states(pools, slots, parents, status, stream=0)
    assert not lib.calls


def test_beams_refuse_what_no_step_could_take(product_lib):
    """When they are made, not after a step has chosen its tokens."""
    slots = orders()[0]
    pool = torch.zeros((9, 4))
    many = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    for s, pools in ((slots, [pool, pool]), (slots, [pool, pool[:8]]), (slots, [pool[:, ::2]]), (slots.long(), [pool]),
                     (many(1, 33), [pool]), (many(257, 4), [pool]), (slots[0], [pool])):
        with pytest.raises(ValueError):
            Beams(s, pools)
    Beams(slots, [torch.zeros((9, 4)) for _ in range(150)])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [65, 130])
def test_reordering_of_many_pools(n):
    dev = device()
    g = torch.Generator().manual_seed(n)
    pools = [torch.randint(0, 200, (11, 1 + i % 7, 4), generator=g).to((F32, torch.uint8, torch.bfloat16)[i % 3]) for i in range(n)]
    slots = torch.randperm(11, generator=g)[:8].view(2, 4).int()
    for parents, want in ((torch.randint(0, 4, (2, 4), generator=g).int(), ss.OK), (torch.full((2, 4), 4).int(), ss.ERR_INVALID_ARGUMENT)):
        got = [p.to(dev) for p in pools]
        status = torch.full((1,), -1, dtype=torch.int32, device=dev)
        ss.reorder_states(got, slots.to(dev), parents.to(dev), status)
        torch.cuda.synchronize()
        assert int(status) == want
        for old, new in zip(pools, got):
            moved = old.clone()
            if want == ss.OK:
                for row, up in zip(slots.tolist(), parents.tolist()):
                    for s, p in zip(row, up):
                        moved[s] = old[row[p]]
            assert torch.equal(new.cpu(), moved)


@pytest.mark.gpu
def test_a_search_over_many_layers():
    """Two steps of a search whose states are in 70 pools: every pool follows the beams."""
    dev = device()
    slots = torch.tensor([[4, 1, 0], [2, 6, 5]], dtype=torch.int32)
    pools = [torch.randn((7, 3 + i % 4), generator=torch.Generator().manual_seed(i)) for i in range(70)]
    search = Beams(slots.to(dev), [p.to(dev) for p in pools])
    logits = torch.randn((2, 6, 50), generator=torch.Generator().manual_seed(99))
    scores = torch.tensor([[0.0, -float("inf"), -float("inf")]] * 2)
    for step in range(2):
        search.advance(logits[step].to(dev))
        torch.cuda.synchronize()
        value, parents, tokens = R.beam(logits[step], scores, None, None, 3)
        scores = value.float()
        assert int(search.status) == ss.OK
        assert torch.equal(search.parents.cpu(), parents) and torch.equal(search.tokens.cpu(), tokens)
        old = [p.clone() for p in pools]
        for b in range(2):
            for j in range(3):
                for p, was in zip(pools, old):
                    p[slots[b, j]] = was[slots[b, parents[b, j]]]
        for p, got in zip(pools, search.pools):
            assert torch.equal(got.cpu(), p)
