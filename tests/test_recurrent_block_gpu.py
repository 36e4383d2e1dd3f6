"""The recurrent block's kernels against 64-bit references (tests/block_ref.py), at the sizes where they can go
wrong: runs of no token, of one, around a checkpoint and over many; odd widths, column ranges and misaligned
rows; saturated gates; rows of zeros and of non-finite values; few rows and ragged tiles."""
import pytest
import torch

import selective_scan_gb300 as ss
from tests import block_ref as R
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN = float("nan")


def randn(seed, *shape, std=1.0, mean=0.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std + mean


def to_dev(t, dev, off=0, extra=0):
    """On the GPU as a column range that starts `off` elements into rows `extra` wider (0, 0: contiguous)."""
    if off == 0 and extra == 0:
        return t.to(dev)
    wide = torch.full((t.shape[0], t.shape[1] + extra), NAN, dtype=t.dtype, device=dev)
    wide[:, off:off + t.shape[1]] = t.to(dev)
    return wide[:, off:off + t.shape[1]]


def cu_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def rec_inputs(seed, lengths, dim, dtype, lower):
    rows = sum(lengths)
    x = randn(seed, rows, dim).to(dtype)
    gate = randn(seed + 1, rows, dim, std=1.5, mean=1.5).to(dtype)
    lo = torch.rand(dim, generator=torch.Generator().manual_seed(seed + 2)) * 0.9 if lower else None
    n = len(lengths)
    slots = torch.randperm(n + 3, generator=torch.Generator().manual_seed(seed + 3))[:n].tolist()
    fresh = [(seed + i) % 2 for i in range(n)]
    pool = randn(seed + 4, n + 3, dim)
    return x, gate, lo, pool, slots, fresh


def poison(pool, slots, fresh):
    """The slots that a call must not read hold NaN on the GPU."""
    p = pool.clone()
    for s in range(pool.shape[0]):
        if s not in slots or fresh[slots.index(s)]:
            p[s] = NAN
    return p


LENGTHS = [[1], [0, 1, 0, 2], [127, 128, 129], [256, 0, 257, 3], [2300], [3, 700, 4500]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("dim,off,extra", [(64, 0, 0), (37, 0, 0), (130, 1, 5), (66, 2, 6), (264, 8, 264)])
def test_recurrence_forward_and_backward(dtype, lengths, dim, off, extra):
    dev = device()
    seed = dim + len(lengths)
    x, gate, lo, pool, slots, fresh = rec_inputs(seed, lengths, dim, dtype, dim != 64)
    cu, rows, n = cu_of(lengths), sum(lengths), len(lengths)
    ref = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
    gx, gg = to_dev(x, dev, off, extra), to_dev(gate, dev, off, extra)
    glo = lo.to(dev) if lo is not None else None
    st = poison(pool, slots, fresh).to(dev)
    y = to_dev(torch.zeros_like(x), dev, off, extra)
    kept = torch.full((ss.gated_recurrence_checkpoints(cu), dim), NAN, device=dev)
    ss.gated_recurrence(y, gx, gg, glo, st, cu, slots, fresh, checkpoints=kept)
    torch.cuda.synchronize()
    R.check(y, ref["y"], "y")
    at = torch.tensor(slots)
    R.check(st[at.to(dev)], tuple(v[at] for v in ref["pool"]), "state")
    others = torch.tensor([s for s in range(n + 3) if s not in slots])
    assert torch.isnan(st.cpu()[others]).all(), "a slot outside the batch was written"
    per = ss.RECURRENCE_CHUNK // ss.RECURRENCE_STEP
    at_row, row = {}, 0  # checkpoint row -> the token that it stands before
    for i in range(n):
        at_row.update({row + k: cu[i] + t for k, t in enumerate(range(0, lengths[i], ss.RECURRENCE_STEP))})
        row += -(-lengths[i] // ss.RECURRENCE_CHUNK) * per
    assert row == kept.shape[0]
    firsts, rows_at = list(at_row.values()), torch.tensor(list(at_row), device=dev)
    R.check(kept[rows_at], (ref["prev"][0][firsts], ref["prev"][2][firsts]), "checkpoints")
    # backward
    dy, de = randn(seed + 8, rows, dim).to(dtype), randn(seed + 9, n, dim)
    want = R.recurrence_backward(x, gate, lo, ref, cu, dy, de)
    dx, dgate = to_dev(torch.zeros_like(x), dev, off, extra), to_dev(torch.zeros_like(x), dev, off, extra)
    dlo = torch.full((dim,), NAN, device=dev) if lo is not None else None
    d0 = torch.full((n, dim), NAN, device=dev)
    ss.gated_recurrence_backward(dx, dgate, dlo, d0, to_dev(dy, dev, off, extra), de.to(dev), gx, gg, glo, kept, cu)
    torch.cuda.synchronize()
    for name, got in (("dx", dx), ("dgate", dgate), ("dstate", d0), ("dlower", dlo)):
        if got is not None:
            R.check(got, want[name], name)


@pytest.mark.parametrize("runs,dim", [(2, 72), (64, 72), (65, 72), (300, 72), (40, 1500)])
def test_recurrence_many_runs_of_different_lengths(runs, dim):
    """Runs whose chunks are taken in turns: longer and shorter ones, some empty, in no order."""
    dev = device()
    g = torch.Generator().manual_seed(runs)
    lengths = [int(v) for v in (torch.rand(runs, generator=g) ** 3 * (3 if runs > 100 or dim > 100 else 9) * 128)]
    lengths[0], lengths[1] = 700, 0
    x, gate, lo, pool, slots, fresh = rec_inputs(runs, lengths, dim, BF16, True)
    cu, rows = cu_of(lengths), sum(lengths)
    ref = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
    gx, gg, glo, st = x.to(dev), gate.to(dev), lo.to(dev), pool.to(dev)
    y, kept = torch.empty_like(gx), torch.empty((ss.gated_recurrence_checkpoints(cu), dim), device=dev)
    ss.gated_recurrence(y, gx, gg, glo, st, cu, slots, fresh, checkpoints=kept)
    dy, de = randn(runs + 8, rows, dim).to(BF16), randn(runs + 9, runs, dim)
    want = R.recurrence_backward(x, gate, lo, ref, cu, dy, de)
    dx, dg, dlo, d0 = torch.empty_like(gx), torch.empty_like(gx), torch.empty_like(glo), torch.empty((runs, dim), device=dev)
    ss.gated_recurrence_backward(dx, dg, dlo, d0, dy.to(dev), de.to(dev), gx, gg, glo, kept, cu)
    torch.cuda.synchronize()
    R.check(y, ref["y"], "y")
    R.check(st, ref["pool"], "state")
    for name, got in (("dx", dx), ("dgate", dg), ("dstate", d0), ("dlower", dlo)):
        R.check(got, want[name], name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,at", [(130, ((0, 0), (1, 1), (2, 3), (3, 6), (5, 7))), (67, ((2, 7), (0, 1), (3, 4), (0, 0), (5, 6)))])
def test_recurrence_matrices_of_different_strides(dtype, dim, at):
    """x, gate, dy and the outputs each start at an offset and have a stride of their own."""
    dev = device()
    lengths = [131, 1, 40]
    x, gate, lo, pool, slots, fresh = rec_inputs(57, lengths, dim, dtype, True)
    cu, rows = cu_of(lengths), sum(lengths)
    ref = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
    dy = randn(58, rows, dim).to(dtype)
    want = R.recurrence_backward(x, gate, lo, ref, cu, dy, None)
    gx, gg, gd = (to_dev(t, dev, *at[i]) for i, t in enumerate((x, gate, dy)))
    y, dx, dg = (to_dev(torch.zeros_like(x), dev, *at[i]) for i in (3, 4, 0))
    st, dlo = pool.to(dev), torch.empty(dim, device=dev)
    kept = torch.empty((ss.gated_recurrence_checkpoints(cu), dim), device=dev)
    ss.gated_recurrence(y, gx, gg, lo.to(dev), st, cu, slots, fresh, checkpoints=kept)
    ss.gated_recurrence_backward(dx, dg, dlo, None, gd, None, gx, gg, lo.to(dev), kept, cu)
    torch.cuda.synchronize()
    R.check(y, ref["y"], "y")
    for name, got in (("dx", dx), ("dgate", dg), ("dlower", dlo)):
        R.check(got, want[name], name)


def test_recurrence_optional_outputs_and_repeat():
    """dlower, dstate and dstate_end left out; the same call twice gives the same bits."""
    dev = device()
    lengths, dim = [500, 3000], 96
    x, gate, lo, pool, slots, fresh = rec_inputs(7, lengths, dim, BF16, True)
    cu = cu_of(lengths)
    ref = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
    gx, gg, glo = x.to(dev), gate.to(dev), lo.to(dev)
    dy = randn(9, sum(lengths), dim).to(BF16)
    runs = []
    for _ in range(2):
        st = pool.to(dev)
        y = torch.empty_like(gx)
        kept = torch.zeros((ss.gated_recurrence_checkpoints(cu), dim), device=dev)
        ss.gated_recurrence(y, gx, gg, glo, st, cu, slots, fresh, checkpoints=kept)
        dx, dg, dlo = torch.empty_like(gx), torch.empty_like(gx), torch.empty_like(glo)
        ss.gated_recurrence_backward(dx, dg, dlo, None, dy.to(dev), None, gx, gg, glo, kept, cu)
        runs.append((y, st, kept, dx, dg, dlo))
    y2 = torch.empty_like(gx)
    ss.gated_recurrence(y2, gx, gg, glo, pool.to(dev), cu, slots, fresh)
    dx2, dg2 = torch.empty_like(gx), torch.empty_like(gx)
    ss.gated_recurrence_backward(dx2, dg2, None, None, dy.to(dev), None, gx, gg, glo, kept, cu)
    torch.cuda.synchronize()
    for a, b in zip(*runs):
        assert_bits_equal(a, b, "repeat")
    assert_bits_equal(y2, y, "without checkpoints")
    assert_bits_equal(dx2, dx, "without dlower")
    assert_bits_equal(dg2, dg, "without dlower")
    want = R.recurrence_backward(x, gate, lo, ref, cu, dy, None)
    R.check(dx, want["dx"], "dx")
    R.check(dlo, want["dlower"], "dlower")


@pytest.mark.parametrize("value", [200.0, -200.0, float("inf"), -float("inf")])
def test_recurrence_saturated_gates(value):
    """f = 1 holds the state, f = lo (or 0) drops it; no inf - inf or 0 / 0 in either direction."""
    dev = device()
    lengths, dim = [300, 5], 64
    x, gate, lo, pool, slots, fresh = rec_inputs(17, lengths, dim, F32, True)
    gate[::3] = value
    lo[:8], lo[8:16] = 0.0, 1.0
    cu = cu_of(lengths)
    ref = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
    st, y = pool.to(dev), torch.empty((305, dim), device=dev)
    kept = torch.empty((ss.gated_recurrence_checkpoints(cu), dim), device=dev)
    ss.gated_recurrence(y, x.to(dev), gate.to(dev), lo.to(dev), st, cu, slots, fresh, checkpoints=kept)
    dy = randn(18, 305, dim)
    want = R.recurrence_backward(x, gate, lo, ref, cu, dy, None)
    dx, dg, dlo, d0 = torch.empty_like(y), torch.empty_like(y), torch.empty(dim, device=dev), torch.empty((2, dim), device=dev)
    ss.gated_recurrence_backward(dx, dg, dlo, d0, dy.to(dev), None, x.to(dev), gate.to(dev), lo.to(dev), kept, cu)
    torch.cuda.synchronize()
    R.check(y, ref["y"], "y")
    for name, got in (("dx", dx), ("dgate", dg), ("dstate", d0), ("dlower", dlo)):
        R.check(got, want[name], name)


def test_recurrence_non_finite_stays_in_its_run_and_channel():
    dev = device()
    lengths, dim = [400, 400, 10], 40
    x, gate, lo, pool, slots, _ = rec_inputs(23, lengths, dim, BF16, False)
    cu, fresh = cu_of(lengths), [1, 1, 1]
    ref = R.recurrence(x, gate, None, pool, cu, slots, fresh)
    x2 = x.clone()
    x2[cu[1] + 7, 5] = NAN
    y, st = torch.empty((810, dim), dtype=BF16, device=dev), pool.to(dev)
    ss.gated_recurrence(y, x2.to(dev), gate.to(dev), None, st, cu, slots, fresh)
    torch.cuda.synchronize()
    bad = torch.isnan(y.cpu())
    want = torch.zeros_like(bad)
    want[cu[1] + 7:cu[2], 5] = True
    assert torch.equal(bad, want)
    keep = [c for c in range(dim) if c != 5]
    R.check(y[:, keep], tuple(v[:, keep] for v in ref["y"]), "other channels")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_recurrence_resumes_and_steps(dtype):
    """Prefill in two calls, then single tokens by the host and the device batch: the runs' one-call result."""
    dev = device()
    lengths, dim = [700, 1, 130], 72
    x, gate, lo, pool, slots, fresh = rec_inputs(31, lengths, dim, dtype, True)
    cu = cu_of(lengths)
    ref = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
    st = poison(pool, slots, fresh).to(dev)
    glo = lo.to(dev)
    got = torch.empty_like(x)
    cuts = [[0, 300, 690, 699, 700], [0, 1, 1, 1, 1], [0, 3, 120, 129, 130]]
    at, empty_before = [0, 0, 0], list(fresh)
    for p in range(2):  # two prefills
        rows = [torch.arange(cu[i] + cuts[i][p], cu[i] + cuts[i][p + 1]) for i in range(3)]
        idx = torch.cat(rows)
        y = torch.empty((len(idx), dim), dtype=dtype, device=dev)
        ss.gated_recurrence(y, x[idx].to(dev), gate[idx].to(dev), glo, st, cu_of([len(r) for r in rows]), slots,
                            fresh if p == 0 else [0, 0, 0])
        got[idx] = y.cpu()
    n_dev, status = torch.tensor([2], dtype=torch.int32, device=dev), torch.full((1,), -1, dtype=torch.int32, device=dev)
    for k in range(10):  # single tokens of the two long runs
        idx = torch.tensor([cu[0] + 690 + k, cu[2] + 120 + k])
        s2 = [slots[0], slots[2]]
        if k % 2:
            y = torch.empty((2, dim), dtype=dtype, device=dev)
            ss.gated_recurrence_step(y, x[idx].to(dev), gate[idx].to(dev), glo, st, s2, [0, 0])
        else:  # a capacity of four, two of them in use
            pad = torch.cat([idx, idx])
            y = torch.full((4, dim), 7.0, dtype=dtype, device=dev)
            ss.gated_recurrence_step_device(y, x[pad].to(dev), gate[pad].to(dev), glo, st,
                                            torch.tensor(s2 + [99, 99], dtype=torch.int32, device=dev),
                                            None if k % 4 else torch.zeros(4, dtype=torch.uint8, device=dev), n_dev, status)
            assert int(status.item()) == ss.OK
            assert (y[2:] == 7.0).all()
        got[idx] = y[:2].cpu()
    R.check(got, ref["y"], "y")
    a = torch.tensor(slots)
    R.check(st[a.to(dev)], tuple(v[a] for v in ref["pool"]), "state")


def test_step_fresh_and_bad_device_batches():
    dev = device()
    dim = 50
    x, gate, _, _, _, _ = rec_inputs(41, [4], dim, BF16, False)
    slots, fresh = [5, 0, 2, 6], [0, 1, 0, 1]
    pool_ = randn(42, 8, dim)
    ref = R.recurrence(x, gate, None, pool_, cu_of([1] * 4), slots, fresh)
    st = poison(pool_, slots, fresh).to(dev)
    y = torch.empty((4, dim), dtype=BF16, device=dev)
    ss.gated_recurrence_step(y, x.to(dev), gate.to(dev), None, st, slots, fresh)
    R.check(y, ref["y"], "y")
    for bad, n, status in (([5, 0, 8, 6], 4, ss.ERR_SLOT_OUT_OF_RANGE), ([5, -1, 2, 6], 4, ss.ERR_SLOT_OUT_OF_RANGE),
                           ([5, 0, 5, 6], 4, ss.ERR_SLOT_SHARED), ([5, 0, 2, 6], 5, ss.ERR_INVALID_ARGUMENT)):
        st = pool_.to(dev)
        y = torch.full((4, dim), 7.0, dtype=BF16, device=dev)
        code = torch.full((1,), -1, dtype=torch.int32, device=dev)
        ss.gated_recurrence_step_device(y, x.to(dev), gate.to(dev), None, st,
                                        torch.tensor(bad, dtype=torch.int32, device=dev),
                                        torch.tensor(fresh, dtype=torch.uint8, device=dev),
                                        torch.tensor([n], dtype=torch.int32, device=dev), code)
        assert int(code.item()) == status, bad
        assert (y == 7.0).all() and torch.equal(st.cpu(), pool_)


@pytest.mark.parametrize("capacity", [3, 130, 256, 300, 1024])
@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (F32, 1500), (BF16, 37)])
def test_step_device_batch_sizes(capacity, dtype, dim):
    """Batches that the step's own CTAs check and larger ones: the result, and what a bad last slot does."""
    dev = device()
    n = capacity - 1
    x, gate, lo, _, _, _ = rec_inputs(capacity, [capacity], dim, dtype, True)
    slots = torch.randperm(capacity + 9, generator=torch.Generator().manual_seed(capacity))[:capacity].tolist()
    fresh = [i % 3 == 0 for i in range(capacity)]
    pool = randn(7, capacity + 9, dim)
    ref = R.recurrence(x[:n], gate[:n], lo, pool, cu_of([1] * n), slots[:n], fresh[:n])
    put = lambda v, t: torch.tensor(v, dtype=t, device=dev)  # noqa: E731
    for bad, status in ((None, ss.OK), (slots[0], ss.ERR_SLOT_SHARED), (capacity + 9, ss.ERR_SLOT_OUT_OF_RANGE)):
        st, y, code = pool.to(dev), torch.full((capacity, dim), 7.0, dtype=dtype, device=dev), put([-1], torch.int32)
        s = list(slots)
        if bad is not None:
            s[n - 1] = bad
        ss.gated_recurrence_step_device(y, x.to(dev), gate.to(dev), lo.to(dev), st, put(s, torch.int32),
                                        put(fresh, torch.uint8), put([n], torch.int32), code)
        assert int(code.item()) == status
        if bad is None:
            R.check(y[:n], ref["y"], "y")
            a = torch.tensor(slots[:n])
            R.check(st[a.to(dev)], tuple(v[a] for v in ref["pool"]), "state")
            rest = [i for i in range(capacity + 9) if i not in slots[:n]]
            assert torch.equal(st.cpu()[rest], pool[rest]) and (y[n:] == 7.0).all()
        else:
            assert torch.equal(st.cpu(), pool) and (y == 7.0).all()


def test_step_device_batch_of_a_large_pool():
    """More slots than the check's bitmap holds: the slots are compared pair by pair."""
    dev = device()
    n, dim, slots_n = 200, 12, 40000
    x, gate, _, _, _, _ = rec_inputs(77, [n], dim, F32, False)
    pool = randn(78, slots_n, dim)
    slots = torch.randperm(slots_n, generator=torch.Generator().manual_seed(79))[:n].tolist()
    ref = R.recurrence(x, gate, None, pool, cu_of([1] * n), slots, [0] * n)
    for twice in (False, True):
        s = slots[:-1] + [slots[3]] if twice else slots
        st, y, code = pool.to(dev), torch.full((n, dim), 7.0, device=dev), torch.full((1,), -1, dtype=torch.int32, device=dev)
        ss.gated_recurrence_step_device(y, x.to(dev), gate.to(dev), None, st, torch.tensor(s, dtype=torch.int32, device=dev),
                                        None, torch.tensor([n], dtype=torch.int32, device=dev), code)
        assert int(code.item()) == (ss.ERR_SLOT_SHARED if twice else ss.OK)
        if twice:
            assert torch.equal(st.cpu(), pool) and (y == 7.0).all()
        else:
            R.check(y, ref["y"], "y")
            R.check(st[slots], tuple(v[slots] for v in ref["pool"]), "state")


def test_recurrence_past_32_bit_offsets():
    dev = device()
    dim, ld = 64, 1 << 28  # row 9 begins past 2^31 elements
    wide = torch.zeros((1, 10 * ld), dtype=BF16, device=dev).view(10, ld)
    x, gate, lo, _, _, _ = rec_inputs(51, [10], dim, BF16, True)
    gx, gg, gy = wide[:, :dim], wide[:, 100:100 + dim], wide[:, 1000:1000 + dim]
    gx.copy_(x.to(dev))
    gg.copy_(gate.to(dev))
    slots = (1 << 31) // dim + 5
    st = torch.zeros((slots + 1, dim), device=dev)
    ss.gated_recurrence(gy, gx, gg, lo.to(dev), st, [0, 10], [slots], [1])
    ref = R.recurrence(x, gate, lo, torch.zeros((1, dim)), [0, 10], [0], [1])
    R.check(gy, ref["y"], "y")
    R.check(st[slots:], ref["pool"], "state")
    kept = torch.zeros((ss.gated_recurrence_checkpoints([0, 10]), dim), device=dev)
    dy = randn(52, 10, dim).to(BF16)
    gdy, dx, dg = wide[:, 2000:2000 + dim], wide[:, 3000:3000 + dim], wide[:, 4000:4000 + dim]
    gdy.copy_(dy.to(dev))
    ss.gated_recurrence_backward(dx, dg, None, None, gdy, None, gx, gg, lo.to(dev), kept, [0, 10])
    want = R.recurrence_backward(x, gate, lo, ref, [0, 10], dy, None)
    R.check(dx, want["dx"], "dx")
    R.check(dg, want["dgate"], "dgate")


def test_recurrence_many_runs_and_no_runs():
    dev = device()
    lengths, dim = [i % 4 for i in range(ss.MAX_SEQS)], 16
    x, gate, lo, pool, slots, fresh = rec_inputs(61, lengths, dim, BF16, True)
    cu = cu_of(lengths)
    ref = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
    st, y = poison(pool, slots, fresh).to(dev), torch.empty(x.shape, dtype=BF16, device=dev)
    ss.gated_recurrence(y, x.to(dev), gate.to(dev), lo.to(dev), st, cu, slots, fresh)
    R.check(y, ref["y"], "y")
    a = torch.tensor(slots)
    R.check(st[a.to(dev)], tuple(v[a] for v in ref["pool"]), "state")
    e = torch.empty((0, dim), dtype=BF16, device=dev)
    dlo = torch.full((dim,), NAN, device=dev)
    ss.gated_recurrence(e, e, e, lo.to(dev), st, [0], [], [])
    ss.gated_recurrence_backward(e, e.clone(), dlo, None, e, None, e, e, lo.to(dev), torch.empty((0, dim), device=dev), [0])
    assert (dlo == 0).all()


# ---------------------------------------------------------------- add + RMS norm

@pytest.mark.parametrize("dtype,stype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 64), (2, 100), (9, 768), (4, 1001), (3, 4104), (2, 9000), (2, 33000)])
@pytest.mark.parametrize("residual", [False, True])
def test_add_rmsnorm(dtype, stype, rows, dim, residual):
    dev = device()
    x, w = randn(dim, rows, dim).to(dtype), randn(dim + 1, dim, std=0.3, mean=1.0)
    r = randn(dim + 2, rows, dim, std=2.0).to(stype) if residual else None
    (s64, serr), yref, rel = R.add_rmsnorm(x, r, w, 1e-5)
    gx, gw = x.to(dev), w.to(dev)
    total = r.to(dev) if residual else torch.empty((rows, dim), dtype=stype, device=dev)
    out = torch.empty_like(gx)
    ss.add_rmsnorm(out, gx, gw, 1e-5, residual=total if residual else None, sum=total)  # the residual in place
    R.check(out, yref, "out")
    R.check(total, (s64, serr), "sum")
    q, scale = torch.empty((rows, dim), dtype=E4M3, device=dev), torch.full((rows,), NAN, device=dev)
    ss.add_rmsnorm(q, gx, gw, 1e-5, residual=r.to(dev) if residual else None, scale=scale)
    sref = yref[0].abs().amax(1) / 448
    R.check(scale, (sref, 2 * rel * sref), "scale")
    # an e4m3 value is off by half a step: 2^-4 relative, 2^-10 below the smallest normal one
    v = yref[0] / scale.cpu().double()[:, None]
    assert ((q.cpu().float().double() - v).abs() <= torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))
            + 4 * rel * v.abs() + 2.0 ** -20).all()
    assert float(q.cpu().float().abs().max()) <= 448
    # backward, from the stored sum
    dy, ds = randn(dim + 3, rows, dim).to(dtype), randn(dim + 4, rows, dim, std=0.5).to(stype)
    src = total.cpu()
    dref, wref = R.add_rmsnorm_backward(src, w, 1e-5, dy, ds if residual else None)
    dx, dr, dw = torch.empty_like(gx), ds.to(dev), torch.full((dim,), NAN, device=dev)
    ss.add_rmsnorm_backward(dx, dr, dw, dy.to(dev), dr if residual else None, total, gw, 1e-5)  # dsum in place
    R.check(dx, dref, "dx")
    R.check(dr, dref, "dresidual")
    R.check(dw, wref, "dweight")


def test_add_rmsnorm_many_rows_backward_repeats():
    dev = device()
    rows, dim = 3001, 264
    s, w, dy = randn(1, rows, dim).to(BF16), randn(2, dim), randn(3, rows, dim).to(BF16)
    _, wref = R.add_rmsnorm_backward(s, w, 1e-5, dy, None)
    got = []
    for _ in range(2):
        dw = torch.empty(dim, device=dev)
        ss.add_rmsnorm_backward(None, None, dw, dy.to(dev), None, s.to(dev), w.to(dev), 1e-5)
        got.append(dw)
    R.check(got[0], wref, "dweight")
    assert_bits_equal(got[0], got[1], "repeat")


@pytest.mark.parametrize("dtype,stype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,dim", [(6001, 33), (5003, 262), (6007, 1001)])
def test_add_rmsnorm_rows_that_start_inside_a_unit(dtype, stype, rows, dim):
    """Rows whose first and last elements share 16 bytes with other rows: those keep to themselves."""
    dev = device()
    x, r, w = randn(dim, rows, dim).to(dtype), randn(dim + 1, rows, dim).to(stype), randn(dim + 2, dim)
    (s64, serr), yref, rel = R.add_rmsnorm(x, r, w, 1e-5)
    x[100], x[rows - 2] = NAN, NAN
    ok = torch.ones(rows, dtype=torch.bool)
    ok[100] = ok[rows - 2] = False
    gx, total, gw = x.to(dev), r.to(dev), w.to(dev)
    out, q, scale = torch.empty_like(gx), torch.empty((rows, dim), dtype=E4M3, device=dev), torch.empty(rows, device=dev)
    ss.add_rmsnorm(q, gx, gw, 1e-5, residual=total, scale=scale)
    ss.add_rmsnorm(out, gx, gw, 1e-5, residual=total, sum=total)
    torch.cuda.synchronize()
    assert torch.isnan(out.cpu()[~ok]).all() and torch.isnan(total.cpu()[~ok].float()).all()
    R.check(total.cpu()[ok], (s64[ok], serr[ok]), "sum")
    R.check(out.cpu()[ok], tuple(v[ok] for v in yref), "out")
    v = (yref[0] / scale.cpu().double()[:, None])[ok]
    assert ((q.cpu().float().double()[ok] - v).abs() <= torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))
            + 4 * rel * v.abs() + 2.0 ** -20).all()
    dy, ds = randn(dim + 3, rows, dim).to(dtype), randn(dim + 4, rows, dim, std=0.5).to(stype)
    src = s64.to(stype)
    dref, wref = R.add_rmsnorm_backward(src, w, 1e-5, dy, ds)
    dx, dr, dw = torch.empty_like(gx), ds.to(dev), torch.full((dim,), NAN, device=dev)
    ss.add_rmsnorm_backward(dx, dr, dw, dy.to(dev), dr, src.to(dev), gw, 1e-5)
    R.check(dx, dref, "dx")
    R.check(dr, dref, "dresidual")
    R.check(dw, wref, "dweight")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 77), (300, 1085), (2, 20001)])
def test_add_rmsnorm_what_lies_behind_the_tensors_is_not_used(dtype, rows, dim):
    """x, the residual, dy and the weights end inside 16 bytes whose rest is NaN."""
    dev = device()

    def followed(t):
        wide = torch.full((t.numel() + 64,), NAN, dtype=t.dtype, device=dev)
        wide[:t.numel()] = t.to(dev).flatten()
        return wide[:t.numel()].view(t.shape)

    x, r, w = randn(1, rows, dim).to(dtype), randn(2, rows, dim).to(dtype), randn(3, dim, std=0.3, mean=1.0)
    (s64, serr), yref, rel = R.add_rmsnorm(x, r, w, 1e-5)
    gx, gr, gw = followed(x), followed(r), followed(w)
    out, total = torch.empty_like(gx), torch.empty_like(gx)
    ss.add_rmsnorm(out, gx, gw, 1e-5, residual=gr, sum=total)
    R.check(out, yref, "out")
    R.check(total, (s64, serr), "sum")
    q, scale = torch.empty((rows, dim), dtype=E4M3, device=dev), torch.full((rows,), NAN, device=dev)
    ss.add_rmsnorm(q, gx, gw, 1e-5, residual=gr, scale=scale)
    sref = yref[0].abs().amax(1) / 448
    R.check(scale, (sref, 2 * rel * sref), "scale")
    dy = randn(4, rows, dim).to(dtype)
    src = total.cpu()
    dref, wref = R.add_rmsnorm_backward(src, w, 1e-5, dy, None)
    dx, dw = torch.empty_like(gx), torch.empty_like(gw)
    ss.add_rmsnorm_backward(dx, None, dw, followed(dy), None, followed(src), gw, 1e-5)
    R.check(dx, dref, "dx")
    R.check(dw, wref, "dweight")


def test_add_rmsnorm_rows_of_zeros_and_non_finite():
    dev = device()
    dim = 300
    x = randn(5, 5, dim)
    x[1] = 0
    x[2, 7] = NAN
    x[3, 299] = float("inf")
    w = randn(6, dim, std=0.1, mean=1.0)
    q, scale = torch.empty((5, dim), dtype=E4M3, device=dev), torch.empty(5, device=dev)
    ss.add_rmsnorm(q, x.to(dev), w.to(dev), 1e-6, scale=scale)
    q, scale = q.cpu().float(), scale.cpu()
    assert (q[1] == 0).all() and scale[1] == 1
    for r in (2, 3):
        assert torch.isnan(scale[r]) and torch.isnan(q[r]).all()
    for r in (0, 4):
        assert torch.isfinite(q[r]).all() and torch.isfinite(scale[r])
    e = torch.empty((0, dim), device=dev)
    dw = torch.full((dim,), NAN, device=dev)
    ss.add_rmsnorm(e, e.clone(), w.to(dev), 1e-6)
    ss.add_rmsnorm_backward(e.clone(), None, dw, e, None, e.clone(), w.to(dev), 1e-6)
    assert (dw == 0).all()


# ---------------------------------------------------------------- linear

def quantise(t):
    s = t.abs().amax(1).clamp_min(1e-8) / 448
    return (t / s[:, None]).to(E4M3), s


SHAPES = [(1, 16, 1), (1, 512, 130), (2, 64, 37), (5, 2048, 512), (16, 128, 128), (17, 144, 65), (33, 80, 300),
          (64, 256, 256), (65, 48, 129), (100, 320, 520), (129, 16, 257), (200, 1024, 100), (300, 208, 515), (520, 64, 260)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("out_type", [BF16, F32])
@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_linear(fp8, out_type, rows, k, n):
    dev = device()
    i = SHAPES.index((rows, k, n))
    activation = ["none", "relu", "silu", "gelu"][(i + fp8) % 4]
    x, w = randn(i, rows, k), randn(i + 50, n, k, std=k ** -0.5)
    bias = randn(i + 60, n, std=0.5) if i % 3 else None
    res = randn(i + 70, rows, n).to(out_type) if i % 2 else None
    xs = wsc = None
    if fp8:
        (x, xs), (w, wsc) = quantise(x), quantise(w)
    else:
        x, w = x.to(BF16), w.to(BF16)
    pref, oref = R.linear(x.float(), w.float(), xs, wsc, bias, res, activation)
    put = lambda t: t.to(dev) if t is not None else None  # noqa: E731
    pad = 16 if fp8 else 8
    if i % 4 == 1:  # a column range of a wider activation
        gx = torch.full((rows, k + 2 * pad), 0.0, device=dev).to(x.dtype)
        gx[:, pad:pad + k] = x.to(dev)
        gx = gx[:, pad:pad + k]
    else:
        gx = x.to(dev)
    off, extra = ((0, 0), (3, 7), (8, 16))[i % 3]
    out = to_dev(torch.zeros((rows, n), dtype=out_type), dev, off, extra)
    pre = torch.full((rows, n), NAN, dtype=BF16, device=dev) if i % 2 == 0 else None
    gres = to_dev(res, dev, off, extra) if res is not None else None
    ss.linear(out, gx, put(w), x_scale=put(xs), w_scale=put(wsc), bias=put(bias), residual=gres, activation=activation,
              pre=pre)
    torch.cuda.synchronize()
    R.check(out, oref, "out")
    if pre is not None:
        R.check(pre, pref, "pre")
    if extra:  # nothing beside the column range is written
        base = out._base
        assert torch.isnan(base[:, :off]).all() and torch.isnan(base[:, off + n:]).all()
    assert ss.library().mamba2_device_timeouts() == 0


@pytest.mark.parametrize("rows", [3, 300])
def test_linear_in_place_residual(rows):
    dev = device()
    x, w, r = randn(1, rows, 64).to(BF16), randn(2, 72, 64, std=0.1).to(BF16), randn(3, rows, 72).to(BF16)
    _, oref = R.linear(x.float(), w.float(), None, None, None, r, "silu")
    out = r.to(dev)
    ss.linear(out, x.to(dev), w.to(dev), residual=out, activation="silu")
    R.check(out, oref, "in place")


def test_linear_repeats_and_large_rows():
    dev = device()
    for rows in (40, 2000):
        x, w = randn(1, rows, 4096).to(BF16).to(dev), randn(2, 1030, 4096, std=0.02).to(BF16).to(dev)
        a, b = torch.empty((rows, 1030), device=dev), torch.empty((rows, 1030), device=dev)
        ss.linear(a, x, w)
        ss.linear(b, x, w)
        assert_bits_equal(a, b, "repeat")
        pick = [0, rows // 2, rows - 1]
        _, oref = R.linear(x[pick].cpu().float(), w.cpu().float(), None, None, None, None, "none")
        R.check(a[pick], oref, "sampled rows")


@pytest.mark.parametrize("rows,k,n", [(1, 8, 1), (3, 64, 37), (64, 128, 64), (130, 72, 129), (300, 264, 520), (520, 40, 100), (1000, 512, 300)])
@pytest.mark.parametrize("activation", ["none", "relu", "silu", "gelu"])
def test_linear_backward(rows, k, n, activation):
    dev = device()
    x, w = randn(1, rows, k).to(BF16), randn(2, n, k, std=0.2).to(BF16)
    dy, pre = randn(3, rows, n).to(BF16), randn(4, rows, n).to(BF16) if activation != "none" else None
    want = R.linear_backward(dy, pre, x, w, activation)
    gx = to_dev(x, dev, 8, 16) if n % 2 else x.to(dev)
    dx, dw, db = torch.empty((rows, k), dtype=BF16, device=dev), torch.empty((n, k), dtype=BF16, device=dev), torch.empty(n, device=dev)
    gpre = pre.to(dev) if pre is not None else None
    ss.linear_backward(dx, dw, db, dy.to(dev), gx, w.to(dev), activation=activation, pre=gpre)
    torch.cuda.synchronize()
    for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
        R.check(got, want[name], name)
    only = torch.empty_like(dw)  # one gradient alone
    ss.linear_backward(None, only, None, dy.to(dev), gx, w.to(dev), activation=activation, pre=gpre)
    assert_bits_equal(only, dw, "dw alone")
    assert ss.library().mamba2_device_timeouts() == 0


def test_linear_backward_of_no_rows():
    dev = device()
    e = lambda c: torch.empty((0, c), dtype=BF16, device=dev)  # noqa: E731
    dw, db = torch.full((24, 16), NAN, dtype=BF16, device=dev), torch.full((24,), NAN, device=dev)
    ss.linear_backward(e(16), dw, db, e(24), e(16), torch.zeros((24, 16), dtype=BF16, device=dev))
    assert (dw == 0).all() and (db == 0).all()


# ---------------------------------------------------------------- streams and graphs

def test_side_stream_and_graph_capture():
    """Forward and backward of every operator on a side stream and in a captured graph replayed on new inputs."""
    dev = device()
    lengths, dim = [700, 0, 300], 128
    x, gate, lo, pool, slots, fresh = rec_inputs(71, lengths, dim, BF16, True)
    cu = cu_of(lengths)
    gx, gg, glo, st0 = x.to(dev), gate.to(dev), lo.to(dev), pool.to(dev)
    w, nw = randn(72, 256, dim, std=0.1).to(BF16).to(dev), randn(73, dim).to(dev)
    dy = randn(74, 1000, 256).to(BF16).to(dev)
    buf = dict(st=torch.empty_like(st0), y=torch.empty_like(gx), n=torch.empty_like(gx), s=torch.empty_like(gx),
               kept=torch.zeros((ss.gated_recurrence_checkpoints(cu), dim), device=dev),
               o=torch.empty((1000, 256), dtype=BF16, device=dev), pre=torch.empty((1000, 256), dtype=BF16, device=dev),
               dn=torch.empty_like(gx), dw=torch.empty_like(w), db=torch.empty(256, device=dev), ds=torch.empty_like(gx),
               dnw=torch.empty_like(nw), dx=torch.empty_like(gx), dg=torch.empty_like(gx), dlo=torch.empty_like(glo))

    def chain(b, stream=None):
        b["st"].copy_(st0)
        ss.gated_recurrence(b["y"], gx, gg, glo, b["st"], cu, slots, fresh, checkpoints=b["kept"], stream=stream)
        ss.add_rmsnorm(b["n"], b["y"], nw, 1e-5, residual=gx, sum=b["s"], stream=stream)
        ss.linear(b["o"], b["n"], w, activation="silu", pre=b["pre"], stream=stream)
        ss.linear_backward(b["dn"], b["dw"], b["db"], dy, b["n"], w, activation="silu", pre=b["pre"], stream=stream)
        ss.add_rmsnorm_backward(b["ds"], None, b["dnw"], b["dn"], None, b["s"], nw, 1e-5, stream=stream)
        ss.gated_recurrence_backward(b["dx"], b["dg"], b["dlo"], None, b["ds"], None, gx, gg, glo, b["kept"], cu,
                                     stream=stream)

    chain(buf)
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in buf.items()}
    side = torch.cuda.Stream()
    for v in buf.values():
        v.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(buf)
    side.synchronize()
    for k in buf:
        assert_bits_equal(buf[k], first[k], f"side stream {k}")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(buf)
    gx.mul_(0.5)
    for v in buf.values():
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    again = {k: torch.zeros_like(v) for k, v in buf.items()}
    chain(again)
    torch.cuda.synchronize()
    for k in buf:
        assert_bits_equal(buf[k], again[k], f"graph {k}")
    assert not torch.equal(buf["y"], first["y"])
