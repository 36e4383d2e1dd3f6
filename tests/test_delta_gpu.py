"""The gated delta rule's kernels against the 64-bit token loop of tests/delta_ref.py, at the sizes where they can go
wrong: runs of no token, of one, around a chunk and over many; widths that fill no tile; shared and single keys; column
ranges of wider rows; decays that forget everything or nothing, betas of 0, 1 and 2; alike keys."""
import math

import pytest
import torch

import selective_scan_gb300 as ss
from tests import delta_ref as R
from tests.gpu_util import device
from tests.util import assert_bits_equal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
EPS = 1e-6


def randn(seed, *shape, std=1.0, mean=0.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std + mean


def cu_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def inputs(seed, lengths, groups, heads, d_state, headdim, dtype, l2):
    rows, n = sum(lengths), len(lengths)
    q = randn(seed, rows, groups, d_state, mean=0.3).to(dtype)
    k = randn(seed + 1, rows, groups, d_state, mean=0.3).to(dtype) if l2 else randn(
        seed + 1, rows, groups, d_state, std=0.7 / math.sqrt(d_state)).to(dtype)
    v = randn(seed + 2, rows, heads, headdim).to(dtype)
    g = -torch.nn.functional.softplus(randn(seed + 3, rows, heads, std=1.5, mean=-2.5))
    beta = torch.sigmoid(randn(seed + 4, rows, heads))
    slots = torch.randperm(n + 3, generator=torch.Generator().manual_seed(seed + 5))[:n].tolist()
    fresh = [(seed + i) % 2 for i in range(n)]
    pool = randn(seed + 6, n + 3, heads, headdim, d_state, std=0.3)
    return q, k, v, g, beta, pool, slots, fresh


def poison(pool, slots, fresh):
    """The slots that a call must not read hold NaN on the GPU."""
    p = pool.clone()
    for s in range(pool.shape[0]):
        if s not in slots or fresh[slots.index(s)]:
            p[s] = NAN
    return p


def in_rows(tensors, dev, pad):
    """The tensors as column ranges of one matrix with `pad` columns before, between and after them."""
    if pad is None:
        return [t.to(dev) for t in tensors]
    rows = tensors[0].shape[0]
    wide = torch.full((rows, sum(t[0].numel() if rows else 0 for t in tensors) + pad * (len(tensors) + 1)), NAN,
                      dtype=tensors[0].dtype, device=dev)
    out, at = [], pad
    for t in tensors:
        n = t.shape[1] * t.shape[2]
        wide[:, at:at + n] = t.to(dev).flatten(1)
        out.append(wide[:, at:at + n].unflatten(1, t.shape[1:]))
        at += n + pad
    return out


def check_forward(seed, lengths, groups, heads, d_state, headdim, dtype, l2, pad=None, g=True, beta=True, ckpt=True,
                  change=None, scale=None):
    dev = device()
    q, k, v, gv, bv, pool, slots, fresh = inputs(seed, lengths, groups, heads, d_state, headdim, dtype, l2)
    gv, bv = (gv if g else None), (bv if beta else None)
    if change:
        q, k, v, gv, bv = change(q, k, v, gv, bv)
    cu, rows, eps = cu_of(lengths), sum(lengths), EPS if l2 else None
    by = d_state ** -0.5 if scale is None else scale
    ref = R.forward(q, k, v, gv, bv, pool, cu, slots, fresh, by, eps, R.LOCAL32 if dtype == F32 else R.LOCAL16)
    gq, gk, gvv, y = in_rows([q, k, v, torch.zeros_like(v)], dev, pad)
    st = poison(pool, slots, fresh).to(dev)
    dg, db = (t.to(dev) if t is not None else None for t in (gv, bv))
    kept = torch.full((ss.gated_delta_rule_checkpoints(cu),) + pool.shape[1:], NAN, device=dev) if ckpt else None
    ss.gated_delta_rule(y, gq, gk, gvv, dg, db, st, cu, slots, fresh, scale=scale, l2_eps=eps, checkpoints=kept)
    torch.cuda.synchronize()
    # bf16 outputs of the tensor cores: the state, the scores and the corrections may each be rounded to bf16
    R.within(y, ref["y"], ref["yerr"] + (3 * R.HALF16 * ref["ymag"] if dtype == BF16 else 0), "y")
    if rows:
        R.near(y, ref["y"], 4e-3 if dtype == BF16 else 2e-6, "y")  # 1.7e-3 a bf16 rounding (rms), four of them at most
    at = torch.tensor(slots)
    R.within(st[at.to(dev)], ref["pool"][at], ref["perr"][at][..., None], "state")
    R.near(st[at.to(dev)], ref["pool"][at], 1e-5 if dtype == BF16 else 2e-6, "state")
    others = torch.tensor([s for s in range(pool.shape[0]) if s not in slots])
    assert torch.isnan(st.cpu()[others]).all(), "a slot outside the batch was written"
    if ckpt:
        R.within(kept, ref["kept"], ref["kerr"][..., None], "checkpoints")
    return ref


SHAPES = [(1, 1, 128, 128), (2, 4, 64, 64), (1, 3, 72, 104), (2, 2, 16, 8), (1, 2, 120, 24), (3, 3, 40, 128)]
LENGTHS = [[1], [0, 1, 0, 2], [63, 64, 65], [128, 0, 129, 3], [700], [5, 300, 64]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("groups,heads,d_state,headdim", SHAPES)
def test_forward(dtype, lengths, groups, heads, d_state, headdim):
    check_forward(d_state + len(lengths), lengths, groups, heads, d_state, headdim, dtype, heads != 3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d_state,headdim", [(136, 128), (256, 64), (128, 256), (200, 136)])
def test_forward_of_wide_heads(dtype, d_state, headdim):
    check_forward(3, [130, 1, 70], 1, 2, d_state, headdim, dtype, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 8, 24])
def test_forward_of_column_ranges(dtype, pad):
    check_forward(11, [70, 1, 200], 2, 4, 72, 40, dtype, True, pad=pad)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("g,beta", [(False, True), (True, False), (False, False)])
def test_forward_without_decay_or_beta(dtype, g, beta):
    check_forward(12, [130, 40], 2, 2, 64, 64, dtype, True, g=g, beta=beta, ckpt=False)


def strong_decay(q, k, v, g, beta):
    """Tokens that forget the state (some wholly), between ones that keep it."""
    g = g.clone()
    g[::7] = -90.0
    g[5::11] = -30000.0
    return q, k, v, g, beta


def alike_keys(q, k, v, g, beta):
    """One key for all, nothing decays: I + A is far from the unit matrix."""
    return q, k[:1].expand_as(k).clone(), v, torch.zeros_like(g), torch.full_like(beta, 0.95)


def corner_betas(q, k, v, g, beta):
    beta = beta.clone()
    beta[::3], beta[1::3] = 0.0, 1.0
    beta[2::6] = 2.0
    return q, k, v, g, beta


def zero_rows(q, k, v, g, beta):
    """Keys and queries of no length."""
    q, k = q.clone(), k.clone()
    q[::5], k[::4] = 0.0, 0.0
    return q, k, v, g, beta


def large_values(q, k, v, g, beta):
    return (q.float() * 3e5).to(q.dtype), (k.float() * 2e-5).to(k.dtype), (v.float() * 1e8).to(v.dtype), g, beta


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("change", [strong_decay, alike_keys, corner_betas, zero_rows, large_values], ids=lambda f: f.__name__)
def test_forward_of_values_at_the_edge(dtype, change):
    check_forward(13, [200, 3, 64], 1, 2, 128, 64, dtype, True, change=change)


def test_forward_scale():
    check_forward(14, [66], 1, 1, 64, 64, BF16, True, scale=-3.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,groups,heads,d_state,headdim", [(1, 1, 1, 128, 128), (5, 2, 6, 72, 104), (33, 1, 2, 16, 8), (300, 1, 1, 64, 64),
                                                            (2, 1, 2, 256, 136)])
@pytest.mark.parametrize("l2", [True, False])
def test_steps(dtype, n, groups, heads, d_state, headdim, l2):
    """The host's and the device's batch, one token after another, against the token loop."""
    dev = device()
    q, k, v, g, beta, pool, slots, fresh = inputs(n, [3] * n, groups, heads, d_state, headdim, dtype, l2)
    eps = EPS if l2 else None
    ref = R.forward(q, k, v, g, beta, pool, cu_of([3] * n), slots, fresh, d_state ** -0.5, eps, R.LOCAL32)
    host, devs = poison(pool, slots, fresh).to(dev), poison(pool, slots, fresh).to(dev)
    slots_dev = torch.tensor(slots, dtype=torch.int32, device=dev)
    num, status = torch.tensor([n], dtype=torch.int32, device=dev), torch.full((1,), -1, dtype=torch.int32, device=dev)
    for t in range(3):
        at = torch.arange(n) * 3 + t
        args = [x[at].to(dev) for x in (q, k, v, g, beta)]
        y, yd = torch.full_like(args[2], NAN), torch.full_like(args[2], NAN)
        now = fresh if t == 0 else [0] * n
        ss.gated_delta_rule_step(y, *args, host, slots, now, l2_eps=eps)
        ss.gated_delta_rule_step_device(yd, *args, devs, slots_dev,
                                        torch.tensor(now, dtype=torch.uint8, device=dev) if t == 0 else None, num, status,
                                        l2_eps=eps)
        torch.cuda.synchronize()
        assert int(status) == ss.OK
        assert_bits_equal(yd.cpu(), y.cpu(), "y")
        R.within(y, ref["y"][at], ref["yerr"][at], "y")
    pick = torch.tensor(slots)
    assert_bits_equal(devs[pick.to(dev)].cpu(), host[pick.to(dev)].cpu(), "state")
    R.within(host[pick.to(dev)], ref["pool"][pick], ref["perr"][pick][..., None], "state")


@pytest.mark.parametrize("n", [4, 300])
def test_device_batches_that_are_refused(n):
    """A bad device batch is reported and touches nothing; rows past the count are left as they were."""
    dev = device()
    q, k, v, g, beta, pool, slots, _ = inputs(n, [1] * n, 1, 1, 64, 64, BF16, True)
    args, st = [x.to(dev) for x in (q, k, v, g, beta)], pool.to(dev)
    status = torch.full((1,), -1, dtype=torch.int32, device=dev)
    good = torch.tensor(slots, dtype=torch.int32, device=dev)

    def step(slots_dev, count):
        y = torch.full_like(args[2], NAN)
        ss.gated_delta_rule_step_device(y, *args, st, slots_dev, None, torch.tensor([count], dtype=torch.int32, device=dev),
                                        status, l2_eps=EPS)
        torch.cuda.synchronize()
        return y, int(status)

    for where, value, want in ((2, -1, ss.ERR_SLOT_OUT_OF_RANGE), (0, n + 3, ss.ERR_SLOT_OUT_OF_RANGE), (1, int(good[0]), ss.ERR_SLOT_SHARED)):
        bad = good.clone()
        bad[where] = value
        y, got = step(bad, n)
        assert got == want and torch.isnan(y).all()
    for count in (-1, n + 1):
        y, got = step(good, count)
        assert got == ss.ERR_INVALID_ARGUMENT and torch.isnan(y).all()
    assert_bits_equal(st.cpu(), pool, "state")
    y, got = step(good, n - 2)
    assert got == ss.OK and torch.isfinite(y[:n - 2]).all() and torch.isnan(y[n - 2:]).all()
    left = torch.tensor([s for s in range(n + 3) if s not in slots[:n - 2]])
    assert_bits_equal(st.cpu()[left], pool[left], "state of the others")


def test_prefill_then_steps_is_prefill():
    """A run cut anywhere gives what the whole run gives."""
    dev = device()
    q, k, v, g, beta, pool, slots, fresh = inputs(21, [150], 2, 4, 64, 64, F32, True)
    args, n = [x.to(dev) for x in (q, k, v, g, beta)], 150
    whole, parts = pool.to(dev), pool.to(dev)
    y, z = torch.empty_like(args[2]), torch.empty_like(args[2])
    ss.gated_delta_rule(y, *args, whole, [0, n], slots, [1], l2_eps=EPS)
    ss.gated_delta_rule(z[:100], *(x[:100] for x in args), parts, [0, 100], slots, [1], l2_eps=EPS)
    for t in range(100, n):
        ss.gated_delta_rule_step(z[t:t + 1], *(x[t:t + 1] for x in args), parts, slots, [0], l2_eps=EPS)
    torch.cuda.synchronize()
    R.near(z, y.cpu().double(), 2e-6, "y")
    R.near(parts, whole.cpu().double(), 2e-6, "state")


# ---------------------------------------------------------------- backward

def check_backward(seed, lengths, groups, heads, d_state, headdim, l2, pad=None, g=True, beta=True, ends=True, change=None,
                   scale=None):
    dev = device()
    q, k, v, gv, bv, pool, slots, fresh = inputs(seed, lengths, groups, heads, d_state, headdim, BF16, l2)
    gv, bv = (gv if g else None), (bv if beta else None)
    if change:
        q, k, v, gv, bv = change(q, k, v, gv, bv)
    cu, rows, n, eps = cu_of(lengths), sum(lengths), len(lengths), EPS if l2 else None
    by = d_state ** -0.5 if scale is None else scale
    fwd = R.forward(q, k, v, gv, bv, pool, cu, slots, fresh, by, eps, R.LOCAL16)
    dy = randn(seed + 8, rows, heads, headdim).to(BF16)
    de = randn(seed + 9, n, heads, headdim, d_state, std=0.3) if ends else None
    want = R.backward(fwd["keep"], cu, dy, de, by, groups)
    gq, gk, gvv, gdy, y, dq, dk, dv = in_rows([q, k, v, dy, torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k),
                                               torch.zeros_like(v)], dev, pad)
    gg, gb = (t.to(dev) if t is not None else None for t in (gv, bv))
    st = pool.to(dev)
    kept = torch.full((ss.gated_delta_rule_checkpoints(cu),) + pool.shape[1:], NAN, device=dev)
    ss.gated_delta_rule(y, gq, gk, gvv, gg, gb, st, cu, slots, fresh, scale=scale, l2_eps=eps, checkpoints=kept)
    dg, db = (torch.full((rows, heads), NAN, dtype=BF16, device=dev) for _ in range(2))
    ds = torch.full((n,) + pool.shape[1:], NAN, device=dev)
    args = [gdy, de.to(dev) if ends else None, gq, gk, gvv, gg, gb, kept, cu]
    ss.gated_delta_rule_backward(dq, dk, dv, dg, db, ds, *args, scale=scale, l2_eps=eps)
    torch.cuda.synchronize()
    got = dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=db, dstate=ds)
    for name, t in got.items():
        value, size = want[name]
        if name == "dstate":
            R.within(t, value, size, name)
            R.near(t, value, 1e-5, name)
            continue
        # at most eight operands one behind another are rounded to bf16, each by 2^-8 of what its terms add up to at most;
        # dg is a running sum over a chunk in 32 bits (192 additions at most, of terms that others of its dg are made of)
        R.within(t, value, 8 * R.HALF16 * size + (192 * R.U * size.amax() if name == "dg" and rows else 0), name)
        if rows > 1 and not change:  # 1.7e-3 a rounding (rms): eight of them and the output's own
            R.near(t, value, 5.1e-3, name, want["terms"].get(name))
    # the same again, without what is optional: the same bits
    more = [torch.empty_like(t) for t in (q.to(dev), k.to(dev), v.to(dev))]
    ss.gated_delta_rule_backward(*more, None, None, None, *args, scale=scale, l2_eps=eps)
    torch.cuda.synchronize()
    for a, b in zip(more, (dq, dk, dv)):
        assert_bits_equal(a.cpu(), b.contiguous().cpu(), "the same call again")


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("groups,heads,d_state,headdim", SHAPES)
def test_backward(lengths, groups, heads, d_state, headdim):
    check_backward(d_state + len(lengths), lengths, groups, heads, d_state, headdim, heads != 3)


@pytest.mark.parametrize("pad", [0, 8, 24])
def test_backward_of_column_ranges(pad):
    check_backward(11, [70, 1, 200], 2, 4, 72, 40, True, pad=pad)


@pytest.mark.parametrize("g,beta,ends", [(False, True, True), (True, False, False), (False, False, False)])
def test_backward_without_decay_beta_or_end_states(g, beta, ends):
    check_backward(12, [130, 40], 2, 2, 64, 64, True, g=g, beta=beta, ends=ends)


@pytest.mark.parametrize("change", [strong_decay, alike_keys, corner_betas, zero_rows], ids=lambda f: f.__name__)
def test_backward_of_values_at_the_edge(change):
    check_backward(13, [200, 3, 64], 1, 2, 128, 64, change is not zero_rows, change=change)


def test_backward_scale():
    check_backward(14, [66], 1, 1, 64, 64, False, scale=-3.0)


def test_backward_of_many_heads_and_runs():
    """Runs and heads enough for every split of a state over warps."""
    check_backward(15, [3] * 40 + [64, 130], 2, 4, 32, 128, True)


@pytest.mark.parametrize("l2", [True, False])
def test_gradients_against_differences(l2):
    """The gradients' projection on a direction against central differences of the 64-bit loop."""
    dev = device()
    lengths, G, H, N, P = [70, 33], 1, 2, 24, 16
    q, k, v, g, beta, pool, slots, _ = inputs(31, lengths, G, H, N, P, BF16, l2)
    fresh, cu, rows, eps = [0, 0], cu_of(lengths), sum(lengths), EPS if l2 else None
    dy, de = randn(32, rows, H, P).to(BF16), randn(33, 2, H, P, N, std=0.3)
    at = torch.tensor(slots)

    def loss(q, k, v, g, beta, pool):
        r = R.forward(q, k, v, g, beta, pool, cu, slots, fresh, N ** -0.5, eps, R.LOCAL16)
        return float((r["y"] * dy.double()).sum() + (r["pool"][at] * de.double()).sum())

    base = [t.double() for t in (q, k, v, g, beta, pool)]
    gin = [t.to(dev) for t in (q, k, v, g, beta)]
    kept = torch.empty((ss.gated_delta_rule_checkpoints(cu),) + pool.shape[1:], device=dev)
    y, st = torch.empty_like(gin[2]), pool.to(dev)
    ss.gated_delta_rule(y, *gin, st, cu, slots, fresh, l2_eps=eps, checkpoints=kept)
    out = [torch.empty_like(gin[0]), torch.empty_like(gin[1]), torch.empty_like(gin[2])] + [torch.empty((rows, H), dtype=BF16, device=dev) for _ in range(2)]
    ds = torch.empty((2, H, P, N), device=dev)
    ss.gated_delta_rule_backward(*out, ds, dy.to(dev), de.to(dev), *gin, kept, cu, l2_eps=eps)
    torch.cuda.synchronize()
    grads = [t.cpu().double() for t in out] + [ds.cpu().double()]
    for i, name in enumerate(("q", "k", "v", "g", "beta", "state")):
        way = randn(40 + i, *base[i].shape).double()
        if name == "state":
            way[[s for s in range(pool.shape[0]) if s not in slots]] = 0
        h = 1e-5
        up, down = [list(base) for _ in range(2)]
        up[i], down[i] = base[i] + h * way, base[i] - h * way
        slope = (loss(*up) - loss(*down)) / (2 * h)
        got = grads[i] * (way if name != "state" else way[at])
        # each gradient is off by 5.1e-3 of its norm at most (above), so a projection by that times both norms
        most = 5.1e-3 * float(grads[i].norm()) * float((way if name != "state" else way[at]).norm()) + 1e-6 * abs(slope)
        assert abs(float(got.sum()) - slope) <= most, (name, float(got.sum()), slope, most)
