"""Host side of the recurrent block's operators (no GPU): every refusal happens before a device pointer is
touched, and the 64-bit references that the GPU tests use agree with hand-worked values and with differences."""
import ctypes

import pytest
import torch

import selective_scan_gb300 as ss
from tests import block_ref as R

P = [0x10000 * (i + 1) for i in range(16)]  # aligned addresses that nothing may touch
INV, NOT, WS = ss.ERR_INVALID_ARGUMENT, ss.ERR_NOT_IMPLEMENTED, ss.ERR_WORKSPACE_TOO_SMALL


def rec(lib, cu=(0, 3, 7), slots=(0, 1), rows=7, dim=64, ld=(64, 64, 64), act=ss.BF16, num_slots=4, p=None, ws=None,
        ws_bytes=0):
    q = list(P[:6]) if p is None else p
    b = ss.Batch(list(cu), list(slots), [0] * len(slots))
    return lib.mamba2_gated_recurrence(*q, num_slots, rows, dim, *ld, act, b.ref(), ws, ws_bytes, None)


def without(i, v=None, n=6):
    q = list(P[:n])
    q[i] = v
    return q


def test_recurrence_refusals(product_lib):
    lib = product_lib
    assert rec(lib, slots=(0, 4)) == ss.ERR_SLOT_OUT_OF_RANGE
    assert rec(lib, slots=(2, 2)) == ss.ERR_SLOT_SHARED
    assert rec(lib, cu=(0, 5, 4)) == ss.ERR_RUNS_DONT_COVER_ROWS
    assert rec(lib, cu=(0, 3, 6)) == ss.ERR_RUNS_DONT_COVER_ROWS
    assert rec(lib, dim=0) == INV and rec(lib, rows=-1) == INV and rec(lib, act=ss.E4M3) == INV
    for k in range(3):
        ld = [64, 64, 64]
        ld[k] = 63
        assert rec(lib, ld=ld) == INV
    for i in (0, 2, 3, 5):  # y, x, gate, state
        assert rec(lib, p=without(i)) == INV, i
    for i in (0, 2, 3):  # element alignment for strided matrices
        assert rec(lib, p=without(i, P[i] + 1)) == INV, i
    for i in (1, 4, 5):
        assert rec(lib, p=without(i, P[i] + 8)) == INV, i
    assert rec(lib, p=without(0, P[2])) == INV and rec(lib, p=without(0, P[3])) == INV
    assert rec(lib, cu=(0,), slots=(), rows=0) == ss.OK
    long = dict(cu=(0, 300, 301), rows=301)
    need = ss.gated_recurrence_workspace_bytes([0, 300, 301], 64)
    if need:
        assert rec(lib, **long) == WS and rec(lib, ws=P[9], ws_bytes=need - 1, **long) == WS
        assert rec(lib, ws=P[9] + 16, ws_bytes=need, **long) == INV


def test_recurrence_checkpoints(product_lib):
    assert (ss.RECURRENCE_STEP, ss.RECURRENCE_CHUNK) == (16, 128)
    assert ss.gated_recurrence_checkpoints([0, 0, 1, 129, 257, 386]) == 8 * (0 + 1 + 1 + 1 + 2)
    assert ss.gated_recurrence_checkpoints([0]) == 0
    for cu in ([1, 2], [0, 3, 2]):
        with pytest.raises(ss.Mamba2Error):
            ss.gated_recurrence_checkpoints(cu)
    assert product_lib.mamba2_gated_recurrence_checkpoints(None, 1) == -1
    assert product_lib.mamba2_gated_recurrence_checkpoints(None, ss.MAX_SEQS + 1) == -1


def test_step_refusals(product_lib):
    lib = product_lib

    def step(slots=(0, 1), cu=None, p=None, dim=64, ld=(64, 64, 64), num_slots=4, act=ss.BF16):
        b = ss.Batch(cu, list(slots), [0] * len(slots))
        return lib.mamba2_gated_recurrence_step(*(p or P[:5]), num_slots, dim, *ld, act, b.ref(), None)

    assert step(slots=(0, 4)) == ss.ERR_SLOT_OUT_OF_RANGE and step(slots=(1, 1)) == ss.ERR_SLOT_SHARED
    assert step(cu=[0, 1, 3]) == ss.ERR_RUNS_DONT_COVER_ROWS and step(cu=[0, 2, 2]) == INV
    assert step(dim=0) == INV and step(ld=(64, 63, 64)) == INV and step(act=7) == INV
    for i in (0, 1, 2, 4):
        assert step(p=without(i, n=5)) == INV, i
    assert step(p=without(3, P[3] + 4, 5)) == INV
    assert step(slots=()) == ss.OK

    def dev(p=None, cap=4, slots=P[8], fresh=P[9], n=P[10], status=P[11], num_slots=4):
        return lib.mamba2_gated_recurrence_step_device(*(p or P[:5]), num_slots, 64, 64, 64, 64, ss.BF16, slots, fresh,
                                                       n, cap, status, None)

    assert dev(cap=0) == INV and dev(cap=ss.MAX_SEQS + 1) == INV and dev(num_slots=-1) == INV
    for kw in ({"slots": None}, {"n": None}, {"status": None}, {"slots": P[8] + 2}, {"n": P[10] + 1},
               {"status": P[11] + 2}, {"p": without(0, n=5)}):
        assert dev(**kw) == INV, kw


def test_recurrence_backward_refusals(product_lib):
    lib = product_lib

    def bwd(p=None, cu=(0, 3, 7), rows=7, dim=64, ld=(64,) * 5, act=ss.BF16, ws=P[12], ws_bytes=1 << 30):
        arr = (ctypes.c_int32 * len(cu))(*cu)
        return lib.mamba2_gated_recurrence_backward(*(p or P[:10]), rows, dim, *ld, act, arr, len(cu) - 1, ws,
                                                    ws_bytes, None)

    for i in (0, 1, 4, 6, 7, 9):
        assert bwd(p=without(i, n=10)) == INV, i
    assert bwd(p=without(8, n=10)) == INV  # dlower without lower
    assert bwd(p=without(0, P[6], 10)) == INV and bwd(p=without(1, P[0], 10)) == INV
    assert bwd(cu=(0, 3, 6)) == ss.ERR_RUNS_DONT_COVER_ROWS and bwd(cu=(1, 3, 7)) == ss.ERR_RUNS_DONT_COVER_ROWS
    assert bwd(ld=(64, 64, 64, 64, 10)) == INV and bwd(dim=-1) == INV
    need = ss.gated_recurrence_workspace_bytes([0, 3, 7], 64, backward=True)
    assert need > 0 and bwd(ws_bytes=need - 1) == WS and bwd(ws=None) == WS and bwd(ws=P[12] + 128) == INV


def test_norm_refusals(product_lib):
    lib = product_lib

    def norm(p=None, rows=4, dim=64, eps=1e-5, act=ss.BF16, st=ss.BF16, ot=ss.E4M3):
        return lib.mamba2_add_rmsnorm(*(p or P[:6]), rows, dim, eps, act, st, ot, None)

    assert norm(dim=0) == INV and norm(rows=-1) == INV and norm(eps=-1.0) == INV and norm(eps=float("nan")) == INV
    assert norm(act=ss.E4M3) == INV and norm(act=ss.F32, st=ss.BF16) == INV and norm(ot=ss.F32) == INV
    for i in (0, 1, 3, 5):
        assert norm(p=without(i)) == INV, i
    assert norm(ot=ss.BF16) == INV  # a scale without an 8-bit output
    for i in range(6):
        assert norm(p=without(i, P[i] + 4)) == INV, i
    assert norm(p=without(0, P[3])) == INV and norm(p=without(2, P[3])) == INV
    assert norm(rows=0) == ss.OK

    def bwd(p=None, rows=4, dim=64, act=ss.BF16, st=ss.BF16, ws=P[12], ws_bytes=1 << 30):
        return lib.mamba2_add_rmsnorm_backward(*(p or P[:7]), rows, dim, 1e-5, act, st, ws, ws_bytes, None)

    for i in (3, 5, 6):
        assert bwd(p=without(i, n=7)) == INV, i
    assert bwd(p=without(0, P[3], 7)) == INV and bwd(p=without(1, P[5], 7)) == INV and bwd(p=without(1, P[0], 7)) == INV
    assert bwd(ws=None) == WS and bwd(ws=P[12] + 8) == INV and bwd(act=ss.F32) == INV


def test_linear_refusals(product_lib):
    lib = product_lib

    def lin(p=None, rows=4, k=64, n=32, ld=(32, 64, 32), it=ss.E4M3, ot=ss.BF16, act=0):
        return lib.mamba2_linear(*(p or P[:8]), rows, k, n, *ld, it, ot, act, None)

    bf = [P[0], P[1], P[2], None, P[4], None, P[6], P[7]]
    assert lin(k=72) == NOT and lin(ld=(32, 72, 32)) == NOT and lin(p=bf, it=ss.F32) == NOT
    assert lin(p=bf, it=ss.BF16, k=60) == NOT
    assert lin(it=9) == INV and lin(ot=ss.E4M3) == INV and lin(act=4) == INV and lin(act=-1) == INV
    assert lin(rows=-1) == INV and lin(n=0) == INV and lin(k=0) == INV and lin(k=-16) == INV
    assert lin(it=ss.BF16) == INV  # scales with bf16 operands
    for i in (0, 2, 3, 4, 5):
        assert lin(p=without(i, n=8)) == INV, i
    for i in (1, 2, 3, 4, 5, 6):
        assert lin(p=without(i, P[i] + 8, 8)) == INV, i
    assert lin(ld=(31, 64, 32)) == INV and lin(ld=(32, 48, 32)) == INV and lin(ld=(32, 64, 16)) == INV
    assert lin(p=without(0, P[2], 8)) == INV and lin(p=without(1, P[0], 8)) == INV
    assert lin(p=without(7, P[0], 8), ld=(32, 64, 40)) == INV  # the residual in place with another stride
    assert lin(rows=0) == ss.OK

    def bwd(p=None, rows=4, k=64, n=32, ld=64, act=2, ws=P[12], ws_bytes=1 << 30):
        return lib.mamba2_linear_backward(*(p or P[:7]), rows, k, n, ld, act, ws, ws_bytes, None)

    assert bwd(k=60) == NOT and bwd(ld=68) == NOT and bwd(act=5) == INV and bwd(n=0) == INV and bwd(ld=56) == INV
    for i in (3, 4, 5, 6):
        assert bwd(p=without(i, n=7)) == INV, i
    assert bwd(p=without(0, P[5], 7)) == INV and bwd(p=without(2, P[2] + 4, 7)) == INV
    need = lib.mamba2_linear_backward_workspace_bytes(4, 64, 32)
    assert need > 0 and bwd(ws_bytes=need - 1) == WS and bwd(ws=None) == WS and bwd(ws=P[12] + 16) == INV


def test_binding_refuses_shapes_and_strides(product_lib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    st = torch.zeros((4, 64))
    with pytest.raises(ValueError):  # rows that overlap
        ss.gated_recurrence(torch.empty_like(x), x[:1].expand(4, 64), x, None, st, [0, 4], [0], [1])
    with pytest.raises(ValueError):  # a transposed matrix
        ss.gated_recurrence(torch.empty((64, 64), dtype=x.dtype), torch.zeros((64, 64), dtype=x.dtype).t(),
                            torch.zeros((64, 64), dtype=x.dtype), None, st, [0, 64], [0], [1])
    with pytest.raises(ValueError):
        ss.gated_recurrence(torch.empty_like(x), x, x[:, :32], None, st, [0, 4], [0], [1])
    with pytest.raises(ValueError):
        ss.gated_recurrence(torch.empty_like(x), x, x, None, st, [0, 4], [0], [1], checkpoints=torch.zeros((2, 64)))
    with pytest.raises(ValueError):
        ss.add_rmsnorm(torch.empty_like(x), x, torch.ones(32), 1e-5)
    with pytest.raises(ValueError):
        ss.linear(torch.empty((4, 8), dtype=x.dtype), x, torch.zeros((8, 32), dtype=x.dtype))
    with pytest.raises(KeyError):
        ss.linear(torch.empty((4, 8), dtype=x.dtype), x, torch.zeros((8, 64), dtype=x.dtype), activation="swish")


# ---------------------------------------------------------------- the references themselves

def test_reference_recurrence_by_hand():
    # sigmoid(0) = 1/2: h = h/2 + x/2; with lo = 1/2: f = 3/4, k = 1/4
    x = torch.tensor([[1.0], [2.0], [-1.0]])
    g = torch.zeros((3, 1))
    pool = torch.tensor([[9.0], [4.0]])
    r = R.recurrence(x, g, None, pool, [0, 2, 3], [1, 0], [0, 1])
    assert r["y"][0].flatten().tolist() == [2.5, 2.25, -0.5]
    assert r["pool"][0].flatten().tolist() == [-0.5, 2.25]
    r = R.recurrence(x, g, torch.tensor([0.5]), pool, [0, 2, 3], [1, 0], [0, 1])
    assert r["y"][0].flatten().tolist() == [3.25, 2.9375, -0.25]


def _differences(fn, t, h=1e-5):
    out = torch.zeros_like(t)
    flat, o = t.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        up = fn()
        flat[i] = keep - h
        o[i] = (up - fn()) / (2 * h)
        flat[i] = keep
    return out


def test_reference_recurrence_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    d = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    cu, slots, fresh = [0, 3, 3, 5], [2, 0, 1], [0, 0, 1]
    x, gate, lo, pool = d(5, 2), d(5, 2), torch.rand(2, generator=g, dtype=torch.float64), d(3, 2)
    dy, de = d(5, 2), d(3, 2)

    def loss():
        r = R.recurrence(x, gate, lo, pool, cu, slots, fresh)
        return ((r["y"][0] * dy).sum() + sum((r["pool"][0][s] * de[i]).sum() for i, s in enumerate(slots))).item()

    b = R.recurrence_backward(x, gate, lo, R.recurrence(x, gate, lo, pool, cu, slots, fresh), cu, dy, de)
    for name, t in (("dx", x), ("dgate", gate), ("dlower", lo)):
        assert torch.allclose(b[name][0], _differences(loss, t), atol=1e-8), name
    dpool = _differences(loss, pool)
    assert torch.allclose(b["dstate"][0][0], dpool[2], atol=1e-8)
    assert torch.allclose(b["dstate"][0][1], dpool[0], atol=1e-8)  # a run of no token hands its gradient on


def test_reference_norm_and_linear_gradients_against_differences():
    g = torch.Generator().manual_seed(4)
    d = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    s, w, dy, ds = d(3, 5), d(5), d(3, 5), d(3, 5)
    loss = lambda: ((R.add_rmsnorm(s, None, w, 1e-3)[1][0] * dy).sum() + (s * ds).sum()).item()  # noqa: E731
    (dx, _), (dw, _) = R.add_rmsnorm_backward(s, w, 1e-3, dy, ds)
    assert torch.allclose(dx, _differences(loss, s), atol=1e-8) and torch.allclose(dw, _differences(loss, w), atol=1e-8)
    for a in ("none", "relu", "silu", "gelu"):
        x, w, b, dy = d(3, 4), d(5, 4), d(5), d(3, 5)
        loss = lambda: (R.linear(x, w, None, None, b, None, a)[1][0] * dy).sum().item()  # noqa: E731
        r = R.linear_backward(dy, R.linear(x, w, None, None, b, None, a)[0][0], x, w, a)
        for name, t in (("dx", x), ("dw", w), ("dbias", b)):
            assert torch.allclose(r[name][0], _differences(loss, t), atol=1e-8), (a, name)
