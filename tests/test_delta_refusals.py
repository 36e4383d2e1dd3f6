"""What the gated delta rule, beam selection and state reordering refuse (no GPU: each comes before a device pointer is
touched), at the C interface and in the binding."""
import ctypes
import re
from pathlib import Path

import pytest
import torch

import selective_scan_gb300 as ss

P = [0x10000 * (i + 1) for i in range(20)]  # aligned addresses that nothing may touch
INV, NOT, SMALL = ss.ERR_INVALID_ARGUMENT, ss.ERR_NOT_IMPLEMENTED, ss.ERR_WORKSPACE_TOO_SMALL
WS = (P[18], 1 << 50)
NAN = float("nan")


def dims(heads=4, headdim=64, d_state=128, groups=2):
    return ctypes.byref(ss.Dims(heads, headdim, d_state, groups, 1))


def calls(lib, ptrs=None, ld=(256, 256, 256, 256), d=None, scale=1.0, eps=-1.0, act=ss.BF16, rows=3, slots=5, batch=None, step=None):
    """The status of each of the three forward calls, or of the one that a bad batch is given for."""
    y, q, k, v, g, beta, state = ptrs or P[:7]
    d = d if d is not None else dims()
    if batch is not None:
        return lib.mamba2_gated_delta_rule(y, None, q, k, v, g, beta, state, slots, rows, *ld, d, scale, eps, act, batch.ref(), *WS, None)
    if step is not None:
        return lib.mamba2_gated_delta_rule_step(y, q, k, v, g, beta, state, slots, *ld, d, scale, eps, act, step.ref(), None)
    b, one = ss.Batch([0, rows], [1], [0]), ss.Batch(None, list(range(rows)), [0] * rows)
    return (lib.mamba2_gated_delta_rule(y, None, q, k, v, g, beta, state, slots, rows, *ld, d, scale, eps, act, b.ref(), *WS, None),
            lib.mamba2_gated_delta_rule_step(y, q, k, v, g, beta, state, slots, *ld, d, scale, eps, act, one.ref(), None),
            lib.mamba2_gated_delta_rule_step_device(y, q, k, v, g, beta, state, slots, *ld, d, scale, eps, act, P[8], None, P[9], rows,
                                                    P[10], None))


def test_constants_are_the_headers():
    root = Path(ss.__file__).resolve().parent.parent / "include"
    delta, beam = (root / "delta.h").read_text(), (root / "beam.h").read_text()
    assert int(re.search(r"#define MAMBA2_DELTA_CHUNK (\d+)", delta).group(1)) == ss.DELTA_CHUNK
    assert int(re.search(r"#define MAMBA2_MAX_BEAMS (\d+)", beam).group(1)) == ss.MAX_BEAMS


@pytest.mark.parametrize("at", range(7))
def test_delta_pointers(product_lib, at):
    for bad in (None, P[at] + 8):
        if bad is None and at in (4, 5):  # g and beta are optional
            continue
        ptrs = P[:7]
        ptrs[at] = bad
        assert calls(product_lib, ptrs) == (INV,) * 3
    if 0 < at < 4:
        ptrs = P[:7]
        ptrs[0] = ptrs[at]  # the output over an input
        assert calls(product_lib, ptrs) == (INV,) * 3


@pytest.mark.parametrize("change,want", [
    (dict(heads=0), INV), (dict(heads=3), INV), (dict(groups=0), INV), (dict(headdim=0), INV), (dict(d_state=-8), INV),
    (dict(heads=65536, groups=1, headdim=8), INV), (dict(heads=65535, groups=1, headdim=65536), INV),
    (dict(headdim=60), NOT), (dict(d_state=124), NOT), (dict(d_state=264), NOT)], ids=str)
def test_delta_dims(product_lib, change, want):
    big = (1 << 40,) * 4
    assert calls(product_lib, d=dims(**change), ld=big) == (want,) * 3
    cu = (ctypes.c_int32 * 2)(0, 300)
    assert product_lib.mamba2_gated_delta_rule_workspace_bytes(cu, 1, dims(**change), ss.BF16, 0) == 0
    assert product_lib.mamba2_gated_delta_rule_workspace_bytes(cu, 1, dims(**change), ss.BF16, 1) == 0


def test_delta_strides_types_and_numbers(product_lib):
    for i in range(4):
        short, odd = [256] * 4, [264] * 4
        short[i], odd[i] = 248, 260
        assert calls(product_lib, ld=short) == (INV,) * 3
        assert calls(product_lib, ld=odd) == (NOT,) * 3
    assert calls(product_lib, act=ss.E4M3) == (INV,) * 3
    assert calls(product_lib, scale=NAN) == (INV,) * 3 and calls(product_lib, eps=NAN) == (INV,) * 3
    assert product_lib.mamba2_gated_delta_rule(*P[:8], 5, -1, 256, 256, 256, 256, dims(), 1.0, 1.0, ss.BF16,
                                               ss.Batch([0, 1], [0], [0]).ref(), *WS, None) == INV


def test_delta_batches(product_lib):
    lib = product_lib
    for batch, want in ((ss.Batch([0, 2], [0], [0]), ss.ERR_RUNS_DONT_COVER_ROWS), (ss.Batch([0, 3], [5], [0]), ss.ERR_SLOT_OUT_OF_RANGE),
                        (ss.Batch([0, 2, 3], [1, 1], [0, 0]), ss.ERR_SLOT_SHARED)):
        assert calls(lib, batch=batch) == want
    assert calls(lib, step=ss.Batch([0, 2, 2, 3], [0, 1, 2], [0] * 3)) == INV
    assert calls(lib, step=ss.Batch(None, [0, 1, 1], [0] * 3)) == ss.ERR_SLOT_SHARED
    for slots, num, status, cap in ((None, P[9], P[10], 3), (P[8], None, P[10], 3), (P[8], P[9], None, 3), (P[8] + 2, P[9], P[10], 3),
                                    (P[8], P[9], P[10], 0), (P[8], P[9], P[10], ss.MAX_SEQS + 1)):
        assert lib.mamba2_gated_delta_rule_step_device(*P[:7], 5, 256, 256, 256, 256, dims(), 1.0, -1.0, ss.BF16, slots, None, num, cap,
                                                       status, None) == INV
    for cu, n in (((1, 2), 1), ((0, 4, 3), 2), ((0, 1), ss.MAX_SEQS + 1), ((0, 1), -1)):
        arr = (ctypes.c_int32 * len(cu))(*cu)
        assert lib.mamba2_gated_delta_rule_checkpoints(arr, n) == -1
        assert lib.mamba2_gated_delta_rule_workspace_bytes(arr, n, dims(), ss.BF16, 0) == 0
    with pytest.raises(ss.Mamba2Error):
        ss.gated_delta_rule_checkpoints([0, 5, 3])
    assert ss.gated_delta_rule_checkpoints([0, 0, 1, 65, 129, 194]) == 0 + 1 + 1 + 1 + 2


def test_delta_calls_of_nothing(product_lib):
    none = ss.Batch([0], [], [])
    assert product_lib.mamba2_gated_delta_rule(*[None] * 8, 0, 0, 0, 0, 0, 0, dims(), 1.0, -1.0, ss.BF16, none.ref(), None, 0, None) == ss.OK
    assert product_lib.mamba2_gated_delta_rule_step(*[None] * 7, 0, 0, 0, 0, 0, dims(), 1.0, -1.0, ss.BF16, none.ref(), None) == ss.OK


def delta_tensors(rows=3, dtype=torch.bfloat16):
    q = torch.zeros((rows, 2, 16), dtype=dtype)
    v = torch.zeros((rows, 4, 8), dtype=dtype)
    return dict(y=v.clone(), q=q, k=q.clone(), v=v, g=torch.zeros((rows, 4)), beta=torch.zeros((rows, 4)), state=torch.zeros((5, 4, 8, 16)))


@pytest.mark.parametrize("name,bad", [
    ("y", lambda t: t[:2]), ("q", lambda t: t[:, :1]), ("k", lambda t: t.float()), ("y", lambda t: t.float()), ("g", lambda t: t[:, :3]),
    ("g", lambda t: t.double()), ("beta", lambda t: t.bfloat16()), ("state", lambda t: t.bfloat16()), ("state", lambda t: t[:, :, :, :8]),
    ("v", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)), ("q", lambda t: torch.cat([t, t], 2)[:, :, ::2]),
    ("k", lambda t: t[:1].expand(3, 2, 16)), ("state", lambda t: t.transpose(2, 3).contiguous().transpose(2, 3))], ids=str)
def test_delta_tensors_of_another_shape_or_type(product_lib, name, bad):
    t = delta_tensors()
    t[name] = bad(t[name])
    with pytest.raises(ValueError):
        ss.gated_delta_rule(**t, cu_seqlens=[0, 3], slots=[0], fresh=[1], stream=0)
    with pytest.raises(ValueError):
        ss.gated_delta_rule_step(**t, slots=[0, 1, 2], fresh=[1] * 3, stream=0)


def test_delta_arguments_of_the_binding(product_lib):
    t = delta_tensors()
    for eps in (-1e-6, NAN):
        with pytest.raises(ValueError):
            ss.gated_delta_rule(**t, cu_seqlens=[0, 3], slots=[0], fresh=[1], l2_eps=eps, stream=0)
    with pytest.raises(ValueError):
        ss.gated_delta_rule(**t, cu_seqlens=[0, 3], slots=[0], fresh=[1], checkpoints=torch.zeros((2, 4, 8, 16)), stream=0)
    with pytest.raises(ValueError):
        ss.gated_delta_rule_step(**t, slots=[0, 1], fresh=[1] * 2, stream=0)
    dev = dict(slots_dev=torch.zeros(3, dtype=torch.int32), fresh_dev=None, num_seqs_dev=torch.zeros(1, dtype=torch.int32),
               status_dev=torch.zeros(1, dtype=torch.int32))
    for name, bad in (("slots_dev", torch.zeros(3, dtype=torch.int64)), ("slots_dev", torch.zeros(2, dtype=torch.int32)),
                      ("fresh_dev", torch.zeros(3, dtype=torch.int32)), ("fresh_dev", torch.zeros(2, dtype=torch.uint8)),
                      ("num_seqs_dev", torch.zeros(2, dtype=torch.int32)), ("status_dev", torch.zeros(1))):
        with pytest.raises(ValueError):
            ss.gated_delta_rule_step_device(**t, **{**dev, name: bad}, stream=0)


BEAM = dict(batch=2, beams=3, out=4, vocab=100, ld=100, eos=7)


def beam(lib, ptrs=None, ws=WS, act=ss.F32, **kw):
    c = {**BEAM, **kw}
    return lib.mamba2_beam_select(*(ptrs or P[:7]), c["batch"], c["beams"], c["out"], c["vocab"], c["ld"], c["eos"], act, *ws, None)


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(beams=0), dict(beams=33), dict(out=0), dict(out=33), dict(vocab=0), dict(vocab=0x7fffffff, ld=1 << 40),
                                dict(ld=99), dict(eos=100), dict(eos=-2), dict(eos=-1), dict(batch=21846), dict(vocab=1, eos=0, out=4),
                                dict(act=ss.E4M3)], ids=str)
def test_beam_arguments(product_lib, kw):
    assert beam(product_lib, **kw) == INV


def test_beam_pointers_and_workspace(product_lib):
    for at in (0, 1, 2, 4, 5):
        for bad in (None, P[at] + 2):
            ptrs = P[:7]
            ptrs[at] = bad
            assert beam(product_lib, ptrs) == INV
    ptrs = P[:7]
    ptrs[0] = ptrs[5]
    assert beam(product_lib, ptrs) == INV
    ptrs = P[:7]
    ptrs[3] = ptrs[6]
    assert beam(product_lib, ptrs) == INV
    assert beam(product_lib, ws=(None, 1 << 40)) == SMALL and beam(product_lib, ws=(P[18], 255)) == SMALL
    assert beam(product_lib, ws=(P[18] + 16, 1 << 40)) == INV
    assert beam(product_lib, [None] * 7, batch=0) == ss.OK
    for kw in (dict(batch=0), dict(beams=33), dict(out=0), dict(vocab=0), dict(batch=21846)):
        c = {**BEAM, **kw}
        assert product_lib.mamba2_beam_select_workspace_bytes(c["batch"], c["beams"], c["out"], c["vocab"]) == 0


def test_beam_tensors(product_lib):
    good = dict(scores_out=torch.zeros((2, 4)), parents=torch.zeros((2, 4), dtype=torch.int32), tokens=torch.zeros((2, 4), dtype=torch.int32),
                logits=torch.zeros((6, 100)), scores=torch.zeros((2, 3)), finished=torch.zeros((2, 3), dtype=torch.uint8),
                finished_out=torch.zeros((2, 4), dtype=torch.uint8), eos=3)
    for name, bad in (("logits", torch.zeros((5, 100))), ("logits", torch.zeros((6, 200))[:, ::2]), ("scores", torch.zeros((2, 3)).double()),
                      ("parents", torch.zeros((2, 4), dtype=torch.int64)), ("tokens", torch.zeros((2, 3), dtype=torch.int32)),
                      ("finished", torch.zeros((2, 4), dtype=torch.uint8)), ("finished_out", torch.zeros((2, 4))), ("eos", 100), ("eos", -1)):
        with pytest.raises(ValueError):
            ss.beam_select(**{**good, name: bad}, stream=0)
    with pytest.raises(TypeError):
        ss.beam_select(**{**good, "logits": torch.zeros((6, 100), dtype=torch.float16)}, stream=0)


def reorder(lib, num_pools=2, num_slots=20, slots=P[3], parents=P[4], batch=2, beams=3, status=P[5], pools=(P[0], P[1]), sizes=(64, 64)):
    a, b = (ctypes.c_void_p * len(pools))(*pools), (ctypes.c_int64 * len(sizes))(*sizes)
    return lib.mamba2_reorder_states(a, b, num_pools, num_slots, slots, parents, batch, beams, status, None)


@pytest.mark.parametrize("kw", [dict(num_pools=-1), dict(num_pools=65), dict(num_slots=-1), dict(slots=None), dict(parents=None), dict(batch=-1),
                                dict(beams=0), dict(beams=33), dict(batch=400), dict(status=None), dict(status=P[5] + 2), dict(slots=P[3] + 1),
                                dict(pools=(P[0], None)), dict(sizes=(64, -1)), dict(sizes=(1 << 43, 64))], ids=str)
def test_reorder_arguments(product_lib, kw):
    assert reorder(product_lib, **kw) == INV


def test_pools_that_overlap(product_lib):
    """One pool twice, or two that share bytes, would be moved twice."""
    for second in (P[0], P[0] + 64 * 19, P[0] - 64 * 19):
        assert reorder(product_lib, pools=(P[0], second)) == INV
    pool, order, status = torch.zeros((9, 4)), torch.zeros((2, 3), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ss.Mamba2Error):
        ss.reorder_states([pool, pool], order, order, status, stream=0)


def test_reorder_tensors(product_lib):
    pool, order, status = torch.zeros((9, 4)), torch.zeros((2, 3), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for pools, slots, parents, st in (([pool, pool[:8]], order, order, status), ([pool], order.long(), order, status),
                                      ([pool], order, order[:1], status), ([pool], order, order, status.long()),
                                      ([pool[:, ::2]], order, order, status)):
        with pytest.raises(ValueError):
            ss.reorder_states(pools, slots, parents, st, stream=0)


def backward(lib, ptrs=None, ld=(256,) * 7, d=None, scale=1.0, eps=-1.0, act=ss.BF16, rows=3, cu=(0, 3), ws=WS):
    arr = (ctypes.c_int32 * max(1, len(cu)))(*cu)
    return lib.mamba2_gated_delta_rule_backward(*(ptrs or P[:14]), rows, *ld, d if d is not None else dims(), scale, eps, act, arr,
                                                len(cu) - 1, *ws, None)


# dq, dk, dv, dg, dbeta, dstate, dy, dstate_end, q, k, v, g, beta, checkpoints
@pytest.mark.parametrize("at", range(14))
def test_backward_pointers(product_lib, at):
    for bad in (None, P[at] + 8):
        if bad is None and at in (3, 4, 5, 7, 11, 12):  # optional
            continue
        ptrs = P[:14]
        ptrs[at] = bad
        assert backward(product_lib, ptrs) == INV
    if at < 5:  # an output over an input, or over another
        for other in list(range(6, 14)) + [i for i in range(5) if i != at]:
            ptrs = P[:14]
            ptrs[at] = ptrs[other]
            assert backward(product_lib, ptrs) == INV
    if at == 5:
        ptrs = P[:14]
        ptrs[5] = ptrs[7]
        assert backward(product_lib, ptrs) == INV


def test_backward_arguments(product_lib):
    lib = product_lib
    for change, want in ((dict(heads=0), INV), (dict(heads=3), INV), (dict(headdim=60), NOT), (dict(headdim=136), NOT), (dict(d_state=136), NOT)):
        assert backward(lib, d=dims(**change), ld=(1 << 20,) * 7) == want
    for i in range(7):
        short, odd = [256] * 7, [264] * 7
        short[i], odd[i] = 248, 260
        assert backward(lib, ld=short) == INV and backward(lib, ld=odd) == NOT
    assert backward(lib, act=ss.F32) == NOT and backward(lib, act=ss.E4M3) == INV
    assert backward(lib, scale=NAN) == INV and backward(lib, eps=NAN) == INV and backward(lib, rows=-1) == INV
    for cu in ((0, 2), (1, 3), (0, 4, 3), (0,)):
        assert backward(lib, cu=cu) == ss.ERR_RUNS_DONT_COVER_ROWS
    assert backward(lib, ws=(None, 1 << 40)) == SMALL and backward(lib, ws=(P[18], 1000)) == SMALL
    assert backward(lib, ws=(P[18] + 128, 1 << 40)) == INV
    assert backward(lib, [None] * 14, rows=0, cu=(0,)) == ss.OK


def test_chunked_forward_workspace(product_lib):
    """bf16 heads of at most 128 x 128 go by chunks, which take a workspace; the others do not."""
    b = ss.Batch([0, 3], [1], [0])
    for ws, want in (((None, 1 << 40), SMALL), ((P[18], 1000), SMALL), ((P[18] + 128, 1 << 40), INV)):
        assert product_lib.mamba2_gated_delta_rule(*P[:8], 5, 3, 256, 256, 256, 256, dims(), 1.0, -1.0, ss.BF16, b.ref(), *ws, None) == want
    assert ss.gated_delta_rule_workspace_bytes([0, 65], 4, 64, 128, 2, torch.bfloat16) > 0
    assert ss.gated_delta_rule_workspace_bytes([0, 65], 4, 64, 128, 2, torch.float32) == 0
    assert ss.gated_delta_rule_workspace_bytes([0, 65], 4, 136, 128, 2, torch.bfloat16) == 0


@pytest.mark.parametrize("name,bad", [("dq", lambda t: t[:2]), ("dk", lambda t: t.float()), ("dv", lambda t: t[:, :2]), ("dg", lambda t: t.float()),
                                      ("dbeta", lambda t: t[:, :3]), ("dstate", lambda t: t[:, :, :, :8]), ("dstate_end", lambda t: t.double()),
                                      ("dy", lambda t: t.float()), ("checkpoints", lambda t: t[:0]), ("q", lambda t: t[:2])], ids=str)
def test_backward_tensors(product_lib, name, bad):
    t = delta_tensors()
    state = t.pop("state")
    y = t.pop("y")
    t.update(dq=t["q"].clone(), dk=t["q"].clone(), dv=y.clone(), dg=t["g"].bfloat16(), dbeta=t["g"].bfloat16(), dstate=state[:1].clone(),
             dy=y.clone(), dstate_end=state[:1].clone(), checkpoints=state[:1].clone())
    t[name] = bad(t[name])
    with pytest.raises(ValueError):
        ss.gated_delta_rule_backward(**t, cu_seqlens=[0, 3], stream=0)
