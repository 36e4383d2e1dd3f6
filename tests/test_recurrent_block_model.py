"""The gated-recurrence block as a user runs it: serving (prefill, decode from a captured graph, 8-bit projections)
and a training step, against the block written out in 64 bits with torch's own derivatives.

The block rounds to bf16 between its operators, so it is compared as a whole: every value by 2-norm. Each of the
at most six roundings on a path is off by at most 2^-9 of the 2-norm on average of its signs (2^-8 at worst); the
bound is 1.5e-2, four such worst roundings. In 8 bits the norm's and the weights' roundings are at most 2^-4 each
and independent from value to value: 6e-2 of the branch, which the stream dilutes."""
import pytest
import torch

import selective_scan_gb300 as ss
from selective_scan_gb300.recurrent_block import RecurrentBlock, RecurrentBlockWeights, quantise_rows
from tests.gpu_util import device
from tests.util import assert_bits_equal, rel_l2

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
BOUND, BOUND8 = 1.5e-2, 6e-2


def weights(d_model, dim, bias=True):
    g = torch.Generator().manual_seed(5)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(s, generator=g) * std + mean  # noqa: E731
    return RecurrentBlockWeights(
        norm_w=n(d_model, std=0.2, mean=1.0), w_x=n(dim, d_model, std=d_model ** -0.5).to(BF16),
        b_x=n(dim, std=0.1) if bias else None, w_gate=n(dim, d_model, std=d_model ** -0.5).to(BF16),
        b_gate=n(dim, std=0.5, mean=1.5) if bias else None,
        lower=torch.rand(dim, generator=g) * 0.8 if bias else None,
        w_out=n(d_model, dim, std=dim ** -0.5).to(BF16), b_out=n(d_model, std=0.1) if bias else None)


def on(w, dev):
    return RecurrentBlockWeights(**{k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in vars(w).items()})


def reference(w, hidden, delta, h0, cu):
    """(out, end states) in 64 bits; the arguments may require gradients."""
    none = lambda t: t if t is not None else 0.0  # noqa: E731
    s = hidden + none(delta)
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + w.eps) * w.norm_w
    p = n @ w.w_x.T + none(w.b_x)
    x, gate = p * torch.sigmoid(p), n @ w.w_gate.T + none(w.b_gate)
    lo = none(w.lower)
    f, k = lo + (1 - lo) * torch.sigmoid(gate), (1 - lo) * torch.sigmoid(-gate)
    rows, ends = [], []
    for i in range(len(cu) - 1):
        h = h0[i]
        for t in range(cu[i], cu[i + 1]):
            h = f[t] * h + k[t] * x[t]
            rows.append(h)
        ends.append(h)
    return torch.stack(rows) @ w.w_out.T + none(w.b_out) + s, torch.stack(ends)


def doubles(w, grad=False):
    return RecurrentBlockWeights(**{k: v.double().requires_grad_(grad) if isinstance(v, torch.Tensor) else v
                                    for k, v in vars(w).items()})


def inputs(rows, d_model, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, d_model), generator=g).to(BF16), torch.randn((rows, d_model), generator=g).to(BF16)


@pytest.mark.parametrize("eight,bias,with_delta", [(False, True, True), (False, False, False), (True, True, True)])
def test_prefill_then_decode_in_a_graph(eight, bias, with_delta):
    dev = device()
    d_model, dim, lengths, steps = 128, 192, [150, 3, 40], 6
    w = weights(d_model, dim, bias)
    full = [n + steps for n in lengths]
    cu = [0, full[0], full[0] + full[1], sum(full)]
    hidden, delta = inputs(cu[-1], d_model)
    h0 = torch.randn((3, dim), generator=torch.Generator().manual_seed(2)).double() * torch.tensor([[0.0], [1.0], [1.0]])
    want, ends = reference(doubles(w), hidden.double(), delta.double() if with_delta else None, h0, cu)
    served = on(w, dev)
    if eight:
        served.w_x, served.x_scale = quantise_rows(served.w_x)
        served.w_gate, served.gate_scale = quantise_rows(served.w_gate)
    block = RecurrentBlock(served)
    slots = [4, 0, 2]
    pool = block.state_pool(5, dev)
    pool[torch.tensor(slots, device=dev)] = h0.float().to(dev)
    pool[4] = float("nan")  # the fresh run's slot is not read
    bound = BOUND8 if eight else BOUND
    head = torch.cat([torch.arange(cu[i], cu[i] + lengths[i]) for i in range(3)])
    take = lambda t, idx: t[idx].to(dev) if with_delta else None  # noqa: E731
    got = block.prefill(hidden[head].to(dev), take(delta, head), pool, [0, 150, 153, 193], slots, [1, 0, 0])
    assert rel_l2(got.cpu(), want[head]) <= bound
    # the rest token by token, replaying one captured step
    step_in, step_delta = torch.zeros((3, d_model), dtype=BF16, device=dev), torch.zeros((3, d_model), dtype=BF16, device=dev)
    batch = [torch.tensor(slots, dtype=torch.int32, device=dev), None, torch.tensor([3], dtype=torch.int32, device=dev),
             torch.zeros(1, dtype=torch.int32, device=dev)]
    keep = pool.clone()
    block.decode(step_in, step_delta if with_delta else None, pool, *batch)  # warm-up
    pool.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_out = block.decode(step_in, step_delta if with_delta else None, pool, *batch)
    for k in range(steps):
        idx = torch.tensor([cu[i] + lengths[i] + k for i in range(3)])
        step_in.copy_(hidden[idx])
        step_delta.copy_(delta[idx])
        graph.replay()
        assert int(batch[3].item()) == ss.OK
        assert rel_l2(step_out.cpu(), want[idx]) <= bound
    assert rel_l2(pool[torch.tensor(slots, device=dev)].cpu(), ends) <= bound


@pytest.mark.parametrize("bias,with_delta", [(True, True), (False, False)])
def test_training_step(bias, with_delta):
    dev = device()
    d_model, dim, cu = 128, 136, [0, 140, 140, 143, 300]
    w = weights(d_model, dim, bias)
    hidden, delta = inputs(300, d_model, 7)
    h0 = torch.randn((4, dim), generator=torch.Generator().manual_seed(8))
    dout = inputs(300, d_model, 9)[0]
    dend = torch.randn((4, dim), generator=torch.Generator().manual_seed(10)) * 0.3
    wd = doubles(w, True)
    hd, h0d = hidden.double().requires_grad_(), h0.double().requires_grad_()
    out, ends = reference(wd, hd, delta.double() if with_delta else None, h0d, cu)
    ((out * dout.double()).sum() + (ends * dend.double()).sum()).backward()
    block = RecurrentBlock(on(w, dev))
    args = [hidden.to(dev), delta.to(dev) if with_delta else None]
    results = []
    for stream in (None, torch.cuda.Stream()):
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pool = h0.to(dev)
        torch.cuda.synchronize()
        y, saved = block.forward(*args, pool, cu, [0, 1, 2, 3], [0, 0, 0, 0], stream=stream)
        g = block.backward(dout.to(dev), saved, dend.to(dev), stream=stream)
        torch.cuda.synchronize()
        results.append((y, pool, g))
    y, pool, g = results[0]
    assert rel_l2(y.cpu(), out.detach()) <= BOUND and rel_l2(pool.cpu(), ends.detach()) <= BOUND
    assert rel_l2(g["hidden"].cpu(), hd.grad) <= BOUND and rel_l2(g["state"].cpu(), h0d.grad) <= BOUND
    for name in ("norm_w", "w_x", "b_x", "w_gate", "b_gate", "lower", "w_out", "b_out"):
        if getattr(w, name) is None:
            assert g[name] is None
        else:
            assert rel_l2(g[name].cpu(), getattr(wd, name).grad) <= BOUND, name
    for name, v in results[1][2].items():  # the same on a side stream
        if v is not None:
            assert_bits_equal(v, g[name], name)
    with pytest.raises(ValueError):
        q = on(w, dev)
        q.w_x, q.x_scale = quantise_rows(q.w_x)
        RecurrentBlock(q).forward(*args, pool, cu, [0, 1, 2, 3], [0] * 4)
