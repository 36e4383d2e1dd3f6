"""The delta-rule block as a user runs it: serving (prefill, decode from a captured graph), a training step against the
block written out in 64 bits with torch's own derivatives, and a beam search over its states.

The block rounds to bf16 between its operators, so it is compared as a whole: every value by 2-norm. Each of the at most
eight roundings on a path is off by at most 2^-9 of the 2-norm on average of its signs (2^-8 at worst); the bound is
2e-2, five such worst roundings. What comes of g passes through exp, whose argument's bf16 rounding is relative to |g|
of at most about 2 here: the same bound."""
import pytest
import torch

import selective_scan_gb300 as ss
from selective_scan_gb300.beams import Beams, sequences
from selective_scan_gb300.delta_block import DeltaBlock, DeltaBlockWeights
from tests.gpu_util import device
from tests.util import assert_bits_equal, rel_l2

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BOUND = 2e-2
TENSORS = ("norm_w", "w_qkv", "w_ab", "b_ab", "A_log", "w_out")


def weights(d_model, groups, heads, d_state, headdim):
    g = torch.Generator().manual_seed(5)
    n = lambda *s, std=1.0, mean=0.0: torch.randn(s, generator=g) * std + mean  # noqa: E731
    wide = 2 * groups * d_state + heads * headdim
    return DeltaBlockWeights(
        norm_w=n(d_model, std=0.2, mean=1.0), w_qkv=n(wide, d_model, std=d_model ** -0.5).to(BF16),
        w_ab=n(2 * heads, d_model, std=d_model ** -0.5).to(BF16),
        b_ab=torch.cat([n(heads, std=0.3, mean=-2.0), n(heads, std=0.3)]), A_log=n(heads, std=0.3),
        w_out=n(d_model, heads * headdim, std=(heads * headdim) ** -0.5).to(BF16), groups=groups, d_state=d_state)


def changed(w, f):
    return DeltaBlockWeights(**{k: f(v) if isinstance(v, torch.Tensor) else v for k, v in vars(w).items()})


def reference(w, hidden, delta, h0, cu):
    """(out, end states) in 64 bits; the arguments may require gradients."""
    heads, groups, N = w.A_log.shape[0], w.groups, w.d_state
    s = hidden + (delta if delta is not None else 0.0)
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + w.eps) * w.norm_w
    p, ab = n @ w.w_qkv.T, n @ w.w_ab.T + w.b_ab
    p = p * torch.sigmoid(p)
    unit = lambda x: x / torch.sqrt((x * x).sum(-1, keepdim=True) + w.l2_eps)  # noqa: E731
    q, k = (unit(x.unflatten(1, (groups, N))).repeat_interleave(heads // groups, 1) for x in (p[:, :groups * N], p[:, groups * N:2 * groups * N]))
    v = p[:, 2 * groups * N:].unflatten(1, (heads, -1))
    a, beta = torch.exp(-torch.exp(w.A_log) * torch.log1p(torch.exp(ab[:, :heads]))), torch.sigmoid(ab[:, heads:])
    rows, ends = [], []
    for i in range(len(cu) - 1):
        S = h0[i]
        for t in range(cu[i], cu[i + 1]):
            S = a[t][:, None, None] * S
            u = beta[t][:, None] * (v[t] - (S * k[t][:, None, :]).sum(-1))
            S = S + u[..., None] * k[t][:, None, :]
            rows.append((S * q[t][:, None, :]).sum(-1).flatten() * N ** -0.5)
        ends.append(S)
    return torch.stack(rows) @ w.w_out.T + s, torch.stack(ends)


def inputs(rows, d_model, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((rows, d_model), generator=g).to(BF16), torch.randn((rows, d_model), generator=g).to(BF16)


@pytest.mark.parametrize("groups,heads,d_state,headdim,with_delta", [(2, 4, 32, 48, True), (1, 1, 128, 128, False)])
def test_prefill_then_decode_in_a_graph(groups, heads, d_state, headdim, with_delta):
    dev = device()
    d_model, lengths, steps = 128, [150, 3, 40], 6
    w = weights(d_model, groups, heads, d_state, headdim)
    full = [n + steps for n in lengths]
    cu = [0, full[0], full[0] + full[1], sum(full)]
    hidden, delta = inputs(cu[-1], d_model)
    h0 = torch.randn((3, heads, headdim, d_state), generator=torch.Generator().manual_seed(2)).double() * 0.3
    h0[0] = 0
    want, ends = reference(changed(w, lambda t: t.double()), hidden.double(), delta.double() if with_delta else None, h0, cu)
    block = DeltaBlock(changed(w, lambda t: t.to(dev)))
    slots = [4, 0, 2]
    at = torch.tensor(slots, device=dev)
    pool = block.state_pool(5, dev)
    pool[at] = h0.float().to(dev)
    pool[4] = float("nan")  # the fresh run's slot is not read
    head = torch.cat([torch.arange(cu[i], cu[i] + lengths[i]) for i in range(3)])
    take = lambda t, idx: t[idx].to(dev) if with_delta else None  # noqa: E731
    got = block.prefill(hidden[head].to(dev), take(delta, head), pool, [0, 150, 153, 193], slots, [1, 0, 0])
    assert rel_l2(got.cpu(), want[head]) <= BOUND
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
        assert rel_l2(step_out.cpu(), want[idx]) <= BOUND
    assert rel_l2(pool[at].cpu(), ends) <= BOUND


@pytest.mark.parametrize("groups,heads,d_state,headdim,with_delta", [(2, 4, 32, 24, True), (1, 2, 64, 64, False)])
def test_training_step(groups, heads, d_state, headdim, with_delta):
    dev = device()
    d_model, cu = 128, [0, 140, 140, 143, 300]
    w = weights(d_model, groups, heads, d_state, headdim)
    hidden, delta = inputs(300, d_model, 7)
    shape = (4, heads, headdim, d_state)
    h0 = torch.randn(shape, generator=torch.Generator().manual_seed(8)) * 0.3
    dout = inputs(300, d_model, 9)[0]
    dend = torch.randn(shape, generator=torch.Generator().manual_seed(10)) * 0.3
    wd = changed(w, lambda t: t.double().requires_grad_())
    hd, h0d = hidden.double().requires_grad_(), h0.double().requires_grad_()
    out, ends = reference(wd, hd, delta.double() if with_delta else None, h0d, cu)
    ((out * dout.double()).sum() + (ends * dend.double()).sum()).backward()
    block = DeltaBlock(changed(w, lambda t: t.to(dev)))
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
    for name in TENSORS:
        assert rel_l2(g[name].cpu(), getattr(wd, name).grad) <= BOUND, name
    for name, v in results[1][2].items():  # the same on a side stream
        assert_bits_equal(v.cpu(), g[name].cpu(), name)


@pytest.mark.parametrize("ends", [False, True])
def test_beam_search_over_the_blocks_states(ends):
    """Prompts, then a captured step replayed: decode, logits, selection, reordering. Every hypothesis that comes out has
    the state and the score that running its own tokens gives; with an end token that one beam starts with."""
    dev = device()
    d_model, vocab, B, beams, steps = 64, 97, 3, 4, 9
    w = changed(weights(d_model, 1, 2, 32, 24), lambda t: t.to(dev))
    block = DeltaBlock(w)
    g = torch.Generator().manual_seed(3)
    table = torch.randn((vocab, d_model), generator=g).to(BF16).to(dev)
    w_head = (torch.randn((vocab, d_model), generator=g) * 0.5).to(BF16).to(dev)
    prompts = [torch.randint(0, vocab, (n,), generator=g) for n in (70, 1, 13)]
    cu = [0, 70, 71, 84]
    slots = torch.randperm(B * beams + 3, generator=g)[:B * beams].view(B, beams).int()
    first = slots[:, 0].tolist()
    pool = block.state_pool(B * beams + 3, dev)
    pool.normal_()  # what the slots held before

    def head(x):
        out = torch.empty((x.shape[0], vocab), dtype=F32, device=dev)
        ss.linear(out, x.contiguous(), w_head)
        return out

    hidden = block.prefill(table[torch.cat(prompts).to(dev)], None, pool, cu, first, [1] * B)
    prompt_pool = pool.clone()
    last = head(hidden[torch.tensor([c - 1 for c in cu[1:]], device=dev)])
    eos = int(last[0].topk(2).indices[1]) if ends else None
    search = Beams(slots.to(dev), [pool], eos=eos)
    search.advance(last.repeat_interleave(beams, 0))
    flat = search.slots.flatten()
    count, status = torch.tensor([B * beams], dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    tokens, parents = [search.tokens.clone()], [search.parents.clone()]

    def step():
        x = block.decode(table[search.tokens.flatten().long()], None, pool, flat, None, count, status)
        search.advance(head(x))

    keep = [t.clone() for t in (pool, search.scores, search.tokens, search.parents) + ((search.finished,) if eos is not None else ())]
    step()  # warm-up
    for t, k in zip((pool, search.scores, search.tokens, search.parents, search.finished), keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        assert int(status) == ss.OK and int(search.status) == ss.OK
        tokens.append(search.tokens.clone())
        parents.append(search.parents.clone())
    found = sequences(tokens, parents).cpu()
    scores, states = search.scores.cpu(), pool[search.slots.long()].cpu()
    assert (scores[:, :-1] >= scores[:, 1:]).all() and torch.isfinite(scores).all()
    ended = 0
    for b in range(B):
        assert len({tuple(s.tolist()) for s in found[b]}) == beams or eos is not None
        for j in range(beams):
            path = found[b, j].tolist()
            if eos is not None and eos in path:
                path = path[:path.index(eos) + 1]
                ended += 1
            # the tokens again from the prompt's state (all but the last have been decoded), token by token as the search did
            again = prompt_pool[first[b]:first[b] + 1].clone()
            one, st = torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
            logp, logits = 0.0, last[b:b + 1]
            for i, tok in enumerate(path):
                logp += float(torch.log_softmax(logits.double(), 1)[0, tok])
                if i + 1 < len(path):
                    x = block.decode(table[tok:tok + 1], None, again, one, None, torch.ones_like(one), st)
                    logits = head(x)
            # fp32 scores, a rounding of at most 2^-24 of the sum a step; a batch of one and of twelve round logits alike,
            # but for the order of fp32 sums of products of bf16 numbers: 1e-3
            assert abs(logp - float(scores[b, j])) <= 1e-3 * max(1.0, abs(logp)), (b, j)
            if len(path) == steps + 1:
                assert rel_l2(states[b, j], again[0].cpu()) <= 1e-2
    if eos is not None:
        over = torch.tensor([[eos in s.tolist() for s in found[b]] for b in range(B)])
        assert torch.equal(search.finished.cpu() != 0, over) and ended == int(over.sum())
