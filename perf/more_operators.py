"""What the operators for recurrent decoding are measured on: the gated delta rule (prefill over packed runs,
single-token step, training), beam search's selection over beams and vocabulary, and the reordering of recurrent
states that follows it.

``own`` false: each operator in elementary torch operations in 32 bits (64 for sums of log decays and for the scores
that decide between candidates), rounded once at the end. ``own`` true: the calls of selective_scan_gb300 that a user
makes. ``exact``: the definition in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
SIZE = {BF16: 2, F32: 4}
L2_EPS = 1e-6
CHUNK = 64  # tokens that the plain form takes at once


def listed():
    return [
        # one user's next token: latency alone
        dict(name="step_1", op="delta", mode="step", seqs=1, groups=16, heads=32, d_state=128, headdim=128, type=BF16,
             l2=True, fused=True),
        # a full decode batch over a pool of twice as many slots
        dict(name="step_256", op="delta", mode="step", seqs=256, groups=8, heads=16, d_state=128, headdim=128,
             type=BF16, l2=True, fused=True),
        # a ragged batch of short prompts at 32 bits, some resumed, some of no token; heads of odd widths
        dict(name="prefill_ragged", op="delta", mode="prefill", tokens=3109, seqs=13, groups=3, heads=6, d_state=72,
             headdim=104, type=F32, l2=False, fused=False),
        # a prefill batch of prompts
        dict(name="prefill_prompts", op="delta", mode="prefill", tokens=16384, seqs=24, groups=8, heads=16,
             d_state=128, headdim=128, type=BF16, l2=True, fused=True),
        # one long document
        dict(name="prefill_long", op="delta", mode="prefill", tokens=32768, seqs=1, groups=16, heads=32, d_state=128,
             headdim=128, type=BF16, l2=True, fused=True),
        # a small training batch, every head with its own keys, as they are
        dict(name="train_small", op="delta", mode="train", tokens=1777, seqs=3, groups=4, heads=4, d_state=64,
             headdim=64, type=BF16, l2=False, fused=False),
        # a training batch: the forward pass that keeps what the backward needs, then the backward
        dict(name="train_batch", op="delta", mode="train", tokens=8192, seqs=8, groups=8, heads=16, d_state=128,
             headdim=128, type=BF16, l2=True, fused=False),
        # one user's beams: latency alone
        dict(name="beam_4", op="beam", batch=1, beams=4, out=4, vocab=50277, type=F32, finished=False),
        # as many candidates as keep a live beam for each that ends
        dict(name="beam_double", op="beam", batch=16, beams=5, out=10, vocab=32001, type=F32, finished=True),
        # a full batch
        dict(name="beam_512", op="beam", batch=64, beams=8, out=8, vocab=131072, type=BF16, finished=True),
        # one layer's states of one user's beams
        dict(name="reorder_4", op="reorder", batch=1, beams=4, layers=1, heads=16, d_state=128, headdim=64, type=BF16),
        # a model's states of a batch of beams
        dict(name="reorder_64", op="reorder", batch=16, beams=4, layers=12, heads=16, d_state=128, headdim=128,
             type=BF16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "beam", "reorder"])
    if op == "delta":
        mode = rng.choice(["step", "prefill", "prefill", "train"])
        groups, per = _log_int(rng, 1, 16), rng.choice([1, 1, 2, 3, 4])
        heads = min(32, groups * per) // groups * groups
        c = dict(op=op, mode=mode, groups=groups, heads=heads, d_state=8 * _log_int(rng, 2, 16),
                 headdim=8 * _log_int(rng, 2, 16), type=rng.choice([BF16, BF16, F32]) if mode != "train" else BF16,
                 l2=rng.random() < 0.7, fused=rng.random() < 0.5)
        c["seqs"] = _log_int(rng, 1, 256 if mode == "step" else 32)
        one = heads * c["d_state"] * c["headdim"]
        if mode == "step":
            c["seqs"] = max(1, min(c["seqs"], 256 * 16 * 128 * 128 // one))
        else:
            most = {"prefill": 32768 * 32, "train": 8192 * 16}[mode] * 128 * 128 // one
            c["tokens"] = _log_int(rng, 1, min({"prefill": 32768, "train": 16384}[mode], most) // (2 if c["type"] == F32 else 1))
        return c
    if op == "beam":
        beams = _log_int(rng, 1, 16)
        vocab = _log_int(rng, 1000, 131072)
        t = rng.choice([BF16, F32])
        return dict(op=op, beams=beams, out=beams * rng.choice([1, 1, 2]), vocab=vocab, type=t,
                    batch=_log_int(rng, 1, max(1, min(64, 64 * 8 * 131072 // (beams * vocab) // (2 if t == F32 else 1)))),
                    finished=rng.random() < 0.5)
    beams, layers = _log_int(rng, 2, 16), _log_int(rng, 1, 16)
    heads, d_state, headdim = _log_int(rng, 1, 32), 8 * _log_int(rng, 2, 16), 8 * _log_int(rng, 2, 16)
    most = 64 * 12 * 16 * 128 * 128 // (beams * layers * heads * d_state * headdim)
    return dict(op=op, beams=beams, layers=layers, heads=heads, d_state=d_state, headdim=headdim,
                batch=_log_int(rng, 1, max(1, min(1024 // beams, most))), type=rng.choice([BF16, F32]))


# ---------------------------------------------------------------- inputs

def _lengths(tokens, seqs, seed):
    """Ragged run lengths that add up to `tokens`; a few of many runs are empty."""
    r = random.Random(seed * 1009 + seqs)
    if seqs == 1:
        return [tokens]
    w = [0.0 if seqs > 4 and r.random() < 0.08 else r.uniform(0.2, 1.8) for _ in range(seqs)]
    if not sum(w):
        w[0] = 1.0
    total, at, cuts = sum(w), 0.0, [0]
    for v in w:
        at += v
        cuts.append(int(round(tokens * at / total)))
    cuts[-1] = tokens
    return [b - a for a, b in zip(cuts[:-1], cuts[1:])]


def _parents(batch, beams, seed):
    r = random.Random(seed * 7919 + beams)
    return [[r.randrange(beams) for _ in range(beams)] for _ in range(batch)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    t = DTYPE[case["type"]]
    s = dict(case)
    r = random.Random(seed * 31 + 7)

    def normal(shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(std).add_(mean)

    def uniform(shape, lo, hi):
        return torch.rand(shape, generator=g, device=dev).mul_(hi - lo).add_(lo)

    if case["op"] == "delta":
        n, H, K, N, P = case["seqs"], case["heads"], case["groups"], case["d_state"], case["headdim"]
        rows = n if case["mode"] == "step" else case["tokens"]
        silu = torch.nn.functional.silu
        q, k, v = silu(normal((rows, K * N), 1.5)), silu(normal((rows, K * N), 1.5)), silu(normal((rows, H * P), 1.5))
        if not case["l2"]:  # keys of about unit length, as a model that does not normalise them keeps them
            k = normal((rows, K * N), 0.8 / math.sqrt(N))
        if case["fused"]:  # ranges of one projection's output
            wide = torch.cat([q, k, v], 1).to(t)
            q, k, v = wide[:, :K * N], wide[:, K * N:2 * K * N], wide[:, 2 * K * N:]
        else:
            q, k, v = q.to(t), k.to(t), v.to(t)
        s["q"], s["k"], s["v"] = q.unflatten(1, (K, N)), k.unflatten(1, (K, N)), v.unflatten(1, (H, P))
        s["g"] = -uniform((H,), 1.0, 16.0) * torch.nn.functional.softplus(normal((rows, H), 1.0, -4.0))
        s["beta"] = torch.sigmoid(normal((rows, H)))
        s["slots"] = r.sample(range(2 * n), n)
        s["pool"] = normal((2 * n, H, P, N), 0.1)
        s["fresh"] = [0] * n if case["mode"] == "step" else [int(r.random() < 0.5) for _ in range(n)]
        s["slots_dev"] = torch.tensor(s["slots"], dtype=torch.int32, device=dev)
        s["fresh_dev"] = torch.tensor(s["fresh"], dtype=torch.uint8, device=dev)
        if case["mode"] == "step":
            s["count_dev"] = torch.tensor([n], dtype=torch.int32, device=dev)
            s["status_dev"] = torch.zeros(1, dtype=torch.int32, device=dev)
        else:
            cu = [0]
            for m in _lengths(rows, n, seed):
                cu.append(cu[-1] + m)
            s["cu"] = cu
            # where the chunks' tokens are (`rows` itself where there is none), and which chunk of which run comes when
            where, turns = [], []
            for i in range(n):
                for c, at in enumerate(range(cu[i], cu[i + 1], CHUNK)):
                    if c == len(turns):
                        turns.append(([], []))
                    turns[c][0].append(i)
                    turns[c][1].append(len(where))
                    where.append([at + j if at + j < cu[i + 1] else rows for j in range(CHUNK)])
            s["where"] = torch.tensor(where, dtype=torch.int64, device=dev).view(-1, CHUNK)
            s["turns"] = [(torch.tensor(a, device=dev), torch.tensor(b, device=dev)) for a, b in turns]
        if case["mode"] == "train":
            s["dy"] = normal((rows, H, P)).to(t)
            s["dstate_end"] = normal((n, H, P, N), 0.1)
    elif case["op"] == "beam":
        B, b, V = case["batch"], case["beams"], case["vocab"]
        logits = normal((B * b, V), 2.5)
        logits[torch.rand((B * b, V), generator=g, device=dev) < 0.02] = -math.inf  # tokens that may not follow
        s["logits"] = logits.to(t)
        s["scores"] = -uniform((B, b), 0.0, 6.0).sort(1).values
        if r.random() < 0.3 and b > 1:  # the first token: one beam, the others not yet in being
            s["scores"][:, 1:] = -math.inf
        s["done"] = (torch.rand((B, b), generator=g, device=dev) < 0.2).to(torch.uint8) if case["finished"] else None
        s["eos"] = r.randrange(V)
    else:
        B, b, L = case["batch"], case["beams"], case["layers"]
        H, N, P = case["heads"], case["d_state"], case["headdim"]
        slots = r.sample(range(B * b + 8), B * b)
        s["slots_dev"] = torch.tensor(slots, dtype=torch.int32, device=dev).view(B, b)
        s["parents"] = torch.tensor(_parents(B, b, seed), dtype=torch.int32, device=dev)
        s["status_dev"] = torch.zeros(1, dtype=torch.int32, device=dev)
        s["pools"] = []
        for _ in range(L):  # a layer's convolution history and its state
            s["pools"] += [normal((B * b + 8, 3, H * P)).to(t), normal((B * b + 8, H, P, N))]
    return s


# ---------------------------------------------------------------- plain forms

def _units(s, q, k):
    """q with the scale and k, divided by their lengths where the model does so."""
    if s["l2"]:
        q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + L2_EPS)
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + L2_EPS)
    return q / math.sqrt(s["d_state"]), k


def _plain_step(s):
    act, pool, slots = s["v"].dtype, s["pool"], s["slots_dev"].long()
    per = s["heads"] // s["groups"]
    q, k = _units(s, s["q"].float(), s["k"].float())
    q, k, v = q.repeat_interleave(per, 1), k.repeat_interleave(per, 1), s["v"].float()
    S = torch.where(s["fresh_dev"].bool()[:, None, None, None], 0, pool[slots]) * torch.exp(s["g"])[:, :, None, None]
    u = s["beta"][:, :, None] * (v - (S * k[:, :, None, :]).sum(-1))
    S = S + u[..., None] * k[:, :, None, :]
    pool[slots] = S
    return [(S * q[:, :, None, :]).sum(-1).to(act), pool]


def _chunked(s, q, k, v, g, beta, S):
    """y and the end states from fp32 inputs, chunks of 64 tokens, all runs' at a time."""
    rows, per, where = v.shape[0], s["heads"] // s["groups"], s["where"]
    q, k = _units(s, q, k)

    def cut(x):  # [chunks, heads, CHUNK, ...], zeros where there is no token
        x = torch.cat([x, x.new_zeros((1,) + x.shape[1:])])[where]
        return x.transpose(1, 2)

    q, k, v, beta = cut(q.repeat_interleave(per, 1)), cut(k.repeat_interleave(per, 1)), cut(v), cut(beta)
    G = cut(g.double()).cumsum(-1)
    low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=v.device).tril()
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
    up, left = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    A = beta[..., None] * (k @ k.transpose(-1, -2)) * D
    eye = torch.eye(CHUNK, device=v.device).expand(A.shape)
    T = eye[..., :1, :]
    for i in range(1, CHUNK):  # (I + A)^-1, a row from those above it
        T = torch.cat([T, eye[..., i:i + 1, :] - A[..., i:i + 1, :i] @ T], -2)
    W, U0 = T @ (beta[..., None] * up * k), T @ (beta[..., None] * v)
    scores = (q @ k.transpose(-1, -2)) * D
    end, ys, order = S, [], []
    for runs, chunks in s["turns"]:
        S0 = end[runs]
        U = U0[chunks] - W[chunks] @ S0.transpose(-1, -2)
        ys.append((up[chunks] * q[chunks]) @ S0.transpose(-1, -2) + scores[chunks] @ U)
        order.append(chunks)
        end = end.index_copy(0, runs, up[chunks, :, -1:] * S0 + U.transpose(-1, -2) @ (left[chunks] * k[chunks]))
    y = torch.cat(ys)[torch.argsort(torch.cat(order))].transpose(1, 2).flatten(0, 1)
    return y[torch.argsort(where.flatten(), stable=True)[:rows]], end


def _plain_delta(s):
    if s["mode"] == "step":
        return _plain_step(s)
    act, pool, slots = s["v"].dtype, s["pool"], s["slots_dev"].long()
    S = torch.where(s["fresh_dev"].bool()[:, None, None, None], 0, pool[slots])
    args = [x.float() for x in (s["q"], s["k"], s["v"], s["g"], s["beta"], S)]
    if s["mode"] == "prefill":
        y, end = _chunked(s, *args)
        pool[slots] = end
        return [y.to(act), pool]
    with torch.enable_grad():
        args = [x.detach().requires_grad_() for x in args]
        y, end = _chunked(s, *args)
        dq, dk, dv, dg, dbeta, dS = torch.autograd.grad([y, end], args, [s["dy"].float(), s["dstate_end"]])
    pool[slots] = end.detach()
    return [y.detach().to(act), pool, dq.to(act), dk.to(act), dv.to(act), dg.to(act), dbeta.to(act), dS]


def _plain_beam(s):
    B, b, V = s["batch"], s["beams"], s["vocab"]
    x = s["logits"].double().view(B, b, V)
    top = x.amax(-1, keepdim=True)
    x = s["scores"].double()[:, :, None] + (x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))))
    x = torch.where(torch.isnan(x), -math.inf, x)
    if s["done"] is not None:  # a finished beam goes on as it is
        only = torch.arange(V, device=x.device) == s["eos"]
        x = torch.where(s["done"].bool()[:, :, None], torch.where(only, s["scores"].double()[:, :, None], -math.inf), x)
    value, at = torch.sort(x.view(B, b * V), dim=1, descending=True, stable=True)
    value, at = value[:, :s["out"]], at[:, :s["out"]]
    parents, tokens = at // V, at % V
    out = [value.float(), parents.int(), tokens.int()]
    if s["done"] is None:
        return out
    return out + [(torch.gather(s["done"], 1, parents).bool() | (tokens == s["eos"])).to(torch.uint8)]


def _plain_reorder(s):
    slots = s["slots_dev"].long()
    source = torch.gather(slots, 1, s["parents"].long())
    for pool in s["pools"]:
        pool[slots.flatten()] = pool[source.flatten()]
    return s["pools"]


# ---------------------------------------------------------------- the framework's calls

def _own_delta(s):
    import selective_scan_gb300 as ss
    q, k, v, g, beta, pool = s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"]
    eps = L2_EPS if s["l2"] else None
    y = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if s["mode"] == "step":
        ss.gated_delta_rule_step_device(y, q, k, v, g, beta, pool, s["slots_dev"], s["fresh_dev"], s["count_dev"],
                                        s["status_dev"], l2_eps=eps)
        return [y, pool]
    if s["mode"] == "prefill":
        ss.gated_delta_rule(y, q, k, v, g, beta, pool, s["cu"], s["slots"], s["fresh"], l2_eps=eps)
        return [y, pool]
    kept = torch.empty((ss.gated_delta_rule_checkpoints(s["cu"]),) + pool.shape[1:], dtype=torch.float32, device=v.device)
    ss.gated_delta_rule(y, q, k, v, g, beta, pool, s["cu"], s["slots"], s["fresh"], l2_eps=eps, checkpoints=kept)
    dq, dk, dv, dg, dbeta = (torch.empty(x.shape, dtype=v.dtype, device=v.device) for x in (q, k, v, g, beta))
    dS = torch.empty_like(s["dstate_end"])
    ss.gated_delta_rule_backward(dq, dk, dv, dg, dbeta, dS, s["dy"], s["dstate_end"], q, k, v, g, beta, kept, s["cu"],
                                 l2_eps=eps)
    return [y, pool, dq, dk, dv, dg, dbeta, dS]


def _own_beam(s):
    import selective_scan_gb300 as ss
    shape, dev = (s["batch"], s["out"]), s["logits"].device
    scores = torch.empty(shape, dtype=torch.float32, device=dev)
    parents, tokens = (torch.empty(shape, dtype=torch.int32, device=dev) for _ in range(2))
    done = torch.empty(shape, dtype=torch.uint8, device=dev) if s["done"] is not None else None
    ss.beam_select(scores, parents, tokens, s["logits"], s["scores"], finished=s["done"], finished_out=done,
                   eos=s["eos"] if done is not None else None)
    return [scores, parents, tokens] + ([done] if done is not None else [])


def _own_reorder(s):
    import selective_scan_gb300 as ss
    ss.reorder_states(s["pools"], s["slots_dev"], s["parents"], s["status_dev"])
    return s["pools"]


def run(state):
    op = state["op"]
    if own:
        return {"delta": _own_delta, "beam": _own_beam, "reorder": _own_reorder}[op](state)
    return {"delta": _plain_delta, "beam": _plain_beam, "reorder": _plain_reorder}[op](state)


# ---------------------------------------------------------------- floors

def work(case):
    e = SIZE[case["type"]]
    if case["op"] == "delta":
        n, H, K, N, P = case["seqs"], case["heads"], case["groups"], case["d_state"], case["headdim"]
        T = n if case["mode"] == "step" else case["tokens"]
        states = 4 * n * H * P * N
        pass_bytes = T * (e * (2 * K * N + 2 * H * P) + 8 * H)  # q, k, v, g, beta in; y out
        # decay, correction (a product and its update) and output: 7 operations a state element and token
        if case["mode"] != "train":
            return {"bytes": pass_bytes + 2 * states, "flops": 7 * T * H * P * N}
        # the loss stands between the two directions, so the inputs are read by each; a state before each 64 tokens is
        # what the backward starts from
        back = T * (e * (4 * K * N + 3 * H * P) + 8 * H + 2 * e * H)
        kept = 2 * 4 * H * P * N * max(T // CHUNK, 1)
        return {"bytes": pass_bytes + back + kept + 4 * states, "flops": 24 * T * H * P * N}
    if case["op"] == "beam":
        B, b, V, k = case["batch"], case["beams"], case["vocab"], case["out"]
        return {"bytes": e * B * b * V + 4 * B * b + 12 * B * k + ((B * b + B * k) if case["finished"] else 0),
                "flops": 4 * B * b * V}
    B, b = case["batch"], case["beams"]
    one = case["layers"] * case["heads"] * case["headdim"] * (3 * e + 4 * case["d_state"])
    moved = sum(p != j for row in _parents(B, b, 1) for j, p in enumerate(row))
    read = sum(len({p for j, p in enumerate(row) if p != j}) for row in _parents(B, b, 1))
    return {"bytes": one * max(moved + read, 1) + 8 * B * b, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_delta(s):
    """Token by token over all runs at once (the runs still going at a token are the first ones)."""
    T, n, H, mode = torch.float64, s["seqs"], s["heads"], s["mode"]
    dev, per = s["pool"].device, s["heads"] // s["groups"]
    cu = list(range(n + 1)) if mode == "step" else s["cu"]
    lens = [b - a for a, b in zip(cu[:-1], cu[1:])]
    longest = max(lens)
    if mode == "train" and 8 * sum(lens) * H * s["headdim"] * s["d_state"] > 100e9:
        return None
    spread = torch.arange(H, device=dev) // per
    qr, kr = s["q"].to(T), s["k"].to(T)
    ql = kl = None
    if s["l2"]:
        ql, kl = torch.sqrt((qr ** 2).sum(-1) + L2_EPS), torch.sqrt((kr ** 2).sum(-1) + L2_EPS)
    qu, ku = (qr / ql[..., None], kr / kl[..., None]) if s["l2"] else (qr, kr)
    c = 1 / math.sqrt(s["d_state"])
    q, k, v = qu[:, spread] * c, ku[:, spread], s["v"].to(T)
    a, beta = torch.exp(s["g"].to(T)), s["beta"].to(T)
    pool = s["pool"].to(T)
    slots = s["slots_dev"].long()
    start = pool[slots]
    start[s["fresh_dev"].bool()] = 0
    order = sorted(range(n), key=lambda i: -lens[i])
    perm = torch.tensor(order, device=dev)
    first = torch.tensor([cu[i] for i in order], device=dev)
    going, alive = [], n
    for t in range(longest):
        while alive and lens[order[alive - 1]] <= t:
            alive -= 1
        going.append(alive)
    S = start[perm]
    y, before, us = torch.zeros_like(v), [], []
    for t, m in enumerate(going):
        at = first[:m] + t
        old = S[:m]
        dec = a[at][..., None, None] * old
        err = v[at] - torch.matmul(dec, k[at][..., None])[..., 0]
        new = dec + (beta[at][..., None] * err)[..., None] * k[at][..., None, :]
        y[at] = torch.matmul(new, q[at][..., None])[..., 0]
        if mode == "train":
            before.append(old.clone())
            us.append(err)
        S[:m] = new
    end = torch.empty_like(S)
    end[perm] = S
    pool[slots] = end
    if mode != "train":
        return [y, pool]
    dy = s["dy"].to(T)
    dS = s["dstate_end"].to(T)[perm]
    dqh, dkh, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(a), torch.zeros_like(a)
    for t in range(longest - 1, -1, -1):
        m = going[t]
        at = first[:m] + t
        old, err = before[t], us[t]
        before[t] = us[t] = None
        dec = a[at][..., None, None] * old
        u = beta[at][..., None] * err
        new = dec + u[..., None] * k[at][..., None, :]
        D = dS[:m] + dy[at][..., None] * q[at][..., None, :]  # of the state after the token
        dqh[at] = torch.matmul(dy[at][..., None, :], new)[..., 0, :]
        du = torch.matmul(D, k[at][..., None])[..., 0]
        dkh[at] = torch.matmul(u[..., None, :], D)[..., 0, :]
        dbeta[at] = (du * err).sum(-1)
        de = beta[at][..., None] * du
        dv[at] = de
        dkh[at] -= torch.matmul(de[..., None, :], dec)[..., 0, :]
        D = D - de[..., None] * k[at][..., None, :]
        dg[at] = (D * dec).sum((-1, -2))
        dS[:m] = a[at][..., None, None] * D
    dstate = torch.empty_like(dS)
    dstate[perm] = dS

    def gather(d, unit, length):
        d = d.unflatten(1, (s["groups"], per)).sum(2)
        return d if length is None else (d - unit * (d * unit).sum(-1, keepdim=True)) / length[..., None]

    return [y, pool, gather(dqh * c, qu, ql), gather(dkh, ku, kl), dv, dg, dbeta, dstate]


def _exact_beam(s):
    B, b, V, n = s["batch"], s["beams"], s["vocab"], s["out"]
    T = torch.float64
    values, places, ends = [], [], []
    for i in range(B):  # a beam's best `out` tokens hold its part of the best `out` of all
        best = []
        for j in range(b):
            old = float(s["scores"][i, j])
            if s["done"] is not None and int(s["done"][i, j]):
                best.append((-old, j * V + s["eos"]))
                best += [(math.inf, j * V + t) for t in range(min(V, n + 1)) if t != s["eos"]]
                continue
            row = s["logits"][i * b + j].to(T)
            logp = row - torch.logsumexp(row, 0) + old
            logp[torch.isnan(logp)] = -math.inf
            floor = torch.topk(logp, min(n, V)).values[-1]
            keep = torch.nonzero(logp >= floor)[:, 0]
            if float(floor) == -math.inf:
                keep = torch.cat([torch.nonzero(logp > floor)[:, 0], torch.nonzero(logp == floor)[:n, 0]])
            best += [(-x, j * V + t) for x, t in zip(logp[keep].tolist(), keep.tolist())]
        best = sorted(best)[:n]
        values.append([-x for x, _ in best])
        places.append([p for _, p in best])
        if s["done"] is not None:
            ends.append([int(s["done"][i, p // V]) or int(p % V == s["eos"]) for p in places[-1]])
    at = torch.tensor(places, dtype=torch.int64)
    out = [torch.tensor(values, dtype=T), (at // V).int(), (at % V).int()]
    return out + [torch.tensor(ends, dtype=torch.uint8)] if s["done"] is not None else out


def _exact_reorder(s):
    slots, parents = s["slots_dev"].tolist(), s["parents"].tolist()
    out = []
    for pool in s["pools"]:
        old, new = pool.to(torch.float64), pool.to(torch.float64)
        for row, up in zip(slots, parents):
            for j, p in enumerate(up):
                new[row[j]] = old[row[p]]
        out.append(new)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "beam": _exact_beam, "reorder": _exact_reorder}[case["op"]](s)
