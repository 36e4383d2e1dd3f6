"""What the recurrent block's operators are measured on: the gated linear recurrence (prefill, single-token
step, training), the RMS norm with the residual's addition (8-bit output, plain output, backward) and the
matrix product with bias, activation and residual (few rows, many rows, 8-bit operands, backward).

``own`` false: each operator in elementary torch operations in 32 bits, rounded once at the end. ``own`` true:
the calls of selective_scan_gb300 that a user makes. ``exact``: the definition in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32, E4M3 = "bf16", "f32", "e4m3"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
SIZE = {BF16: 2, F32: 4, E4M3: 1}
EPS = 1e-5
MAX8 = 448.0  # largest e4m3 value


def listed():
    return [
        # one user's next token: latency alone
        dict(name="step_1", op="recurrence", mode="step", seqs=1, dim=1536, type=BF16, lower=True, fused=True),
        # a full decode batch over a pool of twice as many slots
        dict(name="step_256", op="recurrence", mode="step", seqs=256, dim=2048, type=BF16, lower=True, fused=True),
        # a ragged prefill batch of prompts, some resumed, some of no token, at 32 bits
        dict(name="prefill_ragged", op="recurrence", mode="prefill", tokens=3109, seqs=13, dim=1536, type=F32,
             lower=False, fused=False),
        # one long document
        dict(name="prefill_long", op="recurrence", mode="prefill", tokens=65536, seqs=1, dim=2048, type=BF16,
             lower=True, fused=True),
        # a training batch: the forward pass that keeps what the backward needs, then the backward
        dict(name="train_recurrence", op="recurrence", mode="train", tokens=16384, seqs=8, dim=2048, type=BF16,
             lower=True, fused=False),
        # a decode batch's norm before an 8-bit projection; an odd number of rows
        dict(name="norm_8bit_decode", op="norm", mode="forward", rows=33, dim=1536, type=BF16, sum_type=BF16,
             out_type=E4M3, residual=True),
        # a training forward with the residual stream kept in 32 bits
        dict(name="norm_wide_sum", op="norm", mode="forward", rows=16384, dim=2560, type=BF16, sum_type=F32,
             out_type=BF16, residual=True),
        # its backward pass with everything in bf16
        dict(name="norm_backward", op="norm", mode="backward", rows=16384, dim=2048, type=BF16, sum_type=BF16,
             residual=True),
        # decode projections: a few tokens against a weight that is read once
        dict(name="linear_decode", op="linear", mode="forward", rows=5, inner=2048, out=8192, type=BF16,
             out_type=BF16, bias=True, residual=False, act="silu"),
        # prefill projection with everything in the epilogue
        dict(name="linear_epilogue", op="linear", mode="forward", rows=16384, inner=2048, out=4096, type=BF16,
             out_type=BF16, bias=True, residual=True, act="silu"),
        # the same work with 8-bit operands and their scales; rows that fill no tile
        dict(name="linear_8bit", op="linear", mode="forward", rows=16001, inner=4096, out=4096, type=E4M3,
             out_type=BF16, bias=True, residual=True, act="none"),
        # backward of the expanding projection
        dict(name="linear_backward", op="linear", mode="backward", rows=8192, inner=2048, out=4096, type=BF16,
             bias=True, act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["recurrence", "recurrence", "norm", "linear", "linear"])
    if op == "recurrence":
        mode = rng.choice(["step", "prefill", "train"])
        dim = _log_int(rng, 100, 4096)
        c = dict(op=op, mode=mode, seqs=_log_int(rng, 1, 256 if mode == "step" else 64), dim=dim,
                 type=rng.choice([BF16, BF16, F32]), lower=rng.random() < 0.6, fused=rng.random() < 0.5)
        if mode != "step":
            most = (65536 * 2048 if mode == "prefill" else 16384 * 2048) // dim
            c["tokens"] = _log_int(rng, 1, min(65536, most) // (2 if c["type"] == F32 else 1))
        return c
    if op == "norm":
        mode = rng.choice(["forward", "forward", "backward"])
        dim = _log_int(rng, 96, 8192)
        t = rng.choice([BF16, BF16, F32])
        c = dict(op=op, mode=mode, dim=dim, rows=_log_int(rng, 1, 16384 * 2048 // dim // (2 if t == F32 else 1)),
                 type=t, sum_type=rng.choice([t, F32]), residual=rng.random() < 0.8)
        if mode == "forward":
            c["out_type"] = rng.choice([t, E4M3])
        return c
    mode = rng.choice(["forward", "forward", "backward"])
    t = rng.choice([BF16, E4M3]) if mode == "forward" else BF16
    c = dict(op=op, mode=mode, inner=16 * _log_int(rng, 8, 256), out=_log_int(rng, 128, 8192), type=t,
             bias=rng.random() < 0.6, act=rng.choice(["none", "relu", "silu", "gelu"]))
    most = 16384 * 2048 * 4096 // (2 if mode == "backward" else 1) // (c["inner"] * c["out"])
    if mode == "forward":
        c["rows"] = _log_int(rng, 1, min(16384, most))
        c["out_type"] = rng.choice([BF16, BF16, F32])
        c["residual"] = rng.random() < 0.5
    else:
        c["rows"] = _log_int(rng, min(256, most), min(16384, most))
    return c


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


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(dev).manual_seed(int(seed))
    t = DTYPE[case["type"]]
    s = dict(case)

    def normal(shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(std).add_(mean)

    if case["op"] == "recurrence":
        n, D = case["seqs"], case["dim"]
        rows = n if case["mode"] == "step" else case["tokens"]
        x, gate = torch.nn.functional.silu(normal((rows, D), 1.5)), normal((rows, D), 1.5, 2.0)
        if case["fused"]:  # the two halves of one projection's output
            both = torch.cat([x, gate], 1).to(t)
            s["x"], s["gate"] = both[:, :D], both[:, D:]
        else:
            s["x"], s["gate"] = x.to(t), gate.to(t)
        s["lower_bound"] = torch.rand((D,), generator=g, device=dev).mul_(0.9) if case["lower"] else None
        r = random.Random(seed * 31 + n)
        s["slots"] = r.sample(range(2 * n), n)
        s["pool"] = normal((2 * n, D), 0.5)
        s["fresh"] = [0] * n if case["mode"] == "step" else [int(r.random() < 0.5) for _ in range(n)]
        s["slots_dev"] = torch.tensor(s["slots"], dtype=torch.int32, device=dev)
        s["fresh_dev"] = torch.tensor(s["fresh"], dtype=torch.uint8, device=dev)
        if case["mode"] == "step":
            s["count_dev"] = torch.tensor([n], dtype=torch.int32, device=dev)
            s["status_dev"] = torch.zeros(1, dtype=torch.int32, device=dev)
        else:
            lens = _lengths(rows, n, seed)
            cu = [0]
            for v in lens:
                cu.append(cu[-1] + v)
            s["cu"] = cu
            s["cu_dev"] = torch.tensor(cu, dtype=torch.int64, device=dev)
        if case["mode"] == "train":
            s["dy"] = normal((rows, D)).to(t)
            s["dstate_end"] = normal((n, D), 0.1)
    elif case["op"] == "norm":
        M, D = case["rows"], case["dim"]
        st = DTYPE[case["sum_type"]]
        s["weight"] = normal((D,), 0.2, 1.0)
        if case["mode"] == "forward":
            s["x"] = normal((M, D)).to(t)
            s["res"] = normal((M, D), 2.0).to(st) if case["residual"] else None
        else:
            s["sum"] = normal((M, D), 2.0).to(st)
            s["dy"] = normal((M, D)).to(t)
            s["dsum"] = normal((M, D), 0.5).to(st) if case["residual"] else None
    else:
        M, K, N = case["rows"], case["inner"], case["out"]
        x, w = normal((M, K)), normal((N, K), 1.0 / math.sqrt(K))
        if t == torch.float8_e4m3fn:
            s["x_scale"], s["w_scale"] = x.abs().amax(1) / MAX8, w.abs().amax(1) / MAX8
            s["x"], s["w"] = (x / s["x_scale"][:, None]).to(t), (w / s["w_scale"][:, None]).to(t)
        else:
            s["x_scale"] = s["w_scale"] = None
            s["x"], s["w"] = x.to(t), w.to(t)
        if case["mode"] == "forward":
            s["bias_v"] = normal((N,), 0.2) if case["bias"] else None
            s["res"] = normal((M, N)).to(DTYPE[case["out_type"]]) if case["residual"] else None
        else:
            s["pre"] = normal((M, N)).to(t) if case["act"] != "none" else None
            s["dy"] = normal((M, N)).to(t)
    return s


# ---------------------------------------------------------------- plain forms

def _gates(s, T):
    g = s["gate"].to(T)
    up, down = torch.sigmoid(g), torch.sigmoid(-g)
    if s["lower_bound"] is None:
        return up, down, up, down
    lo = s["lower_bound"].to(T)
    return lo + (1 - lo) * up, (1 - lo) * down, up, down


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 0, h_{-1} = 0, by doubling."""
    d = 1
    while d < a.shape[0]:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_recurrence(s):
    x, pool, act = s["x"].float(), s["pool"], s["x"].dtype
    slots, fresh = s["slots_dev"].long(), s["fresh_dev"].bool()
    f, k, up, down = _gates(s, torch.float32)
    h0 = torch.where(fresh[:, None], torch.zeros_like(pool[slots]), pool[slots])
    if s["mode"] == "step":
        h = f * h0 + k * x
        pool[slots] = h
        return [h.to(act), pool]
    cu = s["cu_dev"]
    lens = cu[1:] - cu[:-1]
    some = lens > 0
    first, last = cu[:-1][some], cu[1:][some] - 1
    b, a = k * x, f.clone()
    b[first] += f[first] * h0[some]
    a[first] = 0
    h = _scan(a, b)
    end = h0.clone()
    end[some] = h[last]
    pool[slots] = end
    if s["mode"] == "prefill":
        return [h.to(act), pool]
    before = torch.roll(h, 1, 0)
    before[first] = h0[some]
    dy = s["dy"].float()
    dy[last] += s["dstate_end"][some]
    nxt = torch.roll(f, -1, 0)
    nxt[last] = 0
    G = _scan(nxt.flip(0), dy.flip(0)).flip(0)
    df = G * (before - x)
    lo = 0 if s["lower_bound"] is None else s["lower_bound"]
    dh0 = s["dstate_end"].clone()
    dh0[some] = f[first] * G[first]
    out = [h.to(act), pool, (k * G).to(act), (df * (1 - lo) * up * down).to(act), dh0]
    if s["lower_bound"] is not None:
        out.append((df * down).double().sum(0).float())
    return out


def _plain_norm(s):
    w, D = s["weight"], s["dim"]
    if s["mode"] == "forward":
        v = s["x"].float()
        if s["res"] is not None:
            v = v + s["res"].float()
        y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * w
        out = [v.to(DTYPE[s["sum_type"]])] if s["res"] is not None else []
        if s["out_type"] != E4M3:
            return out + [y.to(DTYPE[s["out_type"]])]
        top = y.abs().amax(1)
        scale = torch.where(top > 0, top / MAX8, torch.ones_like(top))
        return out + [(y / scale[:, None]).to(torch.float8_e4m3fn), scale]
    v, dy = s["sum"].float(), s["dy"].float()
    inv = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    wd = w * dy
    d = inv * (wd - v * (inv * inv * (wd * v).mean(1, keepdim=True)))
    if s["dsum"] is not None:
        d = d + s["dsum"].float()
    out = [d.to(s["dy"].dtype), (dy * v * inv).double().sum(0).float()]
    return out + [d.to(s["sum"].dtype)] if s["sum"].dtype != s["dy"].dtype else out


def _act(name, v):
    if name == "relu":
        return v.clamp_min(0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return v


def _slope(name, v):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "silu":
        p = torch.sigmoid(v)
        return p * (1 + v * (1 - p))
    return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))


def _plain_linear(s):
    x, w = s["x"].float(), s["w"].float()
    if s["mode"] == "forward":
        v = x @ w.t()
        if s["x_scale"] is not None:
            v = v * s["x_scale"][:, None] * s["w_scale"]
        if s["bias_v"] is not None:
            v = v + s["bias_v"]
        v = _act(s["act"], v)
        if s["res"] is not None:
            v = v + s["res"].float()
        return [v.to(DTYPE[s["out_type"]])]
    dp = s["dy"].float()
    if s["act"] != "none":
        dp = dp * _slope(s["act"], s["pre"].float())
    out = [(dp @ w).to(s["x"].dtype), (dp.t() @ x).to(s["w"].dtype)]
    return out + [dp.double().sum(0).float()] if s["bias"] else out


# ---------------------------------------------------------------- the framework's calls

def _own_recurrence(s):
    import selective_scan_gb300 as ss
    x, gate, lo, pool = s["x"], s["gate"], s["lower_bound"], s["pool"]
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if s["mode"] == "step":
        ss.gated_recurrence_step_device(y, x, gate, lo, pool, s["slots_dev"], s["fresh_dev"], s["count_dev"],
                                        s["status_dev"])
        return [y, pool]
    if s["mode"] == "prefill":
        ss.gated_recurrence(y, x, gate, lo, pool, s["cu"], s["slots"], s["fresh"])
        return [y, pool]
    kept = torch.empty((ss.gated_recurrence_checkpoints(s["cu"]), s["dim"]), dtype=torch.float32, device=x.device)
    ss.gated_recurrence(y, x, gate, lo, pool, s["cu"], s["slots"], s["fresh"], checkpoints=kept)
    dx, dgate, dh0 = torch.empty_like(y), torch.empty_like(y), torch.empty_like(s["dstate_end"])
    dlo = torch.empty_like(lo) if lo is not None else None
    ss.gated_recurrence_backward(dx, dgate, dlo, dh0, s["dy"], s["dstate_end"], x, gate, lo, kept, s["cu"])
    return [y, pool, dx, dgate, dh0] + ([dlo] if lo is not None else [])


def _own_norm(s):
    import selective_scan_gb300 as ss
    if s["mode"] == "forward":
        x, res = s["x"], s["res"]
        out = torch.empty(x.shape, dtype=DTYPE[s["out_type"]], device=x.device)
        total = torch.empty_like(res) if res is not None else None
        scale = torch.empty(x.shape[:1], dtype=torch.float32, device=x.device) if s["out_type"] == E4M3 else None
        ss.add_rmsnorm(out, x, s["weight"], EPS, residual=res, sum=total, scale=scale)
        return [v for v in (total, out, scale) if v is not None]
    v, dy = s["sum"], s["dy"]
    dx, dw = torch.empty_like(dy), torch.empty_like(s["weight"])
    dres = torch.empty_like(v) if v.dtype != dy.dtype else None
    ss.add_rmsnorm_backward(dx, dres, dw, dy, s["dsum"], v, s["weight"], EPS)
    return [u for u in (dx, dw, dres) if u is not None]


def _own_linear(s):
    import selective_scan_gb300 as ss
    x, w = s["x"], s["w"]
    if s["mode"] == "forward":
        out = torch.empty((x.shape[0], w.shape[0]), dtype=DTYPE[s["out_type"]], device=x.device)
        ss.linear(out, x, w, x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias_v"], residual=s["res"],
                  activation=s["act"])
        return [out]
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = torch.empty(w.shape[:1], dtype=torch.float32, device=x.device) if s["bias"] else None
    ss.linear_backward(dx, dw, db, s["dy"], x, w, activation=s["act"], pre=s["pre"])
    return [dx, dw] + ([db] if s["bias"] else [])


def run(state):
    op = state["op"]
    if own:
        return {"recurrence": _own_recurrence, "norm": _own_norm, "linear": _own_linear}[op](state)
    return {"recurrence": _plain_recurrence, "norm": _plain_norm, "linear": _plain_linear}[op](state)


# ---------------------------------------------------------------- floors

def work(case):
    e = SIZE[case["type"]]
    if case["op"] == "recurrence":
        D, n = case["dim"], case["seqs"]
        T = n if case["mode"] == "step" else case["tokens"]
        fixed = 2 * 4 * n * D + (4 * D if case["lower"] else 0)
        if case["mode"] != "train":  # x, gate in; y out; the state in and out
            return {"bytes": 3 * e * T * D + fixed, "flops": 12 * T * D}
        # the loss stands between the two directions, so x and gate are read by each
        return {"bytes": 8 * e * T * D + fixed + 8 * n * D + (8 * D if case["lower"] else 0), "flops": 45 * T * D}
    if case["op"] == "norm":
        M, D, st = case["rows"], case["dim"], SIZE[case["sum_type"]]
        if case["mode"] == "forward":
            o = SIZE[case["out_type"]]
            return {"bytes": M * D * (e + o + (2 * st if case["residual"] else 0)) + 4 * D
                    + (4 * M if case["out_type"] == E4M3 else 0), "flops": 6 * M * D}
        return {"bytes": M * D * (2 * e + st + (st if case["residual"] else 0) + (st if st != e else 0)) + 8 * D,
                "flops": 14 * M * D}
    M, K, N = case["rows"], case["inner"], case["out"]
    if case["mode"] == "forward":
        o = SIZE[case["out_type"]]
        return {"bytes": e * (M * K + N * K) + o * M * N * (2 if case["residual"] else 1)
                + (4 * N if case["bias"] else 0) + (4 * (M + N) if e == 1 else 0), "flops": 2 * M * N * K}
    return {"bytes": e * (2 * M * K + 2 * N * K + M * N * (2 if case["act"] != "none" else 1))
            + (4 * N if case["bias"] else 0), "flops": 4 * M * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_recurrence(s):
    """Token by token over all runs at once (runs padded to the longest)."""
    D, n = s["dim"], s["seqs"]
    T = torch.float64
    pool = s["pool"].to(T)
    slots, fresh = s["slots_dev"].long(), s["fresh_dev"].bool()
    h0 = pool[slots] * (~fresh)[:, None]
    lo = torch.zeros(D, dtype=T, device=pool.device) if s["lower_bound"] is None else s["lower_bound"].to(T)
    cu = list(range(n + 1)) if s["mode"] == "step" else s["cu"]
    lens = [b - a for a, b in zip(cu[:-1], cu[1:])]
    order = sorted(range(n), key=lambda i: -lens[i])  # the runs still going at a token are the first ones
    start = torch.tensor([cu[i] for i in order], device=pool.device)
    going, alive = [], n
    for t in range(max(lens)):
        while alive and lens[order[alive - 1]] <= t:
            alive -= 1
        going.append(alive)
    perm = torch.tensor(order, device=pool.device)
    sg = 1 / (1 + torch.exp(-s["gate"].to(T)))
    sn = 1 / (1 + torch.exp(s["gate"].to(T)))
    f, k, x = lo + (1 - lo) * sg, (1 - lo) * sn, s["x"].to(T)
    h = h0[perm]
    y, prev = torch.empty_like(x), torch.empty_like(x)
    for t, m in enumerate(going):
        at = start[:m] + t
        prev[at] = h[:m]
        h[:m] = f[at] * h[:m] + k[at] * x[at]
        y[at] = h[:m]
    end = torch.empty_like(h)
    end[perm] = h
    pool[slots] = end
    if s["mode"] != "train":
        return [y, pool]
    dy = s["dy"].to(T)
    G = s["dstate_end"].to(T)[perm]  # the gradient that reaches the state after token t
    dx, df = torch.empty_like(x), torch.empty_like(x)
    for t in range(len(going) - 1, -1, -1):
        m = going[t]
        at = start[:m] + t
        c = G[:m] + dy[at]
        dx[at] = k[at] * c
        df[at] = c * (prev[at] - x[at])
        G[:m] = f[at] * c
    dh0 = torch.empty_like(G)
    dh0[perm] = G
    out = [y, pool, dx, df * (1 - lo) * sg * sn, dh0]
    return out + [(df * sn).sum(0)] if s["lower_bound"] is not None else out


def _exact_norm(s):
    T = torch.float64
    w = s["weight"].to(T)
    if s["mode"] == "forward":
        v = s["x"].to(T) + (s["res"].to(T) if s["res"] is not None else 0)
        y = w * v / torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / s["dim"] + EPS)
        out = [v] if s["res"] is not None else []
        if s["out_type"] != E4M3:
            return out + [y]
        scale = torch.linalg.vector_norm(y, math.inf, 1) / MAX8
        scale[scale == 0] = 1
        return out + [y / scale[:, None], scale]
    v, dy = s["sum"].to(T), s["dy"].to(T)
    rms = torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / s["dim"] + EPS)
    u = v / rms
    wd = w * dy
    d = (wd - u * torch.sum(wd * u, 1, keepdim=True) / s["dim"]) / rms
    if s["dsum"] is not None:
        d = d + s["dsum"].to(T)
    out = [d, torch.sum(dy * u, 0)]
    return out + [d] if s["sum"].dtype != s["dy"].dtype else out


def _exact_linear(s):
    T = torch.float64
    x, w = s["x"].to(T), s["w"].to(T)
    if s["x_scale"] is not None:
        x, w = x * s["x_scale"].to(T)[:, None], w * s["w_scale"].to(T)[:, None]
    if s["mode"] == "forward":
        v = torch.matmul(x, w.T)
        if s["bias_v"] is not None:
            v += s["bias_v"].to(T)
        if s["act"] == "relu":
            v = torch.maximum(v, torch.zeros_like(v))
        elif s["act"] == "silu":
            v = v / (1 + torch.exp(-v))
        elif s["act"] == "gelu":
            v = v * torch.special.ndtr(v)
        return [v + s["res"].to(T)] if s["res"] is not None else [v]
    dp = s["dy"].to(T)
    if s["act"] != "none":
        p = s["pre"].to(T)
        e = torch.exp(-p)
        dp = dp * {"relu": lambda: (p > 0).to(T), "silu": lambda: (1 + e + p * e) / (1 + e) ** 2,
                   "gelu": lambda: torch.special.ndtr(p) + p * torch.exp(-p * p / 2) / math.sqrt(2 * math.pi)}[s["act"]]()
    out = [torch.matmul(dp, w), torch.matmul(dp.T, x)]
    return out + [torch.sum(dp, 0)] if s["bias"] else out


def exact(case, seed):
    s = prepare(case, seed)
    return {"recurrence": _exact_recurrence, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](s)
