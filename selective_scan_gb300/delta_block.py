"""A residual block with a gated delta rule from the operators of ``include/delta.h`` and ``include/block.h``: the
residual's addition and RMS norm, one projection to queries, keys and values (with SiLU), one to the heads' decays and
betas, the delta rule over packed runs with keys and queries of unit length, and the output projection that adds the
stream back:

    s       = stream + delta                          n = s / rms(s) * norm_w
    q, k, v = silu(n . w_qkv^T)                       a, b = n . w_ab^T + b_ab
    g       = -exp(A_log) softplus(a)                 beta = sigmoid(b)
    S_t     = e^{g_t} S_{t-1} + beta_t (v_t - e^{g_t} S_{t-1} k_t) k_t^T
    out     = (S_t q_t / sqrt(d_state)) . w_out^T + s

``prefill`` and ``decode`` serve (the latter from a batch in device memory, so that a captured CUDA graph can be
replayed); ``forward`` and ``backward`` train. Every step runs in libmamba2's kernels, but for what is elementwise in
[rows, heads] (g, beta and their derivatives) and the addition of two gradients in ``backward``, which are torch's; this
module orders the calls and allocates the intermediates with torch, on the stream that they run on (``stream``, else the
current one).
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (_on, add_rmsnorm, add_rmsnorm_backward, gated_delta_rule, gated_delta_rule_backward,
               gated_delta_rule_checkpoints, gated_delta_rule_step_device, linear, linear_backward)


@dataclass
class DeltaBlockWeights:
    """``norm_w`` [d_model] f32; ``w_qkv`` [2 groups d_state + heads headdim, d_model] bf16: queries, keys, values;
    ``w_ab`` [2 heads, d_model] bf16 and ``b_ab`` [2 heads] f32: what decays and betas are made of; ``A_log`` [heads]
    f32; ``w_out`` [d_model, heads headdim] bf16. d_state and headdim are multiples of 8."""
    norm_w: torch.Tensor
    w_qkv: torch.Tensor
    w_ab: torch.Tensor
    b_ab: torch.Tensor
    A_log: torch.Tensor
    w_out: torch.Tensor
    groups: int
    d_state: int
    eps: float = 1e-5
    l2_eps: float = 1e-6


@dataclass
class Saved:
    """What ``forward`` keeps for ``backward``."""
    s: torch.Tensor
    n: torch.Tensor
    pre: torch.Tensor
    qkv: torch.Tensor
    ab: torch.Tensor
    g: torch.Tensor
    beta: torch.Tensor
    h: torch.Tensor
    checkpoints: torch.Tensor
    cu_seqlens: list


class DeltaBlock:
    def __init__(self, weights: DeltaBlockWeights):
        self.w = weights
        self.groups, self.d_state = int(weights.groups), int(weights.d_state)
        self.heads = int(weights.A_log.shape[0])
        self.d_model, inner = (int(v) for v in weights.w_out.shape)
        self.headdim = inner // self.heads

    def state_pool(self, num_slots: int, device) -> torch.Tensor:
        """An fp32 state pool of this block: [num_slots, heads, headdim, d_state]."""
        return torch.zeros((num_slots, self.heads, self.headdim, self.d_state), dtype=torch.float32, device=device)

    def _split(self, qkv):
        """Queries, keys and values: column ranges of one matrix, by heads."""
        narrow = self.groups * self.d_state
        return (qkv[:, :narrow].unflatten(1, (self.groups, self.d_state)),
                qkv[:, narrow:2 * narrow].unflatten(1, (self.groups, self.d_state)),
                qkv[:, 2 * narrow:].unflatten(1, (self.heads, self.headdim)))

    def _inputs(self, hidden, delta, pre=None):
        w, rows, dev = self.w, hidden.shape[0], hidden.device
        s = hidden if delta is None else torch.empty_like(hidden)
        n = torch.empty_like(hidden)
        if delta is None:
            add_rmsnorm(n, hidden, w.norm_w, w.eps)
        else:
            add_rmsnorm(n, delta, w.norm_w, w.eps, residual=hidden, sum=s)
        qkv = torch.empty((rows, w.w_qkv.shape[0]), dtype=hidden.dtype, device=dev)
        linear(qkv, n, w.w_qkv, activation="silu", pre=pre)
        ab = torch.empty((rows, 2 * self.heads), dtype=torch.float32, device=dev)
        linear(ab, n, w.w_ab, bias=w.b_ab)
        g = torch.nn.functional.softplus(ab[:, :self.heads]) * -torch.exp(w.A_log)
        return s, n, qkv, ab, g, torch.sigmoid(ab[:, self.heads:])

    def _output(self, h, s):
        out = torch.empty_like(s)
        linear(out, h.flatten(1), self.w.w_out, residual=s)
        return out

    def prefill(self, hidden, delta, pool, cu_seqlens, slots, fresh, stream=None) -> torch.Tensor:
        """hidden (the residual stream) and delta (what the layer before adds to it, or None) [rows, d_model] of
        packed runs -> the stream after the block; the pool is updated at the slots."""
        with _on(stream):
            s, _, qkv, _, g, beta = self._inputs(hidden, delta)
            q, k, v = self._split(qkv)
            h = torch.empty(v.shape, dtype=v.dtype, device=v.device)
            gated_delta_rule(h, q, k, v, g, beta, pool, cu_seqlens, slots, fresh, l2_eps=self.w.l2_eps)
            return self._output(h, s)

    def decode(self, hidden, delta, pool, slots_dev, fresh_dev, num_seqs_dev, status_dev, stream=None) -> torch.Tensor:
        """One token per sequence, the batch in device memory (``gated_delta_rule_step_device``)."""
        with _on(stream):
            s, _, qkv, _, g, beta = self._inputs(hidden, delta)
            q, k, v = self._split(qkv)
            h = torch.empty(v.shape, dtype=v.dtype, device=v.device)
            gated_delta_rule_step_device(h, q, k, v, g, beta, pool, slots_dev, fresh_dev, num_seqs_dev, status_dev,
                                         l2_eps=self.w.l2_eps)
            return self._output(h, s)

    def forward(self, hidden, delta, pool, cu_seqlens, slots, fresh, stream=None):
        """``prefill`` that also returns what ``backward`` needs."""
        with _on(stream):
            pre = torch.empty((hidden.shape[0], self.w.w_qkv.shape[0]), dtype=torch.bfloat16, device=hidden.device)
            s, n, qkv, ab, g, beta = self._inputs(hidden, delta, pre=pre)
            q, k, v = self._split(qkv)
            h = torch.empty(v.shape, dtype=v.dtype, device=v.device)
            kept = torch.empty((gated_delta_rule_checkpoints(cu_seqlens),) + pool.shape[1:], dtype=torch.float32,
                               device=hidden.device)
            gated_delta_rule(h, q, k, v, g, beta, pool, cu_seqlens, slots, fresh, l2_eps=self.w.l2_eps, checkpoints=kept)
            return self._output(h, s), Saved(s, n, pre, qkv, ab, g, beta, h, kept, list(cu_seqlens))

    def backward(self, dout, saved: Saved, dstate_end=None, stream=None) -> dict:
        """Gradients by name from that of the output (and of the runs' end states): ``hidden`` (delta's is the
        same), ``state`` [num_seqs, heads, headdim, d_state], and the weights' by their field names."""
        with _on(stream):
            w, dev, grads = self.w, dout.device, {}
            h = saved.h.flatten(1)
            dh, grads["w_out"] = torch.empty_like(h), torch.empty_like(w.w_out)
            linear_backward(dh, grads["w_out"], None, dout, h, w.w_out)
            q, k, v = self._split(saved.qkv)
            dqkv = torch.empty_like(saved.qkv)
            dq, dk, dv = self._split(dqkv)
            dg, dbeta = (torch.empty(saved.g.shape, dtype=v.dtype, device=dev) for _ in range(2))
            grads["state"] = torch.empty((len(saved.cu_seqlens) - 1, self.heads, self.headdim, self.d_state),
                                         dtype=torch.float32, device=dev)
            gated_delta_rule_backward(dq, dk, dv, dg, dbeta, grads["state"], dh.unflatten(1, (self.heads, self.headdim)),
                                      dstate_end, q, k, v, saved.g, saved.beta, saved.checkpoints, saved.cu_seqlens,
                                      l2_eps=w.l2_eps)
            dg = dg.float()
            grads["A_log"] = (dg * saved.g).sum(0)
            da = dg * torch.sigmoid(saved.ab[:, :self.heads]) * -torch.exp(w.A_log)
            db = dbeta.float() * saved.beta * (1 - saved.beta)
            dab = torch.cat([da, db], 1).to(dout.dtype)
            dn, dn_ab = torch.empty_like(saved.n), torch.empty_like(saved.n)
            grads["w_qkv"], grads["w_ab"] = torch.empty_like(w.w_qkv), torch.empty_like(w.w_ab)
            grads["b_ab"] = torch.empty_like(w.b_ab)
            linear_backward(dn, grads["w_qkv"], None, dqkv, saved.n, w.w_qkv, activation="silu", pre=saved.pre)
            linear_backward(dn_ab, grads["w_ab"], grads["b_ab"], dab, saved.n, w.w_ab)
            dn += dn_ab  # (in bf16: each product's gradient is rounded, and their sum)
            grads["hidden"], grads["norm_w"] = torch.empty_like(dout), torch.empty_like(w.norm_w)
            add_rmsnorm_backward(grads["hidden"], None, grads["norm_w"], dn, dout, saved.s, w.norm_w, w.eps)
            return grads
