"""A gated-recurrence residual block from the operators of ``include/block.h``: the residual's addition and RMS
norm, two projections (the input with SiLU, the gate), the gated recurrence over packed runs, and the output
projection that adds the stream back:

    s   = stream + delta                       n = s / rms(s) * norm_w
    x   = silu(n . w_x^T + b_x)                gate = n . w_gate^T + b_gate
    h_t = f_t h_{t-1} + (1 - f_t) x_t          out = h . w_out^T + b_out + s

``prefill`` and ``decode`` serve (the latter from a batch in device memory, so that a captured CUDA graph can be
replayed); ``forward`` and ``backward`` train. With 8-bit input projections the norm writes its rows in e4m3 with a
scale each, and they take them as they are. Every step runs in libmamba2's kernels, but for the addition of two
gradients in ``backward``, which is torch's; this module orders the calls and allocates the intermediates with torch,
on the stream that they run on (``stream``, else the current one), so that their memory goes to no other stream's work.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import (_on, add_rmsnorm, add_rmsnorm_backward, gated_recurrence, gated_recurrence_backward,
               gated_recurrence_checkpoints, gated_recurrence_step_device, linear, linear_backward)

E4M3 = torch.float8_e4m3fn


def quantise_rows(w: torch.Tensor):
    """(e4m3 weight, fp32 scale per row): each output feature's largest weight maps to 448, the largest e4m3 value."""
    scale = w.float().abs().amax(1).clamp_min(1e-30) / 448.0
    return (w.float() / scale[:, None]).to(E4M3), scale


@dataclass
class RecurrentBlockWeights:
    """``norm_w`` [d_model] f32; ``w_x``, ``w_gate`` [dim, d_model] bf16, or e4m3 with ``x_scale``, ``gate_scale``
    [dim] f32 (``quantise_rows``); ``b_x``, ``b_gate`` [dim] f32 or None; ``lower`` [dim] f32 or None: the forget
    gate's lower bounds; ``w_out`` [d_model, dim] bf16; ``b_out`` [d_model] f32 or None."""
    norm_w: torch.Tensor
    w_x: torch.Tensor
    b_x: Optional[torch.Tensor]
    w_gate: torch.Tensor
    b_gate: Optional[torch.Tensor]
    lower: Optional[torch.Tensor]
    w_out: torch.Tensor
    b_out: Optional[torch.Tensor]
    eps: float = 1e-5
    x_scale: Optional[torch.Tensor] = None
    gate_scale: Optional[torch.Tensor] = None


@dataclass
class Saved:
    """What ``forward`` keeps for ``backward``."""
    s: torch.Tensor
    n: torch.Tensor
    pre_x: torch.Tensor
    x: torch.Tensor
    gate: torch.Tensor
    h: torch.Tensor
    checkpoints: torch.Tensor
    cu_seqlens: list


class RecurrentBlock:
    def __init__(self, weights: RecurrentBlockWeights):
        self.w = weights
        self.dim, self.d_model = (int(v) for v in weights.w_x.shape)

    def state_pool(self, num_slots: int, device) -> torch.Tensor:
        """An fp32 state pool of this block: [num_slots, dim]."""
        return torch.zeros((num_slots, self.dim), dtype=torch.float32, device=device)

    def _inputs(self, hidden, delta, pre_x=None):
        """(s, n, x, gate): the norm and both input projections."""
        w, rows, dev = self.w, hidden.shape[0], hidden.device
        s = hidden if delta is None else torch.empty_like(hidden)
        eight = w.w_x.dtype == E4M3
        n = torch.empty(hidden.shape, dtype=E4M3 if eight else hidden.dtype, device=dev)
        scale = torch.empty(rows, dtype=torch.float32, device=dev) if eight else None
        if delta is None:
            add_rmsnorm(n, hidden, w.norm_w, w.eps, scale=scale)
        else:
            add_rmsnorm(n, delta, w.norm_w, w.eps, residual=hidden, sum=s, scale=scale)
        x = torch.empty((rows, self.dim), dtype=hidden.dtype, device=dev)
        gate = torch.empty_like(x)
        linear(x, n, w.w_x, x_scale=scale, w_scale=w.x_scale, bias=w.b_x, activation="silu", pre=pre_x)
        linear(gate, n, w.w_gate, x_scale=scale, w_scale=w.gate_scale, bias=w.b_gate)
        return s, n, x, gate

    def _output(self, h, s):
        out = torch.empty_like(s)
        linear(out, h, self.w.w_out, bias=self.w.b_out, residual=s)
        return out

    def prefill(self, hidden, delta, pool, cu_seqlens, slots, fresh, stream=None) -> torch.Tensor:
        """hidden (the residual stream) and delta (what the layer before adds to it, or None) [rows, d_model] of
        packed runs -> the stream after the block; the pool is updated at the slots."""
        with _on(stream):
            s, _, x, gate = self._inputs(hidden, delta)
            h = torch.empty_like(x)
            gated_recurrence(h, x, gate, self.w.lower, pool, cu_seqlens, slots, fresh)
            return self._output(h, s)

    def decode(self, hidden, delta, pool, slots_dev, fresh_dev, num_seqs_dev, status_dev, stream=None) -> torch.Tensor:
        """One token per sequence, the batch in device memory (``gated_recurrence_step_device``)."""
        with _on(stream):
            s, _, x, gate = self._inputs(hidden, delta)
            h = torch.empty_like(x)
            gated_recurrence_step_device(h, x, gate, self.w.lower, pool, slots_dev, fresh_dev, num_seqs_dev, status_dev)
            return self._output(h, s)

    def forward(self, hidden, delta, pool, cu_seqlens, slots, fresh, stream=None):
        """``prefill`` that also returns what ``backward`` needs (bf16 weights)."""
        with _on(stream):
            if self.w.w_x.dtype == E4M3:
                raise ValueError("training takes bf16 weights")
            pre = torch.empty((hidden.shape[0], self.dim), dtype=torch.bfloat16, device=hidden.device)
            s, n, x, gate = self._inputs(hidden, delta, pre_x=pre)
            h = torch.empty_like(x)
            kept = torch.empty((gated_recurrence_checkpoints(cu_seqlens), self.dim), dtype=torch.float32,
                               device=hidden.device)
            gated_recurrence(h, x, gate, self.w.lower, pool, cu_seqlens, slots, fresh, checkpoints=kept)
            return self._output(h, s), Saved(s, n, pre, x, gate, h, kept, list(cu_seqlens))

    def backward(self, dout, saved: Saved, dstate_end=None, stream=None) -> dict:
        """Gradients by name from that of the output (and of the runs' end states): ``hidden`` (delta's is the
        same), ``state`` [num_seqs, dim], and the weights' by their field names."""
        with _on(stream):
            w, dev = self.w, dout.device
            g = {}

            def vector(name, like):
                g[name] = torch.empty_like(like) if like is not None else None
                return g[name]

            dh, g["w_out"] = torch.empty_like(saved.h), torch.empty_like(w.w_out)
            linear_backward(dh, g["w_out"], vector("b_out", w.b_out), dout, saved.h, w.w_out)
            dx, dgate = torch.empty_like(dh), torch.empty_like(dh)
            g["state"] = torch.empty((len(saved.cu_seqlens) - 1, self.dim), dtype=torch.float32, device=dev)
            gated_recurrence_backward(dx, dgate, vector("lower", w.lower), g["state"], dh, dstate_end, saved.x,
                                      saved.gate, w.lower, saved.checkpoints, saved.cu_seqlens)
            dn, dn_gate = torch.empty_like(saved.n), torch.empty_like(saved.n)
            g["w_x"], g["w_gate"] = torch.empty_like(w.w_x), torch.empty_like(w.w_gate)
            linear_backward(dn, g["w_x"], vector("b_x", w.b_x), dx, saved.n, w.w_x, activation="silu", pre=saved.pre_x)
            linear_backward(dn_gate, g["w_gate"], vector("b_gate", w.b_gate), dgate, saved.n, w.w_gate)
            dn += dn_gate  # (in bf16: each product's gradient is rounded, and their sum)
            g["hidden"] = torch.empty_like(dout)
            add_rmsnorm_backward(g["hidden"], None, vector("norm_w", w.norm_w), dn, dout, saved.s, w.norm_w, w.eps)
            return g
