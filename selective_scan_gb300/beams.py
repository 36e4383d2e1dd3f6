"""Beam search over recurrent states: the beams of a batch of sequences, each in a slot of every layer's state pools.

A step of the search decodes one token of every beam, selects the best continuations over beams and vocabulary
(``beam_select``) and hands every beam the states of the one that it continues (``reorder_states``). All of it stays in
device memory at addresses that do not change, so a step can be captured in a CUDA graph and replayed. Buffers are
allocated with torch.
"""
from __future__ import annotations

import torch

from . import MAX_BEAMS, MAX_SEQS, _on, _overlap, _pools, beam_select, reorder_states


class Beams:
    """``slots`` [batch, beams] int32 on the device: where the beams' states are, all different, of at most ``MAX_SEQS``
    beams, ``MAX_BEAMS`` a sequence; ``pools``: every layer's pools, each [num_slots, ...], any number of them, none
    overlapping another. What no step could take is a ValueError here. At first only beam 0 of a sequence is in being (its prompt's prefill has left
    the state in ``slots[:, 0]``); the others come out of it with the first step. With ``eos``, a beam that has it goes
    on as it is. ``tokens`` [batch, beams] holds each beam's last token, ``scores`` its summed log-probability,
    ``finished`` whether it has ended, ``status`` the outcome of the last reordering once the stream has passed it."""

    def __init__(self, slots: torch.Tensor, pools, eos=None):
        self.slots, self.pools, self.eos = slots, list(pools), eos
        if slots.dtype != torch.int32 or slots.dim() != 2 or not slots.is_contiguous():
            raise ValueError(f"slots: expected a contiguous [batch, beams] of int32, got {tuple(slots.shape)} of {slots.dtype}")
        if slots.shape[1] < 1 or slots.shape[1] > MAX_BEAMS or slots.numel() > MAX_SEQS:
            raise ValueError(f"slots: at most {MAX_BEAMS} beams a sequence and {MAX_SEQS} in all, got {tuple(slots.shape)}")
        if _overlap(*_pools(self.pools)):
            raise ValueError("two pools overlap")
        dev, shape = slots.device, slots.shape
        self.scores = torch.full(shape, -float("inf"), dtype=torch.float32, device=dev)
        self.scores[:, 0] = 0.0
        self.finished = torch.zeros(shape, dtype=torch.uint8, device=dev) if eos is not None else None
        self.tokens, self.parents = (torch.zeros(shape, dtype=torch.int32, device=dev) for _ in range(2))
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self._scores, self._finished = torch.empty_like(self.scores), (
            torch.empty_like(self.finished) if eos is not None else None)

    def advance(self, logits: torch.Tensor, stream=None) -> torch.Tensor:
        """Takes the step that ``logits`` [batch * beams, vocab] (row b * beams + j is beam j's of sequence b) call
        for; returns ``tokens``. ``parents`` [batch, beams] then tells the beam that each has continued."""
        with _on(stream):
            beam_select(self._scores, self.parents, self.tokens, logits, self.scores, finished=self.finished,
                        finished_out=self._finished, eos=self.eos)
            reorder_states(self.pools, self.slots, self.parents, self.status)
            self.scores.copy_(self._scores)
            if self.finished is not None:
                self.finished.copy_(self._finished)
        return self.tokens


def sequences(tokens, parents) -> torch.Tensor:
    """The beams' token sequences [batch, beams, steps] from every step's ``tokens`` and ``parents`` [batch, beams]."""
    at = torch.arange(tokens[-1].shape[1], device=tokens[-1].device).expand(tokens[-1].shape)
    out = []
    for t, p in zip(reversed(tokens), reversed(parents)):
        out.append(torch.gather(t, 1, at))
        at = torch.gather(p, 1, at).long()
    return torch.stack(out[::-1], 2)
