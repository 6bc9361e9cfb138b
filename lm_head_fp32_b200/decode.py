"""One decode step at the LM head: logits of the last positions with each
request's adapter, the best continuations of its beams, and its states put in
the order of the beams that go on.

  logits = X . W^T + scale[a] (X . A_a^T) . B_a^T   lmhead_fwd_lora (lmhead_fwd
                                                    without adapters)
  next beams = best continuations                   beam_select
  states     = in the order of their parents        beam_reorder

This module only sequences the library calls; the buffers of a step are made
once, so that a step allocates nothing and can be captured into a CUDA graph.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import lmhead


class BeamDecoder:
    """Buffers and calls of a beam search of `entries` requests with `beams` beams
    over the vocabulary of W [V,K] (BF16).

    step() takes X [entries * beams, K] (BF16, the hidden states of the last
    positions) and leaves in

      cand_score / cand_beam / cand_token [entries, 2 * beams]   best first
      scores / parents / tokens           [entries, beams]       the beams that go on

    with `scores` also the input of the next step.  reset() sets the scores of a new
    search: beam 0 alone."""

    def __init__(self, W: torch.Tensor, entries: int, beams: int, eos: int = -1,
                 A: Optional[torch.Tensor] = None, B: Optional[torch.Tensor] = None,
                 scale: Optional[torch.Tensor] = None):
        if (A is None) != (B is None) or (A is None) != (scale is None):
            raise ValueError("A, B and scale are given together")
        self.W, self.A, self.B, self.scale, self.eos = W, A, B, scale, int(eos)
        self.entries, self.beams = int(entries), int(beams)
        V, K = W.shape
        M, C = self.entries * self.beams, 2 * self.beams
        n = lmhead.beam_select_workspace_bytes(self.entries, self.beams, V, C)
        if n < 0:
            raise ValueError(f"{entries} x {beams} beams over {V} tokens are out of range")
        if A is not None:
            m = lmhead.lmhead_lora_workspace_bytes(M, K, V, A.shape[1], A.shape[0])
            if m < 0:
                raise ValueError(f"{A.shape[0]} adapters of rank {A.shape[1]} are out of range")
            n = max(n, m)
            self.u = torch.empty((M, A.shape[1]), dtype=torch.float32, device=W.device)

        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=W.device)

        e, b = self.entries, self.beams
        self.logits = new((M, V), torch.float32)
        self.scores = new((e, b), torch.float32)
        self.cand_score = new((e, C), torch.float32)
        self.cand_beam = new((e, C), torch.int32)
        self.cand_token = new((e, C), torch.int64)
        self.parents = new((e, b), torch.int32)
        self.tokens = new((e, b), torch.int64)
        self.workspace = new((max(n, 256),), torch.uint8)
        self.status = torch.zeros(1, dtype=torch.int32, device=W.device)
        self.reset()

    def reset(self) -> None:
        self.scores.fill_(float("-inf"))
        self.scores[:, 0] = 0.0

    def step(self, X: torch.Tensor, states=(), entry_dim: int = 0,
             adapter: Optional[torch.Tensor] = None, done: Optional[torch.Tensor] = None):
        """One step; `states` (a tensor or a list, see lmhead.beam_reorder) are reordered
        in place.  adapter: [entries * beams] int32, needed where the decoder has
        adapters.  Returns (tokens, parents, scores)."""
        if (adapter is None) != (self.A is None):
            raise ValueError("adapter ids are given where the decoder has adapters, and only there")
        if self.A is None:
            with torch.cuda.device(self.W.device):
                lmhead.lmhead_fwd(X, self.W, self.logits, self.status)
        else:
            lmhead.lmhead_fwd_lora(X, self.W, self.A, self.B, self.scale, adapter, self.u,
                                   self.logits, self.workspace, self.status)
        # the new scores may take the place of the old ones: they are written by
        # the call's last kernel, entry by entry, after that entry's were read
        lmhead.beam_select(self.logits.view(self.entries, self.beams, -1), self.scores,
                           self.cand_score, self.cand_beam, self.cand_token, self.scores,
                           self.parents, self.tokens, self.workspace, eos=self.eos, done=done,
                           status=self.status)
        if isinstance(states, torch.Tensor) or len(states):
            lmhead.beam_reorder(states, self.parents, entry_dim, status=self.status)
        return self.tokens, self.parents, self.scores
