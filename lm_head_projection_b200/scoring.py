"""Scoring through an 8-bit vocabulary head: the last norm, the head and the
log-probabilities in a row, with no [rows, V] logits beyond one block of rows.
"""

from __future__ import annotations

from typing import Optional

import torch

from .fp8 import Fp8Head
from .logprobs import token_logprobs_forward
from .norm import AddRMSNorm

__all__ = ["Fp8Scorer"]


class Fp8Scorer(torch.nn.Module):
    """``norm`` (an :class:`~lm_head_projection_b200.norm.AddRMSNorm`) and
    ``head`` (an :class:`~lm_head_projection_b200.fp8.Fp8Head`) as one call:

    ``forward(x, residual=None, target=None)`` with ``x [..., H]`` and a target per
    row, in row order, adds the residual, norms to e4m3, forms ``block_rows`` rows
    of logits at a time and returns ``{"logp", "entropy", "top_logp", "top_ids",
    "H"}`` of x's leading shape (None for what was not asked for).  The logits,
    which nobody else sees, are fp32 whatever the head's ``out_dtype`` (a bf16 logit
    of 20 is off by up to 0.06, and its log-probability with it).  No gradient."""

    def __init__(self, norm: AddRMSNorm, head: Fp8Head, top_k: int = 0,
                 temperature: float = 1.0, ignore_index: int = -100, block_rows: int = 1024):
        super().__init__()
        if block_rows < 1:
            raise ValueError("block_rows must be at least 1")
        self.norm, self.head = norm, head
        self.top_k, self.temperature = top_k, temperature
        self.ignore_index, self.block_rows = ignore_index, block_rows

    @torch.no_grad()
    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                target: Optional[torch.Tensor] = None) -> dict:
        lead = x.shape[:-1]
        if target is not None and target.numel() != lead.numel():
            raise ValueError(f"target has shape {tuple(target.shape)}, expected {tuple(lead)}")
        codes, scale, h = self.norm.quantized(x, residual)
        codes = codes.reshape(-1, codes.shape[-1])
        scale = scale.reshape(-1, scale.shape[-1])
        y = None if target is None else target.reshape(-1).contiguous()
        rows = codes.shape[0]
        parts = []
        for r0 in range(0, max(rows, 1), self.block_rows):
            r1 = min(rows, r0 + self.block_rows)
            z = self.head.logits(codes[r0:r1], scale[r0:r1], out_dtype=torch.float32)
            parts.append(token_logprobs_forward(z, None if y is None else y[r0:r1],
                                                self.ignore_index, self.temperature, self.top_k))
        out = {"H": h}
        for n in ("logp", "entropy", "top_logp", "top_ids"):
            v = [p[n] for p in parts]
            if v[0] is None:
                out[n] = None
            else:
                t = v[0] if len(v) == 1 else torch.cat(v)
                out[n] = t.reshape((*lead, *t.shape[1:]))
        return out
