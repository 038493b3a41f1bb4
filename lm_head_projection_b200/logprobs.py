"""Log-probabilities of given tokens, entropy and best alternatives of logits.

For rows of logits that exist (a served or scored batch);
:func:`lm_head_projection_b200.selective_logprob` gives the log-probabilities
of a head without them.  ``token_logprobs_forward`` and
``token_logprobs_backward`` marshal torch tensors into the C entry points of
those names; ``token_logprobs`` and the module ``TokenLogProbs`` are the
autograd forms.  There is no PyTorch fallback: the CUDA library does every
step.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import DTYPES, _check_dev, _launch, _on, _ptr

__all__ = ["token_logprobs_forward", "token_logprobs_backward", "token_logprobs",
           "TokenLogProbs", "TokenLogProbsOutput", "MAX_TOP_K"]

MAX_TOP_K = 32


def _check_logits(logits: torch.Tensor, target: Optional[torch.Tensor]):
    if logits.dtype not in DTYPES:
        raise ValueError(f"dtype {logits.dtype} not supported (float32 or bfloat16)")
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, V]")
    rows, V = logits.shape
    if V > 1 and logits.stride(1) != 1 or rows > 1 and logits.stride(0) < V:
        raise ValueError("logits need unit stride along V and rows that do not overlap")
    if target is not None:
        _check_dev("target", target, torch.int64, (rows,), logits.device)
    return rows, V, max(logits.stride(0), V) if rows > 1 else V


def token_logprobs_forward(logits: torch.Tensor, target: Optional[torch.Tensor] = None,
                           ignore_index: int = -100, temperature: float = 1.0, top_k: int = 0,
                           stream: Optional[torch.cuda.Stream] = None) -> dict:
    """One pass over ``logits [rows, V]`` (rows may be padded: any row stride,
    any V): with p = softmax(logits / temperature) per row, returns

    * ``logp [rows]``: ln p of ``target`` (None without a target),
    * ``entropy [rows]``, ``lse [rows]``,
    * ``top_ids`` / ``top_logp [rows, top_k]``: the largest logits, ties to the
      lower index, and their ln p (None with ``top_k`` 0; at most 32),
    * ``stats [rows, 2]``: what :func:`token_logprobs_backward` needs.

    A row whose target is ``ignore_index`` is dropped (0 everywhere, ids -1); a
    target outside [0, V) has logp 0.  Masked logits (-infinity) have
    probability 0; a row of nothing else gives logp, lse and top_logp
    -infinity and entropy 0."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_logprobs_forward(logits, target, ignore_index, temperature, top_k)
    rows, V, ld = _check_logits(logits, target)
    if not 0 <= top_k <= min(MAX_TOP_K, V):
        raise ValueError(f"top_k must lie in [0, {min(MAX_TOP_K, V)}], got {top_k}")
    dev, f32 = logits.device, torch.float32
    # (in the cheapest of torch's ways to allocate: six outputs cost more host
    # time than the launch)
    entropy = logits.new_empty(rows, dtype=f32)
    lse, stats = torch.empty_like(entropy), entropy.new_empty((rows, 2))
    logp = torch.empty_like(entropy) if target is not None else None
    top_logp = entropy.new_empty((rows, top_k)) if top_k else None
    top_ids = logits.new_empty((rows, top_k), dtype=torch.int64) if top_k else None
    _launch("flkl_token_logprobs_forward", dev, logits.data_ptr(), ld, _ptr(target),
            ignore_index, rows, V, DTYPES[logits.dtype], temperature, top_k, _ptr(logp),
            entropy.data_ptr(), lse.data_ptr(), stats.data_ptr(), _ptr(top_logp),
            _ptr(top_ids))
    return {"logp": logp, "entropy": entropy, "lse": lse, "top_logp": top_logp,
            "top_ids": top_ids, "stats": stats}


def token_logprobs_backward(logits: torch.Tensor, target: Optional[torch.Tensor], forward: dict,
                            dlogp: Optional[torch.Tensor] = None,
                            dentropy: Optional[torch.Tensor] = None,
                            dtop_logp: Optional[torch.Tensor] = None, ignore_index: int = -100,
                            temperature: float = 1.0,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The gradient of the logits (their type, ``[rows, V]``; where the logits'
    rows start off the 16-byte boundaries, its rows do so alike, a few elements
    apart) for upstream fp32 gradients of logp, entropy ``[rows]`` and top_logp ``[rows, top_k]``
    (None: none), from the dict that :func:`token_logprobs_forward` returned
    for the same logits, target, ignore_index and temperature."""
    if stream is not None:
        with _on(stream, logits.device):
            return token_logprobs_backward(logits, target, forward, dlogp, dentropy, dtop_logp,
                                           ignore_index, temperature)
    rows, V, ld = _check_logits(logits, target)
    dev, f32 = logits.device, torch.float32
    stats, entropy, top_ids = forward["stats"], forward["entropy"], forward["top_ids"]
    _check_dev("stats", stats, f32, (rows, 2), dev)
    _check_dev("entropy", entropy, f32, (rows,), dev)
    k = 0 if top_ids is None else top_ids.shape[1]
    if k:
        _check_dev("top_ids", top_ids, torch.int64, (rows, k), dev)
    if dlogp is not None:
        if target is None:
            raise ValueError("dlogp needs a target")
        _check_dev("dlogp", dlogp, f32, (rows,), dev)
    if dentropy is not None:
        _check_dev("dentropy", dentropy, f32, (rows,), dev)
    if dtop_logp is not None:
        if not k:
            raise ValueError("dtop_logp needs alternatives (top_k > 0)")
        _check_dev("dtop_logp", dtop_logp, f32, (rows, k), dev)
    # rows one after another, not as far apart as the logits' (which may be one
    # position of many); the same phase within 16 bytes keeps the vector path
    dld = V + (ld - V) % (16 // logits.element_size())
    dlogits = logits.new_empty_strided((rows, V), (dld, 1))
    _launch("flkl_token_logprobs_backward", dev, logits.data_ptr(), ld, _ptr(target),
            ignore_index, rows, V, DTYPES[logits.dtype], temperature, k, stats.data_ptr(),
            entropy.data_ptr(), _ptr(top_ids), _ptr(dlogp), _ptr(dentropy), _ptr(dtop_logp),
            dlogits.data_ptr(), dld)
    return dlogits


class TokenLogProbsOutput(NamedTuple):
    """What :func:`token_logprobs` returns (None for what was not asked for)."""
    logp: Optional[torch.Tensor]
    entropy: torch.Tensor
    top_logp: Optional[torch.Tensor]
    top_ids: Optional[torch.Tensor]


class _TokenLogProbsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, target, ignore_index, temperature, top_k):
        r = token_logprobs_forward(logits, target, ignore_index, temperature, top_k)
        ctx.save_for_backward(logits, target, r["stats"], r["entropy"], r["top_ids"])
        ctx.opts = (ignore_index, temperature)
        ctx.set_materialize_grads(False)
        if r["top_ids"] is not None:
            ctx.mark_non_differentiable(r["top_ids"])
        return r["logp"], r["entropy"], r["top_logp"], r["top_ids"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy, dtop, _ids):
        logits, target, stats, entropy, top_ids = ctx.saved_tensors
        ignore_index, temperature = ctx.opts
        g = [None if t is None else t.contiguous() for t in (dlogp, dentropy, dtop)]
        d = token_logprobs_backward(
            logits, target, {"stats": stats, "entropy": entropy, "top_ids": top_ids}, *g,
            ignore_index=ignore_index, temperature=temperature)
        return d, None, None, None, None


def token_logprobs(logits: torch.Tensor, target: Optional[torch.Tensor] = None,
                   ignore_index: int = -100, temperature: float = 1.0,
                   top_k: int = 0) -> TokenLogProbsOutput:
    """:func:`token_logprobs_forward` as an autograd function of the logits:
    any loss of the log-probabilities, the entropy and the alternatives'
    log-probabilities can follow."""
    return TokenLogProbsOutput(*_TokenLogProbsFunction.apply(logits, target, ignore_index,
                                                             temperature, top_k))


class TokenLogProbs(torch.nn.Module):
    """Module form of :func:`token_logprobs`: ``forward(logits, target=None)``."""

    def __init__(self, ignore_index: int = -100, temperature: float = 1.0, top_k: int = 0):
        super().__init__()
        self.ignore_index, self.temperature, self.top_k = ignore_index, temperature, top_k

    def forward(self, logits, target=None) -> TokenLogProbsOutput:
        return token_logprobs(logits, target, self.ignore_index, self.temperature, self.top_k)
