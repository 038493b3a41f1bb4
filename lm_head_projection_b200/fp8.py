"""The vocabulary head in 8 bits: e4m3 matrices with a scale per block of 128.

``quantize_rows`` (activations: one fp32 scale per row and 128 columns) and
``quantize_blocks`` (weights: one per 128 x 128 block) give codes and scales;
``block_matmul`` multiplies them on the tensor cores with fp32 sums.
``Fp8Head`` holds a head's weight so, quantised once.  Inference and scoring
only: none of this records a gradient.  There is no PyTorch fallback: the CUDA
library does every step.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import DTYPES, _check_dev, _launch, _on, _ptr, _written

__all__ = ["quantize_rows", "quantize_blocks", "block_matmul", "Fp8Head"]

_F8 = torch.float8_e4m3fn


def _quantize(x: torch.Tensor, block_rows: int, stream) -> Tuple[torch.Tensor, torch.Tensor]:
    if stream is not None:
        with _on(stream, x.device):
            return _quantize(x, block_rows, None)
    if x.dtype not in DTYPES:
        raise ValueError(f"dtype {x.dtype} not supported (float32 or bfloat16)")
    if x.dim() < 1:
        raise ValueError("x needs a last dimension")
    _check_dev("x", x, x.dtype, x.shape, x.device)
    K = x.shape[-1]
    rows = x.numel() // K if K else 0
    q = torch.empty_like(x, dtype=_F8)
    kb = -(-K // 128)
    shape = (*x.shape[:-1], kb) if block_rows == 1 else (-(-rows // 128), kb)
    scale = x.new_empty(shape, dtype=torch.float32)
    _launch("flkl_fp8_quantize", x.device, x.data_ptr(), rows, K, DTYPES[x.dtype], block_rows,
            q.data_ptr(), scale.data_ptr())
    return q, scale


def quantize_rows(x: torch.Tensor, stream: Optional[torch.cuda.Stream] = None):
    """``x [..., K]`` -> e4m3 codes of its shape and fp32 scales
    ``[..., ceil(K / 128)]`` (largest magnitude of 128 columns / 448)."""
    return _quantize(x, 1, stream)


def quantize_blocks(w: torch.Tensor, stream: Optional[torch.cuda.Stream] = None):
    """``w [N, K]`` -> e4m3 codes and fp32 scales
    ``[ceil(N / 128), ceil(K / 128)]`` of its 128 x 128 blocks."""
    if w.dim() != 2:
        raise ValueError("w must be a matrix")
    return _quantize(w, 128, stream)


def block_matmul(A: torch.Tensor, a_scale: torch.Tensor, B: torch.Tensor, b_scale: torch.Tensor,
                 bias: Optional[torch.Tensor] = None,
                 out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """``D = A Bᵀ (+ bias)`` of e4m3 matrices ``A [M, K]`` (scales
    ``[M, ceil(K / 128)]``) and ``B [N, K]`` (scales ``[ceil(N / 128),
    ceil(K / 128)]``), in ``out_dtype`` (bfloat16 or float32; ``bias [N]`` has
    it too); fp32 sums, one rounding.  K must be a multiple of 16.  ``out`` is
    written as by an in-place operation of torch's: it must not require a gradient
    while gradients are recorded."""
    if stream is not None:
        with _on(stream, A.device):
            return block_matmul(A, a_scale, B, b_scale, bias, out_dtype, out)
    if out_dtype not in DTYPES:
        raise ValueError(f"out_dtype {out_dtype} not supported (float32 or bfloat16)")
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be matrices")
    dev = A.device
    M, K = A.shape
    N = B.shape[0]
    kb = -(-K // 128)
    _check_dev("A", A, _F8, (M, K), dev)
    _check_dev("B", B, _F8, (N, K), dev)
    _check_dev("a_scale", a_scale, torch.float32, (M, kb), dev)
    _check_dev("b_scale", b_scale, torch.float32, (-(-N // 128), kb), dev)
    if bias is not None:
        _check_dev("bias", bias, out_dtype, (N,), dev)
    given = out is not None
    if not given:
        out = A.new_empty((M, N), dtype=out_dtype)
    else:
        _check_dev("out", out, out_dtype, (M, N), dev)
        if out.requires_grad and torch.is_grad_enabled():
            raise ValueError("out requires a gradient")
    _launch("flkl_fp8_block_matmul", dev, A.data_ptr(), a_scale.data_ptr(), B.data_ptr(),
            b_scale.data_ptr(), _ptr(bias), M, N, K, DTYPES[out_dtype], out.data_ptr())
    if given:
        _written(out)
    return out


class Fp8Head(torch.nn.Module):
    """A vocabulary head ``[V, H]`` held in e4m3 with 128 x 128 scales.

    ``forward(hidden)`` quantises the rows of ``hidden [..., H]`` and gives
    their logits; ``logits(codes, scale)`` takes rows that are quantised
    already (the norm's 8-bit output), and another ``out_dtype`` than the head's
    where the caller wants one.  ``bias [V]`` (float32 or bfloat16) keeps its type
    and is cast to that of the logits where they differ.

    ``Module.to`` and its kin move the head between devices; a change of type
    (``model.to(torch.bfloat16)``, ``.half()``) passes it by, since codes and
    scales are no numbers of that kind."""

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 out_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        if out_dtype not in DTYPES:
            raise ValueError(f"out_dtype {out_dtype} not supported (float32 or bfloat16)")
        if bias is not None and bias.dtype not in DTYPES:
            bias = bias.to(out_dtype)
        codes, scale = quantize_blocks(weight.detach().contiguous())
        self.register_buffer("codes", codes)
        self.register_buffer("scale", scale)
        self.register_buffer("bias", None if bias is None else bias.detach().contiguous())
        self.out_dtype = out_dtype

    def _apply(self, fn, recurse=True):
        def keep_type(t):
            probe = fn(t.new_empty(0))
            return fn(t) if probe.dtype == t.dtype else t.to(probe.device)

        return super()._apply(keep_type, recurse)

    def logits(self, codes: torch.Tensor, scale: torch.Tensor,
               out: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
        K = self.codes.shape[1]
        dt = self.out_dtype if out_dtype is None else out_dtype
        D = block_matmul(codes.reshape(-1, K), scale.reshape(-1, self.scale.shape[1]),
                         self.codes, self.scale,
                         None if self.bias is None else self.bias.to(dt), dt, out)
        return D.reshape((*codes.shape[:-1], D.shape[-1]))

    @torch.no_grad()
    def forward(self, hidden: torch.Tensor) -> torch.Tensor:
        return self.logits(*quantize_rows(hidden.contiguous()))
