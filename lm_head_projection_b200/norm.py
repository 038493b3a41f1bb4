"""RMSNorm / LayerNorm backward with frozen-parameter flags, and RMSNorm with
the residual's addition.

The LoRA normalization pull-request page (*Key Changes*): when a norm's
weight (bias) is frozen, its gradient is neither accumulated nor reduced;
the input gradient does not change.  ``rms_norm_backward`` and
``layer_norm_backward`` marshal torch tensors into the C entry points
``flkl_rms_norm_backward`` / ``flkl_layer_norm_backward``; the autograd
modules below take the flags from ``requires_grad`` of the parameters.

``add_rms_norm`` is the norm that stands before the vocabulary head (and
before any projection of a residual network): h = X + residual, y = W h /
rms(h), with h passed on and y in the input's type or in e4m3 with one scale
per row and 128 columns, as :func:`lm_head_projection_b200.fp8.block_matmul`
reads it; ``add_rms_norm_backward`` and the module ``AddRMSNorm`` differentiate
the former.
There is no PyTorch fallback: the CUDA library does every step.
"""

from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (DTYPES, FLKL_OK, FlklError, _check_dev, _launch, _on, _ptr, _written,
               flkl_layer_norm_backward, flkl_norm_workspace_size, flkl_rms_norm_backward)

__all__ = ["rms_norm_backward", "layer_norm_backward", "RMSNorm", "LayerNorm", "add_rms_norm",
           "add_rms_norm_backward", "AddRMSNorm"]


def _prepare(dY, X, W, accum_fp32):
    if X.dtype not in DTYPES:
        raise ValueError(f"dtype {X.dtype} not supported (float32 or bfloat16)")
    if X.dim() < 1:
        raise ValueError("X needs a last (hidden) dimension")
    H = X.shape[-1]
    rows = X.numel() // H if H else 0
    dev, dt = X.device, X.dtype
    _check_dev("X", X, dt, X.shape, dev)
    _check_dev("dY", dY, dt, X.shape, dev)
    _check_dev("W", W, dt, (H,), dev)
    pdt = torch.float32 if (accum_fp32 or dt == torch.float32) else dt
    return rows, H, dev, dt, pdt


def rms_norm_backward(dY: torch.Tensor, X: torch.Tensor, W: torch.Tensor, eps: float = 1e-6,
                      compute_dW: bool = True, accum_fp32: bool = True,
                      stream: Optional[torch.cuda.Stream] = None) -> dict:
    """dX (and dW unless the weight is frozen) of ``y = W * X / rms(X)``
    over the last dimension; returns ``{"dX", "dW"}`` (dW None when frozen)."""
    if stream is not None:  # what the call allocates belongs to its stream, too
        with _on(stream, X.device):
            return rms_norm_backward(dY, X, W, eps, compute_dW, accum_fp32)
    rows, H, dev, dt, pdt = _prepare(dY, X, W, accum_fp32)
    dX = torch.empty_like(X)
    dW = torch.empty((H,), dtype=pdt, device=dev) if compute_dW else None
    need = flkl_norm_workspace_size(rows, H, compute_dW, False)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    st = torch.cuda.current_stream(dev)
    status = flkl_rms_norm_backward(_ptr(dY), _ptr(X), _ptr(W), rows, H, DTYPES[dt], eps,
                                    compute_dW, accum_fp32, _ptr(dX), _ptr(dW), _ptr(ws), need,
                                    st.cuda_stream)
    if status != FLKL_OK:
        raise FlklError(status, "flkl_rms_norm_backward")
    return {"dX": dX, "dW": dW}


def layer_norm_backward(dY: torch.Tensor, X: torch.Tensor, W: torch.Tensor, eps: float = 1e-5,
                        compute_dW: bool = True, compute_db: bool = True,
                        accum_fp32: bool = True,
                        stream: Optional[torch.cuda.Stream] = None) -> dict:
    """dX, dW and db (None when frozen) of ``y = W * (X - mean) / std + b``
    over the last dimension; returns ``{"dX", "dW", "db"}``."""
    if stream is not None:
        with _on(stream, X.device):
            return layer_norm_backward(dY, X, W, eps, compute_dW, compute_db, accum_fp32)
    rows, H, dev, dt, pdt = _prepare(dY, X, W, accum_fp32)
    dX = torch.empty_like(X)
    dW = torch.empty((H,), dtype=pdt, device=dev) if compute_dW else None
    db = torch.empty((H,), dtype=pdt, device=dev) if compute_db else None
    need = flkl_norm_workspace_size(rows, H, compute_dW, compute_db)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    st = torch.cuda.current_stream(dev)
    status = flkl_layer_norm_backward(_ptr(dY), _ptr(X), _ptr(W), rows, H, DTYPES[dt], eps,
                                      compute_dW, compute_db, accum_fp32, _ptr(dX), _ptr(dW),
                                      _ptr(db), _ptr(ws), need, st.cuda_stream)
    if status != FLKL_OK:
        raise FlklError(status, "flkl_layer_norm_backward")
    return {"dX": dX, "dW": dW, "db": db}


def add_rms_norm(X: torch.Tensor, W: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, quantize: bool = False, inplace: bool = False,
                 stream: Optional[torch.cuda.Stream] = None) -> dict:
    """``h = X + residual`` (rounded to the inputs' type), ``y = W * h / rms(h)``
    over the last dimension, in one pass; returns ``{"Y", "scale", "H"}``.

    ``quantize`` gives Y as ``torch.float8_e4m3fn`` codes with fp32 scales
    ``[..., ceil(H / 128)]`` (largest magnitude of 128 columns / 448); else Y
    has X's type and scale is None.  Without a residual H is X itself;
    ``inplace`` writes h over the residual, which autograd takes as an in-place
    change of it (a backward that saved it raises), and is refused for one that
    requires a gradient while gradients are recorded.  No gradient is recorded: see
    :class:`AddRMSNorm`."""
    if stream is not None:
        with _on(stream, X.device):
            return add_rms_norm(X, W, residual, eps, quantize, inplace)
    if X.dtype not in DTYPES:
        raise ValueError(f"dtype {X.dtype} not supported (float32 or bfloat16)")
    if X.dim() < 1:
        raise ValueError("X needs a last (hidden) dimension")
    H = X.shape[-1]
    rows = X.numel() // H if H else 0
    dev, dt = X.device, X.dtype
    _check_dev("X", X, dt, X.shape, dev)
    _check_dev("W", W, dt, (H,), dev)
    Hs = None
    if residual is not None:
        _check_dev("residual", residual, dt, X.shape, dev)
        if inplace and residual.requires_grad and torch.is_grad_enabled():
            raise ValueError("inplace would overwrite a residual that requires a gradient")
        Hs = residual.detach() if inplace else torch.empty_like(X)
    elif inplace:
        raise ValueError("inplace needs a residual")
    Y = torch.empty_like(X, dtype=torch.float8_e4m3fn if quantize else dt)
    scale = X.new_empty((*X.shape[:-1], -(-H // 128)), dtype=torch.float32) if quantize else None
    _launch("flkl_add_rms_norm_forward", dev, X.data_ptr(), _ptr(residual), W.data_ptr(), rows,
            H, DTYPES[dt], eps, 1 if quantize else 0, Y.data_ptr(), _ptr(scale), _ptr(Hs))
    if inplace:
        _written(residual)
    return {"Y": Y, "scale": scale, "H": X if Hs is None else Hs}


def add_rms_norm_backward(dY: torch.Tensor, H: torch.Tensor, W: torch.Tensor,
                          dH: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          compute_dW: bool = True, accum_fp32: bool = True,
                          stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of :func:`add_rms_norm` from its ``H``: dX, the gradient of X
    and of the residual alike, with ``dH`` (what arrives at h from its other
    use) added; and dW unless the weight is frozen.  Returns ``{"dX", "dW"}``."""
    if stream is not None:
        with _on(stream, dY.device):
            return add_rms_norm_backward(dY, H, W, dH, eps, compute_dW, accum_fp32)
    rows, hidden, dev, dt, pdt = _prepare(dY, H, W, accum_fp32)
    if dH is not None:
        _check_dev("dH", dH, dt, H.shape, dev)
    dX = torch.empty_like(H)
    dW = H.new_empty(hidden, dtype=pdt) if compute_dW else None
    if dev.type == "cuda" and dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):  # the size goes by the current device
            need = flkl_norm_workspace_size(rows, hidden, compute_dW, False)
    else:
        need = flkl_norm_workspace_size(rows, hidden, compute_dW, False)
    ws = H.new_empty(need, dtype=torch.uint8) if need else None
    _launch("flkl_add_rms_norm_backward", dev, dY.data_ptr(), _ptr(dH), H.data_ptr(),
            W.data_ptr(), rows, hidden, DTYPES[dt], eps, 1 if compute_dW else 0,
            1 if accum_fp32 else 0, dX.data_ptr(), _ptr(dW), _ptr(ws), need)
    return {"dX": dX, "dW": dW}


class _AddRMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, residual, W, eps):
        r = add_rms_norm(X, W, residual, eps)
        ctx.save_for_backward(r["H"], W)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return r["Y"], r["H"]

    @staticmethod
    @once_differentiable
    def backward(ctx, dY, dH):
        H, W = ctx.saved_tensors
        if dY is None:
            return dH, dH, None, None
        r = add_rms_norm_backward(dY.contiguous(), H, W,
                                  None if dH is None else dH.contiguous(), ctx.eps,
                                  compute_dW=ctx.needs_input_grad[2])
        dW = None if r["dW"] is None else r["dW"].to(W.dtype)
        return r["dX"], r["dX"], dW, None


class _RMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, eps):
        ctx.save_for_backward(X, W)
        ctx.eps = eps
        # forward in torch (not a hot path here; the backward is the kernel)
        Xf = X.float()
        r = torch.rsqrt(Xf.pow(2).mean(-1, keepdim=True) + eps)
        return (Xf * r * W.float()).to(X.dtype)

    @staticmethod
    def backward(ctx, dY):
        X, W = ctx.saved_tensors
        r = rms_norm_backward(dY.contiguous(), X, W, ctx.eps, compute_dW=ctx.needs_input_grad[1])
        dW = None if r["dW"] is None else r["dW"].to(W.dtype)
        return r["dX"], dW, None


class _LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, b, eps):
        ctx.save_for_backward(X, W)
        ctx.eps = eps
        Xf = X.float()
        mu = Xf.mean(-1, keepdim=True)
        var = (Xf - mu).pow(2).mean(-1, keepdim=True)
        return ((Xf - mu) * torch.rsqrt(var + eps) * W.float() + b.float()).to(X.dtype)

    @staticmethod
    def backward(ctx, dY):
        X, W = ctx.saved_tensors
        r = layer_norm_backward(dY.contiguous(), X, W, ctx.eps,
                                compute_dW=ctx.needs_input_grad[1],
                                compute_db=ctx.needs_input_grad[2])
        dW = None if r["dW"] is None else r["dW"].to(W.dtype)
        db = None if r["db"] is None else r["db"].to(W.dtype)
        return r["dX"], dW, db, None


class RMSNorm(torch.nn.Module):
    """RMSNorm whose backward skips dW when ``weight.requires_grad`` is False."""

    def __init__(self, hidden: int, eps: float = 1e-6, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device=device))
        self.eps = eps

    def forward(self, x):
        return _RMSNormFunction.apply(x.contiguous(), self.weight, self.eps)


class LayerNorm(torch.nn.Module):
    """LayerNorm whose backward skips dW / db for frozen weight / bias."""

    def __init__(self, hidden: int, eps: float = 1e-5, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(hidden, dtype=dtype, device=device))
        self.eps = eps

    def forward(self, x):
        return _LayerNormFunction.apply(x.contiguous(), self.weight, self.bias, self.eps)


class AddRMSNorm(torch.nn.Module):
    """RMSNorm of ``x + residual``: ``forward(x, residual) -> (y, h)`` with
    gradients (dW skipped for a frozen weight); ``quantized(x, residual=None)
    -> (codes, scale, h)`` gives y in e4m3 for the 8-bit head, without."""

    def __init__(self, hidden: int, eps: float = 1e-6, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device=device))
        self.eps = eps

    def forward(self, x, residual):
        return _AddRMSNormFunction.apply(x.contiguous(), residual.contiguous(), self.weight,
                                         self.eps)

    @torch.no_grad()
    def quantized(self, x, residual=None):
        r = add_rms_norm(x.contiguous(), self.weight,
                         None if residual is None else residual.contiguous(), self.eps,
                         quantize=True)
        return r["Y"], r["scale"], r["H"]
