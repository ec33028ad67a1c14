"""Layers over the 8-bit block-scaled product and the RMS norm.

``RMSNorm``        y = h / rms(h) * w with h = x + residual, differentiable.
``FP8Linear``      y = x W^T, the frozen weight in e4m3 with a scale per 128 x 128
                   block; activations (and, backward, gradients) are quantized
                   with a scale per row and 128 columns.
``FP8NormLinear``  the two together: the norm writes the 8-bit activations the
                   product reads, with no bf16 copy of them in between.

As in ``nn``: the quantized weight is frozen and gets no gradient ("bitsandbytes"
page, 4-bit/LoRA paragraph: frozen quantized base weights with trainable
parameters beside them); inputs are bf16 or fp32 of any leading shape; no bias.
Quantization of activations counts as the identity in the backward pass.
Gradients are of first order: a derivative of one (``create_graph=True``) raises.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from ._ops import (FP8_FORMATS, FP8Tensor, nf4_fp8_matmul, nf4_fp8_quantize, nf4_rmsnorm_bwd, nf4_rmsnorm_fwd,
                   nf4_rmsnorm_fwd_fp8)


def _rows(t: torch.Tensor, cols: int) -> torch.Tensor:
    """[.., cols] as a matrix the kernels take (contiguous rows, 16-byte aligned start); copied if it is not one."""
    m = t.reshape(-1, cols)
    ok = (cols <= 1 or m.stride(1) == 1) and (m.shape[0] <= 1 or m.stride(0) >= cols) and m.data_ptr() % 16 == 0
    return m if ok else m.clone(memory_format=torch.contiguous_format)


def _check_input(x: torch.Tensor, cols: int, name: str = "x"):
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"{name} must be bfloat16 or float32 (got {x.dtype})")
    if x.shape[-1] != cols:
        raise ValueError(f"{name} has {x.shape[-1]} features, the layer expects {cols}")


def _check_residual(x: torch.Tensor, residual: Optional[torch.Tensor]):
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError(f"residual must be {tuple(x.shape)} {x.dtype} (got {tuple(residual.shape)} {residual.dtype})")


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps: float, out_dtype):
        H = weight.shape[0]
        y, h, rstd = nf4_rmsnorm_fwd(_rows(x, H), weight, None if residual is None else _rows(residual, H), eps, out_dtype)
        ctx.save_for_backward(h, weight, rstd)
        ctx.has_residual = residual is not None
        y = y.reshape(x.shape)
        return (y, h.reshape(x.shape)) if ctx.has_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gh=None):
        h, weight, rstd = ctx.saved_tensors
        H = weight.shape[0]
        dx, dw = nf4_rmsnorm_bwd(_rows(gy, H), h, weight, rstd, None if gh is None else _rows(gh, H))
        dx = dx.reshape(gy.shape)
        return dx, dw, dx if ctx.has_residual else None, None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             out_dtype: Optional[torch.dtype] = None):
    """y, or with ``residual`` (y, h): h = x + residual is the residual stream that goes on."""
    _check_input(x, weight.shape[0])
    _check_residual(x, residual)
    return _RMSNorm.apply(x, weight, residual, eps, out_dtype or x.dtype)


class RMSNorm(torch.nn.Module):
    """Root-mean-square norm with a trainable weight, optionally of x + residual."""

    def __init__(self, features: int, eps: float = 1e-6, dtype: torch.dtype = torch.bfloat16, device="cuda"):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=dtype, device=device))

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        return rms_norm(x, self.weight, residual, self.eps)

    def extra_repr(self) -> str:
        return f"{self.weight.shape[0]}, eps={self.eps}"


def _input_gradient(gy: torch.Tensor, wt: FP8Tensor, fmt: str, dtype: torch.dtype) -> torch.Tensor:
    """dx = gy W with gy quantized per row and 128 columns; wt is W transposed."""
    return nf4_fp8_matmul(nf4_fp8_quantize(_rows(gy, wt.cols), 1, fmt), wt, dtype)


class _FP8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w: FP8Tensor, wt: Optional[FP8Tensor], out_dtype, grad_fmt: str):
        y = nf4_fp8_matmul(nf4_fp8_quantize(_rows(x, w.cols)), w, out_dtype)
        ctx.wt, ctx.fmt, ctx.shape, ctx.dtype = wt, grad_fmt, x.shape, x.dtype
        return y.reshape(*x.shape[:-1], w.rows)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        return _input_gradient(gy, ctx.wt, ctx.fmt, ctx.dtype).reshape(ctx.shape), None, None, None, None


def _check_layer(w: FP8Tensor, wt: Optional[FP8Tensor], out_dtype, grad_fmt: str):
    if w.block_rows != 128 or w.data.dtype != torch.float8_e4m3fn:
        raise ValueError("the weight must be an e4m3 FP8Tensor with 128 x 128 blocks")
    if wt is not None and (wt.shape != (w.cols, w.rows) or wt.block_rows != 128):
        raise ValueError(f"the transposed weight must be {(w.cols, w.rows)} (got {wt.shape})")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
    if grad_fmt not in FP8_FORMATS:
        raise ValueError(f"grad_fmt must be one of {tuple(FP8_FORMATS)} (got {grad_fmt!r})")


def fp8_linear(x: torch.Tensor, w: FP8Tensor, wt: Optional[FP8Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, grad_fmt: str = "e4m3") -> torch.Tensor:
    """y = x W^T for bf16/fp32 x [.., w.cols]; differentiable in x where ``wt`` (``w.t()``) is given."""
    _check_layer(w, wt, out_dtype, grad_fmt)
    _check_input(x, w.cols)
    if wt is None and x.requires_grad and torch.is_grad_enabled():
        raise ValueError("the input gradient needs the transposed weight (wt=w.t(), laid out once)")
    return _FP8Linear.apply(x, w, wt, out_dtype, grad_fmt)


class FP8Linear(torch.nn.Module):
    """A bias-free linear layer whose frozen weight is e4m3 with a scale per 128 x 128 block.

    ``trainable_input`` keeps the transposed weight beside it for the input
    gradient (two bytes a weight in all, as bf16 has; one without).
    """

    def __init__(self, qweight: FP8Tensor, trainable_input: bool = True, out_dtype: torch.dtype = torch.bfloat16,
                 grad_fmt: str = "e4m3"):
        super().__init__()
        _check_layer(qweight, None, out_dtype, grad_fmt)
        self.qweight = qweight
        self.qweight_t = qweight.t() if trainable_input else None
        self.out_dtype, self.grad_fmt = out_dtype, grad_fmt

    @property
    def in_features(self) -> int:
        return self.qweight.cols

    @property
    def out_features(self) -> int:
        return self.qweight.rows

    @classmethod
    def from_weight(cls, weight: torch.Tensor, **kw) -> "FP8Linear":
        """Quantizes a [out_features, in_features] bf16/fp32 device weight."""
        if weight.dim() != 2:
            raise ValueError("weight must be 2-D [out_features, in_features]")
        return cls(nf4_fp8_quantize(_rows(weight.detach(), weight.shape[1]), 128), **kw)

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, **kw) -> "FP8Linear":
        if linear.bias is not None:
            raise ValueError("FP8Linear has no bias; the layer to convert has one")
        return cls.from_weight(linear.weight, **kw)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return fp8_linear(x, self.qweight, self.qweight_t, self.out_dtype, self.grad_fmt)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}, out_dtype={self.out_dtype}"


class _FP8NormLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, w: FP8Tensor, wt: Optional[FP8Tensor], out_dtype, grad_fmt):
        H = w.cols
        q, h, rstd = nf4_rmsnorm_fwd_fp8(_rows(x, H), weight, None if residual is None else _rows(residual, H), eps)
        y = nf4_fp8_matmul(q, w, out_dtype).reshape(*x.shape[:-1], w.rows)
        ctx.save_for_backward(h, weight, rstd)
        ctx.wt, ctx.fmt, ctx.has_residual, ctx.shape = wt, grad_fmt, residual is not None, x.shape
        return (y, h.reshape(x.shape)) if ctx.has_residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gh=None):
        h, weight, rstd = ctx.saved_tensors
        dn = _input_gradient(gy, ctx.wt, ctx.fmt, h.dtype)             # of the norm's output
        dx, dw = nf4_rmsnorm_bwd(dn, h, weight, rstd, None if gh is None else _rows(gh, h.shape[1]))
        dx = dx.reshape(ctx.shape)
        return dx, dw, dx if ctx.has_residual else None, None, None, None, None, None


class FP8NormLinear(torch.nn.Module):
    """y = rms_norm(x [+ residual]) W^T; returns y, or with a residual (y, h) with h = x + residual.

    The norm's output goes to the product in e4m3 with a scale per 128 columns.
    Layers that share the norm (q, k, v; gate and up) take one weight of their
    rows one below the other, and split y.
    """

    def __init__(self, qweight: FP8Tensor, eps: float = 1e-6, trainable: bool = True,
                 out_dtype: torch.dtype = torch.bfloat16, grad_fmt: str = "e4m3", norm_dtype: torch.dtype = torch.bfloat16):
        super().__init__()
        _check_layer(qweight, None, out_dtype, grad_fmt)
        self.qweight, self.eps = qweight, eps
        self.qweight_t = qweight.t() if trainable else None
        self.out_dtype, self.grad_fmt = out_dtype, grad_fmt
        self.weight = torch.nn.Parameter(torch.ones(qweight.cols, dtype=norm_dtype, device=qweight.device),
                                         requires_grad=trainable)

    @classmethod
    def from_weight(cls, weight: torch.Tensor, **kw) -> "FP8NormLinear":
        if weight.dim() != 2:
            raise ValueError("weight must be 2-D [out_features, in_features]")
        return cls(nf4_fp8_quantize(_rows(weight.detach(), weight.shape[1]), 128), **kw)

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None):
        _check_input(x, self.qweight.cols)
        _check_residual(x, residual)
        if self.qweight_t is None and torch.is_grad_enabled() and (
                x.requires_grad or (residual is not None and residual.requires_grad) or self.weight.requires_grad):
            raise ValueError("gradients need the transposed weight: build the layer with trainable=True")
        return _FP8NormLinear.apply(x, self.weight, residual, self.eps, self.qweight, self.qweight_t, self.out_dtype,
                                    self.grad_fmt)

    def extra_repr(self) -> str:
        return f"in_features={self.qweight.cols}, out_features={self.qweight.rows}, eps={self.eps}"
