"""torch.autograd wrappers of the QLoRA linear layer and of RMSNorm.

Marshalling only: the forward is one ``qlora_linear_fwd_save`` call, which
also keeps the adapter activations bf16(scale X A^T) [M, r], and the backward
one ``qlora_linear_bwd_saved`` call that takes them instead of forming them
again (``qlora_linear_fwd`` / ``qlora_linear_bwd`` without an adapter)
(QLoRA vs ChatGPT page, capability
"training pipeline": the 4-bit base is frozen and dequantized on the fly,
gradients go to the low-rank adapter and the input). It lets a caller compose
projections into a larger model with autograd, recompute them under
``torch.utils.checkpoint``, and gives the base weight no gradient.

Tensors: X bf16 [M, K] (any leading shape, flattened to M rows), A fp32
[r, K], B fp32 [N, r], on the weight's device. The output is bf16 [..., N].

``rmsnorm`` is the norm in front of the projections, with the residual's
addition: one ``qlora_rmsnorm_fwd`` call and one ``qlora_rmsnorm_bwd`` call.

A backward pass may be captured into a HIP graph. As with any of torch's, no
eager graph of the same leaves may be alive then: its gradient accumulation
belongs to another stream, and torch ends the process.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (NF4Weight, qlora_linear_bwd, qlora_linear_bwd_saved, qlora_linear_fwd, qlora_linear_fwd_save,
               qlora_rmsnorm_bwd, qlora_rmsnorm_fwd)


class QLoRALinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, A, B, W: NF4Weight, scale: float):
        lead = X.shape[:-1]
        X2 = X.reshape(-1, X.shape[-1]).contiguous()
        if A is not None:
            Y, Hs = qlora_linear_fwd_save(X2, W, A, B, scale)
        else:
            Y, Hs = qlora_linear_fwd(X2, W, A, B, scale), None
        ctx.save_for_backward(X2, A, B, Hs)
        ctx.W, ctx.scale, ctx.lead = W, scale, lead
        return Y.reshape(*lead, W.rows)

    @staticmethod
    def backward(ctx, dY):
        X2, A, B, Hs = ctx.saved_tensors
        dY2 = dY.reshape(-1, ctx.W.rows).to(torch.bfloat16).contiguous()
        if Hs is not None:
            dX, dA, dB = qlora_linear_bwd_saved(dY2, X2, Hs, ctx.W, A, B, ctx.scale)
        else:
            dX, dA, dB = qlora_linear_bwd(dY2, X2, ctx.W, A, B, ctx.scale)
        return dX.reshape(*ctx.lead, ctx.W.cols), dA, dB, None, None


def qlora_linear(X, W: NF4Weight, A=None, B=None, scale: float = 0.0):
    """Y = X W-hat^T + scale (X A^T) B^T with autograd to X, A and B."""
    return QLoRALinearFn.apply(X, A, B, W, float(scale))


def _rows(t, cols):
    """``t`` as contiguous rows of ``cols``, 16-byte aligned as the library
    takes them: a gradient may be a view that begins anywhere."""
    t = t.reshape(-1, cols).contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _second_grad(t, shape):
    """``t``, already the gradient of X, as that of a residual of this shape. The
    same tensor, which torch copies for one of the two, or a copy: a view of it
    would leave both leaves with one gradient's memory."""
    return t if t.shape == shape else t.reshape(shape).clone()


class RMSNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, weight, residual, eps: float):
        cols = X.shape[-1]
        flat = _rows(X, cols)
        res = None
        if residual is not None:
            if residual.shape[-1:] != X.shape[-1:] or residual.numel() != X.numel():
                raise ValueError(f"residual must hold the rows of X {tuple(X.shape)}, got {tuple(residual.shape)}")
            res = _rows(residual, cols)
            ctx.residual_shape = residual.shape
        Y, H, rstd = qlora_rmsnorm_fwd(flat, weight, eps, residual=res)
        ctx.save_for_backward(H, weight, rstd)
        ctx.set_materialize_grads(False)
        if residual is None:
            return Y.reshape(X.shape)
        return Y.reshape(X.shape), H.reshape(X.shape)

    @staticmethod
    @once_differentiable   # a second derivative is refused, not taken for zero
    def backward(ctx, dY, dH=None):
        H, weight, rstd = ctx.saved_tensors
        with_residual = ctx.needs_input_grad[2]
        if dY is None:   # only H went on, X and the residual take its gradient
            return dH, None, _second_grad(dH, ctx.residual_shape) if with_residual else None, None
        shape = dY.shape
        dY = _rows(dY, H.shape[1])
        if dH is not None:
            dH = _rows(dH, H.shape[1])
        dX, dW = qlora_rmsnorm_bwd(dY, H, weight, rstd, dH=dH)
        dX = dX.reshape(shape)
        return dX, dW.to(weight.dtype), _second_grad(dX, ctx.residual_shape) if with_residual else None, None


def rmsnorm(X, weight, residual=None, eps: float = 1e-6):
    """RMSNorm of bf16 X [..., D] with autograd to X, weight [D] (fp32 or bf16)
    and residual (as many rows of D, in any leading shape). Without a residual
    the result is Y; with one it is (Y, H), H = bf16(X + residual) being the
    residual stream that goes on."""
    return RMSNormFn.apply(X, weight, residual, float(eps))
