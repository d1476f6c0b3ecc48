"""torch.autograd wrappers of the QLoRA linear layer, of the gated feed-forward
block, of RMSNorm and of rotary positions.

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
``qlora_gated`` is the feed-forward block up to its down projection, ``rope``
the rotary positions of queries and keys, each one call a pass.

A backward pass may be captured into a HIP graph. As with any of torch's, no
eager graph of the same leaves may be alive then: its gradient accumulation
belongs to another stream, and torch ends the process.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (NF4Weight, qlora_gated_bwd, qlora_gated_fwd, qlora_gated_fwd_save, qlora_linear_bwd, qlora_linear_bwd_saved,
               qlora_linear_fwd, qlora_linear_fwd_save, qlora_rmsnorm_bwd, qlora_rmsnorm_fwd, qlora_rope_bwd, qlora_rope_fwd)


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


class GatedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, Ag, Bg, Au, Bu, gate: NF4Weight, up: NF4Weight, scale: float, keep: bool):
        X2 = _rows(X, X.shape[-1])
        args = (gate, up, Ag, Bg, Au, Bu, scale)
        shape = (*X.shape[:-1], gate.rows)
        if not keep:
            return qlora_gated_fwd(X2, *args).reshape(shape)
        H, G, U, Hs = qlora_gated_fwd_save(X2, *args)
        ctx.save_for_backward(X2, G, U, Hs, Ag, Bg, Au, Bu)
        ctx.weights, ctx.scale, ctx.shape = (gate, up), scale, X.shape
        return H.reshape(shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dH):
        X2, G, U, Hs, *factors = ctx.saved_tensors
        dH = _rows(dH.to(torch.bfloat16), G.shape[1])
        dX, *grads = qlora_gated_bwd(dH, X2, G, U, Hs, *ctx.weights, *factors, ctx.scale)
        return (dX.reshape(ctx.shape), *grads, None, None, None, None)


def qlora_gated(X, gate: NF4Weight, up: NF4Weight, Ag=None, Bg=None, Au=None, Bu=None, scale: float = 0.0):
    """H = silu(G) * U, G = X Wg-hat^T + scale (X Ag^T) Bg^T and U likewise, with
    autograd to X (bf16, any leading shape) and the adapters (fp32 or bf16, all
    four or none): the feed-forward block up to its down projection in one
    ``qlora_gated_fwd_save`` and one ``qlora_gated_bwd`` call. Where no gradient
    is asked for nothing is kept: ``qlora_gated_fwd``."""
    # through the function all the same: torch refuses forward-mode tangents there, which a call past it would drop
    keep = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (X, Ag, Bg, Au, Bu))
    return GatedFn.apply(X, Ag, Bg, Au, Bu, gate, up, float(scale), keep)


class RopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, positions, freqs, amplitude: float, interleaved: bool):
        ctx.save_for_backward(positions, freqs)
        ctx.how = (amplitude, interleaved)
        ctx.set_materialize_grads(False)
        return qlora_rope_fwd(Q, K, positions, freqs, amplitude, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dQ, dK):
        given = [None if t is None else t if t.stride(-1) == 1 else t.contiguous() for t in (dQ, dK)]
        first = given[0] if given[0] is not None else given[1]
        if first is None:
            return (None,) * 6
        second = given[1] if given[0] is not None else None
        a, b = qlora_rope_bwd(first, second, *ctx.saved_tensors, *ctx.how)
        return (a, b, None, None, None, None) if given[0] is not None else (None, a, None, None, None, None)


def rope(Q, K, positions, freqs, amplitude: float = 1.0, interleaved: bool = False):
    """(Q, K) with rotary positions, with autograd to both: heads [..., heads,
    dim] in fp32 or bf16, positions [...] of the same leading shape (int32 or
    int64), freqs and amplitude of ``qlora_rope_freqs``. K may be None."""
    def flat(t):
        t = t.reshape(-1, *t.shape[-2:])
        return t if t.stride(2) == 1 else t.contiguous()
    q, k = RopeFn.apply(flat(Q), None if K is None else flat(K), positions.reshape(-1).contiguous(), freqs, float(amplitude), bool(interleaved))
    return q.reshape(Q.shape), None if k is None else k.reshape(K.shape)
