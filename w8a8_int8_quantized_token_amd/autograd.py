"""Differentiable forms of the linear, the gated product, and the norm and
rotation of queries and keys.

Quantization is differentiated straight through: the forward pass runs on the
codes, the backward pass treats the rounding as the identity.  What the
backward passes keep is the int8 codes and their scales (half the bytes of
bf16 activations), or nothing of the activations where weights are frozen.

A backward pass is refused while a HIP graph is being captured: autograd would
also run the leaves' accumulation nodes, which belong to the stream they were
first used on; with an eager graph of the same leaves alive that ends the
process.  Capture the forward pass, and ``linear_backward``,
``gated_linear_backward`` and ``qk_norm_rope_backward`` themselves, which have
no such nodes.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import block_ops, ops


def _not_captured(name: str) -> None:
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"the backward pass of {name} cannot be captured into a graph; capture the "
                           "*_backward entry points instead")


def _aligned(grad):
    """An output's gradient, contiguous and at an address that 16-byte loads
    take: it may arrive as a piece of a larger tensor."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


class _FrozenLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, wq, w_scale, bias):
        ctx.save_for_backward(wq, w_scale)
        return block_ops.linear_dynamic(x, wq, w_scale, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _not_captured("a W8A8 linear")
        wq, w_scale = ctx.saved_tensors
        dx, _, _ = block_ops.linear_backward(dy.contiguous(), None, None, wq, w_scale, dw=False, dbias=False)
        return dx, None, None, None


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        with torch.cuda.device_of(x):
            wq, w_scale = ops.quantize_weight(weight)
            xq, x_scale = ops.quantize_act(x)
            ctx.save_for_backward(xq, x_scale, wq, w_scale)
            return ops.linear(xq, x_scale, wq, w_scale, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _not_captured("linear_ste")
        return block_ops.linear_backward(dy.contiguous(), *ctx.saved_tensors, dx=ctx.needs_input_grad[0],
                                         dw=ctx.needs_input_grad[1], dbias=ctx.needs_input_grad[2])


class _Gated(torch.autograd.Function):
    """Gated product of bf16 x by codes (frozen) or by a bf16 weight quantized here."""

    @staticmethod
    def forward(ctx, x, weight, w_scale, bias, act):
        wq = weight
        with torch.cuda.device_of(x):
            if weight.dtype != torch.int8:
                wq, w_scale = ops.quantize_weight(weight)
            xq, x_scale = ops.quantize_act(x)
        ctx.act = act
        ctx.save_for_backward(xq, x_scale, wq, w_scale, bias)
        return block_ops.gated_linear(xq, x_scale, wq, w_scale, bias, act=act)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _not_captured("a gated product")
        need = ctx.needs_input_grad
        dx, dw, db = block_ops.gated_linear_backward(dy.contiguous(), *ctx.saved_tensors, act=ctx.act, dx=need[0],
                                                     dw=need[1], dbias=need[3])
        return dx, dw, None, db, None


class _QKNormRope(torch.autograd.Function):
    """Packed QKV rows -> normed and rotated q, k, and v."""

    @staticmethod
    def forward(ctx, qkv, q_weight, k_weight, cos, sin, positions, heads, eps, interleaved):
        Hq, Hk, D = heads
        q, k, v = _split(qkv, heads)
        ctx.save_for_backward(qkv, q_weight, k_weight, cos, sin, positions)
        ctx.heads, ctx.eps, ctx.interleaved = heads, eps, interleaved
        q, k = block_ops.qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)
        return q, k, v.clone()

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk, dv):
        _not_captured("the norm and rotation")
        qkv, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        q, k, _ = _split(qkv, ctx.heads)
        dqkv = torch.empty_like(qkv)
        gq, gk, gv = _split(dqkv, ctx.heads)
        weights = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        _, _, gqw, gkw = block_ops.qk_norm_rope_backward(_aligned(dq), _aligned(dk), q, k, q_weight, k_weight,
                                                         cos, sin, positions, ctx.eps, ctx.interleaved, weights,
                                                         q_grad=gq, k_grad=gk)
        gv.copy_(dv)
        need = ctx.needs_input_grad
        return (dqkv, gqw.to(torch.bfloat16) if need[1] else None, gkw.to(torch.bfloat16) if need[2] else None,
                *(None,) * 6)


def _split(qkv, heads):
    Hq, Hk, D = heads
    M = qkv.shape[0]
    return (qkv[:, :Hq * D].view(M, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(M, Hk, D),
            qkv[:, (Hq + Hk) * D:].view(M, Hk, D))


def linear_ste(x, weight, bias=None):
    """bf16 x [M,K], weight [N,K], bias [N] -> bf16 y [M,N] through int8
    codes, differentiable in all three (straight through the rounding): the
    linear of quantization-aware training."""
    return _Linear.apply(x, weight, bias)


def gated_linear_ste(x, weight, bias=None, act: str = "silu"):
    """The gated product of bf16 x [M,K] by a bf16 weight [2N,K] (gate rows,
    then up rows) through int8 codes, differentiable in x, weight and bias."""
    return _Gated.apply(x, weight, None, bias, act)
