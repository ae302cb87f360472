"""torch.autograd wrappers over the C ABI.

fused_add_rmsnorm(x, residual, w, eps, weight_bias) -> (out, new_residual)
    forward: rmsnorm_fwd_ex, which also saves each row's scale (rstd);
    backward: rmsnorm_vjp_ex on the saved new_residual with that rstd, giving
    one gradient for x and residual (they enter as a sum) and gw.
rms_norm(x, w, eps, weight_bias) -> out
    forward: rmsnorm_fwd_ex without a residual; backward: rmsnorm_vjp_ex.
block_norm(y, residual, w_post, w_pre, eps, weight_bias, gate, scale) -> (out, new_residual)
    forward: rmsnorm_block_fwd with both scales saved; backward:
    rmsnorm_block_vjp on y and the saved new_residual.
rope(q, k, positions, inv_freq, attn_scale, interleaved) -> (q_out, k_out)
    forward: rmsnorm_rope; backward: the same rotation inverted.
Inputs whose rows sit a stride apart (slices of wider buffers) are used in
place; fp16, bf16 and fp32.

The kernels accumulate gw in fp32; it is returned in w's dtype, as autograd
expects a gradient of a parameter's own dtype.  Gradients that do not reach
an output arrive as None and are not materialised.

Source: "Fused residual-add RMSNorm and fused RoPE + KV-append decode
kernels", Background (two-output FusedAddRMSNorm); "RMSNormVJP backward
writes a full {n_rows, D} gw_temp intermediate", POC (the gradients of
rms_norm through autograd).
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .api import (rmsnorm_block_fwd, rmsnorm_block_vjp, rmsnorm_fwd_ex, rmsnorm_rope,
                  rmsnorm_vjp_ex, rows_layout_ok)


def _rows(t):
    """t itself when the kernels take its layout (rows a stride apart), else a
    dense copy (e.g. an expanded gradient of a sum)."""
    return t if rows_layout_ok(t) else t.contiguous()


class FusedAddRMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, w, eps: float, weight_bias: float):
        ctx.set_materialize_grads(False)
        out, new_res, rstd = rmsnorm_fwd_ex(_rows(x), w.contiguous(), eps, weight_bias,
                                            _rows(residual), rstd=True)
        ctx.save_for_backward(new_res, w, rstd)
        ctx.eps = eps
        ctx.weight_bias = weight_bias
        return out, new_res

    @staticmethod
    def backward(ctx, g_out, g_res):
        new_res, w, rstd = ctx.saved_tensors
        if g_out is None:
            g_h = None if g_res is None else g_res.contiguous()
            gw = torch.zeros_like(w) if ctx.needs_input_grad[2] else None
        else:
            g_h, gw32 = rmsnorm_vjp_ex(new_res, w.contiguous(), _rows(g_out), ctx.eps,
                                       ctx.weight_bias, None if g_res is None else _rows(g_res),
                                       rstd=rstd)
            gw = gw32.to(w.dtype) if ctx.needs_input_grad[2] else None
        gx = g_h if ctx.needs_input_grad[0] else None
        gr = g_h if ctx.needs_input_grad[1] else None
        return gx, gr, gw, None, None


class RMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, eps: float, weight_bias: float):
        x = _rows(x)
        out, _, rstd = rmsnorm_fwd_ex(x, w.contiguous(), eps, weight_bias, rstd=True)
        ctx.save_for_backward(x, w, rstd)
        ctx.eps = eps
        ctx.weight_bias = weight_bias
        return out

    @staticmethod
    def backward(ctx, g_out):
        x, w, rstd = ctx.saved_tensors
        gx, gw32 = rmsnorm_vjp_ex(x, w.contiguous(), _rows(g_out), ctx.eps, ctx.weight_bias,
                                  rstd=rstd)
        return (gx if ctx.needs_input_grad[0] else None,
                gw32.to(w.dtype) if ctx.needs_input_grad[1] else None, None, None)


def _heads(t):
    """t itself when its heads' elements are contiguous, else a dense copy."""
    return t if t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


class RopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, attn_scale: float, interleaved: bool):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions, inv_freq)
        ctx.attn_scale = attn_scale
        ctx.interleaved = interleaved
        return rmsnorm_rope(_heads(q), None if k is None else _heads(k), positions, inv_freq,
                            attn_scale=attn_scale, interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_q, g_k):
        positions, inv_freq = ctx.saved_tensors
        both = [g for g in (g_q, g_k) if g is not None]
        turned = (None, None)
        if both:  # a gradient that is missing takes no part
            turned = rmsnorm_rope(_heads(both[0]), _heads(both[1]) if len(both) == 2 else None, positions,
                                  inv_freq, attn_scale=ctx.attn_scale, interleaved=ctx.interleaved,
                                  inverse=True)
        got = iter(turned)
        return (next(got) if g_q is not None else None, next(got) if g_k is not None else None,
                None, None, None, None)


class BlockNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, w_post, w_pre, eps: float, weight_bias: float, gate, scale: float):
        ctx.set_materialize_grads(False)
        y = _rows(y)
        gate_rows = None if gate is None else _rows(gate)
        out, new_res, rstd = rmsnorm_block_fwd(
            y, _rows(residual), None if w_post is None else w_post.contiguous(), w_pre.contiguous(),
            eps, weight_bias, gate_rows, scale, rstd=True)
        ctx.save_for_backward(y, new_res, w_post, w_pre, gate, rstd)
        ctx.eps = eps
        ctx.weight_bias = weight_bias
        ctx.scale = scale
        return out, new_res

    @staticmethod
    @once_differentiable
    def backward(ctx, g_out, g_res):
        if g_out is None and g_res is None:
            return (None,) * 8
        y, new_res, w_post, w_pre, gate, rstd = ctx.saved_tensors
        if g_out is None:  # only new_residual was used
            g_out = torch.zeros_like(new_res)
        g_y, g_h, gw_post, gw_pre, g_gate = rmsnorm_block_vjp(
            y, new_res, None if w_post is None else w_post.contiguous(), w_pre.contiguous(),
            _rows(g_out), ctx.eps, ctx.weight_bias, None if gate is None else _rows(gate), ctx.scale,
            None if g_res is None else _rows(g_res), rstd=rstd)
        need = ctx.needs_input_grad
        return (g_y if need[0] else None, g_h if need[1] else None,
                gw_post.to(w_post.dtype) if need[2] else None,
                gw_pre.to(w_pre.dtype) if need[3] else None, None, None,
                g_gate.to(gate.dtype) if need[6] else None, None)


def fused_add_rmsnorm(x, residual, w, eps: float, weight_bias: float = 0.0):
    """(out, new_residual) with h = x + residual and
    out = h * rsqrt(mean(h^2) + eps) * (weight_bias + w); differentiable."""
    return FusedAddRMSNormFunction.apply(x, residual, w, eps, weight_bias)


def rms_norm(x, w, eps: float, weight_bias: float = 0.0):
    """x * rsqrt(mean(x^2) + eps) * (weight_bias + w); differentiable."""
    return RMSNormFunction.apply(x, w, eps, weight_bias)


def block_norm(y, residual, w_post, w_pre, eps: float, weight_bias: float = 0.0, gate=None,
               scale: float = 1.0):
    """(out, new_residual) with h = residual + scale * gate * norm(y; w_post) and
    out = norm(h; w_pre): the norms after a block and before the next one, with
    the block's gate and residual scale; differentiable in y, residual, both
    weights and the gate (scale is a constant)."""
    return BlockNormFunction.apply(y, residual, w_post, w_pre, eps, weight_bias, gate, scale)


def rope(q, k, positions, inv_freq, attn_scale: float = 1.0, interleaved: bool = False):
    """(q_out, k_out): q and k (which may be None) rotated to their positions, as
    rmsnorm_rope; differentiable in q and k."""
    return RopeFunction.apply(q, k, positions, inv_freq, attn_scale, interleaved)
