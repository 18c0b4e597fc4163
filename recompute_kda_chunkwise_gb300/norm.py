"""The norm between blocks (include/kda_serving.h, kda_block_norm_fwd / _bwd):

    u     = w_post * RMS(y) * sigmoid(z)
    h_out = residual_scale * h + block_scale * u
    n     = w_pre * RMS(h_out)

over the last dimension. Any of z, h, w_post, w_pre may be left out; without
h and w_pre it is the gated output norm of a delta-rule layer.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._serving import bind, done
from .kda import _dense


def block_norm_fwd(y, *, z=None, h=None, w_post=None, w_pre=None, residual_scale: float = 1.0, block_scale: float = 1.0,
                   eps: float = 1e-5, out=None):
    """Forward. y, z, h: [..., width] in one dtype; w_post, w_pre: [width]
    fp32. Returns (h_out, n); n is None without w_pre. ``out`` may hold
    (h_out, n), either of them None, and h_out may be h."""
    h_out, n = (None, None) if out is None else out
    return done(bind().norm_fwd(y, z, h, w_post, w_pre, residual_scale, block_scale, eps, h_out, n), "kda_block_norm_fwd")


def block_norm_bwd(y, *, z=None, h=None, w_post=None, w_pre=None, dh_out=None, dn=None, residual_scale: float = 1.0,
                   block_scale: float = 1.0, eps: float = 1e-5, workspace=None):
    """Backward, from the forward's inputs and the gradients of h_out and n
    (zero when None). Returns dict dy, dz, dh, dw_post, dw_pre (None for what
    was not given)."""
    r = done(bind().norm_bwd(y, z, h, w_post, w_pre, dh_out, dn, residual_scale, block_scale, eps, workspace),
             "kda_block_norm_bwd")
    return dict(zip(("dy", "dz", "dh", "dw_post", "dw_pre"), r))


class BlockNormFunction(torch.autograd.Function):
    """Autograd wrapper: saves the inputs only. Differentiable once: a second
    derivative through it raises."""

    @staticmethod
    def forward(ctx, y, z, h, w_post, w_pre, residual_scale, block_scale, eps):
        h_out, n = block_norm_fwd(y, z=z, h=h, w_post=w_post, w_pre=w_pre, residual_scale=residual_scale,
                                  block_scale=block_scale, eps=eps)
        ctx.save_for_backward(y, z, h, w_post, w_pre)
        ctx.args = dict(residual_scale=residual_scale, block_scale=block_scale, eps=eps)
        ctx.set_materialize_grads(False)
        return h_out if n is None else (h_out, n)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh_out, dn=None):
        y, z, h, w_post, w_pre = ctx.saved_tensors
        c = lambda t: None if t is None else _dense(t)  # noqa: E731
        g = block_norm_bwd(y, z=z, h=h, w_post=w_post, w_pre=w_pre, dh_out=c(dh_out), dn=c(dn), **ctx.args)
        return g["dy"], g["dz"], g["dh"], g["dw_post"], g["dw_pre"], None, None, None


def block_norm(y, *, z=None, h=None, w_post=None, w_pre=None, residual_scale: float = 1.0, block_scale: float = 1.0,
               eps: float = 1e-5):
    """Differentiable (once) block norm. Returns h_out, or (h_out, n) with w_pre."""
    return BlockNormFunction.apply(y, z, h, w_post, w_pre, residual_scale, block_scale, eps)
