"""The norm between blocks (include/kda_serving.h, kda_block_norm_fwd / _bwd):

    u     = w_post * RMS(y) * sigmoid(z)
    h_out = residual_scale * h + block_scale * u
    n     = w_pre * RMS(h_out)

over the last dimension. Any of z, h, w_post, w_pre may be left out; without
h and w_pre it is the gated output norm of a delta-rule layer.
"""
from __future__ import annotations

import torch

from . import kda as _kda
from ._serving import NormProblem, check, library, maybe, need, stream


def _problem(y, a, b, eps):
    if y.dim() < 1 or y.dtype not in _kda._DTYPE_CODE:
        raise ValueError(f"y must be [..., width] in bfloat16 or float32 (got {y.dtype} {tuple(y.shape)})")
    D = y.shape[-1]
    return NormProblem(y.numel() // D if D else 0, D, _kda._DTYPE_CODE[y.dtype], a, b, eps), y.shape, D


def block_norm_fwd(y, *, z=None, h=None, w_post=None, w_pre=None, residual_scale: float = 1.0, block_scale: float = 1.0,
                   eps: float = 1e-5, out=None):
    """Forward. y, z, h: [..., width] in one dtype; w_post, w_pre: [width]
    fp32. Returns (h_out, n); n is None without w_pre. ``out`` may hold
    (h_out, n) and h_out may be h."""
    p, shape, D = _problem(y, residual_scale, block_scale, eps)
    dev, dt, f32 = y.get_device(), y.dtype, torch.float32
    args = [need(y, "y", shape, dt, dev), maybe(z, "z", shape, dt, dev), maybe(h, "h", shape, dt, dev),
            maybe(w_post, "w_post", (D,), f32, dev), maybe(w_pre, "w_pre", (D,), f32, dev)]
    if out is None:
        h_out = torch.empty_like(y)
        n = torch.empty_like(y) if w_pre is not None else None
    else:
        h_out, n = out
    st = library().kda_block_norm_fwd(p, *args, need(h_out, "h_out", shape, dt, dev),
                                      maybe(n, "n", shape, dt, dev), stream(dev))
    if st:
        check(st, "kda_block_norm_fwd")
    return h_out, n


def block_norm_bwd(y, *, z=None, h=None, w_post=None, w_pre=None, dh_out=None, dn=None, residual_scale: float = 1.0,
                   block_scale: float = 1.0, eps: float = 1e-5, workspace=None):
    """Backward, from the forward's inputs and the gradients of h_out and n
    (zero when None). Returns dict dy, dz, dh, dw_post, dw_pre (None for what
    was not given)."""
    p, shape, D = _problem(y, residual_scale, block_scale, eps)
    dev, dt, f32 = y.get_device(), y.dtype, torch.float32
    args = [need(y, "y", shape, dt, dev), maybe(z, "z", shape, dt, dev), maybe(h, "h", shape, dt, dev),
            maybe(w_post, "w_post", (D,), f32, dev), maybe(w_pre, "w_pre", (D,), f32, dev),
            maybe(dh_out, "dh_out", shape, dt, dev), maybe(dn, "dn", shape, dt, dev)]
    g = {"dy": torch.empty_like(y), "dz": None if z is None else torch.empty_like(z),
         "dh": None if h is None else torch.empty_like(h),
         "dw_post": None if w_post is None else torch.empty_like(w_post),
         "dw_pre": None if w_pre is None else torch.empty_like(w_pre)}
    lib = library()
    size = lib.kda_block_norm_workspace_bytes(p, w_post is not None, w_pre is not None)
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=y.device) if size else None
    else:
        _kda._check_buffer(workspace, size, y, "workspace")
    st = lib.kda_block_norm_bwd(p, *args, *(None if t is None else t.data_ptr() for t in g.values()),
                                None if workspace is None else workspace.data_ptr(), stream(dev))
    if st:
        check(st, "kda_block_norm_bwd")
    return g


class BlockNormFunction(torch.autograd.Function):
    """Autograd wrapper: saves the inputs only."""

    @staticmethod
    def forward(ctx, y, z, h, w_post, w_pre, residual_scale, block_scale, eps):
        h_out, n = block_norm_fwd(y, z=z, h=h, w_post=w_post, w_pre=w_pre, residual_scale=residual_scale,
                                  block_scale=block_scale, eps=eps)
        ctx.save_for_backward(y, z, h, w_post, w_pre)
        ctx.args = dict(residual_scale=residual_scale, block_scale=block_scale, eps=eps)
        ctx.set_materialize_grads(False)
        return h_out if n is None else (h_out, n)

    @staticmethod
    def backward(ctx, dh_out, dn=None):
        y, z, h, w_post, w_pre = ctx.saved_tensors
        c = lambda t: None if t is None else t.contiguous()  # noqa: E731
        g = block_norm_bwd(y, z=z, h=h, w_post=w_post, w_pre=w_pre, dh_out=c(dh_out), dn=c(dn), **ctx.args)
        return g["dy"], g["dz"], g["dh"], g["dw_post"], g["dw_pre"], None, None, None


def block_norm(y, *, z=None, h=None, w_post=None, w_pre=None, residual_scale: float = 1.0, block_scale: float = 1.0,
               eps: float = 1e-5):
    """Differentiable block norm. Returns h_out, or (h_out, n) with w_pre."""
    return BlockNormFunction.apply(y, z, h, w_post, w_pre, residual_scale, block_scale, eps)
