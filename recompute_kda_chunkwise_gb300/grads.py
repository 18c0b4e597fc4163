"""The global gradient norm over many tensors, and clipping by it
(include/kda_blocks.h, kda_grad_norm / kda_clip_grads).

Tensors are dense CUDA tensors of one device in bf16 or fp32, of any number
and size. The norm stays on the device: nothing waits for it.
"""
from __future__ import annotations

from ._serving import bind, done


def grad_norm(grads, *, workspace=None):
    """sqrt of the sum of squares over all tensors of the list, as an fp32 CUDA
    tensor without dimensions (0 for an empty list)."""
    return done(bind().norm_of_grads(grads, workspace), "kda_grad_norm")


def clip_grads(grads, max_norm, *, out=None, workspace=None):
    """out[i] = grads[i] * min(1, max_norm / norm); returns the norm before
    clipping, as ``grad_norm`` does. ``out``: tensors of the gradients' shapes
    and strides, bf16 or fp32, one for each; the gradients themselves when
    None. No output may overlap anything but its own gradient. A norm that is
    not finite clips nothing: the caller sees it in the result. workspace: a
    uint8 CUDA buffer of 8192 bytes for every 1000 tensors or part of them."""
    return done(bind().clip(grads, max_norm, out, workspace), "kda_clip_grads")
