"""Causal attention of packed sequences, for training and for scoring
(include/kda_blocks.h, kda_attention_fwd / _bwd). Thin binding.

Token i of a sequence attends to its sequence's tokens up to itself. q
[S, Hq, D], k and v [S, Hkv, D] in bf16, D 64 or 128, Hq a multiple of Hkv;
each may be a slice of a fused projection (contiguous within a token).

cu_seqlens goes from 0 to S without decreasing: rows behind the last sequence
(padding) are given a sequence of their own, or sliced off. It is checked on the
device. Where it is refused, every output that the call itself makes is NaN, a
given ``out`` is left as it was, and ``status`` says so: an int32 CUDA tensor of
one zero, read with ``kda.query_device_status``; without one, the head of the
workspace holds that word. A value that is not finite may reach tokens of its own
sequence that do not see it, never another sequence.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from ._serving import AttentionProblem, bind, done, library
from .kda import _dense


def attention_fwd(q, k, v, cu_seqlens, *, scale=None, out=None, workspace=None, status=None):
    """Forward. cu_seqlens int32 [N+1]; scale: D ** -0.5 when None. workspace: a
    uint8 CUDA buffer of at least attention_workspace_bytes, whose head holds
    the call's status word where no status is given; allocated when None. out may hold o, and may be a
    contiguous q; it and the workspace overlap nothing else. Returns (o [S, Hq, D], lse
    fp32 [Hq, S]: the logarithm of each query's sum of exponentials)."""
    return done(bind().packed_fwd(q, k, v, cu_seqlens, scale, out, workspace, status), "kda_attention_fwd")


def attention_bwd(q, k, v, o, lse, d_o, cu_seqlens, *, scale=None, workspace=None, status=None):
    """Gradients (dq, dk, dv) from the forward's inputs and outputs and the
    gradient d_o of o. The same bits every time."""
    return done(bind().packed_bwd(q, k, v, o, lse, d_o, cu_seqlens, scale, workspace, status), "kda_attention_bwd")


def attention_workspace_bytes(q, k, cu_seqlens, *, backward=False) -> int:
    """Bytes of workspace for attention_fwd (attention_bwd) with tensors of these shapes."""
    S, Hq, D = q.shape
    p = AttentionProblem(S, Hq * D, k.shape[1] * D, k.shape[1] * D, cu_seqlens.numel() - 1, Hq, k.shape[1], D, 0, 1.0, None)
    lib = library()
    return int((lib.kda_attention_bwd_workspace_bytes if backward else lib.kda_attention_fwd_workspace_bytes)(ctypes.byref(p)))


class AttentionFunction(torch.autograd.Function):
    """Autograd wrapper: saves the inputs, o and lse. Differentiable once: a
    second derivative through it raises."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale, status=None):
        o, lse = attention_fwd(q, k, v, cu_seqlens, scale=scale, status=status)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.scale, ctx.status = scale, status
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o):
        q, k, v, o, lse, cu_seqlens = ctx.saved_tensors
        return *attention_bwd(q, k, v, o, lse, _dense(d_o), cu_seqlens, scale=ctx.scale, status=ctx.status), None, None, None


def attention(q, k, v, cu_seqlens, *, scale=None, status=None):
    """Differentiable (once) causal attention of packed sequences. Returns o.
    cu_seqlens that are refused (they do not end at S, for one) give NaN, and
    are recorded in ``status``, by the forward and the backward."""
    return AttentionFunction.apply(q, k, v, cu_seqlens, scale, status)
