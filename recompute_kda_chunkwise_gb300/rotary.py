"""Rotary positions (include/kda_blocks.h, kda_rotary): the channels of every
query and key head turn in pairs by an angle that grows with the position.

    rope = Rotary(128, base=10000.0, scaling="by_parts", factor=8.0, trained=4096)
    q, k = rotary(rope, q, k, cu_seqlens=cu_seqlens)        # autograd
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from ._serving import bind, done
from .kda import _dense


class Rotary:
    """Which channels turn, how fast and in which layout; made once, on one device.

    dim          channels of a head that turn: the first ``dim`` (even)
    base         pair i turns by base ** (-2 i / dim) radians a position
    interleaved  pairs are channels (2i, 2i + 1) instead of (i, i + dim / 2)
    scaling      how a context of ``factor`` times the trained length is reached:
                 "linear": every frequency divided by factor;
                 "ntk": base * factor ** (dim / (dim - 2)), which divides the slowest
                 by factor and leaves the fastest (dim > 2);
                 "by_parts": a pair that makes ``low`` turns or fewer within ``trained``
                 positions is divided by factor, one that makes ``high`` or more is
                 left, with a ramp between that is linear in the number of turns;
                 rotated channels are scaled by 0.1 ln(factor) + 1. (Weights that
                 were trained with a ramp over the pairs' index want ``frequencies``.)
    frequencies  radians a position for each pair, instead of base and scaling
    magnitude    scales the rotated channels (None: 1, or by_parts' value)

    Frequencies are worked out in double precision and kept in ``turns``, as
    int64 units of 2^-64 of a turn (the device's 64-bit products with a position
    are exact modulo whole turns)."""

    def __init__(self, dim, *, base=10000.0, interleaved=False, scaling=None, factor=1.0, trained=None, low=1.0, high=32.0,
                 frequencies=None, magnitude=None, device="cuda"):
        if dim < 2 or dim % 2:
            raise ValueError(f"dim must be even and at least 2 (got {dim})")
        if frequencies is not None:
            if scaling is not None:
                raise ValueError("frequencies are given as they are: no scaling")
            f = [float(x) for x in (frequencies.tolist() if torch.is_tensor(frequencies) else frequencies)]
            if len(f) != dim // 2:
                raise ValueError(f"{dim // 2} frequencies are needed (got {len(f)})")
        else:
            if not (base > 0 and math.isfinite(base)):
                raise ValueError(f"base must be positive (got {base})")
            if not (factor >= 1 and math.isfinite(factor)):
                raise ValueError(f"factor must be at least 1 (got {factor})")
            if scaling == "ntk":
                if dim == 2:
                    raise ValueError("ntk scaling needs more than one pair")
                base = base * factor ** (dim / (dim - 2))
            f = [base ** (-2 * i / dim) for i in range(dim // 2)]
            if scaling == "linear":
                f = [x / factor for x in f]
            elif scaling == "by_parts":
                if trained is None or trained <= 0 or not low < high:
                    raise ValueError("by_parts scaling needs the trained length, and low < high")
                keep = [min(max((trained * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
                f = [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]
                if magnitude is None:
                    magnitude = 0.1 * math.log(factor) + 1.0
            elif scaling not in (None, "ntk"):
                raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'by_parts' (got {scaling!r})")
        if not all(math.isfinite(x) for x in f):
            raise ValueError("frequencies must be finite")
        self.dim, self.interleaved = dim, bool(interleaved)
        self.magnitude = 1.0 if magnitude is None else float(magnitude)
        self.frequencies = f
        units = [round(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64) % (1 << 64) for x in f]
        self.turns = torch.tensor([u - (1 << 64) if u >= 1 << 63 else u for u in units], dtype=torch.int64, device=device)


def _call(rope, q, k, inverse, positions, cu_seqlens, out, status):
    q_out, k_out = (None, None) if out is None else out
    return done(bind().rotary(rope.turns, rope.interleaved, rope.magnitude, q, k, inverse, positions, cu_seqlens, q_out, k_out,
                              status), "kda_rotary")


def rotary_fwd(rope, q, k=None, *, positions=None, cu_seqlens=None, out=None, status=None):
    """Rotates q [S, Hq, D] and k [S, Hkv, D] (bf16 or fp32; slices of a fused
    projection fit: a token's heads and channels have to be contiguous). A
    token's position is positions[s] (int32 [S]) or its index in its sequence
    of cu_seqlens (int32 [N+1]); one of the two is given. Tokens that it puts into no
    sequence (padding) are zeros in an output that the call makes, are left as they
    were in a given one, and are recorded in status (an int32 CUDA tensor of one
    zero, read with ``kda.query_device_status``). Returns (q', k'),
    contiguous; k' is None without k. ``out`` may hold (q', k'), either of
    them None; each may be its contiguous input, and overlaps nothing else."""
    return _call(rope, q, k, 0, positions, cu_seqlens, out, status)


def rotary_bwd(rope, dq, dk=None, *, positions=None, cu_seqlens=None, out=None, status=None):
    """Gradients of q and k from those of q' and k': the opposite rotation."""
    return _call(rope, dq, dk, 1, positions, cu_seqlens, out, status)


class RotaryFunction(torch.autograd.Function):
    """Autograd wrapper. Differentiable once: a second derivative through it raises."""

    @staticmethod
    def forward(ctx, rope, q, k, positions, cu_seqlens, status=None):
        ctx.save_for_backward(positions, cu_seqlens)
        ctx.rope, ctx.status = rope, status
        qr, kr = rotary_fwd(rope, q, k, positions=positions, cu_seqlens=cu_seqlens, status=status)
        return qr if k is None else (qr, kr)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk=None):
        positions, cu_seqlens = ctx.saved_tensors
        dq, dk = rotary_bwd(ctx.rope, _dense(dq), None if dk is None else _dense(dk), positions=positions,
                            cu_seqlens=cu_seqlens, status=ctx.status)
        return None, dq, dk, None, None, None


def rotary(rope, q, k=None, *, positions=None, cu_seqlens=None, status=None):
    """Differentiable (once) rotation. Returns q', or (q', k') with k. Tokens
    that cu_seqlens puts into no sequence are zeros, and so are their gradients;
    the forward and the backward record them in status."""
    return RotaryFunction.apply(rope, q, k, positions, cu_seqlens, status)
