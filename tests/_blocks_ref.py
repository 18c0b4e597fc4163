"""Plain float64 implementations (CPU tensors in, CPU float64 out) of the operators of
include/kda_blocks.h, written from the definitions there, and the error bars of their tests. Shares
no code with the kernels.

Bars count roundings: half a step of bf16 is 2^-8 of the value at most, of fp32 2^-24. What is left
over for fp32 arithmetic (exponentials of 2^-22, sums of a few hundred products) is 2^-12 of the
same sums of absolute values: 16 times less than one bf16 rounding, and far more than it needs."""
import math

import torch

from _serving_ref import check, d, half_ulp  # noqa: F401  (for the tests)

BF, FINE = 2.0 ** -8, 2.0 ** -12


# ---- rotary positions ----

def turn(x, positions, frequencies, magnitude=1.0, interleaved=False, sign=1):
    """x [S, H, D] and the bar of its rotation: sine and cosine within 2^-22 (2 steps of fp32 and the
    angle's), magnitude and products rounded: 2^-21 of |a| + |b| covers them."""
    y, bar = d(x).clone(), torch.zeros(x.shape, dtype=torch.float64)
    f = torch.tensor(frequencies, dtype=torch.float64)
    half = len(frequencies)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    u, v = y[..., a].clone(), y[..., b].clone()
    angle = torch.as_tensor(positions).double()[:, None, None] * f
    c, s = magnitude * torch.cos(angle), sign * magnitude * torch.sin(angle)
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    bar[..., a] = bar[..., b] = 2.0 ** -21 * magnitude * (u.abs() + v.abs())
    return y, bar


# ---- causal attention of packed sequences ----

def attention(q, k, v, cu, scale, d_o=None):
    """dict of o, lse and, with d_o, dq, dk, dv; and dict of their bars."""
    q, k, v, d_o = (d(t) for t in (q, k, v, d_o))
    S, Hq, D = q.shape
    group = Hq // k.shape[1]
    out = dict(o=torch.zeros_like(q), lse=torch.zeros(Hq, S, dtype=torch.float64))
    if d_o is not None:
        out.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v))
    bar = {n: torch.zeros_like(t) for n, t in out.items()}
    for lo, hi in zip(cu[:-1], cu[1:]):
        for h in range(Hq):
            r, g = slice(lo, hi), h // group
            x, y, z = q[r, h], k[r, g], v[r, g]
            later = torch.ones(hi - lo, hi - lo, dtype=torch.bool).triu(1)
            s = (x @ y.T * scale).masked_fill(later, -math.inf)
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None]) if hi > lo else s
            out["lse"][h, r], out["o"][r, h] = lse, p @ z
            # the scores' fp32 sums: 2^-20 of the absolute ones (128 additions of half a step, at random)
            if hi > lo:
                bar["lse"][h, r] = 2.0 ** -20 * (1 + lse.abs() + scale * (x.abs() @ y.abs().T).amax(1))
            bar["o"][r, h] = (BF + FINE) * (p @ z.abs())
            if d_o is None:
                continue
            w = d_o[r, h]
            o = p @ z
            delta, dp = (w * o).sum(1, keepdim=True), w @ z.T
            ds = p * (dp - delta)
            out["dv"][r, g] += p.T @ w
            out["dq"][r, h] = scale * ds @ y
            out["dk"][r, g] += scale * ds.T @ x
            # dS is rounded, and so was the o that delta is formed from
            e = (BF + FINE) * ds.abs() + p * BF * (w.abs() * o.abs()).sum(1, keepdim=True) + \
                FINE * p * (w.abs() @ z.abs().T + (w.abs() * o.abs()).sum(1, keepdim=True))
            bar["dv"][r, g] += (BF + FINE) * (p.T @ w.abs())
            bar["dq"][r, h] = scale * e @ y.abs()
            bar["dk"][r, g] += scale * e.T @ x.abs()
    return out, bar


def check_all(got, ref, bar):
    for n, t in got.items():
        check(t, ref[n], bar[n], n)
        # and as a whole: roundings of either sign leave the error well below their largest, 2^-8 of the terms
        fine = torch.isfinite(ref[n])
        if fine.any():
            err = (d(t) - ref[n])[fine].pow(2).mean().sqrt()
            assert err <= 0.01 * ref[n][fine].pow(2).mean().sqrt() + 0.25 * bar[n][fine].pow(2).mean().sqrt(), (n, err)


# ---- gradient norm ----

def norm(grads):
    """In pieces that neither overflow nor vanish in float64."""
    return math.sqrt(math.fsum(d(t).reshape(-1).square().sum().item() for t in grads))
