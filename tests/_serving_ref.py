"""Plain float64 implementations of the serving operators (CPU tensors in,
CPU float64 out), written from the definitions in include/kda_serving.h, and
the error bars of their tests. Shares no code with the kernels."""
import math

import torch


def d(t):
    return None if t is None else t.detach().cpu().double()


def half_ulp(ref, dtype):
    """Half a unit in the last place of ``ref`` stored as ``dtype``."""
    bits = {torch.bfloat16: 8, torch.float32: 24}[dtype]
    return torch.ldexp(torch.ones_like(ref), torch.frexp(ref)[1] - 1 - bits) * (ref != 0)


def check(x, ref, bar, what):
    """|x - ref| within ``bar`` (a number times the RMS of ref, or a tensor)
    beyond the rounding of x's own dtype; NaN and infinities in the same places."""
    got = d(x)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if ref.numel() == 0:
        return
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: not finite in other places"
    rms = ref[fine].pow(2).mean().sqrt() if fine.any() else torch.tensor(0.0)
    bar = bar if torch.is_tensor(bar) else bar * rms
    # the computed value, up to ``bar`` from ref, is what is rounded: half an ulp of the largest it may be
    over = (got - ref).abs() - half_ulp(ref.abs() + bar, x.dtype) - bar
    worst = over[fine].max().item() if fine.any() else 0.0
    assert worst <= 1e-6 * rms + 1e-30, f"{what}: {worst:.3e} over the bar (RMS {rms:.3e})"


def step(q, k, v, g, gates, A_log, dt_bias, cu, states, index, commit, scale=1.0, lower=-5.0, eps=1e-6):
    """o [S, H, D] and the new pool. Inactive sequences (index < 0) give zero rows."""
    q, k, v, g, A_log, dt_bias, pool = (d(t) for t in (q, k, v, g, A_log, dt_bias, states))
    gates = [torch.sigmoid(d(t)) for t in gates]
    pool, o = pool.clone(), torch.zeros_like(q)
    for n in range(len(cu) - 1):
        slot = n if index is None else int(index[n])
        if slot < 0:
            continue
        S, length = pool[slot].clone(), cu[n + 1] - cu[n]
        upto = length if commit is None else min(int(commit[n]), length)
        for i in range(length):
            t = cu[n] + i
            kh = k[t] / (k[t].square().sum(-1, keepdim=True) + eps).sqrt()
            qh = scale * q[t] / (q[t].square().sum(-1, keepdim=True) + eps).sqrt()
            b, w = (gates[0][t], gates[1][t]) if len(gates) == 2 else (gates[0][t][:, None],) * 2
            S = S * torch.exp(lower * torch.sigmoid(A_log.exp()[:, None] * (g[t] + dt_bias)))[:, :, None]
            r = w * v[t] - torch.einsum("hkv,hk->hv", S, b * kh)
            S = S + kh[:, :, None] * r[:, None, :]
            o[t] = torch.einsum("hkv,hk->hv", S, qh)
            if i + 1 == upto:
                pool[slot] = S
    return o, pool


def block_norm(y, z, h, w_post, w_pre, a, b, eps):
    """(h_out, n) as differentiable float64 expressions of float64 tensors."""
    u = y * (y.square().mean(-1, keepdim=True) + eps).rsqrt()
    if w_post is not None:
        u = u * w_post
    if z is not None:
        u = u * torch.sigmoid(z)
    ho = b * u if h is None else a * h + b * u
    n = None if w_pre is None else ho * (ho.square().mean(-1, keepdim=True) + eps).rsqrt() * w_pre
    return ho, n


def verify(target, draft, x, num, u, noise):
    """tokens, accepted (int tensors)."""
    target, draft, u, noise = (d(t) for t in (target, draft, u, noise))
    N, T1, V = target.shape
    tokens, accepted = torch.full((N, T1), -1, dtype=torch.int64), torch.zeros(N, dtype=torch.int64)
    for n in range(N):
        count = T1 - 1 if num is None else min(max(int(num[n]), 0), T1 - 1)
        a = 0
        while a < count:
            t = int(x[n, a])
            if not 0 <= t < V:
                break
            q = 1.0 if draft is None else float(draft[n, a, t])
            if not float(u[n, a]) * q < float(target[n, a, t]):
                break
            tokens[n, a] = t
            a += 1
        r = target[n, a].clone()
        if a < count:
            if draft is not None:
                r = r - draft[n, a]
            elif 0 <= int(x[n, a]) < V:
                r[int(x[n, a])] = 0
            if not (r > 0).any():
                r = target[n, a]
        best, at = -1.0, 0
        score = torch.where(r > 0, r / noise[n], torch.tensor(-1.0, dtype=torch.float64))
        for i in (score == score[~score.isnan()].max()).nonzero()[:1].flatten().tolist():
            best, at = float(score[i]), i
        tokens[n, a] = at if best >= 0 else 0
        accepted[n] = a
    return tokens, accepted


def attention(q, k_pages, v_pages, table, lens, cu, scale):
    """o and, per element, sum_t p_t |v_t| (the size of what the rounding of
    the probabilities can change)."""
    q, k_pages, v_pages = d(q), k_pages.cpu(), v_pages.cpu()
    o, size = torch.zeros_like(q), torch.zeros_like(q)
    page, Hkv = k_pages.shape[1], k_pages.shape[2]
    group = q.shape[1] // Hkv
    for n in range(len(cu) - 1):
        new, total = cu[n + 1] - cu[n], int(lens[n])
        if new == 0 or total <= 0:
            continue
        ids = table[n, : -(-total // page)].long().cpu()
        k = k_pages[ids].flatten(0, 1)[:total].double()
        v = v_pages[ids].flatten(0, 1)[:total].double()
        for i in range(new):
            seen = total - new + i + 1
            if seen <= 0:
                continue
            t = cu[n] + i
            s = torch.einsum("hgd,thd->hgt", q[t].view(Hkv, group, -1), k[:seen]) * scale
            p = torch.softmax(s, -1)
            o[t] = torch.einsum("hgt,thd->hgd", p, v[:seen]).flatten(0, 1)
            size[t] = torch.einsum("hgt,thd->hgd", p, v[:seen].abs()).flatten(0, 1)
    return o, size


def attention_bar(size):
    """Probabilities are rounded to bf16 (8 significant bits: 2^-8 of each at
    most); scores and sums are fp32 (below 2^-15 of a probability for the
    sizes tested)."""
    return size * (2.0 ** -8 + 2.0 ** -14)


def cu_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def inf_like(t):
    return torch.full_like(t, math.inf)
