"""Cases for the operators of attention blocks from training to serving: rotary positions, the paged
append that rotates on the way, causal attention of packed sequences with its gradient, and the
global gradient norm with clipping.

``run`` is one pass through an operator. With ``own`` false it uses elementary torch operations in
fp32 (the plain forms below; angles in fp64, since fp32 loses those of far positions); with ``own``
true it calls this package. ``exact`` is each operator's definition in float64, written separately.
Sizes: head counts 12, 16, 64 and head dims 64 / 128 are the package's own workloads'; the others are
generic.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda"


def listed():
    return [
        # --- rotary positions of queries and keys ---
        # one decoded token far into a context: latency
        dict(name="rotary_one_token", op="rotary", S=1, N=1, Hq=16, Hkv=16, D=128, R=128, layout="half", scaling="linear",
             dtype="bf16", at="positions", far=1_000_000, mode="fwd"),
        # an attention layer in training: packed sequences, the whole head, context extended eightfold
        dict(name="rotary_train", op="rotary", S=8192, N=3, Hq=64, Hkv=8, D=128, R=128, layout="half", scaling="by_parts",
             dtype="bf16", at="cu", far=0, mode="train"),
        # fp32, a part of the head that no vector width divides, interleaved pairs, an odd number of tokens
        dict(name="rotary_part_f32", op="rotary", S=1777, N=1, Hq=12, Hkv=3, D=64, R=42, layout="pairs", scaling="ntk",
             dtype="f32", at="positions", far=50_000, mode="train"),
        # --- new tokens into a paged cache, keys (and the queries) rotated on the way ---
        # decode: 32 sequences of unequal length, one new token each
        dict(name="append_decode", op="append", N=32, L=1, ragged=False, kv=16384, Hq=64, Hkv=8, D=128, R=128, layout="half",
             scaling="by_parts", page=64),
        # chunked prefill: sequences with chunks of up to 2048 new tokens, small pages, half of the head
        dict(name="append_chunk", op="append", N=4, L=2048, ragged=True, kv=8192, Hq=64, Hkv=8, D=128, R=64, layout="pairs",
             scaling="none", page=16),
        # --- causal attention of packed sequences ---
        # one short sequence, training: latency
        dict(name="attn_short", op="attn", lens="77", Hq=16, Hkv=16, D=128, mode="train"),
        # a packed batch of unequal sequences, training: one token, less than a tile, odd lengths
        dict(name="attn_packed", op="attn", lens="4096 1 2777 130 3001 64 1999 513 3803", Hq=16, Hkv=4, D=64, mode="train"),
        # one long sequence with grouped heads, training: the largest
        dict(name="attn_long", op="attn", lens="8192", Hq=64, Hkv=8, D=128, mode="train"),
        # scoring of two documents: forward only, a key/value head for each query head
        dict(name="attn_score", op="attn", lens="5000 3192", Hq=16, Hkv=16, D=128, mode="fwd"),
        # --- the global gradient norm, and clipping by it ---
        # the gradients of a small stack, fp32
        dict(name="clip_small", op="clip", layers=2, width=256, dtype="f32", into="same", mode="clip"),
        # the gradients of a large stack: bf16 matrices, fp32 vectors, clipped into fp32 for the optimizer
        dict(name="clip_large", op="clip", layers=7, width=4096, dtype="bf16", into="f32", mode="clip"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attn", "attn", "clip"])
    layout, scaling = rng.choice(["half", "pairs"]), rng.choice(["none", "linear", "ntk", "by_parts"])
    if op == "rotary":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 3, 8, 16])
        Hq = Hkv * rng.choice([1, 3, 4])
        return dict(op=op, S=_log(rng, 1, 75_000_000 // ((Hq + Hkv) * D)), N=_log(rng, 1, 16), Hq=Hq, Hkv=Hkv, D=D,
                    R=rng.choice([D, D, D // 2, 2 * rng.randint(2, D // 2)]), layout=layout, scaling=scaling,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), at=rng.choice(["positions", "cu"]),
                    far=_log(rng, 100, 1_000_000), mode=rng.choice(["fwd", "train"]))
    if op == "append":
        kv = _log(rng, 1, 16384)
        Hkv = rng.choice([1, 2, 4, 8])
        L = min(kv, rng.choice([1, rng.randint(2, 8), _log(rng, 8, 2048)]))
        D = rng.choice([64, 128])
        return dict(op=op, N=_log(rng, 1, 32) if L <= 8 else rng.randint(1, 4), L=L, ragged=rng.random() < 0.7, kv=kv,
                    Hq=Hkv * rng.choice([1, 3, 4, 8]), Hkv=Hkv, D=D, R=rng.choice([D, D, D // 2, 2 * rng.randint(2, D // 2)]),
                    layout=layout, scaling=scaling, page=rng.choice([8, 16, 24, 32, 64, 128, 256]))
    if op == "attn":
        D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 3, 4, 8])
        # query heads times squared lengths within the largest listed case's
        most = min(16384, int((8192 * 8192 * 64 / Hq) ** 0.5))
        total, lens = _log(rng, 1, most), []
        parts = rng.choice([1, 1, 3, 12])
        for i in range(parts):
            left = total - sum(lens)
            lens.append(left if i == parts - 1 else rng.randint(0, left) if rng.random() < 0.8 else 0)
        rng.shuffle(lens)
        return dict(op=op, lens=" ".join(map(str, lens)), Hq=Hq, Hkv=Hkv, D=D, mode=rng.choice(["fwd", "train", "train"]))
    width, mode = _log(rng, 16, 4096), rng.choice(["clip", "clip", "norm"])
    layers = _log(rng, 1, min(7 if mode == "clip" else 40, 500_000_000 // (8 * width * width) + 1))
    return dict(op=op, layers=layers, width=width, dtype=rng.choice(["bf16", "f32"]), into=rng.choice(["same", "f32"]), mode=mode)


# ---- lengths and shapes that a case fixes ----

def _seq_lens(c):
    """Lengths of the packed sequences of a rotary case."""
    r = random.Random(31 * c["S"] + c["N"])
    cuts = sorted(r.randint(0, c["S"]) for _ in range(c["N"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [c["S"]])]


def _new_lens(c):
    """New tokens of each sequence of an append: the largest first."""
    n, most = c["N"], c["L"]
    if most == 1 or not c["ragged"]:
        return [most] * n
    r = random.Random(1000 * n + most)
    return [most] + [r.randint(0, most) for _ in range(n - 1)]


def _kv_lens(c, new):
    """Cached length of each sequence, its new tokens included."""
    r = random.Random(77 * c["N"] + c["kv"])
    return [c["kv"] if i == 0 else max(n, r.randint(c["kv"] // 4, c["kv"])) for i, n in enumerate(new)]


def _attn_lens(c):
    """Lengths of the packed sequences of an attention case."""
    return [int(n) for n in c["lens"].split()]


def _shapes(c):
    """Gradients of a stack: per layer a wide projection, an output projection and small vectors."""
    w, out = c["width"], []
    out.append((2 * w + 1, w))
    for _ in range(c["layers"]):
        out += [(w, 5 * w), (w, 16), (16,), (16, 7), (w, w), (w,), (w,), (1,)]
    return out


# ---- inputs ----

def _cu(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=_DEV)


_SCALING = {"none": {}, "linear": dict(scaling="linear", factor=4.0), "ntk": dict(scaling="ntk", factor=4.0),
            "by_parts": dict(scaling="by_parts", factor=8.0, trained=4096)}


def _frequencies(c):
    """Radians per position [R / 2] in fp64, and the magnitude of the rotated channels."""
    R, base, mag = c["R"], 10000.0, 1.0
    how = _SCALING[c["scaling"]]
    if c["scaling"] == "ntk" and R > 2:
        base = base * how["factor"] ** (R / (R - 2))
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    if c["scaling"] == "linear":
        f = [x / how["factor"] for x in f]
    elif c["scaling"] == "by_parts":
        # whole turns within the trained length: up to 1 stretched by the factor, from 32 on left alone
        keep = [min(max((how["trained"] * x / (2 * math.pi) - 1.0) / (32.0 - 1.0), 0.0), 1.0) for x in f]
        f = [x * (k + (1 - k) / how["factor"]) for x, k in zip(f, keep)]
        mag = 0.1 * math.log(how["factor"]) + 1.0
    return f, mag


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    normal = lambda *s, std=1.0: torch.randn(*s, generator=g, device=_DEV) * std  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op in ("rotary", "append"):
        if own:
            from recompute_kda_chunkwise_gb300.rotary import Rotary
            s["rope"] = Rotary(case["R"], base=10000.0, interleaved=case["layout"] == "pairs", **_SCALING[case["scaling"]])
        f, s["magnitude"] = _frequencies(case)
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device=_DEV)
        D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
        dt = _DT[case.get("dtype", "bf16")]
    if op == "rotary":
        S = case["S"]
        # queries, keys and values as the projection leaves them, side by side in a row
        fused = normal(S, (Hq + 2 * Hkv) * D).to(dt)
        s["q"], s["k"] = fused[:, :Hq * D].view(S, Hq, D), fused[:, Hq * D:(Hq + Hkv) * D].view(S, Hkv, D)
        s["cu"] = _cu(_seq_lens(case)) if case["at"] == "cu" else None
        s["positions"] = torch.randint(0, case["far"] + 1, (S,), generator=g, device=_DEV, dtype=torch.int32) \
            if case["at"] == "positions" else None
        if case["mode"] == "train":
            s["dq"], s["dk"] = normal(S, Hq, D).to(dt), normal(S, Hkv, D).to(dt)
    elif op == "append":
        page = case["page"]
        new = _new_lens(case)
        kv = _kv_lens(case, new)
        S, need = sum(new), [-(-x // page) for x in kv]
        fused = normal(S, (Hq + 2 * Hkv) * D).to(dt)
        parts = fused.split([Hq * D, Hkv * D, Hkv * D], 1)
        s["q"], s["k"], s["v"] = (t.view(S, -1, D) for t in parts)
        pages = sum(need) + 5
        s["k_pages"], s["v_pages"] = normal(pages, page, Hkv, D).to(dt), normal(pages, page, Hkv, D).to(dt)
        order = torch.randperm(pages, generator=g, device=_DEV).to(torch.int32)
        s["table"] = torch.zeros(case["N"], max(need), dtype=torch.int32, device=_DEV)
        at = 0
        for i, n in enumerate(need):
            s["table"][i, :n] = order[at:at + n]
            at += n
        s["lens"] = torch.tensor(kv, dtype=torch.int32, device=_DEV)
        s["cu"] = _cu(new)
    elif op == "attn":
        S, Hq, Hkv, D = sum(_attn_lens(case)), case["Hq"], case["Hkv"], case["D"]
        s["q"], s["k"], s["v"] = (normal(S, h, D).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        s["cu"] = _cu(_attn_lens(case))
        s["scale"] = D ** -0.5
        if case["mode"] == "train":
            s["do"] = normal(S, Hq, D, std=0.5).to(torch.bfloat16)
    else:
        dt = _DT[case["dtype"]]
        r = random.Random(int(seed))
        s["grads"] = []
        for shape in _shapes(case):  # matrices in the case's type, vectors in fp32, sizes of gradients far apart
            t = torch.randn(shape, generator=g, device=_DEV, dtype=dt if len(shape) > 1 else torch.float32)
            s["grads"].append(t.mul_(10.0 ** r.uniform(-5, -1)))
        s["out"] = [torch.empty_like(t, dtype=torch.float32 if case["into"] == "f32" else t.dtype) for t in s["grads"]] \
            if case["mode"] == "clip" else None
        # about half of the norm of gradients of these sizes
        s["max_norm"] = 0.01 * sum(t.numel() for t in s["grads"]) ** 0.5
    return s


# ---- one pass ----

def run(s):
    return {"rotary": _run_rotary, "append": _run_append, "attn": _run_attn, "clip": _run_clip}[s["case"]["op"]](s)


def _angles(s, positions):
    a = positions.double()[:, None] * s["freqs"]
    return (torch.cos(a) * s["magnitude"]).float()[:, None], (torch.sin(a) * s["magnitude"]).float()[:, None]


def _rotate(x, cos, sin, case):
    """One tensor [S, H, D]; the gradient is the rotation by the opposite angles."""
    R = case["R"]
    y = x.float().clone()
    if case["layout"] == "pairs":
        a, b = y[..., 0:R:2].clone(), y[..., 1:R:2].clone()
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = y[..., :R // 2].clone(), y[..., R // 2:R].clone()
        y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, a * sin + b * cos
    return y.to(x.dtype)


def _run_rotary(s):
    c = s["case"]
    train = c["mode"] == "train"
    if own:
        from recompute_kda_chunkwise_gb300 import rotary
        q, k = rotary.rotary_fwd(s["rope"], s["q"], s["k"], positions=s["positions"], cu_seqlens=s["cu"])
        out = {"q": q, "k": k}
        if train:
            out["dq"], out["dk"] = rotary.rotary_bwd(s["rope"], s["dq"], s["dk"], positions=s["positions"], cu_seqlens=s["cu"])
        return out
    pos = s["positions"]
    if pos is None:
        tok = torch.arange(c["S"], device=_DEV, dtype=torch.int32)
        pos = tok - s["cu"][torch.searchsorted(s["cu"][1:], tok, right=True)]
    cos, sin = _angles(s, pos)
    out = {"q": _rotate(s["q"], cos, sin, c), "k": _rotate(s["k"], cos, sin, c)}
    if train:
        out["dq"], out["dk"] = _rotate(s["dq"], cos, -sin, c), _rotate(s["dk"], cos, -sin, c)
    return out


def _run_append(s):
    c = s["case"]
    if own:
        from recompute_kda_chunkwise_gb300 import decode
        q = decode.paged_append_rotary(s["rope"], s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    cu, lens, page = s["cu"].long(), s["lens"].long(), c["page"]
    tok = torch.arange(s["q"].shape[0], device=_DEV)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    pos = lens[seq] - (cu[seq + 1] - tok)
    cos, sin = _angles(s, pos)
    slot = s["table"][seq, pos // page].long()
    s["k_pages"][slot, pos % page] = _rotate(s["k"], cos, sin, c)
    s["v_pages"][slot, pos % page] = s["v"]
    return {"q": _rotate(s["q"], cos, sin, c), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _run_attn(s):
    c = s["case"]
    train = c["mode"] == "train"
    if own:
        from recompute_kda_chunkwise_gb300 import attention
        o, lse = attention.attention_fwd(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"])
        out = {"o": o, "lse": lse}
        if train:
            out["dq"], out["dk"], out["dv"] = attention.attention_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], s["cu"], scale=s["scale"])
        return out
    S, Hq, Hkv, D, scale = s["q"].shape[0], c["Hq"], c["Hkv"], c["D"], s["scale"]
    group, f32 = Hq // Hkv, dict(dtype=torch.float32, device=_DEV)
    o, lse = torch.empty(S, Hq, D, **f32), torch.empty(Hq, S, **f32)
    if train:
        dq, dk, dv = torch.empty(S, Hq, D, **f32), torch.zeros(S, Hkv, D, **f32), torch.zeros(S, Hkv, D, **f32)
    a = 0
    for L in _attn_lens(c):
        if L == 0:
            continue
        b = a + L
        later = torch.ones(L, L, dtype=torch.bool, device=_DEV).triu(1)
        step = max(1, min(Hkv, (1 << 28) // (L * L * group)))  # key/value heads at a time, as memory allows
        for h in range(0, Hkv, step):
            hs = min(step, Hkv - h)
            q = s["q"][a:b, h * group:(h + hs) * group].float().reshape(L, hs, group, D).permute(1, 2, 0, 3)
            k, v = (s[n][a:b, h:h + hs].float().permute(1, 0, 2)[:, None] for n in ("k", "v"))
            sc = (torch.matmul(q, k.transpose(-1, -2)) * scale).masked_fill_(later, -math.inf)
            top = sc.amax(-1, keepdim=True)
            p = sc.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            p = p.div_(total)
            y = torch.matmul(p, v)
            o[a:b, h * group:(h + hs) * group] = y.permute(2, 0, 1, 3).reshape(L, hs * group, D)
            lse[h * group:(h + hs) * group, a:b] = (top + total.log()).reshape(hs * group, L)
            if train:
                do = s["do"][a:b, h * group:(h + hs) * group].float().reshape(L, hs, group, D).permute(1, 2, 0, 3)
                dv[a:b, h:h + hs] = torch.matmul(p.transpose(-1, -2), do).sum(1).permute(1, 0, 2)
                ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * y).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                dq[a:b, h * group:(h + hs) * group] = torch.matmul(ds, k).permute(2, 0, 1, 3).reshape(L, hs * group, D)
                dk[a:b, h:h + hs] = torch.matmul(ds.transpose(-1, -2), q).sum(1).permute(1, 0, 2)
        a = b
    out = {"o": o.to(torch.bfloat16), "lse": lse}
    if train:
        out.update(dq=dq.to(torch.bfloat16), dk=dk.to(torch.bfloat16), dv=dv.to(torch.bfloat16))
    return out


def _run_clip(s):
    if own:
        from recompute_kda_chunkwise_gb300 import grads
        if s["case"]["mode"] == "norm":
            return {"norm": grads.grad_norm(s["grads"])}
        return {"norm": grads.clip_grads(s["grads"], s["max_norm"], out=s["out"]), "out": s["out"]}
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).double().sum().sqrt()
    if s["case"]["mode"] == "norm":
        return {"norm": norm.float()}
    factor = torch.where(torch.isfinite(norm), (s["max_norm"] / norm).clamp_max(1.0), 1.0).float()
    for t, y in zip(s["grads"], s["out"]):
        y.copy_(t.float() * factor)
    return {"norm": norm.float(), "out": s["out"]}


# ---- what one pass cannot do without ----

def work(case):
    op = case["op"]
    if op == "rotary":
        e, n = (2 if case["dtype"] == "bf16" else 4), case["S"] * (case["Hq"] + case["Hkv"])
        ways = 2 if case["mode"] == "train" else 1
        return {"bytes": ways * 2 * e * n * case["D"], "flops": ways * 3 * n * case["R"]}
    if op == "append":
        S = sum(_new_lens(case))
        return {"bytes": 2 * S * case["D"] * (2 * case["Hq"] + 4 * case["Hkv"]), "flops": 3 * S * (case["Hq"] + case["Hkv"]) * case["R"]}
    if op == "attn":
        S, Hq, Hkv, D = sum(_attn_lens(case)), case["Hq"], case["Hkv"], case["D"]
        pairs = sum(n * (n + 1) // 2 for n in _attn_lens(case))
        # forward: q, k, v, o, lse; backward: those and do, dq, dk, dv
        nbytes, flops = 2 * D * S * (2 * Hq + 2 * Hkv) + 4 * S * Hq, 4 * pairs * Hq * D
        if case["mode"] == "train":
            nbytes, flops = nbytes + 2 * D * S * (4 * Hq + 4 * Hkv) + 4 * S * Hq, flops + 10 * pairs * Hq * D
        return {"bytes": nbytes, "flops": flops}
    n = total = 0
    for shape in _shapes(case):
        size = math.prod(shape)
        e = 2 if case["dtype"] == "bf16" and len(shape) > 1 else 4
        n += size
        total += size * (e + (0 if case["mode"] == "norm" else 4 if case["into"] == "f32" else e))
    return {"bytes": total, "flops": n * (2 if case["mode"] == "norm" else 3)}


# ---- each operator's definition in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "attn": _exact_attn, "clip": _exact_clip}[case["op"]](case, s)


def _turned(x, pos, case, sign=1):
    """x [S, H, D] with channel pairs as complex numbers, times magnitude * exp(i sign angle)."""
    f, mag = _frequencies(case)
    R = case["R"]
    angle = sign * torch.tensor(pos, dtype=torch.float64, device=_DEV)[:, None] * torch.tensor(f, dtype=torch.float64, device=_DEV)
    z = torch.polar(torch.full_like(angle, mag), angle)[:, None]
    y = x.double().clone()
    if case["layout"] == "pairs":
        w = torch.view_as_complex(y[..., :R].reshape(*y.shape[:2], R // 2, 2).contiguous()) * z
        y[..., :R] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * z
        y[..., :R] = torch.cat([w.real, w.imag], -1)
    return y


def _exact_rotary(case, s):
    if case["at"] == "cu":
        pos = [i for n in _seq_lens(case) for i in range(n)]
    else:
        pos = s["positions"].tolist()
    out = {"q": _turned(s["q"], pos, case), "k": _turned(s["k"], pos, case)}
    if case["mode"] == "train":
        out.update(dq=_turned(s["dq"], pos, case, -1), dk=_turned(s["dk"], pos, case, -1))
    return out


def _exact_append(case, s):
    new = _new_lens(case)
    kv = _kv_lens(case, new)
    pos = [t - n + i for n, t in zip(new, kv) for i in range(n)]
    k = _turned(s["k"], pos, case)
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    at = 0
    for i, n in enumerate(new):
        p = torch.tensor(pos[at:at + n], device=_DEV, dtype=torch.int64)
        rows = s["table"][i].long()[p // case["page"]] * case["page"] + p % case["page"]
        k_pages.view(-1, case["Hkv"], case["D"])[rows] = k[at:at + n]
        v_pages.view(-1, case["Hkv"], case["D"])[rows] = s["v"][at:at + n].double()
        at += n
    return {"q": _turned(s["q"], pos, case), "k_pages": k_pages, "v_pages": v_pages}


def _exact_attn(case, s):
    train, group, scale = case["mode"] == "train", case["Hq"] // case["Hkv"], s["scale"]
    f64 = {n: torch.zeros(t.shape, dtype=torch.float64, device=_DEV) for n, t in (("o", s["q"]), ("dq", s["q"]), ("dk", s["k"]), ("dv", s["v"]))}
    lse = torch.zeros(case["Hq"], s["q"].shape[0], dtype=torch.float64, device=_DEV)
    a = 0
    for L in _attn_lens(case):
        b = a + L
        for h in range(case["Hq"]):
            q, k, v = s["q"][a:b, h].double(), s["k"][a:b, h // group].double(), s["v"][a:b, h // group].double()
            do = s["do"][a:b, h].double() if train else None
            for i in range(0, L, 2048):  # rows i .. j of the sequence see its keys 0 .. j
                j = min(L, i + 2048)
                sc = torch.einsum("id,jd->ij", q[i:j], k[:j]) * scale
                sc[torch.arange(j, device=_DEV)[None] > torch.arange(i, j, device=_DEV)[:, None]] = -math.inf
                lse[h, a + i:a + j] = torch.logsumexp(sc, 1)
                p = torch.softmax(sc, 1)
                f64["o"][a + i:a + j, h] = p @ v[:j]
                if train:
                    f64["dv"][a:a + j, h // group] += p.T @ do[i:j]
                    dp = do[i:j] @ v[:j].T
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                    f64["dq"][a + i:a + j, h] = ds @ k[:j]
                    f64["dk"][a:a + j, h // group] += ds.T @ q[i:j]
        a = b
    out = {"o": f64["o"], "lse": lse}
    if train:
        out.update(dq=f64["dq"], dk=f64["dk"], dv=f64["dv"])
    return out


def _exact_clip(case, s):
    total = 0.0
    for t in s["grads"]:
        total += torch.linalg.vector_norm(t.double()).item() ** 2
    norm = torch.tensor(math.sqrt(total), dtype=torch.float64, device=_DEV)
    if case["mode"] == "norm":
        return {"norm": norm}
    factor = min(1.0, s["max_norm"] / norm.item())
    return {"norm": norm, "out": [t.double() * factor for t in s["grads"]]}
