"""Cases for the serving and block operators: the recurrent gated delta rule, the fused block norm,
attention of a chunk of new tokens over a paged cache, and verification of drafted tokens.

``run`` is one pass through an operator. With ``own`` false it uses elementary torch operations in
fp32 (the plain forms below); with ``own`` true it calls this package. ``exact`` is each operator's
definition in float64, written separately. Sizes: head counts 12, 16, 64, 96 and head dims 64 / 128
are the package's own workloads'; the others are generic.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_DEV = "cuda"
EPS_L2 = 1e-6      # epsilon of the delta rule's q/k norms
EPS_RMS = 1e-5     # epsilon of the block norms
LOWER = -5.0       # lower bound of the delta rule's safe gate
ACCEPT = 0.8       # share of drafted tokens the target accepts with the inputs below (for work())


def listed():
    return [
        # --- the recurrent gated delta rule: one decode step over a pool of states ---
        # one sequence, one token: the latency of single-stream decoding
        dict(name="step_one_token", op="step", gates="kda", dtype="bf16", N=1, H=16, D=128, T=1),
        # a full decode batch at the long-context workload's 96 heads, one token each
        dict(name="step_batch", op="step", gates="kda", dtype="bf16", N=128, H=96, D=128, T=1),
        # speculative decoding with GDN-2's gates: up to 6 tokens a sequence, part of them committed
        dict(name="step_drafts_gdn2", op="step", gates="gdn2", dtype="bf16", N=48, H=16, D=128, T=6),
        # the small fp32 preset's heads: an odd batch with ragged lengths
        dict(name="step_f32_ragged", op="step", gates="kda", dtype="f32", N=201, H=12, D=64, T=3),
        # --- the block norm: norm after the block, its gate, the scaled residual, the next norm ---
        # the output norm of a delta-rule layer in training: per head, sigmoid gate (8192 x 96 rows)
        dict(name="norm_heads_train", op="norm", form="gate", mode="train", dtype="bf16", rows=8192 * 96, D=128),
        # between two blocks of a decode step
        dict(name="norm_decode", op="norm", form="residual", mode="fwd", dtype="bf16", rows=5, D=2048),
        # between two blocks in training, every part in use
        dict(name="norm_train", op="norm", form="full", mode="train", dtype="bf16", rows=8192, D=4096),
        # odd width and row count in fp32
        dict(name="norm_odd_f32", op="norm", form="full", mode="train", dtype="f32", rows=777, D=1537),
        # --- verification of drafted tokens ---
        # one stream, a small vocabulary
        dict(name="verify_one", op="verify", N=1, T=3, V=32000, draft="probs"),
        # a full batch over a large vocabulary
        dict(name="verify_batch", op="verify", N=256, T=5, V=131072, draft="probs"),
        # --- attention of new tokens over a paged cache ---
        # decode: 32 sequences of unequal length, one new token each
        dict(name="attn_decode", op="attn", N=32, L=1, ragged=False, kv=16384, Hq=64, Hkv=8, D=128, page=64),
        # chunked prefill: 2 sequences, chunks of up to 2048 new tokens over what came before
        dict(name="attn_chunk", op="attn", N=2, L=2048, ragged=True, kv=8192, Hq=64, Hkv=8, D=128, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "norm", "verify", "attn"])
    if op == "step":
        c = dict(op=op, gates=rng.choice(["kda", "gdn2"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                 N=_log(rng, 1, 256), H=rng.choice([1, 3, 8, 12, 16, 32]), D=rng.choice([64, 128]), T=rng.randint(1, 8))
        return c
    if op == "norm":
        form = rng.choice(["gate", "residual", "full"])
        if form == "gate":
            D, rows = rng.choice([64, 128]), _log(rng, 1, 400_000)
        else:
            D = rng.choice([_log(rng, 1, 8192), 8 * _log(rng, 8, 1024)])
            rows = _log(rng, 1, max(1, 16_000_000 // D))
        if D == 3072:
            D += 8
        return dict(op=op, form=form, mode=rng.choice(["fwd", "train"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    rows=rows, D=D)
    if op == "verify":
        V = _log(rng, 100, 160_000)
        return dict(op=op, N=_log(rng, 1, 256), T=rng.randint(1, 8), V=V + (V == 3072), draft=rng.choice(["probs", "probs", "none"]))
    kv = _log(rng, 1, 16384)
    Hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 8])
    L = min(kv, rng.choice([1, rng.randint(2, 8), _log(rng, 8, 2048)]))
    N = _log(rng, 1, 32) if L <= 8 else rng.randint(1, 3)
    return dict(op=op, N=N, L=L, ragged=rng.random() < 0.7, kv=kv + (kv == 3072), Hq=Hkv * group, Hkv=Hkv,
                D=rng.choice([64, 128]), page=rng.choice([8, 16, 24, 32, 64, 128, 256]))


# ---- lengths that a case fixes ----

def _lengths(c):
    """Tokens per sequence (new tokens of attention, tokens of a step): the largest first."""
    n, most = c["N"], c["T"] if c["op"] == "step" else c["L"]
    if most == 1 or not c.get("ragged", True):
        return [most] * n
    r = random.Random(1000 * n + most)
    return [most] + [r.randint(0, most) for _ in range(n - 1)]


def _kv_lens(c, new):
    """Cached length of each sequence, its new tokens included."""
    r = random.Random(77 * c["N"] + c["kv"])
    return [c["kv"] if i == 0 else max(l, r.randint(c["kv"] // 4, c["kv"])) for i, l in enumerate(new)]


# ---- inputs ----

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    return g


def _cu(lengths):
    cu = [0]
    for l in lengths:
        cu.append(cu[-1] + l)
    return torch.tensor(cu, dtype=torch.int32, device=_DEV)


def prepare(case, seed):
    g = _gen(seed)
    normal = lambda *s, std=1.0: torch.randn(*s, generator=g, device=_DEV) * std  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op == "step":
        dt, H, D, N = _DT[case["dtype"]], case["H"], case["D"], case["N"]
        lens = _lengths(case)
        S = sum(lens)
        s["cu"] = _cu(lens)
        for name in ("q", "k", "v", "g"):
            s[name] = normal(S, H, D).to(dt)
        if case["gates"] == "kda":
            s["beta"] = normal(S, H).to(dt)
        else:
            s["erase"], s["write"] = normal(S, H, D).to(dt), normal(S, H, D).to(dt)
        s["A_log"], s["dt_bias"] = normal(H, std=0.3), normal(H, D, std=0.3) - 2.0
        slots = N + 3  # a pool with a few free slots, in the order that admissions left
        s["state"] = normal(slots, H, D, D, std=0.5)
        s["index"] = torch.randperm(slots, generator=g, device=_DEV)[:N].to(torch.int32)
        # with drafts, the tokens verified in the step before come first and are committed
        lens_t = torch.tensor(lens, device=_DEV)
        s["commit"] = None if case["T"] == 1 else \
            (torch.rand(N, generator=g, device=_DEV) * (lens_t + 1)).floor().to(torch.int32)
    elif op == "norm":
        dt, R, D = _DT[case["dtype"]], case["rows"], case["D"]
        form, train = case["form"], case["mode"] == "train"
        s["y"] = normal(R, D, std=0.7).to(dt)
        s["w_post"] = 1.0 + normal(D, std=0.1)
        s["z"] = normal(R, D).to(dt) if form in ("gate", "full") else None
        s["h"] = normal(R, D, std=2.0).to(dt) if form != "gate" else None
        s["w_pre"] = 1.0 + normal(D, std=0.1) if form != "gate" else None
        s["dh_out"] = normal(R, D, std=0.1).to(dt) if train else None
        s["dn"] = normal(R, D, std=0.1).to(dt) if train and form != "gate" else None
        s["scales"] = (1.0, 1.0) if form == "gate" else (0.9, 0.5)
    elif op == "verify":
        N, T, V = case["N"], case["T"], case["V"]
        logits = normal(N, T + 1, V, std=2.0)
        s["target"] = torch.softmax(logits, -1)
        if case["draft"] == "probs":
            logits = logits[:, :T] + 0.5 * normal(N, T, V)
            s["draft"] = torch.softmax(logits, -1)
            noise = torch.empty(N, T, V, device=_DEV).exponential_(generator=g)
            s["tokens"] = (s["draft"] / noise).argmax(-1).to(torch.int32)
        else:  # drafts looked up in the text so far: no probabilities; many of them likely tokens
            s["draft"] = None
            likely = logits[:, :T].argmax(-1)
            s["tokens"] = likely.to(torch.int32)
            s["target"][:, :T] *= 0.3  # the rest of the mass on the likely token
            s["target"][:, :T].scatter_add_(2, likely[..., None], torch.full((N, T, 1), 0.7, device=_DEV))
        s["num"] = torch.randint(0, T + 1, (N,), generator=g, device=_DEV, dtype=torch.int32) if N > 1 else \
            torch.full((1,), T, dtype=torch.int32, device=_DEV)
        s["u"] = torch.rand(N, T, generator=g, device=_DEV)
        s["noise"] = torch.empty(N, V, device=_DEV).exponential_(generator=g).clamp_min_(1e-30)
    else:
        N, D, Hq, Hkv, page = case["N"], case["D"], case["Hq"], case["Hkv"], case["page"]
        new = _lengths(case)
        kv = _kv_lens(case, new)
        S, width = sum(new), -(-max(kv) // page)
        need = [-(-x // page) for x in kv]
        pages = sum(need) + 5
        bf = torch.bfloat16
        s["q"], s["k"], s["v"] = normal(S, Hq, D).to(bf), normal(S, Hkv, D).to(bf), normal(S, Hkv, D).to(bf)
        s["k_pages"] = normal(pages, page, Hkv, D).to(bf)
        s["v_pages"] = normal(pages, page, Hkv, D).to(bf)
        order = torch.randperm(pages, generator=g, device=_DEV).to(torch.int32)
        table = torch.zeros(N, width, dtype=torch.int32, device=_DEV)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["table"] = table
        s["lens"] = torch.tensor(kv, dtype=torch.int32, device=_DEV)
        s["cu"] = _cu(new)
        s["scale"] = D ** -0.5
    return s


# ---- one pass ----

def run(s):
    return {"step": _run_step, "norm": _run_norm, "verify": _run_verify, "attn": _run_attn}[s["case"]["op"]](s)


def _run_step(s):
    c = s["case"]
    if own:
        from recompute_kda_chunkwise_gb300 import decode
        if c["gates"] == "kda":
            o = decode.kda_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["A_log"], s["dt_bias"], s["cu"], s["state"],
                                state_index=s["index"], commit=s["commit"], lower_bound=LOWER, eps=EPS_L2)
        else:
            o = decode.gdn2_step(s["q"], s["k"], s["v"], s["g"], s["erase"], s["write"], s["A_log"], s["dt_bias"], s["cu"],
                                 s["state"], state_index=s["index"], commit=s["commit"], lower_bound=LOWER, eps=EPS_L2)
        return {"o": o, "state": s["state"]}
    T, dt = c["T"], s["q"].dtype
    q, k, v, g = (s[n].float() for n in ("q", "k", "v", "g"))
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + EPS_L2)
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + EPS_L2)
    decay = torch.exp(LOWER * torch.sigmoid(torch.exp(s["A_log"])[:, None] * (g + s["dt_bias"])))
    if c["gates"] == "kda":
        beta = torch.sigmoid(s["beta"].float())[..., None]
        kb, vw = k * beta, v * beta
    else:
        kb, vw = k * torch.sigmoid(s["erase"].float()), v * torch.sigmoid(s["write"].float())
    lens = s["cu"][1:] - s["cu"][:-1]
    state = s["state"][s["index"]]
    kept = state
    o = torch.zeros_like(q)
    for t in range(T):  # the recurrence itself: each token needs the state that the one before left
        live = lens > t
        at = (s["cu"][:-1] + t).clamp_max(q.shape[0] - 1)
        p = state * decay[at][..., None]
        r = vw[at] - (p * kb[at][..., None]).sum(-2)
        state = p + k[at][..., None] * r[..., None, :]
        rows = (state * q[at][..., None]).sum(-2)
        o = torch.where(_rows_of(at, live, q.shape[0]), _spread(rows, at, live, q.shape[0]), o)
        keep = live if s["commit"] is None else (s["commit"] > t) & live
        kept = torch.where(keep[:, None, None, None], state, kept)
    s["state"][s["index"]] = kept
    return {"o": o.to(dt), "state": s["state"]}


def _rows_of(at, live, S):
    m = torch.zeros(S + 1, dtype=torch.bool, device=at.device)
    m[torch.where(live, at, S)] = True
    return m[:S, None, None]


def _spread(rows, at, live, S):
    out = rows.new_zeros((S + 1,) + rows.shape[1:])
    out[torch.where(live, at, S)] = rows
    return out[:S]


def _run_norm(s):
    c = s["case"]
    a, b = s["scales"]
    train, gate = c["mode"] == "train", c["form"] == "gate"
    if own:
        from recompute_kda_chunkwise_gb300 import norm
        h_out, n = norm.block_norm_fwd(s["y"], z=s["z"], h=s["h"], w_post=s["w_post"], w_pre=s["w_pre"],
                                       residual_scale=a, block_scale=b, eps=EPS_RMS)
        out = {"h_out": h_out} if gate else {"h_out": h_out, "n": n}
        if train:
            out.update({k: v for k, v in norm.block_norm_bwd(
                s["y"], z=s["z"], h=s["h"], w_post=s["w_post"], w_pre=s["w_pre"], dh_out=s["dh_out"], dn=s["dn"],
                residual_scale=a, block_scale=b, eps=EPS_RMS).items() if v is not None})
        return out
    dt = s["y"].dtype
    y = s["y"].float()
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS_RMS)
    yn = y * ry
    u = yn * s["w_post"]
    if s["z"] is not None:
        sg = torch.sigmoid(s["z"].float())
        u = u * sg
    h = b * u if gate else a * s["h"].float() + b * u
    out = {"h_out": h.to(dt)}
    if not gate:
        rh = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS_RMS)
        hn = h * rh
        out["n"] = (hn * s["w_pre"]).to(dt)
    if train:
        dh = s["dh_out"].float()
        if not gate:
            dn = s["dn"].float()
            out["dw_pre"] = (dn * hn).sum(0)
            d = dn * s["w_pre"]
            dh = dh + rh * (d - hn * (d * hn).mean(-1, keepdim=True))
            out["dh"] = (a * dh).to(dt)
        du = b * dh
        if s["z"] is not None:
            out["dz"] = (du * yn * s["w_post"] * sg * (1 - sg)).to(dt)
            du = du * sg
        out["dw_post"] = (du * yn).sum(0)
        d = du * s["w_post"]
        out["dy"] = (ry * (d - yn * (d * yn).mean(-1, keepdim=True))).to(dt)
    return out


def _run_verify(s):
    if own:
        from recompute_kda_chunkwise_gb300 import decode
        tokens, accepted = decode.verify_drafts(s["target"], s["draft"], s["tokens"], s["num"], s["u"], s["noise"])
        return {"tokens": tokens, "accepted": accepted}
    p, x, num = s["target"], s["tokens"].long(), s["num"]
    N, T1, V = p.shape
    T = T1 - 1
    steps = torch.arange(T1, device=p.device)
    px = p[:, :T].gather(2, x[..., None])[..., 0]
    qx = s["draft"].gather(2, x[..., None])[..., 0] if s["draft"] is not None else torch.ones_like(px)
    ok = (s["u"] * qx < px) & (steps[:T] < num[:, None])
    accepted = ok.long().cumprod(1).sum(1)
    rows = torch.arange(N, device=p.device)
    last = p[rows, accepted]
    at = accepted.clamp_max(T - 1)
    if s["draft"] is not None:
        rest = (last - s["draft"][rows, at]).clamp_min(0)
    else:
        rest = last.scatter(1, x[rows, at][:, None], 0.0)
    rest = torch.where((accepted < num)[:, None], rest, last)
    rest = torch.where((rest > 0).any(1, keepdim=True), rest, last)
    token = (rest / s["noise"]).argmax(1)
    padded = torch.cat([x, x.new_full((N, 1), -1)], 1)
    tokens = torch.where(steps < accepted[:, None], padded, torch.where(steps == accepted[:, None], token[:, None], -1))
    return {"tokens": tokens.to(torch.int32), "accepted": accepted.to(torch.int32)}


def _run_attn(s):
    c = s["case"]
    if own:
        from recompute_kda_chunkwise_gb300 import decode
        decode.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"])
        o = decode.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"], scale=s["scale"])
        return {"o": o, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    page, group, L = c["page"], c["Hq"] // c["Hkv"], c["L"]
    S, width = s["q"].shape[0], s["table"].shape[1]
    cu, lens, dev = s["cu"].long(), s["lens"].long(), s["q"].device
    new = cu[1:] - cu[:-1]
    tok = torch.arange(S, device=dev)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    pos = lens[seq] - new[seq] + tok - cu[seq]  # position of each new token
    slot = s["table"][seq, pos // page].long()
    s["k_pages"][slot, pos % page] = s["k"]
    s["v_pages"][slot, pos % page] = s["v"]
    o = torch.zeros(S, c["Hq"], c["D"], device=dev)
    ks = torch.arange(width * page, device=dev)
    for n in range(c["N"] if L > 8 else 0):  # long chunks: one sequence at a time, as a padded batch would not fit
        rows = cu[n] + torch.arange(L, device=dev)
        live = rows < cu[n + 1]
        rows = rows.clamp_max(S - 1)
        k = s["k_pages"][s["table"][n].long()].reshape(-1, c["Hkv"], c["D"]).float()
        v = s["v_pages"][s["table"][n].long()].reshape(-1, c["Hkv"], c["D"]).float()
        qn = s["q"][rows].float().reshape(L, c["Hkv"], group, c["D"]).transpose(0, 1).reshape(c["Hkv"], L * group, c["D"])
        sc = torch.matmul(qn, k.permute(1, 2, 0)) * s["scale"]
        sc = sc.masked_fill(ks > pos[rows].repeat_interleave(group)[:, None], -math.inf)
        w = torch.exp(sc - sc.amax(-1, keepdim=True))
        w = w / w.sum(-1, keepdim=True)
        r = torch.matmul(w, v.transpose(0, 1)).reshape(c["Hkv"], L, group, c["D"]).transpose(0, 1).reshape(L, c["Hq"], c["D"])
        o = torch.where(_rows_of(rows, live, S), _spread(r, rows, live, S), o)
    if L <= 8:
        rows = cu[:-1, None] + torch.arange(L, device=dev)
        live = rows < cu[1:, None]
        rows = rows.clamp_max(S - 1)
        k = s["k_pages"][s["table"].long()].reshape(c["N"], -1, c["Hkv"], c["D"]).float()
        v = s["v_pages"][s["table"].long()].reshape(c["N"], -1, c["Hkv"], c["D"]).float()
        qn = s["q"][rows].float().reshape(c["N"], L, c["Hkv"], group, c["D"])
        qn = qn.transpose(1, 2).reshape(c["N"], c["Hkv"], L * group, c["D"])
        sc = torch.matmul(qn, k.permute(0, 2, 3, 1)) * s["scale"]
        last = lens[:, None] - new[:, None] + torch.arange(L, device=dev)
        sc = sc.masked_fill(ks > last.repeat_interleave(group, 1)[:, None, :, None], -math.inf)
        w = torch.exp(sc - sc.amax(-1, keepdim=True))
        w = w / w.sum(-1, keepdim=True)
        r = torch.matmul(w, v.transpose(1, 2)).reshape(c["N"], c["Hkv"], L, group, c["D"]).transpose(1, 2).reshape(-1, c["Hq"], c["D"])
        o = _spread(r, rows.reshape(-1), live.reshape(-1), S)
    return {"o": o.to(s["q"].dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ---- what one pass cannot do without ----

def work(case):
    op = case["op"]
    if op == "step":
        e, H, D, N = (2 if case["dtype"] == "bf16" else 4), case["H"], case["D"], case["N"]
        S = sum(_lengths(case))
        wide = 5 if case["gates"] == "kda" else 7  # q, k, v, g, o (and the two gates)
        states = N * H * D * D * 4 * (2 if case["T"] == 1 else 1 + case["T"] / (case["T"] + 1))  # a commit of 0 writes none
        return {"bytes": states + S * H * D * e * wide + (S * H * e if case["gates"] == "kda" else 0), "flops": S * H * D * D * 7}
    if op == "norm":
        e, n = (2 if case["dtype"] == "bf16" else 4), case["rows"] * case["D"]
        reads, writes = {"gate": (2, 1), "residual": (2, 2), "full": (3, 2)}[case["form"]]
        r, w = {"gate": (3, 2), "residual": (4, 2), "full": (5, 3)}[case["form"]]
        if case["mode"] == "train":
            reads, writes = reads + r, writes + w
        return {"bytes": e * n * (reads + writes), "flops": n * (12 if case["mode"] == "fwd" else 45)}
    if op == "verify":
        N, T, V = case["N"], case["T"], case["V"]
        # the one row of target probabilities and noise, and the draft's row where a draft was refused
        mean = sum(1 - ACCEPT ** n for n in range(T + 1)) / (T + 1) if N > 1 else 1 - ACCEPT ** T
        return {"bytes": N * V * 4 * (2 + (mean if case["draft"] == "probs" else 0)), "flops": N * V * 3}
    new = _lengths(case)
    kv = _kv_lens(case, new)
    pairs = sum(l * (t - l) + l * (l + 1) // 2 for l, t in zip(new, kv))
    S, D = sum(new), case["D"]
    seen = sum(t for l, t in zip(new, kv) if l)
    return {"bytes": 2 * D * (2 * S * case["Hq"] + 4 * S * case["Hkv"] + 2 * seen * case["Hkv"]), "flops": 4 * pairs * case["Hq"] * D}


# ---- each operator's definition in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return None  # whole numbers only
    if op == "step":
        return _exact_step(case, s)
    if op == "norm":
        return _exact_norm(case, s)
    return _exact_attn(case, s)


def _exact_step(case, s):
    f = {n: s[n].double() for n in ("q", "k", "v", "g", "beta", "erase", "write", "A_log", "dt_bias") if s.get(n) is not None}
    pool = s["state"].double()
    o = torch.zeros_like(f["q"])
    cu, index = s["cu"].tolist(), s["index"].tolist()
    commit = [None] * case["N"] if s["commit"] is None else s["commit"].tolist()
    for n in range(case["N"]):
        S = pool[index[n]].clone()  # [H, D(k), D(v)]
        count = cu[n + 1] - cu[n]
        upto = count if commit[n] is None else commit[n]
        for t in range(cu[n], cu[n + 1]):
            kh = f["k"][t] / (f["k"][t].pow(2).sum(-1, keepdim=True) + EPS_L2).sqrt()
            qh = f["q"][t] / (f["q"][t].pow(2).sum(-1, keepdim=True) + EPS_L2).sqrt()
            rate = f["A_log"].exp()[:, None] * (f["g"][t] + f["dt_bias"])
            S = S * torch.exp(LOWER / (1 + torch.exp(-rate)))[:, :, None]
            if case["gates"] == "kda":
                beta = 1 / (1 + torch.exp(-f["beta"][t]))
                erase, write = beta[:, None], beta[:, None]
            else:
                erase, write = 1 / (1 + torch.exp(-f["erase"][t])), 1 / (1 + torch.exp(-f["write"][t]))
            new = write * f["v"][t] - torch.einsum("hkv,hk->hv", S, erase * kh)
            S = S + torch.einsum("hk,hv->hkv", kh, new)
            o[t] = torch.einsum("hkv,hk->hv", S, qh)
            if t - cu[n] + 1 == upto:
                pool[index[n]] = S
    return {"o": o, "state": pool}


def _exact_norm(case, s):
    a, b = s["scales"]
    leaf = {n: s[n].double().requires_grad_(case["mode"] == "train") for n in ("y", "z", "h", "w_post", "w_pre") if s[n] is not None}
    D = case["D"]
    y = leaf["y"]
    u = leaf["w_post"] * y / ((y ** 2).sum(-1, keepdim=True) / D + EPS_RMS) ** 0.5
    if "z" in leaf:
        u = u / (1 + torch.exp(-leaf["z"]))
    h = b * u + (a * leaf["h"] if "h" in leaf else 0)
    n = leaf["w_pre"] * h / ((h ** 2).sum(-1, keepdim=True) / D + EPS_RMS) ** 0.5 if "w_pre" in leaf else None
    out = {"h_out": h.detach()}
    if n is not None:
        out["n"] = n.detach()
    if case["mode"] == "train":
        loss = (h * s["dh_out"].double()).sum() + (0 if n is None else (n * s["dn"].double()).sum())
        grads = torch.autograd.grad(loss, list(leaf.values()))
        out.update({"d" + k: v for k, v in zip(leaf, grads)})
    return out


def _exact_attn(case, s):
    page, group = case["page"], case["Hq"] // case["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    for n in range(case["N"]):
        l, t = cu[n + 1] - cu[n], lens[n]
        if not l:
            continue
        ids = s["table"][n, : -(-t // page)].long()
        k = s["k_pages"][ids].flatten(0, 1)[:t].clone()
        v = s["v_pages"][ids].flatten(0, 1)[:t].clone()
        k[t - l:], v[t - l:] = s["k"][cu[n]:cu[n + 1]], s["v"][cu[n]:cu[n + 1]]
        for i in range(0, l, 512):
            j = min(l, i + 512)
            for hk in range(case["Hkv"]):
                q = s["q"][cu[n] + i:cu[n] + j, hk * group:(hk + 1) * group].double()
                sc = torch.einsum("lgd,td->lgt", q, k[:, hk].double()) * s["scale"]
                hidden = torch.arange(t, device=o.device)[None] > (t - l + torch.arange(i, j, device=o.device))[:, None]
                sc[hidden[:, None].expand_as(sc)] = -math.inf
                o[cu[n] + i:cu[n] + j, hk * group:(hk + 1) * group] = torch.einsum("lgt,td->lgd", torch.softmax(sc, -1), v[:, hk].double())
    k_pages = s["k_pages"].clone()
    v_pages = s["v_pages"].clone()
    for n in range(case["N"]):
        l, t = cu[n + 1] - cu[n], lens[n]
        for i in range(l):
            p = t - l + i
            k_pages[s["table"][n, p // page], p % page] = s["k"][cu[n] + i]
            v_pages[s["table"][n, p // page], p % page] = s["v"][cu[n] + i]
    return {"o": o, "k_pages": k_pages.double(), "v_pages": v_pages.double()}
