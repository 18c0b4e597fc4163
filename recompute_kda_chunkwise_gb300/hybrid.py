"""A small language-model stack of delta-rule and attention blocks with random
weights: the package's operators together, as a program uses them.

    python -m recompute_kda_chunkwise_gb300.hybrid

trains a stack of delta-rule blocks for a few steps (``kda`` and ``block_norm``
with gradients), then serves a stack with attention blocks between them:
prefill (``kda_fwd`` to a pool of states, ``paged_append`` and
``paged_attention``), and decoding with drafted tokens (``kda_step``, the paged
cache, ``verify_drafts``). Projections are plain matrix products.
"""
from __future__ import annotations

import torch

from . import decode
from . import kda as K
from .norm import block_norm, block_norm_fwd

EPS = 1e-5


class Block(torch.nn.Module):
    """Projections of one block: a delta-rule layer (per head: query, key,
    value, raw decay, raw output gate; raw beta) or grouped-query attention."""

    def __init__(self, dim, heads, head_dim, kind, kv_heads=None, gen=None, device="cuda"):
        super().__init__()
        self.kind, self.heads, self.head_dim, self.kv_heads = kind, heads, head_dim, kv_heads or heads
        wide = heads * head_dim

        def weight(n_in, n_out):
            w = torch.randn(n_in, n_out, generator=gen, device=device) * n_in ** -0.5
            return torch.nn.Parameter(w.to(torch.bfloat16))

        if kind == "delta":
            self.proj = weight(dim, 5 * wide)
            self.beta = weight(dim, heads)
            self.A_log = torch.nn.Parameter(torch.zeros(heads, device=device))
            self.dt_bias = torch.nn.Parameter(torch.full((heads, head_dim), -2.0, device=device))
            self.out_norm = torch.nn.Parameter(torch.ones(head_dim, device=device))
        else:
            self.proj = weight(dim, wide + 2 * self.kv_heads * head_dim)
        self.out = weight(wide, dim)
        self.post = torch.nn.Parameter(torch.ones(dim, device=device))  # norm after the block
        self.pre = torch.nn.Parameter(torch.ones(dim, device=device))   # norm before the next one

    def delta_inputs(self, n):
        S, H, D = n.shape[0], self.heads, self.head_dim
        q, k, v, g, z = (t.reshape(S, H, D).contiguous() for t in (n @ self.proj).split(H * D, 1))
        return q, k, v, g, z, n @ self.beta


class Stack(torch.nn.Module):
    """Blocks joined by block_norm: h += post-norm of a block's output, and the
    next block reads the pre-norm of h."""

    def __init__(self, vocab=512, dim=256, heads=2, head_dim=128, kinds=("delta", "delta"), kv_heads=1, seed=0,
                 device="cuda"):
        super().__init__()
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        self.blocks = torch.nn.ModuleList(Block(dim, heads, head_dim, k, kv_heads, gen, device) for k in kinds)
        self.embed = torch.nn.Parameter((torch.randn(vocab, dim, generator=gen, device=device) * dim ** -0.5).to(torch.bfloat16))
        self.first = torch.nn.Parameter(torch.ones(dim, device=device))

    def start(self, tokens):
        h = self.embed[tokens]
        _, n = block_norm(torch.zeros_like(h), h=h, w_pre=self.first)
        return h, n

    def forward(self, tokens, cu_seqlens):
        """Logits [S, vocab] of packed sequences; every block a delta rule."""
        h, n = self.start(tokens)
        for b in self.blocks:
            q, k, v, g, z, beta = b.delta_inputs(n)
            o = K.kda(q, k, v, g, beta, b.A_log, b.dt_bias, cu_seqlens)
            o = block_norm(o, z=z, w_post=b.out_norm, eps=EPS)
            h, n = block_norm(o.flatten(1) @ b.out, h=h, w_post=b.post, w_pre=b.pre, block_scale=0.5, eps=EPS)
        return n @ self.embed.T


def train_step(model, tokens, cu_seqlens, targets, lr=1e-3):
    """One step of gradient descent; returns the loss."""
    loss = torch.nn.functional.cross_entropy(model(tokens, cu_seqlens).float(), targets)
    grads = torch.autograd.grad(loss, list(model.parameters()))
    with torch.no_grad():
        for p, g in zip(model.parameters(), grads):
            p -= lr * g.to(p.dtype)
    return loss.detach()


class Server:
    """Decoding state of a stack: a pool of delta-rule states and paged caches.

    Between two calls a sequence has ``committed`` tokens in its states and
    cache, and pending ones, verified but not committed: the last step's accepted drafts and
    the token it drew. A step feeds pending tokens and drafts together and
    commits the pending ones but the last; refused drafts leave no trace.

    ``capacity`` is the number of tokens that a sequence's pages hold: max_len
    in whole pages (None without attention blocks: states have no length)."""

    def __init__(self, model, sequences, max_len, page=16):
        self.m, self.n = model, sequences
        dev = model.embed.device
        b0 = model.blocks[0]
        H, D = b0.heads, b0.head_dim
        width = -(-max_len // page)
        self.states = [torch.zeros(sequences, H, D, D, device=dev) if b.kind == "delta" else None for b in model.blocks]
        self.caches = [tuple(torch.zeros(sequences * width, page, b.kv_heads, D, dtype=torch.bfloat16, device=dev)
                             for _ in range(2)) if b.kind == "attn" else None for b in model.blocks]
        self.table = torch.arange(sequences * width, dtype=torch.int32, device=dev).view(sequences, width)
        self.committed = [0] * sequences
        self.capacity = width * page if any(b.kind == "attn" for b in model.blocks) else None

    @torch.no_grad()
    def run(self, tokens, lengths, commit=None):
        """Probabilities [S, vocab] after each of the packed tokens. commit
        None: a prefill (chunked delta rule, every token committed). Raises
        ValueError, with nothing changed, for a sequence that its pages do not hold."""
        for i, (c, l) in enumerate(zip(self.committed, lengths)):
            if self.capacity is not None and c + l > self.capacity:
                raise ValueError(f"sequence {i} would have {c + l} tokens: its pages hold {self.capacity}")
        m, dev = self.m, self.table.device
        cu = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)
        lens = torch.tensor([c + l for c, l in zip(self.committed, lengths)], dtype=torch.int32, device=dev)
        kept = lengths if commit is None else commit
        commit_t = None if commit is None else torch.tensor(commit, dtype=torch.int32, device=dev)
        h, n = m.start(tokens)
        for i, b in enumerate(m.blocks):
            if b.kind == "delta":
                q, k, v, g, z, beta = b.delta_inputs(n)
                if commit is None:
                    o, _, _ = K.kda_fwd(q, k, v, g, beta, b.A_log, b.dt_bias, cu, save_ctx=False,
                                        h0=self.states[i].clone(), final_state=self.states[i])
                else:
                    o = decode.kda_step(q, k, v, g, beta, b.A_log, b.dt_bias, cu, self.states[i], commit=commit_t)
                o, _ = block_norm_fwd(o, z=z, w_post=b.out_norm, eps=EPS)
            else:
                S, D = n.shape[0], b.head_dim
                q, k, v = (t.reshape(S, -1, D).contiguous()
                           for t in (n @ b.proj).split([b.heads * D, b.kv_heads * D, b.kv_heads * D], 1))
                kp, vp = self.caches[i]
                decode.paged_append(k, v, kp, vp, self.table, lens, cu)
                o = decode.paged_attention(q, kp, vp, self.table, lens, cu)
            h, n = block_norm_fwd(o.flatten(1) @ b.out, h=h, w_post=b.post, w_pre=b.pre, block_scale=0.5, eps=EPS)
        self.committed = [c + k for c, k in zip(self.committed, kept)]
        return torch.softmax((n @ m.embed.T).float(), -1)


def lookup_drafts(tokens, most):
    """Drafts without a model: what followed the last earlier occurrence of the last token."""
    for i in range(len(tokens) - 2, -1, -1):
        if tokens[i] == tokens[-1]:
            return tokens[i + 1: i + 1 + most]
    return []


def generate(server, prompts, steps, drafts=3, seed=0, greedy=False):
    """Continues each prompt (lists of tokens) by at least ``steps`` tokens, up
    to ``drafts`` drafted at a time. Returns the sequences and the number of
    model calls after the prefill. A sequence that is done goes on as long as
    others are not and its pages hold more."""
    # places that are left of each sequence's pages
    room = [None if server.capacity is None else server.capacity - c for c in server.committed]
    for i, (p, r) in enumerate(zip(prompts, room)):  # the last token that is drawn is not fed
        if r is not None and len(p) + steps - 1 > r:
            raise ValueError(f"prompt {i} has {len(p)} tokens: {steps} more tokens need {len(p) + steps - 1} places and "
                             f"its pages hold {r}")
    dev, vocab = server.table.device, server.m.embed.shape[0]
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    out = [list(p) for p in prompts]
    N = len(prompts)

    def draw(target, drafted, counts):
        if greedy:  # all of the mass on the likeliest token
            target = torch.nn.functional.one_hot(target.argmax(-1), vocab).float()
        T = drafted.shape[1]
        tokens, accepted = decode.verify_drafts(
            target, None, drafted, counts, torch.rand(N, T, generator=gen, device=dev),
            torch.empty(N, vocab, device=dev).exponential_(generator=gen).clamp_min_(1e-20))
        return tokens.tolist(), accepted.tolist()

    lengths = [len(p) for p in prompts]
    probs = server.run(torch.tensor([t for p in prompts for t in p], device=dev), lengths)
    last = torch.tensor(lengths).cumsum(0) - 1
    first, _ = draw(probs[last.to(dev)][:, None].contiguous(), torch.zeros(N, 0, dtype=torch.int32, device=dev), None)
    pending = [[f[0]] for f in first]
    for i in range(N):
        out[i] += pending[i]
    calls = 0
    while min(len(o) - l for o, l in zip(out, lengths)) < steps:
        # len(out) counts the pending tokens: what is left of the pages is for drafts, and a sequence whose pending
        # tokens do not fit (it has more than it was asked for) rests
        resting = [r is not None and len(o) > r for o, r in zip(out, room)]
        drafted = [[] if rests else lookup_drafts(o, drafts if r is None else min(drafts, r - len(o)))
                   for o, r, rests in zip(out, room, resting)]
        feed = [[] if r else p + d for p, d, r in zip(pending, drafted, resting)]
        sizes = [len(f) for f in feed]
        # everything before the last pending token was verified in an earlier call
        probs = server.run(torch.tensor([t for f in feed for t in f], device=dev), sizes,
                           [0 if r else len(p) - 1 for p, r in zip(pending, resting)])
        T = max(len(d) for d in drafted)
        target = torch.zeros(N, T + 1, vocab, device=dev)
        drafted_t = torch.zeros(N, T, dtype=torch.int32)
        at = 0
        for i in range(N):
            if resting[i]:
                continue
            first_row = at + len(pending[i]) - 1
            target[i, : len(drafted[i]) + 1] = probs[first_row: at + sizes[i]]
            drafted_t[i, : len(drafted[i])] = torch.tensor(drafted[i], dtype=torch.int32)
            at += sizes[i]
        counts = torch.tensor([len(d) for d in drafted], dtype=torch.int32, device=dev)
        tokens, accepted = draw(target, drafted_t.to(dev), counts)
        for i in range(N):
            if resting[i]:
                continue
            fresh = tokens[i][: accepted[i] + 1]
            out[i] += fresh
            pending[i] = pending[i][-1:] + fresh
        calls += 1
    return out, calls


def main():
    torch.manual_seed(0)
    model = Stack()
    tokens = torch.randint(0, 512, (600,), device="cuda")
    cu = torch.tensor([0, 250, 600], dtype=torch.int32, device="cuda")
    for i in range(3):
        print(f"training step {i}: loss {train_step(model, tokens, cu, tokens.roll(-1)).item():.4f}")
    model = Stack(kinds=("delta", "delta", "attn", "delta"), heads=4, kv_heads=2)
    prompts = [[5, 6, 7, 8] * 12, [1, 2, 3] * 7, list(range(40))]
    out, calls = generate(Server(model, 3, 256), prompts, steps=24, greedy=True)
    new = [o[len(p):] for o, p in zip(out, prompts)]
    print(f"{sum(map(len, new))} tokens in {calls} calls: {[t[:8] for t in new]}")


if __name__ == "__main__":
    main()
