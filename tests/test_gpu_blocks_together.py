"""The operators of attention blocks together, as a program uses them: a stack with rotary positions
is trained and served, and both see the same model."""
import pytest
import torch

import _blocks_ref as R

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def stack(**kw):
    from recompute_kda_chunkwise_gb300 import hybrid
    from recompute_kda_chunkwise_gb300.rotary import Rotary
    kw = {**dict(kinds=("delta", "attn"), heads=4, kv_heads=2, seed=3, rope=Rotary(96, scaling="by_parts", factor=4.0, trained=64)), **kw}
    return hybrid.Stack(**kw)


def test_serving_computes_what_training_does():
    """Prefill in parts and single tokens over the paged cache against the packed forward."""
    from recompute_kda_chunkwise_gb300 import hybrid
    model = stack()
    tokens = torch.arange(150, device="cuda") * 11 % 512
    with torch.no_grad():
        want = torch.softmax(model(tokens, torch.tensor([0, 150], dtype=I32, device="cuda")).float(), -1)
    server = hybrid.Server(model, 1, 160)
    got = [server.run(tokens[:100], [100]), server.run(tokens[100:149], [49]), server.run(tokens[149:], [1], [1])]
    # bf16 activations of calls of different lengths round apart
    assert (torch.cat(got) - want).abs().max() <= 0.05 * want.max()


def test_training_runs_and_its_gradients_are_finite_and_reach_every_weight():
    from recompute_kda_chunkwise_gb300 import hybrid
    model = stack(kinds=("attn", "delta", "attn"))
    tokens = torch.randint(0, 512, (333,), device="cuda")
    cu = torch.tensor([0, 100, 101, 333], dtype=I32, device="cuda")
    loss = torch.nn.functional.cross_entropy(model(tokens, cu).float(), tokens.roll(-1))
    for name, g in zip(dict(model.named_parameters()), torch.autograd.grad(loss, list(model.parameters()))):
        assert g.isfinite().all() and g.abs().max() > 0, name
    assert hybrid.train_step(model, tokens, cu, tokens.roll(-1), max_norm=0.5).isfinite()


def test_clipping_in_a_training_step():
    from recompute_kda_chunkwise_gb300 import hybrid
    tokens = torch.randint(0, 512, (200,), device="cuda")
    cu = torch.tensor([0, 200], dtype=I32, device="cuda")
    one, other = stack(), stack()
    # a bound that nothing reaches: the same step as without one
    hybrid.train_step(one, tokens, cu, tokens.roll(-1), lr=0.1)
    hybrid.train_step(other, tokens, cu, tokens.roll(-1), lr=0.1, max_norm=1e9)
    assert all(torch.equal(a, b) for a, b in zip(one.parameters(), other.parameters()))
    # one that all of them do: a step no longer than lr * max_norm and the rounding of the weights
    before = [p.detach().clone() for p in one.parameters()]
    hybrid.train_step(one, tokens, cu, tokens.roll(-1), lr=1.0, max_norm=1e-3)
    step = R.norm([(a.double() - b.double()) for a, b in zip(one.parameters(), before)])
    rounding = R.norm([b.double() * (2.0 ** -8 if b.dtype == BF else 2.0 ** -24) for b in before])
    assert step <= 1e-3 * (1 + 2.0 ** -8) + rounding


def test_an_attention_block_against_float64():
    """rotary, attention and their gradients in a chain."""
    from recompute_kda_chunkwise_gb300.attention import attention
    from recompute_kda_chunkwise_gb300.rotary import Rotary, rotary
    g = torch.Generator(device="cuda").manual_seed(9)
    lens, Hq, Hk, D = [70, 1, 200], 4, 2, 64
    S = sum(lens)
    fused = torch.randn(S, (Hq + 2 * Hk) * D, generator=g, device="cuda").to(BF).requires_grad_()
    d_o = torch.randn(S, Hq, D, generator=g, device="cuda").to(BF)
    cu = torch.tensor([0, 70, 71, 271], dtype=I32, device="cuda")
    rope = Rotary(64, interleaved=True)
    q, k, v = (t.view(S, -1, D) for t in fused.split([Hq * D, Hk * D, Hk * D], 1))
    o = attention(*rotary(rope, q, k, cu_seqlens=cu), v, cu)
    (got,) = torch.autograd.grad(o, fused, d_o)
    # the same chain in float64, with its own gradient
    x = fused.detach().cpu().double().requires_grad_()
    a, b, c = (t.view(S, -1, D) for t in x.split([Hq * D, Hk * D, Hk * D], 1))
    pos = torch.cat([torch.arange(n) for n in lens]).double()[:, None, None] * torch.tensor(rope.frequencies, dtype=torch.float64)

    def turned(t):
        z = torch.view_as_complex(t.reshape(S, -1, D // 2, 2)) * torch.polar(torch.ones_like(pos), pos)
        return torch.view_as_real(z).reshape(S, -1, D)

    outs, lo = [], 0
    for n in lens:
        r = slice(lo, lo + n)
        s = torch.einsum("ihd,jhd->hij", turned(a)[r], turned(b)[r].repeat_interleave(2, 1)) * D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -torch.inf)
        outs.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), c[r].repeat_interleave(2, 1)))
        lo += n
    ref = torch.cat(outs)
    (want,) = torch.autograd.grad(ref, x, d_o.cpu().double())
    # six roundings to bf16 on the way (q', k', P, o, dS, dq'), each 2^-8 at most, and the outputs' own
    for y, z in ((o, ref), (got, want)):
        assert (R.d(y) - z.detach()).pow(2).mean().sqrt() <= 7 * 2.0 ** -8 * z.detach().pow(2).mean().sqrt()


def test_captured_block_and_eager_ones_side_by_side():
    """Explicit forward and backward calls in a graph, eager calls on another stream meanwhile."""
    from recompute_kda_chunkwise_gb300 import attention as A, grads as G
    from recompute_kda_chunkwise_gb300.rotary import Rotary, rotary_bwd, rotary_fwd
    g = torch.Generator(device="cuda").manual_seed(2)
    S, Hq, Hk, D = 300, 4, 2, 128
    q, k, v, d_o = (torch.randn(S, h, D, generator=g, device="cuda").to(BF) for h in (Hq, Hk, Hk, Hq))
    cu = torch.tensor([0, 130, 300], dtype=I32, device="cuda")
    rope = Rotary(D)

    def block(q, k, v):
        x, y = rotary_fwd(rope, q, k, cu_seqlens=cu)
        o, lse = A.attention_fwd(x, y, v, cu)
        dx, dy, dv = A.attention_bwd(x, y, v, o, lse, d_o, cu)
        dq, dk = rotary_bwd(rope, dx, dy, cu_seqlens=cu)
        out = [dq, dk, dv]
        return G.clip_grads(out, 1.0), o, *out

    want = [t.clone() for t in block(q, k, v)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ins = [torch.zeros_like(t) for t in (q, k, v)]
    with torch.cuda.stream(s):
        block(*ins)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = block(*ins)
        for a, b in zip(ins, (q, k, v)):
            a.copy_(b)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            graph.replay()
        eager = block(q, k, v)
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, eager):
            assert torch.equal(a, b) and torch.equal(a, c)
