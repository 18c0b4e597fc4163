"""Gradients that arrive as slices of a larger tensor: contiguous, but not where vectors begin."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def rand(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def cases():
    from recompute_kda_chunkwise_gb300 import kda as K
    from recompute_kda_chunkwise_gb300.attention import attention
    from recompute_kda_chunkwise_gb300.norm import block_norm
    from recompute_kda_chunkwise_gb300.rotary import Rotary, rotary
    S, H, D = 40, 2, 128
    cu = torch.tensor([0, 15, S], dtype=I32, device="cuda")
    q, k, v, g = (rand(i, S, H, D) for i in range(4))
    beta, A_log, bias = rand(7, S, H), torch.zeros(H, device="cuda"), torch.zeros(H, D, device="cuda")
    yield "attention", lambda *t: (attention(*t, cu),), (q, k, v)
    yield "rotary", lambda *t: rotary(Rotary(64), *t, cu_seqlens=cu), (q, k)
    yield "rotary, no keys", lambda *t: (rotary(Rotary(64), *t, cu_seqlens=cu),), (q,)
    yield "block_norm", lambda y, h, w: block_norm(y, h=h, w_pre=w), (q, k, torch.ones(D, device="cuda"))
    yield "kda", lambda *t: (K.kda(*t, A_log, bias, cu),), (q, k, v, g, beta)
    yield "gdn2", lambda *t: (K.gdn2(*t, A_log, bias, cu),), (q, k, v, g, rand(8, S, H, D), rand(9, S, H, D))


@pytest.mark.parametrize("n", range(6))
def test_slices_of_a_larger_gradient(n):
    name, op, ins = list(cases())[n]
    ins = [t.requires_grad_() for t in ins]
    outs = op(*ins)
    want = torch.autograd.grad(outs, ins, [rand(20 + i, *o.shape, dtype=o.dtype) for i, o in enumerate(outs)], retain_graph=True)
    lead = torch.zeros(3, device="cuda", dtype=outs[0].dtype)
    joined = torch.cat([t for o in outs for t in (lead, o.flatten())])
    d = torch.cat([t for i, o in enumerate(outs) for t in (lead, rand(20 + i, *o.shape, dtype=o.dtype).flatten())])
    got = torch.autograd.grad(joined, ins, d)
    assert all(torch.equal(a, b) for a, b in zip(got, want)), name
