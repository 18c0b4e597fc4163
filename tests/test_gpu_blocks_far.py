"""Tensors of more than 2^31 elements: what lies behind that is computed as it is by itself."""
import pytest
import torch

import _blocks_ref as R

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, dtype=BF, device="cuda").normal_(generator=g)


def test_packed_attention_and_rotary():
    from recompute_kda_chunkwise_gb300 import attention as A, kda as K, rotary as T
    Hq, Hk, D = 64, 4, 128
    lens = [331] * 798 + [257, 1, 300]
    S, tail = sum(lens), 558  # the last three sequences
    assert (S - tail) * Hq * D > 2 ** 31
    q, k, v, d_o = (rand(i, S, h, D) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).cuda()
    status = torch.zeros(1, dtype=I32, device="cuda")
    rope = T.Rotary(D)
    near = [t[-tail:].clone() for t in (q, k, v, d_o)]
    near_cu = torch.tensor([0, 257, 258, 558], dtype=I32, device="cuda")
    x, y = T.rotary_fwd(rope, q, k, cu_seqlens=cu, out=(q, k), status=status)
    a, b = T.rotary_fwd(rope, *near[:2], cu_seqlens=near_cu)
    assert torch.equal(x[-tail:], a) and torch.equal(y[-tail:], b)
    o, lse = A.attention_fwd(x, y, v, cu, status=status)
    dq, dk, dv = A.attention_bwd(x, y, v, o, lse, d_o, cu, status=status)
    assert K.query_device_status(status) == 0
    want, want_lse = A.attention_fwd(a, b, near[2], near_cu)
    assert torch.equal(o[-tail:], want) and torch.equal(lse[:, -tail:], want_lse)
    ref, bar = R.attention(a, b, near[2], near_cu.tolist(), D ** -0.5, near[3])
    R.check_all(dict(dq=dq[-tail:], dk=dk[-tail:], dv=dv[-tail:]), ref, bar)


def test_clipping():
    from recompute_kda_chunkwise_gb300 import grads as G
    n = 2 ** 31 + 12_345
    t = torch.ones(n, dtype=BF, device="cuda")
    t[-1] = 3.0
    ref = (n + 8) ** 0.5
    assert abs(G.clip_grads([t], ref / 2).item() - ref) <= ref * 2.0 ** -20
    assert (t[-20:-1] == 0.5).all() and t[-1] == 1.5 and t[2 ** 31] == 0.5 and t[0] == 0.5
