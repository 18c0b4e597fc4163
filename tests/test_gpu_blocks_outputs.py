"""Outputs of the operators of include/kda_blocks.h that the caller gives, and what becomes of outputs and the
status where lengths are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)


def cache(Hk=2, D=64):
    pages = [rand(i, 4, 16, Hk, D) for i in (11, 12)]
    return (*pages, torch.arange(4, dtype=I32, device="cuda")[None], torch.tensor([40], dtype=I32, device="cuda"),
            torch.tensor([0, 10], dtype=I32, device="cuda"))


def writes():
    """(name, a call that writes `x` in place, x)."""
    from recompute_kda_chunkwise_gb300 import attention as A, decode, rotary as T
    rope, cu = T.Rotary(64), torch.tensor([0, 10], dtype=I32, device="cuda")
    q, k, v = rand(1, 10, 4, 64), rand(2, 10, 2, 64), rand(3, 10, 2, 64)
    kp, vp, *rest = cache()
    other = rand(4, 10, 4, 64)
    yield "rotary q", lambda x: T.rotary_fwd(rope, x, k, cu_seqlens=cu, out=(x, None)), q
    yield "rotary k", lambda x: T.rotary_fwd(rope, q, x, cu_seqlens=cu, out=(None, x)), k
    yield "rotary_bwd", lambda x: T.rotary_bwd(rope, x, cu_seqlens=cu, out=(x, None)), q
    yield "append q", lambda x: decode.paged_append_rotary(rope, x, k, v, kp, vp, *rest, out=x), q
    yield "append keys", lambda x: decode.paged_append_rotary(rope, q, k, v, x, vp, *rest), kp
    yield "append values", lambda x: decode.paged_append_rotary(rope, q, k, v, kp, x, *rest), vp
    yield "attention", lambda x: A.attention_fwd(q, k, v, cu, out=x), other


@pytest.mark.parametrize("n", range(7))
def test_a_graph_that_saved_an_output_notices(n):
    name, call, x = list(writes())[n]
    w = torch.ones_like(x, requires_grad=True)
    y = (w * x).sum()
    call(x)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():
        call(x.clone())


@pytest.mark.parametrize("D", [64, 128])
def test_attention_may_write_over_its_queries(D):
    from recompute_kda_chunkwise_gb300 import attention as A
    lens = [300, 1, 700, 129] * 3
    q, k, v = rand(1, sum(lens), 16, D), rand(2, sum(lens), 4, D), rand(3, sum(lens), 4, D)
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).cuda()
    o, lse = A.attention_fwd(q, k, v, cu)
    x = q.clone()
    y, lse2 = A.attention_fwd(x, k, v, cu, out=x)
    assert y.data_ptr() == x.data_ptr() and torch.equal(x, o) and torch.equal(lse, lse2)
