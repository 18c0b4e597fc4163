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


def test_outputs_over_other_tensors_are_refused():
    from recompute_kda_chunkwise_gb300 import attention as A, decode, rotary as T
    rope, cu, S = T.Rotary(64), torch.tensor([0, 10], dtype=I32, device="cuda"), 10
    pos = torch.arange(S, dtype=I32, device="cuda")
    q, k, v, d_o = (rand(i, S, 4, 64) for i in range(4))
    kp, vp, *rest = cache(4)
    flat = rand(5, 4 * S * 256)
    at = lambda i: flat[i:i + S * 256].view(S, 4, 64)  # noqa: E731
    fused = rand(6, S, 3 * 256)
    a, b, c = (fused[:, i * 256:(i + 1) * 256].view(S, 4, 64) for i in range(3))
    first = fused[:1].view(3, 4, 64)[0:1]
    keep = [t.clone() for t in (q, k, v, kp, vp, flat, fused, pos)]

    def ints(n):  # int32 tensors inside an output
        return flat.view(I32)[64:64 + n]

    for call, what in (
            (lambda: T.rotary_fwd(rope, q, k, positions=pos, out=(k, None)), "q_out overlaps k"),
            (lambda: T.rotary_fwd(rope, q, k, positions=pos, out=(None, q)), "k_out overlaps q"),
            (lambda: T.rotary_fwd(rope, q, q, positions=pos, out=(q, None)), "q_out overlaps k"),
            (lambda: T.rotary_fwd(rope, q, k, positions=pos, out=(at(0), at(0))), "k_out overlaps q_out"),
            (lambda: T.rotary_fwd(rope, q, k, positions=pos, out=(at(0), at(S * 256 - 8))), "k_out overlaps q_out"),
            (lambda: T.rotary_fwd(rope, at(0), positions=pos, out=(at(8), None)), "q_out overlaps q"),
            (lambda: T.rotary_bwd(rope, at(8), positions=pos, out=(at(0), None)), "q_out overlaps q"),
            (lambda: T.rotary_fwd(rope, q, positions=ints(S), out=(at(0), None)), "q_out overlaps positions"),
            (lambda: T.rotary_fwd(rope, a, positions=pos, out=(fused.view(-1)[:S * 256].view(S, 4, 64), None)), "q_out overlaps q"),
            (lambda: decode.paged_append_rotary(rope, q, k, v, kp, vp, *rest, out=k), "q_out overlaps k"),
            (lambda: decode.paged_append_rotary(rope, q, k, v, kp, vp, *rest, out=v), "q_out overlaps v"),
            (lambda: decode.paged_append_rotary(rope, q, k, v, kp, kp, *rest), "v_pages overlaps k_pages"),
            (lambda: decode.paged_append_rotary(rope, q, kp.view(-1, 4, 64)[:S], v, kp, vp, *rest), "k_pages overlaps k"),
            (lambda: decode.paged_append_rotary(rope, q, k, v, kp, vp, *rest, out=vp.view(-1, 4, 64)[:S]), "v_pages overlaps q_out"),
            (lambda: A.attention_fwd(q, k, v, cu, out=v), "out overlaps v"),
            (lambda: A.attention_fwd(q, k, v, cu, out=k), "out overlaps k"),
            (lambda: A.attention_fwd(a, b, c, cu, out=fused.view(-1)[:S * 256].view(S, 4, 64)), "out overlaps q"),
            (lambda: A.attention_fwd(at(0), k, v, cu, out=at(8)), "out overlaps q"),
            (lambda: A.attention_fwd(at(0), k, v, cu, workspace=flat.view(torch.uint8)), "workspace overlaps q"),
            (lambda: A.attention_fwd(q, k, v, cu, out=at(0), workspace=flat.view(torch.uint8)), "workspace overlaps out"),
            (lambda: A.attention_bwd(q, k, v, at(0), torch.zeros(4, S, device="cuda"), d_o, cu,
                                     workspace=flat.view(torch.uint8)), "workspace overlaps o")):
        with pytest.raises(ValueError, match=what):
            call()
    assert all(torch.equal(x, y) for x, y in zip(keep, (q, k, v, kp, vp, flat, fused, pos)))
    # what lies beside one another, or in the gaps of a strided tensor, does not overlap
    T.rotary_fwd(rope, q, k, positions=pos, out=(at(0), at(S * 256)))
    T.rotary_fwd(rope, first, positions=pos[:1], out=(fused[:1, 256:512].view(1, 4, 64), None))
    A.attention_fwd(q, k, v, cu, out=at(2 * S * 256), workspace=flat[:S * 256].view(torch.uint8))
    # nor does what lies behind the part of a long workspace that the call needs
    A.attention_fwd(q, k, v, cu, out=at(2 * S * 256), workspace=flat.view(torch.uint8))


def spoil(*like):
    """What the allocator hands out next holds sevens."""
    t = [torch.full_like(x, 7.0) for x in like]
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (3, 3)])  # gradients of keys with and without parts to add up
@pytest.mark.parametrize("ends", [[0, 90], [0, 40, 90], [0, 101], [0, 60, 40, 100], [1, 100]])
def test_refused_lengths_reach_the_caller_of_attention(ends, Hq, Hk, D):
    """Padding rows behind the last sequence, among others."""
    from recompute_kda_chunkwise_gb300 import attention as A, kda as K
    S = 100
    q, k, v, d_o = rand(1, S, Hq, D), rand(2, S, Hk, D), rand(3, S, Hk, D), rand(4, S, Hq, D)
    cu = torch.tensor(ends, dtype=I32, device="cuda")
    leaves = [t.requires_grad_() for t in (q, k, v)]
    status = torch.zeros(1, dtype=I32, device="cuda")
    spoil(q, k, v)
    o = A.attention(q, k, v, cu, status=status)
    assert K.query_device_status(status) == 6 and o.isnan().all()
    status.zero_()
    spoil(q, k, v)
    grads = torch.autograd.grad(o, leaves, d_o)
    assert K.query_device_status(status) == 6 and all(g.isnan().all() for g in grads)
    # without a status; a given output is left as it was
    assert A.attention(q, k, v, cu).isnan().all()
    out = torch.full_like(q, 5.0)
    ws = torch.empty(A.attention_workspace_bytes(q, k, cu), dtype=torch.uint8, device="cuda")
    _, lse = A.attention_fwd(q.detach(), k.detach(), v.detach(), cu, out=out, workspace=ws)
    assert (out == 5).all() and lse.isnan().all() and K.query_device_status(ws) == 6
    # the caller's word takes it instead of the workspace's, and the first error stays
    A.attention_fwd(q.detach(), k.detach(), v.detach(), cu, workspace=ws, status=status)
    assert K.query_device_status(ws) == 0 and K.query_device_status(status) == 6
    good = torch.tensor([0, 40, S], dtype=I32, device="cuda")
    o = A.attention(q, k, v, good, status=status)
    assert o.isfinite().all() and K.query_device_status(status) == 6
    status.zero_()
    torch.autograd.grad(A.attention(q, k, v, good, status=status), leaves, d_o)
    assert K.query_device_status(status) == 0


def test_refused_lengths_of_many_rows():
    from recompute_kda_chunkwise_gb300 import attention as A
    S, Hq, Hk, D = 20_000, 16, 4, 64
    q, k, v, d_o = rand(1, S, Hq, D), rand(2, S, Hk, D), rand(3, S, Hk, D), rand(4, S, Hq, D)
    for ends in ([0, S - 1], [0, 7000, S - 1]):
        cu = torch.tensor(ends, dtype=I32, device="cuda")
        o, lse = A.attention_fwd(q, k, v, cu)
        assert o.isnan().all() and lse.isnan().all()
        assert all(g.isnan().all() for g in A.attention_bwd(q, k, v, d_o, lse, d_o, cu))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("S,D,dim", [(10, 64, 64), (10, 64, 42), (5000, 128, 96), (40, 512, 510)])
def test_tokens_of_no_sequence_are_zeros_after_rotary(S, D, dim, interleaved, dtype):
    """Padding rows in front, between and behind; their gradients are zeros too."""
    from recompute_kda_chunkwise_gb300 import kda as K, rotary as T
    rope = T.Rotary(dim, interleaved=interleaved)
    q, k = rand(1, S, 3, D).to(dtype).requires_grad_(), rand(2, S, 2, D).to(dtype).requires_grad_()
    cu = torch.tensor([2, 4, 4, S - 3], dtype=I32, device="cuda")
    pad = torch.ones(S, dtype=torch.bool, device="cuda")
    pad[2:S - 3] = False
    pos = torch.cat([torch.arange(-2, 2), torch.arange(S - 4)]).to(I32).cuda()
    status = torch.zeros(1, dtype=I32, device="cuda")
    spoil(q, k, q, k)
    x, y = T.rotary(rope, q, k, cu_seqlens=cu, status=status)
    assert K.query_device_status(status) == 6
    want = T.rotary_fwd(rope, q, k, positions=pos)
    for got, ref in zip((x, y), want):
        assert (got[pad] == 0).all() and torch.equal(got[~pad], ref[~pad])
    w, z = torch.randn_like(q), torch.randn_like(k)
    want = T.rotary_bwd(rope, w, z, positions=pos)
    status.zero_()
    spoil(q, k, q, k)
    for got, ref in zip(torch.autograd.grad((x, y), (q, k), (w, z)), want):
        assert (got[pad] == 0).all() and torch.equal(got[~pad], ref[~pad])
    assert K.query_device_status(status) == 6
    # one output given, the other made by the call
    out = torch.full_like(k, 9.0)
    spoil(q)
    x, _ = T.rotary_fwd(rope, q.detach(), k.detach(), cu_seqlens=cu, out=(None, out))
    assert (x[pad] == 0).all() and (out[pad] == 9).all() and torch.equal(out[~pad], y[~pad])


def test_skipped_queries_of_an_append_are_zeros():
    from recompute_kda_chunkwise_gb300 import decode, kda as K, rotary as T
    kp, vp, table, lens, _ = cache()
    q, k, v = rand(1, 10, 6, 64), rand(2, 10, 2, 64), rand(3, 10, 2, 64)
    table[0, 2] = 9  # positions 32 to 47 have no page
    cu = torch.tensor([0, 10], dtype=I32, device="cuda")
    keep, status = [t.clone() for t in (kp, vp)], torch.zeros(1, dtype=I32, device="cuda")
    spoil(q)
    x = decode.paged_append_rotary(T.Rotary(64), q, k, v, kp, vp, table, lens, cu, status=status)  # positions 30 to 39
    assert K.query_device_status(status) == 6 and (x[2:] == 0).all() and (x[:2] != 0).any()
    assert torch.equal(kp[2:], keep[0][2:]) and torch.equal(vp[2:], keep[1][2:])
    assert torch.equal(vp[1, 14:], v[:2])
