"""Rotary positions and the paged append that rotates, against float64."""
import pytest
import torch

import _blocks_ref as R

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def rand(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(dim, layout, scaling):
    from recompute_kda_chunkwise_gb300.rotary import Rotary
    how = {None: {}, "linear": dict(factor=3.0), "ntk": dict(factor=4.0), "by_parts": dict(factor=8.0, trained=512)}[scaling]
    return Rotary(dim, interleaved=layout == "pairs", scaling=scaling, **how)


@pytest.mark.parametrize("scaling", [None, "by_parts"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("S,Hq,Hk,D,dim", [(1, 1, 0, 64, 64), (1, 16, 16, 128, 128), (7, 3, 1, 64, 42), (333, 4, 2, 128, 64),
                                           (1200, 2, 1, 8, 2), (700, 1, 1, 64, 64), (65, 12, 12, 96, 80), (9, 5, 2, 512, 512)])
def test_forward_and_gradient(S, Hq, Hk, D, dim, dtype, layout, scaling):
    from recompute_kda_chunkwise_gb300 import rotary
    g = gen(S + dim)
    rope = make(dim, layout, scaling)
    q, k = rand(g, S, Hq, D, dtype=dtype), rand(g, S, Hk, D, dtype=dtype) if Hk else None
    pos = torch.randint(0, 2_000_000, (S,), generator=g, device="cuda", dtype=I32)
    pos[0] = -3
    for fn, sign in ((rotary.rotary_fwd, 1), (rotary.rotary_bwd, -1)):
        for x, y in zip((q, k), fn(rope, q, k, positions=pos)):
            assert (y is None) == (x is None)
            if x is not None:
                ref, bar = R.turn(x, pos.cpu(), rope.frequencies, rope.magnitude, rope.interleaved, sign)
                R.check(y, ref, bar, "rotated")
                assert torch.equal(y[..., dim:], x[..., dim:])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("dim", [2, 4, 6, 8, 12, 20, 24, 26, 40, 44, 46, 60, 62, 64, 66, 68, 70, 72])
def test_every_width_of_a_half(dim, dtype):
    """Halves of 1 to 36 channels: single elements, words, half and whole vectors, and what passes behind them;
    both outside place and over the inputs, and beside the paged append."""
    from recompute_kda_chunkwise_gb300 import decode, rotary
    g = gen(dim)
    S, Hq, Hk, D, page = 77, 6, 2, 128 if dtype == BF else 72, 16
    q, k, v = (rand(g, S, h, D, dtype=dtype) for h in (Hq, Hk, Hk))
    rope = make(dim, "half", "ntk" if dim > 2 else None)
    cu = torch.tensor([0, S], dtype=I32, device="cuda")
    yq, yk = rotary.rotary_fwd(rope, q, k, cu_seqlens=cu)
    for x, y in ((q, yq), (k, yk)):
        ref, bar = R.turn(x, list(range(S)), rope.frequencies, 1.0, False)
        R.check(y, ref, bar, "rotated")
        assert torch.equal(y[..., dim:], x[..., dim:])
    zq, zk = q.clone(), k.clone()
    rotary.rotary_fwd(rope, zq, zk, cu_seqlens=cu, out=(zq, zk))
    assert torch.equal(zq, yq) and torch.equal(zk, yk)
    if dtype == BF:
        kp, vp = (rand(g, 5, page, Hk, D) for _ in range(2))
        table, lens = torch.arange(5, dtype=I32, device="cuda")[None], torch.tensor([S], dtype=I32, device="cuda")
        tail = kp.view(-1, Hk, D)[S:].clone()
        aq = decode.paged_append_rotary(rope, q, k, v, kp, vp, table, lens, cu)
        assert torch.equal(aq, yq) and torch.equal(kp.view(-1, Hk, D)[:S], yk) and torch.equal(vp.view(-1, Hk, D)[:S], v)
        assert torch.equal(kp.view(-1, Hk, D)[S:], tail)


@pytest.mark.parametrize("layout,dim", [("half", 128), ("pairs", 128), ("half", 42)])
def test_packed_slices_in_place_and_autograd(layout, dim):
    """Slices of a fused projection, positions from cu_seqlens, outputs over their inputs."""
    from recompute_kda_chunkwise_gb300 import rotary
    g = gen(3)
    lens = [0, 5, 1, 0, 130, 33]
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).cuda()
    pos = [i for n in lens for i in range(n)]
    S, Hq, Hk, D = sum(lens), 6, 2, 128
    fused = rand(g, S, (Hq + 2 * Hk) * D)
    before = fused.clone()
    q, k = fused[:, :Hq * D].view(S, Hq, D), fused[:, Hq * D:(Hq + Hk) * D].view(S, Hk, D)
    rope = make(dim, layout, "linear")
    yq, yk = rotary.rotary_fwd(rope, q, k, cu_seqlens=cu)
    for x, y in ((q, yq), (k, yk)):
        ref, bar = R.turn(x, pos, rope.frequencies, 1.0, rope.interleaved)
        R.check(y, ref, bar, "packed")
    assert torch.equal(fused, before)
    cq, ck = q.contiguous(), k.contiguous()
    zq, zk = rotary.rotary_fwd(rope, cq, ck, cu_seqlens=cu, out=(cq, ck))
    assert zq.data_ptr() == cq.data_ptr() and torch.equal(cq, yq) and torch.equal(zk, yk)
    # autograd: the opposite rotation, also of gradients that are not contiguous
    lq, lk = q.detach().clone().requires_grad_(), k.detach().clone().requires_grad_()
    aq, ak = rotary.rotary(rope, lq, lk, cu_seqlens=cu)
    w = rand(g, D, Hq, S).permute(2, 1, 0)
    dq, dk = torch.autograd.grad((aq * w).sum() + ak.sum(), (lq, lk))
    eq, ek = rotary.rotary_bwd(rope, w.contiguous(), torch.ones_like(k).contiguous(), cu_seqlens=cu)
    assert torch.equal(aq, yq) and torch.equal(dq, eq) and torch.equal(dk, ek)
    one = rotary.rotary(rope, lq, cu_seqlens=cu)
    assert torch.equal(one, yq)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        torch.autograd.grad(one.square().sum(), lq, create_graph=True)[0].sum().backward()


def test_angles_of_far_positions():
    """fp32 frequencies or products would be off by whole turns there."""
    from recompute_kda_chunkwise_gb300.rotary import Rotary, rotary_fwd
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 0, 1], dtype=I32, device="cuda")
    rope = Rotary(64)
    x = torch.ones(5, 1, 64, device="cuda")
    y, _ = rotary_fwd(rope, x, positions=pos)
    # the product of a double and an integer of 31 bits, and its cosine, are off by 2^-22 of a radian there
    ref, bar = R.turn(x, pos.cpu(), rope.frequencies)
    R.check(y, ref, bar + 2.0 ** -20, "far positions")


def test_custom_frequencies_magnitude_and_values_that_are_not_finite():
    from recompute_kda_chunkwise_gb300.rotary import Rotary, rotary_fwd
    rope = Rotary(8, frequencies=[0.0, 7.25, -0.5, 1e-9], magnitude=0.5)
    x = rand(gen(1), 40, 2, 16)
    x[3, 0, 1], x[4, 1, 12] = float("nan"), float("inf")
    y, _ = rotary_fwd(rope, x, positions=torch.arange(40, dtype=I32, device="cuda"))
    ref, bar = R.turn(x, torch.arange(40), rope.frequencies, 0.5)
    R.check(y, ref, bar.nan_to_num(), "custom")


def test_tokens_of_no_sequence_keep_their_rows():
    from recompute_kda_chunkwise_gb300 import kda as K, rotary
    rope = make(64, "half", None)
    x = rand(gen(2), 10, 2, 64)
    out, status = torch.full_like(x, 9.0), torch.zeros(1, dtype=I32, device="cuda")
    cu = torch.tensor([0, 4, 8], dtype=I32, device="cuda")  # two padding rows at the end
    rotary.rotary_fwd(rope, x, cu_seqlens=cu, out=(out, None), status=status)
    assert K.query_device_status(status) == 6
    ref, bar = R.turn(x[:8], [0, 1, 2, 3] * 2, rope.frequencies)
    R.check(out[:8], ref, bar, "held")
    assert (out[8:] == 9).all()


def test_many_sequences():
    from recompute_kda_chunkwise_gb300 import rotary
    lens = [(i * 7) % 5 for i in range(3000)]
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).cuda()
    x = rand(gen(5), sum(lens), 1, 64)
    rope = make(64, "pairs", None)
    y, _ = rotary.rotary_fwd(rope, x, cu_seqlens=cu)
    ref, bar = R.turn(x, [i for n in lens for i in range(n)], rope.frequencies, 1.0, True)
    R.check(y, ref, bar, "many")


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("layout,dim", [("half", 128), ("pairs", 64), ("half", 42), ("pairs", 30)])
@pytest.mark.parametrize("new,kv,page", [([1], [1], 8), ([1, 1, 1], [17, 300, 64], 64), ([70, 0, 5, 1], [200, 3, 5, 129], 24)])
def test_paged_append(new, kv, page, layout, dim, with_q):
    from recompute_kda_chunkwise_gb300 import decode
    g = gen(page + dim)
    N, S, Hq, Hk, D = len(new), sum(new), 6, 2, 128
    fused = rand(g, S, (Hq + 2 * Hk) * D)
    q, k, v = (t.view(S, -1, D) for t in fused.split([Hq * D, Hk * D, Hk * D], 1))
    need = [-(-t // page) for t in kv]
    pages = sum(need) + 3
    kp, vp = rand(g, pages, page, Hk, D), rand(g, pages, page, Hk, D)
    table = torch.zeros(N, max(need), dtype=I32)
    order = torch.randperm(pages).to(I32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    lens, cu = torch.tensor(kv, dtype=I32, device="cuda"), torch.tensor([0] + new).cumsum(0).to(I32).cuda()
    rope = make(dim, layout, "ntk")
    pos = [t - n + i for n, t in zip(new, kv) for i in range(n)]
    ek, bk = R.turn(k, pos, rope.frequencies, 1.0, rope.interleaved)
    ref_k, ref_v, bar = R.d(kp), R.d(vp), torch.zeros(kp.shape, dtype=torch.float64)
    for t, (p, n) in enumerate(zip(pos, [i for i, n in enumerate(new) for _ in range(n)])):
        where = int(table[n, p // page]), p % page
        ref_k[where], ref_v[where], bar[where] = ek[t], R.d(v[t]), bk[t]
    o = decode.paged_append_rotary(rope, q if with_q else None, k, v, kp, vp, table.cuda(), lens, cu)
    R.check(kp, ref_k, bar, "keys")
    assert torch.equal(R.d(vp), ref_v)
    assert (o is not None) == with_q
    if with_q:
        ref, b = R.turn(q, pos, rope.frequencies, 1.0, rope.interleaved)
        R.check(o, ref, b, "queries")


def test_append_without_rotation_is_paged_append_and_bad_pages_are_skipped():
    from recompute_kda_chunkwise_gb300 import decode, kda as K
    from recompute_kda_chunkwise_gb300.rotary import Rotary
    g = gen(8)
    k, v = rand(g, 6, 2, 64), rand(g, 6, 2, 64)
    caches = [rand(gen(9), 5, 8, 2, 64) for _ in range(4)]
    table = torch.tensor([[1, 7, 0], [-1, 2, 4]], dtype=I32, device="cuda")  # page 7 is outside, -1 too
    lens = torch.tensor([10, 30], dtype=I32, device="cuda")  # sequence 1 reaches past its table
    cu = torch.tensor([0, 3, 6], dtype=I32, device="cuda")
    words = [torch.zeros(1, dtype=I32, device="cuda") for _ in range(2)]
    decode.paged_append(k, v, caches[0], caches[1], table, lens, cu, status=words[0])
    rope = Rotary(64, frequencies=[0.0] * 32)
    q = rand(g, 6, 4, 64)
    out = torch.full_like(q, 3.0)
    decode.paged_append_rotary(rope, q, k, v, caches[2], caches[3], table, lens, cu, out=out, status=words[1])
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    assert [K.query_device_status(w) for w in words] == [6, 6]
    skipped = torch.tensor([False, True, True, True, True, True])
    assert (out[skipped] == 3).all() and torch.equal(out[~skipped], q[~skipped])


def test_captured_on_another_stream():
    from recompute_kda_chunkwise_gb300 import rotary
    rope = make(128, "half", None)
    q, k = rand(gen(1), 50, 4, 128), rand(gen(2), 50, 2, 128)
    pos = torch.arange(50, dtype=I32, device="cuda")
    want = rotary.rotary_fwd(rope, q, k, positions=pos + 7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rotary.rotary_fwd(rope, q, k, positions=pos)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = rotary.rotary_fwd(rope, q, k, positions=pos)
        pos += 7
        graph.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    from recompute_kda_chunkwise_gb300 import rotary
    from recompute_kda_chunkwise_gb300.kda import KdaError
    rope = make(64, "half", None)
    x, cu = rand(gen(1), 10, 2, 64), torch.tensor([0, 10], dtype=I32, device="cuda")
    pos = torch.arange(10, dtype=I32, device="cuda")
    with pytest.raises(ValueError, match="one of positions"):
        rotary.rotary_fwd(rope, x)
    with pytest.raises(ValueError, match="one of positions"):
        rotary.rotary_fwd(rope, x, positions=pos, cu_seqlens=cu)
    with pytest.raises(ValueError, match="positions"):
        rotary.rotary_fwd(rope, x, positions=pos.long())
    with pytest.raises(ValueError, match="contiguous within a token"):
        rotary.rotary_fwd(rope, x.transpose(0, 1).contiguous().transpose(0, 1), positions=pos)
    with pytest.raises(ValueError, match="k must be"):
        rotary.rotary_fwd(rope, x, x[:5], positions=pos)
    with pytest.raises(ValueError, match="q_out"):
        rotary.rotary_fwd(rope, x, positions=pos, out=(x[:, :1], None))
    with pytest.raises(ValueError, match="k_out"):
        rotary.rotary_fwd(rope, x, positions=pos, out=(None, x))
    with pytest.raises(KdaError, match="rotary_dim"):
        rotary.rotary_fwd(make(66, "half", None), x, positions=pos)
    with pytest.raises(KdaError, match="aligned"):
        rotary.rotary_fwd(rope, torch.zeros(10 * 128 + 4, dtype=BF, device="cuda")[4:].view(10, 2, 64), positions=pos)
    with pytest.raises(KdaError, match="stride"):
        rotary.rotary_fwd(rope, torch.zeros(10, 132, dtype=BF, device="cuda")[:, :128].view(10, 2, 64), positions=pos)
    none = rotary.rotary_fwd(rope, x[:0], x[:0], cu_seqlens=cu * 0)
    assert none[0].shape == (0, 2, 64) and none[1].shape == (0, 2, 64)


@pytest.mark.parametrize("dtype,D,dim", [(BF, 512, 510), (BF, 512, 300), (BF, 512, 302), (BF, 264, 262), (BF, 512, 508),
                                         (torch.float32, 512, 510), (torch.float32, 512, 300), (torch.float32, 512, 506)])
@pytest.mark.parametrize("S,Hq,Hk", [(1, 1, 0), (5, 3, 2), (130, 9, 1)])
def test_heads_of_more_items_than_threads(S, Hq, Hk, dtype, D, dim):
    """Halves that are cut into single elements or words: a CTA goes over its tile more than once."""
    from recompute_kda_chunkwise_gb300 import rotary
    g = gen(S + dim)
    rope = make(dim, "half", "linear")
    q, k = rand(g, S, Hq, D, dtype=dtype), rand(g, S, Hk, D, dtype=dtype) if Hk else None
    cu = torch.tensor([0, S // 2, S], dtype=I32, device="cuda")
    pos = list(range(S // 2)) + list(range(S - S // 2))
    for fn, sign in ((rotary.rotary_fwd, 1), (rotary.rotary_bwd, -1)):
        for x, y in zip((q, k), fn(rope, q, k, cu_seqlens=cu)):
            if x is not None:
                ref, bar = R.turn(x, pos, rope.frequencies, 1.0, False, sign)
                R.check(y, ref, bar, "rotated")
                assert torch.equal(y[..., dim:], x[..., dim:])
    z = q.clone()
    rotary.rotary_fwd(rope, z, cu_seqlens=cu, out=(z, None))
    assert torch.equal(z, rotary.rotary_fwd(rope, q, cu_seqlens=cu)[0])
