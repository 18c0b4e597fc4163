"""Causal attention of packed sequences and its gradient, against float64."""
import pytest
import torch

import _blocks_ref as R

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def inputs(lens, Hq, Hk, D, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h: (torch.randn(sum(lens), h, D, generator=g, device="cuda") * std).to(BF)  # noqa: E731
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(I32).cuda()
    return r(Hq), r(Hk), r(Hk), r(Hq), cu


def run(q, k, v, d_o, cu, scale=None):
    from recompute_kda_chunkwise_gb300 import attention as A, kda as K
    fw = torch.empty(A.attention_workspace_bytes(q, k, cu), dtype=torch.uint8, device="cuda")
    bw = torch.empty(A.attention_workspace_bytes(q, k, cu, backward=True), dtype=torch.uint8, device="cuda")
    o, lse = A.attention_fwd(q, k, v, cu, scale=scale, workspace=fw)
    dq, dk, dv = A.attention_bwd(q, k, v, o, lse, d_o, cu, scale=scale, workspace=bw)
    torch.cuda.synchronize()
    assert K.query_device_status(fw) == 0 and K.query_device_status(bw) == 0
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 1), (6, 2)])
@pytest.mark.parametrize("lens", [(1,), (2,), (77,), (128,), (129,), (256,), (257,), (384,), (640,), (1, 1, 1), (300, 1, 0, 128, 513),
                                  (0, 0, 65), (255, 127, 130)])
def test_forward_and_gradients(lens, Hq, Hk, D):
    q, k, v, d_o, cu = inputs(lens, Hq, Hk, D, seed=sum(lens))
    R.check_all(run(q, k, v, d_o, cu), *R.attention(q, k, v, cu.tolist(), D ** -0.5, d_o))


@pytest.mark.parametrize("lens,Hq,Hk,D", [((1500,), 3, 3, 128), ((1100, 900), 8, 1, 64), ((2100,), 2, 1, 128)])
def test_longer_sequences(lens, Hq, Hk, D):
    """Many tiles an item and, with these heads, several items a CTA or none."""
    q, k, v, d_o, cu = inputs(lens, Hq, Hk, D, seed=7)
    R.check_all(run(q, k, v, d_o, cu), *R.attention(q, k, v, cu.tolist(), D ** -0.5, d_o))


def test_more_items_than_ctas():
    q, k, v, d_o, cu = inputs((150, 400, 129, 300), 48, 16, 64, seed=11)
    R.check_all(run(q, k, v, d_o, cu), *R.attention(q, k, v, cu.tolist(), 0.125, d_o))


@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (0.02, 3.0), (0.5, 2.0)])
def test_sharp_and_flat_probabilities(scale, std):
    """Maxima that move by more than 2^8 between tiles, and rows that one key takes all of."""
    q, k, v, d_o, cu = inputs((530,), 2, 1, 128, seed=5, std=std)
    k[::97] *= 4
    R.check_all(run(q, k, v, d_o, cu, scale), *R.attention(q, k, v, cu.tolist(), scale, d_o))


@pytest.mark.parametrize("lens,Hq,Hk", [((1023,), 2, 1), ((640, 100, 897, 0, 128), 4, 2), ((260, 384, 129, 500), 48, 16)])
@pytest.mark.parametrize("D", [128, 64])
def test_maxima_that_rise_with_every_tile(lens, Hq, Hk, D):
    """Scores that rise by some 17 octaves a tile, or fall, as the query's sign is: outputs are rescaled at every
    tile, while other tiles' products are under way; items of one stream and of two, in turn on one CTA."""
    q, k, v, d_o, cu = inputs(lens, Hq, Hk, D, seed=D, std=0.5)
    u = torch.ones(D, device="cuda") * D ** -0.5
    sign = torch.where(torch.rand(q.shape[:2], generator=torch.Generator().manual_seed(3)) < 0.7, 3.0, -3.0).cuda()
    at = torch.cat([torch.arange(n) for n in lens]).cuda().float()
    q = (q.float() + sign[..., None] * u).to(BF)
    k = (k.float() + 0.25 * at[:, None, None] * u).to(BF)
    R.check_all(run(q, k, v, d_o, cu, 0.125), *R.attention(q, k, v, cu.tolist(), 0.125, d_o))


def test_slices_of_a_projection_and_autograd():
    from recompute_kda_chunkwise_gb300.attention import attention
    lens, Hq, Hk, D = (200, 131), 4, 2, 128
    q, k, v, d_o, cu = inputs(lens, Hq, Hk, D, seed=3)
    want = run(q, k, v, d_o, cu)
    fused = torch.cat([t.flatten(1) for t in (q, k, v)], 1).requires_grad_()
    parts = [t.view(sum(lens), -1, D) for t in fused.split([Hq * D, Hk * D, Hk * D], 1)]
    o = attention(*parts, cu)
    assert torch.equal(o, want["o"])
    # a gradient that is not contiguous
    (g,) = torch.autograd.grad(o, fused, d_o.transpose(0, 1).contiguous().transpose(0, 1))
    assert torch.equal(g, torch.cat([want[n].flatten(1) for n in ("dq", "dk", "dv")], 1))
    x = q.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        torch.autograd.grad(attention(x, k, v, cu).square().sum(), x, create_graph=True)[0].sum().backward()


@pytest.mark.parametrize("D", [64, 128])
def test_other_sequences_do_not_matter(D):
    """NaN and infinities in the neighbours of a tile's rows; the same bits as without them."""
    lens = (130, 100, 300)
    q, k, v, d_o, cu = inputs(lens, 4, 2, D, seed=13)
    clean = run(q, k, v, d_o, cu)
    lo, hi = 130, 230
    for t, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan")), (d_o, float("-inf"))):
        t[:lo] = bad
        t[hi:] = bad
    dirty = run(q, k, v, d_o, cu)
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(clean[n][lo:hi], dirty[n][lo:hi]), n
    assert torch.equal(clean["lse"][:, lo:hi], dirty["lse"][:, lo:hi])


def test_one_sequence_does_not_read_what_lies_behind_it():
    """The tensors are slices of larger ones full of NaN."""
    S, H, D = 150, 2, 128
    q, k, v, d_o, cu = inputs((S,), H, H, D, seed=17)
    want = run(q, k, v, d_o, cu)
    wide = torch.full((S + 300, 4, H, D), float("nan"), dtype=BF, device="cuda")
    for i, t in enumerate((q, k, v)):
        wide[:S, i] = t
    got = run(*(wide[:S, i] for i in range(3)), d_o, cu)
    for n in want:
        assert torch.equal(want[n], got[n]), n


def test_the_same_bits_every_time_and_whatever_is_beside():
    q, k, v, d_o, cu = inputs((700, 64, 333), 8, 2, 128, seed=19)
    a, b = run(q, k, v, d_o, cu), run(q, k, v, d_o, cu)
    alone = run(*(t[700:764].contiguous() for t in (q, k, v, d_o)), torch.tensor([0, 64], dtype=I32, device="cuda"))
    for n in a:
        assert torch.equal(a[n], b[n]), n
        # o, lse, dq: a sequence's own; dk, dv are summed by parts of the head group, and their number goes by the call's size
        if n in ("o", "dq"):
            assert torch.equal(a[n][700:764], alone[n]), n


def test_lengths_that_do_not_fit_leave_outputs_alone():
    from recompute_kda_chunkwise_gb300 import attention as A, kda as K
    q, k, v, d_o, cu = inputs((40, 60), 2, 1, 64, seed=1)
    o, lse = A.attention_fwd(q, k, v, cu)
    for bad in ([0, 100], [0, 60, 40, 100], [0, 40, 101], [1, 40, 100], [0, -1, 100], [0, 40, 90], [0, 99], [2, 100]):
        cu = torch.tensor(bad, dtype=I32, device="cuda")
        if bad == [0, 100]:
            continue
        for n in range(2):
            ws = torch.empty(A.attention_workspace_bytes(q, k, cu, backward=n == 1), dtype=torch.uint8, device="cuda")
            if n == 0:
                out = torch.full_like(q, 5.0)
                A.attention_fwd(q, k, v, cu, out=out, workspace=ws)
                assert (out == 5).all()
            else:
                A.attention_bwd(q, k, v, o, lse, d_o, cu, workspace=ws)
            assert K.query_device_status(ws) == 6, bad


def test_a_single_key_has_no_gradient_through_its_probability():
    """Sequences of one token: P is 1 and dS zero, whatever the scores are; dq and dk are zero exactly."""
    for D, H in ((64, 3), (128, 2)):
        q, k, v, d_o, cu = inputs((1, 1, 1, 1, 1), 2 * H, H, D, seed=D, std=3.0)
        got = run(q, k, v, d_o, cu)
        assert torch.equal(got["o"], v.repeat_interleave(2, 1))
        assert (got["dq"] == 0).all() and (got["dk"] == 0).all()


def test_no_tokens():
    q, k, v, d_o, cu = inputs((0, 0), 2, 1, 64)
    got = run(q, k, v, d_o, cu)
    assert got["o"].shape == (0, 2, 64) and got["dk"].shape == (0, 1, 64)


def test_many_sequences():
    lens = [(i * 13) % 9 for i in range(1500)]
    q, k, v, d_o, cu = inputs(lens, 2, 1, 64, seed=23)
    R.check_all(run(q, k, v, d_o, cu), *R.attention(q, k, v, cu.tolist(), 0.125, d_o))


def test_scores_that_are_not_finite():
    """A query whose scores are all -inf has no softmax: NaN, in its own rows."""
    q, k, v, d_o, cu = inputs((90,), 1, 1, 64, seed=29)
    q[5] = 0
    q[5, 0, 0], k[:, 0, 0] = float("-inf"), k[:, 0, 0].abs() + 1
    from recompute_kda_chunkwise_gb300.attention import attention_fwd
    o, lse = attention_fwd(q, k, v, cu)
    assert o[5].isnan().all() and lse[0, 5] == float("-inf")
    rest = torch.arange(90) != 5
    ref, bar = R.attention(q, k, v, [0, 90], 0.125)
    R.check(o[rest.cuda()], ref["o"][rest], bar["o"][rest], "the other rows")


def test_captured_with_other_work_on_another_stream():
    from recompute_kda_chunkwise_gb300 import attention as A
    q, k, v, d_o, cu = inputs((300, 50), 4, 2, 128, seed=31)
    want = run(q, k, v, d_o, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = torch.zeros_like(q)
    with torch.cuda.stream(s):
        o, lse = A.attention_fwd(x, k, v, cu)
        A.attention_bwd(x, k, v, o, lse, d_o, cu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            o, lse = A.attention_fwd(x, k, v, cu)
            g = A.attention_bwd(x, k, v, o, lse, d_o, cu)
        x.copy_(q)
        graph.replay()
        graph.replay()
    s.synchronize()
    for a, n in zip((o, lse, *g), ("o", "lse", "dq", "dk", "dv")):
        assert torch.equal(a, want[n]), n


def test_more_tiles_than_buckets_in_the_list():
    """A sequence of more than 1024 tiles beside a short one: tiles are sorted by buckets of lengths. A few
    rows of the long one against float64; the short one as alone."""
    from recompute_kda_chunkwise_gb300 import attention as A
    lens, D = (140_000, 70), 64
    q, k, v, d_o, cu = inputs(lens, 1, 1, D, seed=37)
    got = run(q, k, v, d_o, cu)
    ref, bar = R.attention(*(t[140_000:] for t in (q, k, v)), [0, 70], 0.125, d_o[140_000:])
    R.check_all({n: t[140_000:] if n != "lse" else t[:, 140_000:] for n, t in got.items()}, ref, bar)
    x, y, z, w = (t[:140_000, 0].double() for t in (q, k, v, d_o))
    for r in (0, 1, 127, 128, 65_535, 131_071, 139_999):
        s = (y[:r + 1] @ x[r]) * 0.125
        p = torch.softmax(s, 0)
        o, dp = p @ z[:r + 1], z[:r + 1] @ w[r]
        delta = w[r] @ o
        ds = p * (dp - delta)
        fine = R.BF + R.FINE
        R.check(got["o"][r, 0], R.d(o), R.d(fine * (p @ z[:r + 1].abs())), f"o {r}")
        e = fine * ds.abs() + p * (fine * (w[r].abs() * o.abs()).sum() + R.FINE * (z[:r + 1].abs() @ w[r].abs()))
        R.check(got["dq"][r, 0], R.d(0.125 * (ds @ y[:r + 1])), R.d(0.125 * (e @ y[:r + 1].abs())), f"dq {r}")
    # the last keys are seen by the last queries only
    lo = 140_000 - 40
    p = torch.exp(x[lo:] @ y[lo:].T * 0.125 - got["lse"][0, lo:140_000].double()[:, None]).tril()
    R.check(got["dv"][lo:140_000, 0], R.d(p.T @ w[lo:]), R.d((R.BF + R.FINE) * (p.T @ w[lo:].abs())), "dv")


def test_refusals():
    from recompute_kda_chunkwise_gb300 import attention as A
    from recompute_kda_chunkwise_gb300.kda import KdaError
    q, k, v, d_o, cu = inputs((40,), 4, 2, 64)
    with pytest.raises(ValueError, match="bfloat16"):
        A.attention_fwd(q.float(), k, v, cu)
    with pytest.raises(ValueError, match="v must be"):
        A.attention_fwd(q, k, v[:, :1], cu)
    with pytest.raises(ValueError, match="k must be"):
        A.attention_fwd(q, k[:30], v, cu)
    with pytest.raises(ValueError, match="cu_seqlens"):
        A.attention_fwd(q, k, v, cu.long())
    with pytest.raises(ValueError, match="workspace"):
        A.attention_bwd(q, k, v, q, torch.zeros(4, 40, device="cuda"), d_o, cu, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="lse"):
        A.attention_bwd(q, k, v, q, torch.zeros(40, 4, device="cuda"), d_o, cu)
    with pytest.raises(ValueError, match="d_o"):
        A.attention_bwd(q, k, v, q, torch.zeros(4, 40, device="cuda"), d_o.transpose(0, 1).contiguous().transpose(0, 1), cu)
    for bad, what in ((dict(scale=0.0), "scale"), (dict(scale=-0.1), "scale")):
        with pytest.raises(KdaError, match=what):
            A.attention_fwd(q, k, v, cu, **bad)
    with pytest.raises(KdaError, match="multiple"):
        A.attention_fwd(q[:, :3], k, v, cu)
    with pytest.raises(KdaError, match="k_stride"):
        A.attention_fwd(q, k[:1].expand(40, 2, 64), v, cu)
    with pytest.raises(KdaError, match="head_dim"):
        A.attention_fwd(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous(), cu)


def test_two_streams_at_once_and_a_workspace_of_two_graphs():
    from recompute_kda_chunkwise_gb300 import attention as A
    cases = [inputs((900,), 8, 2, 128, seed=41), inputs((500, 31, 77), 8, 8, 64, seed=43)]
    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(5):
        for i, (s, (q, k, v, d_o, cu)) in enumerate(zip(streams, cases)):
            with torch.cuda.stream(s):
                o, lse = A.attention_fwd(q, k, v, cu)
                got[i] = (o, lse, *A.attention_bwd(q, k, v, o, lse, d_o, cu))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, w[n]) for a, n in zip(g, ("o", "lse", "dq", "dk", "dv")))
    ws = torch.empty(max(A.attention_workspace_bytes(c[0], c[1], c[4], backward=True) for c in cases), dtype=torch.uint8, device="cuda")
    ws.fill_(255)  # nothing of it is read before it is written
    s, graphs, got = streams[0], [], []
    with torch.cuda.stream(s):
        for q, k, v, d_o, cu in cases:
            o, lse = A.attention_fwd(q, k, v, cu, workspace=ws)
            A.attention_bwd(q, k, v, o, lse, d_o, cu, workspace=ws)
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                o, lse = A.attention_fwd(q, k, v, cu, workspace=ws)
                got.append((o, lse, *A.attention_bwd(q, k, v, o, lse, d_o, cu, workspace=ws)))
        for _ in range(2):
            for g in graphs:
                g.replay()
    s.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, w[n]) for a, n in zip(g, ("o", "lse", "dq", "dk", "dv")))
