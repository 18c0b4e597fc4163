"""The global gradient norm over many tensors and clipping by it, against float64."""
import math

import pytest
import torch

import _blocks_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def make(shapes, seed=0, std=lambda i: 1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * std(i)).to(BF if i % 3 else F32) for i, s in enumerate(shapes)]


SHAPES = [
    [(1,)],
    [(7, 13), (1,), (8192,), (8193,), (31,), (3, 5, 7)],
    [(0,), (100_003,), (0, 4), (64, 64)],
    [(1000, 1000), (513, 77)] + [(17,)] * 40,
    [(5,)] * 130 + [(70_000,)],
    [(3,)] * 2300,
]


def check_norm(n, ref):
    # squares and sums of 32 of them in fp32: 2^-24 for each of 10 additions in a chain and the square, halved by
    # the root; the norm's own rounding
    assert n.shape == () and n.dtype == F32
    assert abs(n.item() - ref) <= ref * 2.0 ** -20, (n.item(), ref)


@pytest.mark.parametrize("shapes", SHAPES)
def test_norm_and_clipping(shapes):
    from recompute_kda_chunkwise_gb300 import grads as G
    ts = make(shapes, len(shapes), std=lambda i: 10.0 ** (i % 7 - 5))
    ref = R.norm(ts)
    check_norm(G.grad_norm(ts), ref)
    assert torch.equal(G.grad_norm(tuple(ts)), G.grad_norm(ts))
    for most in (0.37 * ref, 1.01 * ref, 0.0, math.inf):
        f = min(1.0, most / ref)
        for other in (None, BF, F32):
            src = [t.clone() for t in ts]
            out = None if other is None else [torch.empty_like(t, dtype=other) for t in ts]
            check_norm(G.clip_grads(src, most, out=out), ref)
            for t, s, y in zip(ts, src, src if out is None else out):
                # the norm, the factor and the product each rounded, then the output
                if f == 1.0:
                    assert torch.equal(y, t.to(y.dtype))
                else:
                    R.check(y, R.d(t) * f, R.d(t).abs() * f * 2.0 ** -19, "clipped")
                if out is not None:
                    assert torch.equal(s, t)


def test_views_that_are_not_aligned_and_transposed():
    from recompute_kda_chunkwise_gb300 import grads as G
    base = [torch.randn(40_001, device="cuda").to(t) for t in (BF, F32)]
    ts = [base[0][1:33_000], base[1][3:39_999], base[0][33_001:33_004], torch.randn(70, 90, device="cuda").T]
    ref = R.norm(ts)
    keep = [t.clone() for t in ts]
    edge = base[0][0].item(), base[0][33_000].item(), base[1][2].item(), base[1][39_999].item()
    check_norm(G.clip_grads(ts, ref / 2), ref)
    for t, k in zip(ts, keep):
        R.check(t, R.d(k) / 2, R.d(k).abs() * 2.0 ** -19, "clipped")
    assert edge == (base[0][0].item(), base[0][33_000].item(), base[1][2].item(), base[1][39_999].item())


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e18, 1e30])
def test_sizes_whose_squares_leave_fp32(size):
    from recompute_kda_chunkwise_gb300 import grads as G
    ts = [torch.randn(5000, device="cuda") * size, (torch.randn(333, device="cuda") * size).to(BF)]
    ref = R.norm(ts)
    check_norm(G.grad_norm(ts), ref)
    out = [t.clone() for t in ts]
    G.clip_grads(out, ref * 0.25)
    for t, y in zip(ts, out):
        R.check(y, R.d(t) / 4, R.d(t).abs() * 2.0 ** -19 + 2.0 ** -149, "clipped")


def test_a_factor_below_fp32s_normal_range():
    from recompute_kda_chunkwise_gb300 import grads as G
    t = torch.full((4,), 1e38, device="cuda")
    G.clip_grads([t], 1e-3)
    R.check(t, torch.full((4,), 5e-4, dtype=torch.float64), 5e-4 * 2.0 ** -19, "clipped")


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_not_finite_clips_nothing(bad):
    from recompute_kda_chunkwise_gb300 import grads as G
    ts = make([(300,), (9000,)], 3)
    ts[1][8999] = bad
    keep = [t.clone() for t in ts]
    n = G.clip_grads(ts, 1e-3)
    assert not math.isfinite(n.item()) and math.isnan(n.item()) == math.isnan(bad)
    out = [torch.empty_like(t) for t in ts]
    G.clip_grads(ts, 1e-3, out=out)
    for t, k, o in zip(ts, keep, out):
        assert torch.equal(t.nan_to_num(1.0), k.nan_to_num(1.0)) and torch.equal(o.nan_to_num(1.0), k.nan_to_num(1.0))


def test_zeros_and_no_tensors():
    from recompute_kda_chunkwise_gb300 import grads as G
    z = [torch.zeros(100, device="cuda")]
    assert G.clip_grads(z, 1.0).item() == 0 and (z[0] == 0).all()
    assert G.grad_norm([]).item() == 0 and G.clip_grads([], 1.0).item() == 0
    assert G.grad_norm([torch.zeros(0, device="cuda")]).item() == 0


def test_refusals():
    from recompute_kda_chunkwise_gb300 import grads as G
    from recompute_kda_chunkwise_gb300.kda import KdaError
    t = torch.ones(64, device="cuda")
    for bad, what in ((t, "list"), ([t, t.cpu()], "CUDA"), ([t.half()], "bfloat16"), ([t[::2]], "dense"), ([None], "tensor")):
        with pytest.raises(ValueError, match=what):
            G.grad_norm(bad)
    for grads, out in (([t, t], None), ([t, t[1:]], None), ([t[:32], t[32:]], [t[32:], t[:32]]),
                       ([t[:32], t[33:]], [t[1:33], torch.ones(31, device="cuda")])):
        with pytest.raises(ValueError, match="overlaps"):
            G.clip_grads(grads, 1.0, out=out)
    with pytest.raises(ValueError, match="shape"):
        G.clip_grads([t], 1.0, out=[t[:3]])
    with pytest.raises(ValueError, match="as many"):
        G.clip_grads([t], 1.0, out=[])
    for most in (-1.0, math.nan):
        with pytest.raises(KdaError, match="max_norm"):
            G.clip_grads([t], most)
    assert (t == 1).all()
    assert G.grad_norm([t, t]).item() == pytest.approx(128 ** 0.5)  # a norm may count a tensor twice


def test_the_same_bits_every_time_and_captured():
    from recompute_kda_chunkwise_gb300 import grads as G
    ts = make([(300_001,), (70, 70), (5,)], 9)
    out = [torch.empty_like(t) for t in ts]
    want = G.clip_grads(ts, 0.5, out=out).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [torch.zeros_like(t) for t in ts]
    with torch.cuda.stream(s):
        G.clip_grads(ts, 0.5, out=got)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            n = G.clip_grads(ts, 0.5, out=got)
        for g in got:
            g.zero_()
        graph.replay()
    s.synchronize()
    assert torch.equal(n, want) and all(torch.equal(a, b) for a, b in zip(got, out))


def test_a_graph_that_saved_a_clipped_tensor_notices():
    from recompute_kda_chunkwise_gb300 import grads as G
    w, x = torch.ones(8, device="cuda", requires_grad=True), torch.full((8,), 3.0, device="cuda")
    y = (w * x).sum()
    G.clip_grads([x], 1.0)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    with torch.inference_mode():
        z = torch.full((4,), 2.0, device="cuda")
        assert G.clip_grads([z], 1.0).item() == 4.0 and z.tolist() == [0.5] * 4


def test_workspace_of_the_caller_shared_by_two_graphs():
    from recompute_kda_chunkwise_gb300 import grads as G
    ws = torch.empty(8192, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        G.grad_norm([torch.ones(3, device="cuda")], workspace=ws[:100])
    a, b = make([(50_000,), (9,)], 1), make([(123,), (40_000,), (7, 7)], 2)
    want = [G.grad_norm(a).item(), G.grad_norm(b).item()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphs, norms = [], []
        for ts in (a, b):
            G.grad_norm(ts, workspace=ws)
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                norms.append(G.grad_norm(ts, workspace=ws))
        for _ in range(3):
            for g in graphs:
                g.replay()
    s.synchronize()
    assert [n.item() for n in norms] == want


@pytest.mark.parametrize("dtype,bits", [(F32, [0x8000]), (F32, [0x8000, 0]), (F32, [1]), (F32, [0x10000, 0x8000]), (BF, [1]), (BF, [0x8000, 1])])
def test_the_smallest_gradients_count(dtype, bits):
    """fp32 whose only bit of 16 or more lies where bf16 has its sign, beside other subnormals; zeros of either sign."""
    from recompute_kda_chunkwise_gb300 import grads as G
    n = 100_000
    word = torch.int32 if dtype == F32 else torch.int16
    x = torch.tensor([b - (1 << 16) if dtype == BF and b >> 15 else b for b in bits], dtype=word, device="cuda")
    t = x.repeat(n // len(bits)).view(dtype)
    t[1::2].neg_()
    ref = R.norm([t])
    assert ref > 0
    # the norm is a subnormal or near one: half a step there beside what check_norm allows
    assert abs(G.grad_norm([t]).item() - ref) <= ref * 2.0 ** -20 + 2.0 ** -150
    out = [torch.empty(n, device="cuda")]
    G.clip_grads([t], ref / 2, out=out)
    R.check(out[0], R.d(t) / 2, R.d(t).abs() * 2.0 ** -19 + 2.0 ** -150, "clipped")
    assert G.grad_norm([torch.full((40,), -0.0, device="cuda", dtype=dtype)]).item() == 0
