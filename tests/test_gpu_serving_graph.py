"""The serving operators inside a CUDA graph: replayed on new inputs they give
what a call gives."""
import pytest
import torch

from recompute_kda_chunkwise_gb300 import decode, norm
from tests import test_gpu_norm, test_gpu_paged, test_gpu_step, test_gpu_verify

pytestmark = pytest.mark.gpu


def captured(f):
    """A graph of f() and its outputs (after a warm-up on a side stream)."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


@pytest.mark.parametrize("gdn2", [False, True])
def test_step(gdn2):
    x = test_gpu_step.make([1, 4, 0, 2], 2, 128, torch.bfloat16, gdn2, seed=1)
    states = x["states"].clone()
    graph, o = captured(lambda: test_gpu_step.call(x, states))
    for seed in (2, 3):
        y = test_gpu_step.make([1, 4, 0, 2], 2, 128, torch.bfloat16, gdn2, seed=seed)
        for k in ("q", "k", "v", "g", "A_log", "dt_bias", "index"):
            x[k].copy_(y[k])
        for a, b in zip(x["gates"], y["gates"]):
            a.copy_(b)
        states.copy_(y["states"])
        want = test_gpu_step.call(y, y["states"])
        graph.replay()
        assert torch.equal(o, want) and torch.equal(states, y["states"])


@pytest.mark.parametrize("D", [128, 4096, 1537])
def test_block_norm(D):
    def both(x, dho, dn):
        kw = {k: x[k] for k in ("z", "h", "w_post", "w_pre")}
        return (*norm.block_norm_fwd(x["y"], **kw), *norm.block_norm_bwd(x["y"], dh_out=dho, dn=dn, **kw).values())

    x, dho, dn = test_gpu_norm.make(300, D, torch.bfloat16, "zhpn", seed=1)
    graph, out = captured(lambda: both(x, dho, dn))
    y, dho2, dn2 = test_gpu_norm.make(300, D, torch.bfloat16, "zhpn", seed=2)
    for k in x:
        x[k].copy_(y[k])
    dho.copy_(dho2)
    dn.copy_(dn2)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, both(y, dho2, dn2)))


def test_verify():
    x = {k: v.cuda() for k, v in test_gpu_verify.make(5, 3, 1000, seed=1).items()}
    names = ("target", "draft", "x", "num", "u", "noise")
    graph, out = captured(lambda: decode.verify_drafts(*(x[k] for k in names)))
    y = {k: v.cuda() for k, v in test_gpu_verify.make(5, 3, 1000, seed=2).items()}
    for k in names:
        x[k].copy_(y[k])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, decode.verify_drafts(*(y[k] for k in names))))


def test_append_and_attention():
    """Lengths and pages are read by the replay, so one graph serves a growing cache."""
    new, lens = [2, 40], [300, 700]
    x = test_gpu_paged.make(new, lens, 4, 2, 128, 16, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(42, 2, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))

    def step():
        decode.paged_append(k, v, x["kp"], x["vp"], x["table"], x["lens"], x["cu_t"])
        return decode.paged_attention(x["q"], x["kp"], x["vp"], x["table"], x["lens"], x["cu_t"])

    graph, o = captured(step)
    for cut in (5, 17):
        x["lens"].copy_(torch.tensor([n - cut for n in lens], dtype=torch.int32))
        k.normal_(generator=g)
        want = step()
        graph.replay()
        assert torch.equal(o, want)
