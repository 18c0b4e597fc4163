"""Calls from a thread that has had no business with the GPU: every operator that makes tensor maps, which
need a current context. Autograd's thread is one where a gradient is its first work."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)


def calls():
    from recompute_kda_chunkwise_gb300 import attention as A, decode, kda as K
    S, Hq, Hk = 200, 4, 2
    cu, two = torch.tensor([0, S], dtype=I32, device="cuda"), torch.tensor([0, 80, S], dtype=I32, device="cuda")
    for D in (64, 128):
        q, k, v, d_o = rand(1, S, Hq, D), rand(2, S, Hk, D), rand(3, S, Hk, D), rand(4, S, Hq, D)
        for c in (cu, two):
            o, lse = A.attention_fwd(q, k, v, c)
            yield f"attention_fwd {D} {c.numel()}", lambda q=q, k=k, v=v, c=c: A.attention_fwd(q, k, v, c)
            yield f"attention_bwd {D} {c.numel()}", lambda q=q, k=k, v=v, c=c, o=o, lse=lse, d_o=d_o: A.attention_bwd(q, k, v, o, lse, d_o, c)
        pages = rand(5, 13, 16, Hk, D), rand(6, 13, 16, Hk, D)
        rest = torch.arange(13, dtype=I32, device="cuda")[None], cu[1:].clone(), cu
        yield f"paged_attention {D}", lambda q=q, pages=pages, rest=rest: (decode.paged_attention(q, *pages, *rest),)
    q, k, v, g = (rand(i, S, 2, 128) for i in range(4))
    beta, A_log, bias = rand(7, S, 2), torch.zeros(2, device="cuda"), torch.zeros(2, 128, device="cuda")
    d_o = rand(8, S, 2, 128)

    def delta(grad):
        ts = [t.detach().requires_grad_(grad) for t in (q, k, v, g, beta)]
        o = K.kda(*ts, A_log, bias, cu)
        return torch.autograd.grad(o, ts, d_o) if grad else (o,)

    def without_ctx():
        """The C entry without a ctx, whose first kernel is the forward's own."""
        import ctypes
        lib, out = K.load_library(), torch.empty_like(q)
        p = K._problem_from(q, beta, cu, 1.0, -5.0, 1e-6, K.KDA_FLAG_NO_CHECKPOINTS)
        r = lib.kda_fwd(ctypes.byref(p), *(ctypes.c_void_p(t.data_ptr()) for t in (q, k, v, g, beta, A_log, bias)), None,
                        ctypes.c_void_p(out.data_ptr()), None, None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert r == 0, lib.kda_last_error_message().decode()
        return (out,)

    yield "kda without ctx", without_ctx
    yield "kda", lambda: delta(False)
    yield "kda and its gradient", lambda: delta(True)


@pytest.mark.parametrize("n", range(13))
def test_the_first_call_of_a_thread(n):
    name, call = list(calls())[n]
    want, got = call(), []
    torch.cuda.synchronize()

    def work():
        try:
            got.append(call())
        except Exception as e:  # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not isinstance(got[0], Exception), (name, got[0])
    assert all(torch.equal(a, b) for a, b in zip(got[0], want)), name


def test_a_gradient_as_the_first_work_of_autograds_thread():
    """In a process of its own, where that thread is new."""
    import subprocess
    import sys
    code = """
import torch
from recompute_kda_chunkwise_gb300.attention import attention
q, k, v = (torch.randn(70, 2, 64, device="cuda").bfloat16().requires_grad_() for _ in range(3))
cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
d_o = torch.ones_like(q)
g = torch.autograd.grad(attention(q, k, v, cu), (q, k, v), d_o)
assert all(t.isfinite().all() for t in g)
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


@pytest.mark.parametrize("warm", [True, False])
def test_autograd_captured_into_a_graph(warm):
    """Forward and gradient through the autograd functions in a captured graph; warm False: autograd's thread has
    done nothing before the capture."""
    import subprocess
    import sys
    code = f"""
import torch
from recompute_kda_chunkwise_gb300 import attention as A, kda as K, rotary as T
S, H, D = 300, 4, 64
q, k, v = (torch.randn(S, h, D, device="cuda").bfloat16().requires_grad_() for h in (H, 2, 2))
d_o = torch.randn(S, H, D, device="cuda").bfloat16()
cu = torch.tensor([0, 130, S], dtype=torch.int32, device="cuda")
status = torch.zeros(1, dtype=torch.int32, device="cuda")
rope = T.Rotary(D)

def step():
    x, y = T.rotary(rope, q, k, cu_seqlens=cu, status=status)
    o = A.attention(x, y, v, cu, status=status)
    return (o, *torch.autograd.grad(o, (q, k, v), d_o))

def plain():
    x, y = T.rotary_fwd(rope, q, k, cu_seqlens=cu)
    o, lse = A.attention_fwd(x, y, v, cu)
    dx, dy, dv = A.attention_bwd(x, y, v, o, lse, d_o, cu)
    return (o, *T.rotary_bwd(rope, dx, dy, cu_seqlens=cu), dv)

want = [t.detach().clone() for t in plain()]
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(s):
    if {warm}:
        step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for t in got:
        t.detach().zero_()
    graph.replay()
    graph.replay()
s.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
with torch.no_grad():
    cu[2] = S - 1  # refused at the replay
with torch.cuda.stream(s):
    graph.replay()
s.synchronize()
assert K.query_device_status(status) == 6 and all(t.isnan().all() for t in (got[0], got[3]))
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
