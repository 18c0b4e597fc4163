"""Refusals of the operators of include/kda_blocks.h before any launch (no GPU
needed), and what the float64 reference of their tests is checked by."""
import ctypes
import math

import pytest
import torch

import _blocks_ref as R
from recompute_kda_chunkwise_gb300 import _serving as B, attention, build as kbuild, decode, grads, rotary


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return B.library()


AL, NUL, MIS = ctypes.c_void_p(0x1000), ctypes.c_void_p(0), ctypes.c_void_p(0x1002)


def msg(lib):
    return lib.kda_last_error_message().decode()


def test_struct_layouts():
    assert ctypes.sizeof(B.RotaryProblem) == 88 and B.RotaryProblem.freqs.offset == 64
    assert ctypes.sizeof(B.AttentionProblem) == 64 and B.AttentionProblem.cu_seqlens.offset == 56


def rotary_problem(**kw):
    f = dict(total_tokens=4, q_stride=256, k_stride=128, num_seqs=1, num_heads=4, num_kv_heads=2, head_dim=64, rotary_dim=64,
             dtype=0, interleaved=0, inverse=0, magnitude=1.0, reserved=0.0, freqs=0x1000, positions=0x1000, cu_seqlens=0)
    return B.RotaryProblem(**{**f, **kw})


def test_rotary_refusals(lib):
    def call(q=AL, k=AL, qo=ctypes.c_void_p(0x2000), ko=ctypes.c_void_p(0x3000), status=NUL, **kw):
        return lib.kda_rotary(ctypes.byref(rotary_problem(**kw)), q, k, qo, ko, status, NUL)

    assert call(dtype=7) == 2 and call(head_dim=4) == 2 and call(head_dim=60) == 2 and call(head_dim=520) == 2
    for r in (0, 1, 63, 66, -2):
        assert call(rotary_dim=r) == 1 and "rotary_dim" in msg(lib)
    assert call(num_heads=0) == 1 and call(num_kv_heads=-1) == 1 and call(total_tokens=-1) == 1
    assert call(q_stride=255) == 1 and "q_stride" in msg(lib)
    assert call(q_stride=260) == 1 and call(k_stride=64) == 1 and "k_stride" in msg(lib)
    assert call(magnitude=math.inf) == 1 and call(freqs=0) == 1 and call(freqs=0x1004) == 1 and "freqs" in msg(lib)
    assert call(interleaved=2) == 1 and call(inverse=-1) == 1
    assert call(positions=0) == 1 and "cu_seqlens" in msg(lib)
    assert call(positions=0, cu_seqlens=0x1000, num_seqs=0) == 1 and call(positions=0x1002) == 1
    assert call(q=NUL) == 1 and call(q=MIS) == 1 and call(k=NUL) == 1 and call(qo=NUL) == 1 and call(ko=MIS) == 1
    assert call(status=MIS) == 1 and "status" in msg(lib)
    assert call(qo=AL, q_stride=512) == 1 and "contiguous" in msg(lib)
    assert call(total_tokens=0, q=NUL) == 0


def test_append_rotary_refusals(lib):
    ok = dict(S=4, pages=9, N=1, Hq=4, Hkv=2, D=64, dtype=0, page=16, width=3, scale=0.1, cu=0x1000, table=0x1000, lens=0x1000)

    def call(q=AL, qo=ctypes.c_void_p(0x2000), k=AL, vs=128, paged={}, **kw):
        p = B.PagedProblem(*{**ok, **paged}.values())
        return lib.kda_paged_append_rotary(ctypes.byref(p), ctypes.byref(rotary_problem(**kw)), vs, q, k, AL, qo, AL, AL, NUL, NUL)

    assert call(paged=dict(page=12)) == 2 and call(paged=dict(D=96)) == 2 and call(paged=dict(dtype=1)) == 2
    assert call(rotary_dim=66) == 1 and call(inverse=1) == 1 and "inverse" in msg(lib)
    assert call(q=NUL) == 1 and "together" in msg(lib)
    assert call(qo=NUL) == 1 and call(k=NUL) == 1 and call(vs=64) == 1 and "v_stride" in msg(lib)
    assert call(k_stride=100) == 1 and call(q_stride=8) == 1 and call(freqs=0) == 1


def test_attention_refusals(lib):
    ok = dict(total_tokens=4, q_stride=256, k_stride=128, v_stride=128, num_seqs=1, num_heads=4, num_kv_heads=2, head_dim=64,
              dtype=0, scale=0.1, cu_seqlens=0x1000)

    def call(q=AL, ws=AL, lse=AL, **kw):
        return lib.kda_attention_fwd(ctypes.byref(B.AttentionProblem(**{**ok, **kw})), q, AL, AL, AL, lse, ws, NUL)

    assert call(dtype=1) == 2 and call(head_dim=96) == 2 and call(head_dim=256) == 2
    assert call(num_heads=3) == 1 and "multiple" in msg(lib)
    assert call(num_kv_heads=0) == 1 and call(num_seqs=0) == 1 and call(num_seqs=1 << 20) == 1 and call(total_tokens=-1) == 1
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=s) == 1 and "scale" in msg(lib)
    assert call(q_stride=128) == 1 and call(v_stride=132) == 1 and "v_stride" in msg(lib)
    assert call(cu_seqlens=0) == 1 and call(q=NUL) == 1 and call(q=MIS) == 1 and call(ws=NUL) == 1 and call(lse=ctypes.c_void_p(2)) == 1
    assert lib.kda_attention_bwd(ctypes.byref(B.AttentionProblem(**ok)), AL, AL, AL, AL, AL, AL, AL, NUL, AL, AL, NUL) == 1
    assert "dk" in msg(lib)
    p = B.AttentionProblem(**{**ok, "total_tokens": 1000, "num_seqs": 3})
    assert lib.kda_attention_fwd_workspace_bytes(ctypes.byref(p)) >= 256 + 16 * (1000 // 256 + 3)
    # delta, and two parts of dk and dv each in fp32
    assert lib.kda_attention_bwd_workspace_bytes(ctypes.byref(p)) >= 256 + 4 * 1000 * 4 + 4 * 2 * 2 * 1000 * 128
    p.scale = -1.0
    assert lib.kda_attention_fwd_workspace_bytes(ctypes.byref(p)) == 0


def test_clip_refusals(lib):
    def call(num=1, size=8, dtype=1, ptr=0x1000, out=0x2000, out_dtype=1, most=1.0, norm=AL, ws=AL):
        g, o = (ctypes.c_void_p * 1)(ptr), (ctypes.c_void_p * 1)(out)
        return lib.kda_clip_grads(num, g, (ctypes.c_int64 * 1)(size), (ctypes.c_int32 * 1)(dtype), o,
                                  (ctypes.c_int32 * 1)(out_dtype), most, norm, ws, NUL)

    assert call(most=-1.0) == 1 and call(most=math.nan) == 1 and "max_norm" in msg(lib)
    assert call(num=-1) == 1 and call(size=-1) == 1 and call(size=1 << 60) == 1 and call(dtype=3) == 2 and call(out_dtype=-1) == 2
    assert call(ptr=0) == 1 and call(out=0) == 1 and call(ptr=0x1002) == 1 and "aligned" in msg(lib)
    assert call(out=0x1000, out_dtype=0) == 1 and "place" in msg(lib)
    assert call(norm=NUL) == 1 and call(ws=NUL) == 1 and call(ws=MIS) == 1
    assert lib.kda_grad_norm_workspace_bytes(1) == 8192 and lib.kda_grad_norm_workspace_bytes(1001) == 16384
    assert lib.kda_grad_norm(1, None, None, None, AL, AL, NUL) == 1


def test_binding_refuses_cpu_tensors_shapes_and_strides(lib):
    bf, i32 = torch.bfloat16, torch.int32
    t, cu = torch.zeros(3, 2, 64, dtype=bf), torch.tensor([0, 3], dtype=i32)
    rope = rotary.Rotary(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        rotary.rotary_fwd(rope, t, cu_seqlens=cu)
    with pytest.raises(ValueError, match="must be"):
        rotary.rotary_fwd(rope, t[0], cu_seqlens=cu)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        rotary.rotary_fwd(rope, t.half(), cu_seqlens=cu)
    with pytest.raises(ValueError, match="CUDA"):
        attention.attention_fwd(t, t, t, cu)
    with pytest.raises(ValueError, match="q must be"):
        attention.attention_fwd(t[0], t, t, cu)
    pages = torch.zeros(4, 16, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        decode.paged_append_rotary(rope, t, t, t, pages, pages, cu[None], cu[1:], cu)
    with pytest.raises(ValueError, match="CUDA"):
        grads.grad_norm([t])
    with pytest.raises(ValueError, match="list"):
        grads.clip_grads(t, 1.0)


def test_rotary_plans():
    base = rotary.Rotary(8, device="cpu")
    assert base.frequencies == [1.0, 0.1, 0.01, 0.001] or base.frequencies == pytest.approx([1.0, 0.1, 0.01, 0.001])
    # turns are 64-bit fractions: frequency / 2 pi
    assert [t / 2.0 ** 64 for t in base.turns.tolist()] == pytest.approx([f / (2 * math.pi) for f in base.frequencies], rel=1e-15)
    half = rotary.Rotary(2, frequencies=[math.pi * 1.5], device="cpu")  # three quarters of a turn: negative as int64
    assert half.turns.tolist() == [-(1 << 62)]
    assert rotary.Rotary(8, scaling="linear", factor=4.0, device="cpu").frequencies == pytest.approx([0.25, 0.025, 0.0025, 0.00025])
    ntk = rotary.Rotary(8, scaling="ntk", factor=4.0, device="cpu").frequencies
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(0.001 / 4)
    parts = rotary.Rotary(8, scaling="by_parts", factor=4.0, trained=1000, device="cpu")
    turns = [1000 * f / (2 * math.pi) for f in base.frequencies]  # 159, 15.9, 1.59, 0.159
    assert parts.frequencies[0] == 1.0 and parts.frequencies[3] == pytest.approx(0.001 / 4)
    keep = (turns[1] - 1) / 31
    assert parts.frequencies[1] == pytest.approx(0.1 * (keep + (1 - keep) / 4))
    assert parts.magnitude == pytest.approx(0.1 * math.log(4) + 1) and ntk and base.magnitude == 1.0
    assert rotary.Rotary(8, scaling="by_parts", factor=4.0, trained=1000, magnitude=1.0, device="cpu").magnitude == 1.0
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, scaling="other"), dict(dim=8, base=0.0), dict(dim=8, scaling="by_parts"),
                dict(dim=8, factor=0.5), dict(dim=2, scaling="ntk"), dict(dim=8, frequencies=[1.0]),
                dict(dim=8, frequencies=[1.0, 2.0, 3.0, math.nan]), dict(dim=8, frequencies=[1.0] * 4, scaling="linear")):
        with pytest.raises(ValueError):
            rotary.Rotary(device="cpu", **bad)


def test_reference_gradients_against_differences():
    torch.manual_seed(0)
    S, Hq, Hk, D, cu, scale = 9, 4, 2, 3, [0, 5, 5, 9], 0.7
    q, k, v, w = (torch.randn(S, h, D, dtype=torch.float64) for h in (Hq, Hk, Hk, Hq))
    got, _ = R.attention(q, k, v, cu, scale, w)
    for n, t in (("dq", q), ("dk", k), ("dv", v)):
        for i in range(0, t.numel(), 5):
            def loss(x):
                s = t.clone()
                s.view(-1)[i] += x
                return (R.attention(*(s if u is t else u for u in (q, k, v)), cu, scale)[0]["o"] * w).sum().item()
            assert (loss(1e-6) - loss(-1e-6)) / 2e-6 == pytest.approx(got[n].reshape(-1)[i].item(), abs=1e-7), (n, i)
    # a rotation's gradient is the opposite rotation
    x, y = torch.randn(4, 2, 8, dtype=torch.float64), torch.randn(4, 2, 8, dtype=torch.float64)
    f, pos = [1.0, 0.3, 0.01], [0, 5, 7, 9]
    a = (R.turn(x, pos, f, 1.5, True)[0] * y).sum()
    b = (R.turn(y, pos, f, 1.5, True, -1)[0] * x).sum()
    assert a.item() == pytest.approx(b.item())


def test_fresh_outputs_and_status_refusals(lib):
    p = B.AttentionProblem(4, 256, 128, 128, 1, 4, 2, 64, 0, 0.1, 0x1000)
    fwd = lambda fresh, status: lib.kda_attention_fwd_fresh(ctypes.byref(p), *([AL] * 6), fresh, status, NUL)  # noqa: E731
    bwd = lambda fresh, status: lib.kda_attention_bwd_fresh(ctypes.byref(p), *([AL] * 10), fresh, status, NUL)  # noqa: E731
    for call, bad in ((fwd, (-1, 4)), (bwd, (-1, 2))):
        for fresh in bad:
            assert call(fresh, NUL) == 1 and "fresh" in msg(lib)
        assert call(1, MIS) == 1 and "status" in msg(lib)
    r = rotary_problem(fresh=4)
    assert lib.kda_rotary(ctypes.byref(r), AL, AL, AL, AL, NUL, NUL) == 1 and "fresh" in msg(lib)
    assert B.RotaryProblem.fresh.offset == B.RotaryProblem.reserved.offset == 60
