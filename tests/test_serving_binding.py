"""Refusals of the serving operators before any launch (no GPU needed): the
binding's checks and the C ABI's."""
import ctypes

import pytest
import torch

from recompute_kda_chunkwise_gb300 import _serving as B, build as kbuild, decode, kda as K, norm


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return B.library()


AL, NUL, MIS = ctypes.c_void_p(0x1000), ctypes.c_void_p(0), ctypes.c_void_p(0x1002)


def msg(lib):
    return lib.kda_last_error_message().decode()


def test_struct_layouts():
    assert ctypes.sizeof(B.NormProblem) == 32 and B.NormProblem.eps.offset == 24
    assert ctypes.sizeof(B.PagedProblem) == 72 and B.PagedProblem.cu_seqlens.offset == 48


def test_step_refusals(lib):
    cu = torch.tensor([0, 4], dtype=torch.int32)  # host tensor: never dereferenced
    p = K.make_problem(4, 1, 2, 64, torch.bfloat16, cu)

    def call(p, *, states=AL, slots=1, index=NUL, commit=NUL, q=AL, o=AL, status=NUL):
        return lib.kda_step(ctypes.byref(p), q, AL, AL, AL, AL, AL, AL, states, slots, index, commit, o, status, NUL)

    assert call(p, q=NUL) == 1 and "q is NULL" in msg(lib)
    assert call(p, states=MIS) == 1 and "states" in msg(lib)
    assert call(p, o=NUL) == 1
    assert call(p, slots=0) == 1 and "num_slots" in msg(lib)
    assert call(p, slots=1 << 45) == 1 and "num_slots" in msg(lib)
    assert call(p, index=MIS) == 1 and "aligned" in msg(lib)
    for flags in (K.KDA_FLAG_FORCE_SIMT, K.KDA_FLAG_CHANNEL_GATES, K.KDA_FLAG_CHUNK16):
        assert call(K.make_problem(4, 1, 2, 64, torch.bfloat16, cu, flags=flags)) == 1 and "flags" in msg(lib)
    assert call(K.make_problem(4, 2, 2, 64, torch.bfloat16, cu)) == 1  # two sequences, one slot, no index
    assert call(K.make_problem(4, 1, 2, 96, torch.bfloat16, cu)) == 2
    assert call(K.make_problem(4, 1, 2, 64, torch.bfloat16, cu, lower_bound=-9.0)) == 2
    assert lib.kda_gdn2_step(ctypes.byref(p), *([AL] * 9), 1, NUL, NUL, AL, NUL, NUL) == 1 and "CHANNEL" in msg(lib)
    assert call(K.make_problem(0, 1, 2, 64, torch.bfloat16, cu), q=NUL, o=NUL) == 0  # no tokens: nothing to do


def test_norm_refusals(lib):
    def call(fields, **kw):
        a = dict(y=AL, z=NUL, h=NUL, w_post=NUL, w_pre=NUL, h_out=AL, n=NUL)
        a.update(kw)
        return lib.kda_block_norm_fwd(ctypes.byref(B.NormProblem(*fields)), *a.values(), NUL)

    ok = (4, 64, 0, 1.0, 1.0, 1e-5)
    assert call((4, 0, 0, 1.0, 1.0, 1e-5)) == 2 and "width" in msg(lib)
    assert call((4, 8193, 0, 1.0, 1.0, 1e-5)) == 2
    assert call((4, 64, 5, 1.0, 1.0, 1e-5)) == 2 and "dtype" in msg(lib)
    assert call((-1, 64, 0, 1.0, 1.0, 1e-5)) == 1
    assert call((4, 64, 0, float("nan"), 1.0, 1e-5)) == 1
    assert call((4, 64, 0, 1.0, 1.0, -1e-5)) == 1
    assert call(ok, y=NUL) == 1 and "y is NULL" in msg(lib)
    assert call(ok, h_out=NUL) == 1
    assert call(ok, w_pre=AL) == 1 and "n is NULL" in msg(lib)
    assert call(ok, n=AL) == 1 and "without" in msg(lib)
    assert call(ok, z=MIS) == 1 and "aligned" in msg(lib)
    assert call((0, 64, 0, 1.0, 1.0, 1e-5), y=NUL, h_out=NUL) == 0

    def bwd(fields, **kw):
        a = dict(y=AL, z=NUL, h=NUL, w_post=NUL, w_pre=NUL, dho=AL, dn=NUL, dy=AL, dz=NUL, dh=NUL, dwp=NUL, dwn=NUL, ws=NUL)
        a.update(kw)
        return lib.kda_block_norm_bwd(ctypes.byref(B.NormProblem(*fields)), *a.values(), NUL)

    assert bwd(ok, dy=NUL) == 1 and bwd(ok, z=AL) == 1 and bwd(ok, dz=AL) == 1 and bwd(ok, h=AL) == 1
    assert bwd(ok, dn=AL) == 1 and "dn" in msg(lib)
    assert bwd(ok, w_post=AL) == 1 and "dw_post" in msg(lib)
    assert bwd(ok, w_post=AL, dwp=AL) == 1 and "workspace" in msg(lib)
    p = B.NormProblem(*ok)
    assert lib.kda_block_norm_workspace_bytes(ctypes.byref(p), 0, 0) == 0
    assert lib.kda_block_norm_workspace_bytes(ctypes.byref(p), 1, 0) >= 64 * 4


def test_verify_refusals(lib):
    def call(N=1, T=2, V=10, **kw):
        a = dict(target=AL, draft=AL, x=AL, num=AL, u=AL, noise=AL, tokens=AL, accepted=AL, status=NUL)
        a.update(kw)
        return lib.kda_verify_drafts(N, T, V, *a.values(), NUL)

    assert call(N=0) == 1 and call(T=-1) == 1 and call(V=0) == 1 and call(V=(1 << 30) + 1) == 1
    for name in ("target", "x", "u", "noise", "tokens", "accepted"):
        assert call(**{name: NUL}) == 1 and "NULL" in msg(lib), name
        assert call(**{name: MIS}) == 1 and "aligned" in msg(lib), name


def test_paged_refusals(lib):
    ok = dict(S=4, pages=9, N=1, Hq=4, Hkv=2, D=64, dtype=0, page=16, width=3, scale=0.1, cu=0x1000, table=0x1000, lens=0x1000)

    def call(q=AL, ws=AL, **kw):
        p = B.PagedProblem(*{**ok, **kw}.values())
        return lib.kda_paged_attention(ctypes.byref(p), q, AL, AL, AL, ws, NUL)

    assert call(dtype=1) == 2 and call(D=96) == 2
    for page in (0, 4, 12, -8):
        assert call(page=page) == 2 and "page_size" in msg(lib)
    assert call(Hq=3) == 1 and "multiple" in msg(lib)
    assert call(Hkv=0) == 1 and call(N=0) == 1 and call(width=0) == 1 and call(pages=0) == 1 and call(S=-1) == 1
    assert call(scale=float("inf")) == 1 and "scale" in msg(lib)
    assert call(cu=0) == 1 and call(table=0x1001) == 1 and call(lens=0) == 1
    assert call(q=NUL) == 1 and call(q=MIS) == 1 and call(ws=NUL) == 1
    p = B.PagedProblem(*{**ok, "page": 12}.values())
    assert lib.kda_paged_attention_workspace_bytes(ctypes.byref(p)) == 0
    assert lib.kda_paged_append(ctypes.byref(B.PagedProblem(*ok.values())), NUL, AL, AL, AL, NUL, NUL) == 1


def test_binding_refuses_cpu_tensors_shapes_and_strides(lib):
    bf, i32 = torch.bfloat16, torch.int32
    S, H, D = 3, 2, 64
    t = torch.zeros(S, H, D, dtype=bf)
    cu = torch.tensor([0, 3], dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        decode.kda_step(t, t, t, t, torch.zeros(S, H, dtype=bf), torch.zeros(H), torch.zeros(H, D), cu, torch.zeros(1, H, D, D))
    with pytest.raises(ValueError, match="q must be"):
        decode.kda_step(t[0], t, t, t, t, t, t, cu, t)
    with pytest.raises(ValueError, match="CUDA"):
        norm.block_norm_fwd(t)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        norm.block_norm_fwd(t.half())
    with pytest.raises(ValueError, match="CUDA"):
        decode.verify_drafts(torch.zeros(1, 2, 8), None, torch.zeros(1, 1, dtype=i32), None, torch.zeros(1, 1), torch.zeros(1, 8))
    with pytest.raises(ValueError, match="target"):
        decode.verify_drafts(torch.zeros(1, 8), None, None, None, None, None)
    pages = torch.zeros(4, 16, H, D, dtype=bf)
    table = torch.zeros(1, 2, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        decode.paged_attention(t, pages, pages, table, cu[1:], cu)
    with pytest.raises(ValueError, match="CUDA"):
        decode.paged_append(t, t, pages, pages, table, cu[1:], cu)
    with pytest.raises(ValueError, match="q must be"):
        decode.paged_attention(t[0], pages, pages, table, cu[1:], cu)
