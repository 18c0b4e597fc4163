"""Calls of the operators of include/kda_blocks.h on more than one device from one process, against a
pretended CUDA runtime of two devices with 152 and 100 SMs (no GPU needed)."""
import ctypes
import os
import subprocess

import pytest

from recompute_kda_chunkwise_gb300 import _serving as B, build as kbuild

AL = ctypes.c_void_p(0x1000)  # never dereferenced: the pretended runtime runs nothing
NUL = ctypes.c_void_p(0)
KDA_ERR_CUDA = 4


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    kbuild.build()
    so = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    objs = [os.path.join(kbuild.BUILD, f) for f in ("kda_packed.o", "kda_packed_fwd.o", "kda_packed_bwd.o", "kda_rotary.o",
                                                     "kda_clip.o", "kda_paged.o", "kda_paged_attention.o")]
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_fake_cuda_runtime_blocks.cpp")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(kbuild._nvcc())))
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-z,defs,-Bsymbolic", "-I", kbuild.INCLUDE, "-I",
                    os.path.join(cuda, "include"), src, *objs, "-o", so], check=True)
    return so


@pytest.fixture
def lib(built, tmp_path):
    """A fresh copy of the library: nothing is kept from the test before."""
    so = str(tmp_path / "libfake.so")
    with open(built, "rb") as f, open(so, "wb") as g:
        g.write(f.read())
    lib = ctypes.CDLL(so)
    lib.kda_clip_grads.argtypes = [ctypes.c_int32] + [ctypes.c_void_p] * 5 + [ctypes.c_double] + [ctypes.c_void_p] * 3
    return lib


def problem(D, seqs=1, S=5000):
    return B.AttentionProblem(S, 64 * D, 8 * D, 8 * D, seqs, 64, 8, D, 0, 0.1, 0x1000)


def fwd(lib, D, seqs=1, S=5000):
    return lib.kda_attention_fwd(ctypes.byref(problem(D, seqs, S)), *([AL] * 6), NUL)


def bwd(lib, D, seqs=1, S=5000):
    return lib.kda_attention_bwd(ctypes.byref(problem(D, seqs, S)), *([AL] * 10), NUL)


def clip(lib, n):
    g, o = (ctypes.c_void_p * 1)(0x1000), (ctypes.c_void_p * 1)(0x1000)
    return lib.kda_clip_grads(1, g, (ctypes.c_int64 * 1)(n), (ctypes.c_int32 * 1)(1), o, (ctypes.c_int32 * 1)(1), 1.0, AL, AL, NUL)


# kernels of a call with one sequence: the forward; sums, dq, dk and dv, their parts; squares and scaling
@pytest.mark.parametrize("call,size,kernels", [(fwd, 64, 1), (fwd, 128, 1), (bwd, 64, 3), (bwd, 128, 3), (clip, 10 ** 9, 2)])
def test_every_device_is_set_up(lib, call, size, kernels):
    for device in (0, 1, 0, 1):
        lib.fake_device(device)
        before = lib.fake_launches()
        assert call(lib, size) == 0 and lib.fake_launches() == before + kernels
        if call is not clip:
            assert lib.fake_grid() == (152, 100)[device]
        else:
            assert lib.fake_grid() == 3 * (152, 100)[device]


@pytest.mark.parametrize("call", [fwd, bwd])
def test_launches_follow_the_problem(lib, call):
    lib.fake_device(0)
    for seqs, S, kernels in ((1, 5000, 1), (3, 5000, 2), (1, 40, 1), (3, 0, 0)):
        before = lib.fake_launches()
        assert call(lib, 128, seqs, S) == 0
        # a list of tiles for several sequences; the backward's three kernels, and its parts' sums where groups are cut
        want = kernels if call is fwd or kernels == 0 else kernels + 2 + (S == 40)
        assert lib.fake_launches() == before + want, (seqs, S)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_a_setting_that_failed_is_made_again(lib, call):
    lib.fake_device(0)
    lib.fake_fail(1)
    assert call(lib, 128) == KDA_ERR_CUDA
    assert call(lib, 128) == 0


@pytest.mark.parametrize("call,regs", [(fwd, 168), (bwd, 96)])
def test_a_kernel_built_with_too_few_registers_is_not_launched(lib, call, regs):
    """One that splits them between its warpgroups would wait for the missing ones."""
    lib.fake_device(0)
    for D in (64, 128):
        lib.fake_registers(regs - 8)
        before = lib.fake_launches()
        assert call(lib, D) == KDA_ERR_CUDA and lib.fake_launches() == before
        lib.fake_registers(regs)
        assert call(lib, D) == 0
