"""Launches to more than one device from one process: what a kernel's launch
sets or asks belongs to a device. The launch code runs against a pretended CUDA
runtime of two devices (tests/_fake_cuda_runtime.cpp); no GPU needed."""
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
    objs = [os.path.join(kbuild.BUILD, f) for f in ("kda_norm.o", "kda_paged_attention.o", "kda_paged.o")]
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_fake_cuda_runtime.cpp")
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
    return ctypes.CDLL(so)


def fwd(lib, width):
    p = B.NormProblem(300, width, 1, 1.0, 1.0, 1e-5)
    return lib.kda_block_norm_fwd(ctypes.byref(p), AL, AL, AL, AL, AL, AL, AL, NUL)


def bwd(lib, width):
    p = B.NormProblem(300, width, 1, 1.0, 1.0, 1e-5)
    return lib.kda_block_norm_bwd(ctypes.byref(p), *([AL] * 13), NUL)


def attention(lib, D):
    p = B.PagedProblem(4, 9, 1, 4, 2, D, 0, 16, 3, 0.1, 0x1000, 0x1000, 0x1000)
    return lib.kda_paged_attention(ctypes.byref(p), AL, AL, AL, AL, AL, NUL)


CALLS = [(fwd, 4096), (fwd, 128), (bwd, 4096), (bwd, 128), (bwd, 4097), (attention, 64), (attention, 128)]


@pytest.mark.parametrize("call,size", CALLS)
def test_every_device_is_set_up(lib, call, size):
    for device in (0, 1, 0, 1):
        lib.fake_device(device)
        before = lib.fake_launches()
        assert call(lib, size) == 0, f"device {device}"
        assert lib.fake_launches() > before
    done = lib.fake_settings()
    for device in (0, 1):
        lib.fake_device(device)
        assert call(lib, size) == 0
    assert lib.fake_settings() == done  # once a device is enough


@pytest.mark.parametrize("call,size", CALLS)
def test_a_failed_setting_is_reported_and_not_kept(lib, call, size):
    lib.fake_fail(1)
    assert call(lib, size) == KDA_ERR_CUDA and lib.fake_launches() == 0
    assert call(lib, size) == 0 and lib.fake_launches() > 0


def test_the_grid_follows_the_devices_sms(lib):
    for device, sms in ((0, 152), (1, 100)):
        lib.fake_device(device)
        assert attention(lib, 128) == 0 and lib.fake_grid() == sms
        assert fwd(lib, 4096) == 0 and lib.fake_grid() == sms // 8 * 8
