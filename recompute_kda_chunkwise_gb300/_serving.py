"""ctypes declarations of include/kda_serving.h, shared by the bindings in
``decode`` and ``norm``. As in ``kda``: argument marshalling only, no CPU path."""
from __future__ import annotations

import ctypes

import torch

from . import kda as _kda

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class NormProblem(ctypes.Structure):
    """Mirror of ``kda_norm_problem``."""
    _fields_ = [("rows", _i64), ("width", _i32), ("dtype", _i32), ("residual_scale", _f32), ("block_scale", _f32),
                ("eps", _f32)]


class PagedProblem(ctypes.Structure):
    """Mirror of ``kda_paged_problem``."""
    _fields_ = [("total_tokens", _i64), ("num_pages", _i64), ("num_seqs", _i32), ("num_heads", _i32),
                ("num_kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32), ("page_size", _i32), ("max_pages", _i32),
                ("scale", _f32), ("cu_seqlens", _vp), ("page_table", _vp), ("kv_lens", _vp)]


_lib = None


def library():
    """The CUDA library with the serving entry points declared."""
    global _lib
    if _lib is None:
        lib = _kda.load_library()
        P, N, G = (ctypes.POINTER(t) for t in (_kda.KdaProblem, NormProblem, PagedProblem))
        for name, res, args in (
                ("kda_step", ctypes.c_int, [P] + [_vp] * 8 + [_i64] + [_vp] * 5),
                ("kda_gdn2_step", ctypes.c_int, [P] + [_vp] * 9 + [_i64] + [_vp] * 5),
                ("kda_block_norm_fwd", ctypes.c_int, [N] + [_vp] * 8),
                ("kda_block_norm_workspace_bytes", ctypes.c_size_t, [N, _i32, _i32]),
                ("kda_block_norm_bwd", ctypes.c_int, [N] + [_vp] * 14),
                ("kda_verify_drafts", ctypes.c_int, [_i32] * 3 + [_vp] * 10),
                ("kda_paged_append", ctypes.c_int, [G] + [_vp] * 6),
                ("kda_paged_attention_workspace_bytes", ctypes.c_size_t, [G]),
                ("kda_paged_attention", ctypes.c_int, [G] + [_vp] * 6)):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


check = _kda._check


# The raw handle of the current stream of a device index: these calls take a
# few microseconds on the GPU, so their host side is kept as short.
stream = torch._C._cuda_getCurrentRawStream


def off(t, dtype, device, shape) -> bool:
    """Whether ``t`` is not the contiguous tensor of ``dtype`` and ``shape`` on
    CUDA device ``device`` (an index) that the kernels index."""
    return t.dtype is not dtype or t.get_device() != device or t.shape != shape or not t.is_contiguous()


def refuse(named, dtype, device, shape):
    """Raises for the first of the (name, tensor) pairs that is off()."""
    shape = tuple(shape)
    for name, t in named:
        if device < 0 or off(t, dtype, device, shape):
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {shape}"
                             f"{f' on cuda:{device}' if device >= 0 else ''} (got {t.dtype} {tuple(t.shape)} on "
                             f"{t.device}{'' if t.is_contiguous() else ', strided'})")


def need(t, name, shape, dtype, device):
    """The address of a tensor the kernels index by ``shape``."""
    if device < 0 or off(t, dtype, device, shape):
        refuse(((name, t),), dtype, device, shape)
    return t.data_ptr()


def maybe(t, name, shape, dtype, device):
    return None if t is None else need(t, name, shape, dtype, device)
