"""What the bindings in ``decode`` and ``norm`` share: the ctypes declarations of
include/kda_serving.h and the compiled host side. As in ``kda``: argument
marshalling only, no CPU path."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

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


_bind = None


def bind():
    """The binding's compiled host side (csrc/kda_bind.cpp), joined to the library's entry points."""
    global _bind
    if _bind is None:
        lib = library()
        path = os.path.join(os.path.dirname(_kda.LIB_PATH), "_kda_bind.so")
        if not os.path.exists(path):
            raise RuntimeError(f"KDA binding not built: {path} is missing "
                               "(run recompute_kda_chunkwise_gb300.build.build())")
        loader = importlib.machinery.ExtensionFileLoader("_kda_bind", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_kda_bind", loader))
        loader.exec_module(m)
        m.init(*(ctypes.cast(getattr(lib, n), _vp).value for n in (
            "kda_step", "kda_gdn2_step", "kda_block_norm_fwd", "kda_block_norm_workspace_bytes", "kda_block_norm_bwd",
            "kda_verify_drafts", "kda_paged_append", "kda_paged_attention_workspace_bytes", "kda_paged_attention")))
        _bind = m
    return _bind


def done(result, where):
    """What a function of bind() returned; an int is the entry point's error status."""
    if type(result) is int:
        check(result, where)
    return result
