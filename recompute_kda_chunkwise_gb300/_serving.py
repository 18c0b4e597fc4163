"""What the bindings in ``decode``, ``norm``, ``rotary``, ``attention`` and ``grads``
share: the ctypes declarations of include/kda_serving.h and include/kda_blocks.h
and the compiled host side. As in ``kda``: argument
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


class _Fresh(ctypes.Union):
    _fields_ = [("fresh", _i32), ("reserved", _f32)]  # the second: its name in programs from before it had a use, 0


class RotaryProblem(ctypes.Structure):
    """Mirror of ``kda_rotary_problem``."""
    _anonymous_ = ("_fresh",)
    _fields_ = [("total_tokens", _i64), ("q_stride", _i64), ("k_stride", _i64), ("num_seqs", _i32), ("num_heads", _i32),
                ("num_kv_heads", _i32), ("head_dim", _i32), ("rotary_dim", _i32), ("dtype", _i32), ("interleaved", _i32),
                ("inverse", _i32), ("magnitude", _f32), ("_fresh", _Fresh), ("freqs", _vp), ("positions", _vp),
                ("cu_seqlens", _vp)]


class AttentionProblem(ctypes.Structure):
    """Mirror of ``kda_attention_problem``."""
    _fields_ = [("total_tokens", _i64), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("num_seqs", _i32),
                ("num_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32), ("scale", _f32),
                ("cu_seqlens", _vp)]


_lib = None


def library():
    """The CUDA library with the serving entry points declared."""
    global _lib
    if _lib is None:
        lib = _kda.load_library()
        P, N, G, R, A = (ctypes.POINTER(t) for t in (_kda.KdaProblem, NormProblem, PagedProblem, RotaryProblem, AttentionProblem))
        for name, res, args in (
                ("kda_step", ctypes.c_int, [P] + [_vp] * 8 + [_i64] + [_vp] * 5),
                ("kda_gdn2_step", ctypes.c_int, [P] + [_vp] * 9 + [_i64] + [_vp] * 5),
                ("kda_block_norm_fwd", ctypes.c_int, [N] + [_vp] * 8),
                ("kda_block_norm_workspace_bytes", ctypes.c_size_t, [N, _i32, _i32]),
                ("kda_block_norm_bwd", ctypes.c_int, [N] + [_vp] * 14),
                ("kda_verify_drafts", ctypes.c_int, [_i32] * 3 + [_vp] * 10),
                ("kda_paged_append", ctypes.c_int, [G] + [_vp] * 6),
                ("kda_paged_attention_workspace_bytes", ctypes.c_size_t, [G]),
                ("kda_paged_attention", ctypes.c_int, [G] + [_vp] * 6),
                ("kda_rotary", ctypes.c_int, [R] + [_vp] * 6),
                ("kda_paged_append_rotary", ctypes.c_int, [G, R, _i64] + [_vp] * 8),
                ("kda_attention_fwd_workspace_bytes", ctypes.c_size_t, [A]),
                ("kda_attention_fwd", ctypes.c_int, [A] + [_vp] * 7),
                ("kda_attention_fwd_fresh", ctypes.c_int, [A] + [_vp] * 6 + [_i32] + [_vp] * 2),
                ("kda_attention_bwd_workspace_bytes", ctypes.c_size_t, [A]),
                ("kda_attention_bwd", ctypes.c_int, [A] + [_vp] * 11),
                ("kda_attention_bwd_fresh", ctypes.c_int, [A] + [_vp] * 10 + [_i32] + [_vp] * 2),
                ("kda_grad_norm_workspace_bytes", ctypes.c_size_t, [_i32]),
                ("kda_grad_norm", ctypes.c_int, [_i32] + [_vp] * 6),
                ("kda_clip_grads", ctypes.c_int, [_i32] + [_vp] * 5 + [ctypes.c_double] + [_vp] * 3)):
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
            "kda_verify_drafts", "kda_paged_append", "kda_paged_attention_workspace_bytes", "kda_paged_attention",
            "kda_rotary", "kda_paged_append_rotary", "kda_attention_fwd_workspace_bytes", "kda_attention_fwd_fresh",
            "kda_attention_bwd_workspace_bytes", "kda_attention_bwd_fresh", "kda_grad_norm_workspace_bytes", "kda_grad_norm",
            "kda_clip_grads")))
        _bind = m
    return _bind


def done(result, where):
    """What a function of bind() returned; an int is the entry point's error status."""
    if type(result) is int:
        check(result, where)
    return result
