"""Serving operators (include/kda_serving.h): the recurrent step of the gated
delta rule over a pool of states, attention of new tokens over a paged cache,
and the verification of drafted tokens. Thin binding: checks and marshalling.

Lengths, slots and pages stay on the device; the kernels check them and
record what they refuse in ``status`` (an int32 CUDA tensor of one zero, read
with ``kda.query_device_status``). Tensors are contiguous CUDA tensors of one
device; anything else raises ValueError before a launch.
"""
from __future__ import annotations

import ctypes

from ._serving import PagedProblem, bind, done, library


def kda_step(q, k, v, g, beta, A_log, dt_bias, cu_seqlens, states, *, state_index=None, commit=None,
             scale: float = 1.0, lower_bound: float = -5.0, eps: float = 1e-6, out=None, status=None):
    """The recurrence of ``kda.kda_fwd`` token by token over a pool of states.

    Arguments as for ``kda.kda_fwd``; ``states`` [slots, H, D, D] fp32 is
    updated in place: sequence n continues from slot ``state_index[n]`` (int32;
    n itself when None; negative: an inactive sequence, zero outputs) and
    leaves there the state after its first ``commit[n]`` tokens (int32; all
    when None). Outputs cover every token, so drafted tokens go behind the
    committed ones. Returns o."""
    return done(bind().step(q, k, v, g, beta, None, A_log, dt_bias, cu_seqlens, states, state_index, commit, scale,
                            lower_bound, eps, out, status), "kda_step")


def gdn2_step(q, k, v, g, erase, write, A_log, dt_bias, cu_seqlens, states, *, state_index=None, commit=None,
              scale: float = 1.0, lower_bound: float = -5.0, eps: float = 1e-6, out=None, status=None):
    """``kda_step`` for GDN-2 (channel-wise erase and write gates)."""
    return done(bind().step(q, k, v, g, erase, write, A_log, dt_bias, cu_seqlens, states, state_index, commit, scale,
                            lower_bound, eps, out, status), "kda_gdn2_step")


def verify_drafts(target, draft, draft_tokens, num_drafts, u, noise, *, status=None):
    """Verifies drafted tokens (kda_verify_drafts). target [N, T+1, V] and
    draft [N, T, V] fp32 probabilities (draft None: drafts without a
    distribution), draft_tokens [N, T] int32, num_drafts [N] int32 (None: T),
    u [N, T] uniform and noise [N, V] unit-exponential random numbers. Returns
    (tokens [N, T+1] int32: the accepted drafts, the next token, then -1;
    accepted [N] int32)."""
    return done(bind().verify(target, draft, draft_tokens, num_drafts, u, noise, status), "kda_verify_drafts")


def paged_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens, *, status=None):
    """Writes the new tokens' k, v [S, Hkv, D] to the end of their sequences in
    the cache (kda_paged_append): kv_lens [N] counts them already."""
    done(bind().append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens, status), "kda_paged_append")


def paged_attention(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, *, scale=None, out=None, workspace=None):
    """Causal attention of the new tokens q [S, Hq, D] over the paged cache
    (kda_paged_attention), whose kv_lens [N] positions end with them. scale:
    D ** -0.5 when None. workspace: a uint8 CUDA buffer of at least
    paged_attention_workspace_bytes, whose head holds the call's status word;
    allocated when None. Returns o [S, Hq, D]."""
    return done(bind().attention(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, scale, out, workspace),
                "kda_paged_attention")


def paged_attention_workspace_bytes(q, k_pages, page_table, kv_lens, cu_seqlens) -> int:
    """Bytes of workspace for paged_attention with tensors of these shapes."""
    S, Hq, D = q.shape
    pages, size, Hkv, _ = k_pages.shape
    N, width = page_table.shape
    p = PagedProblem(S, pages, N, Hq, Hkv, D, 0, size, width, 1.0, None, None, None)
    return int(library().kda_paged_attention_workspace_bytes(ctypes.byref(p)))
