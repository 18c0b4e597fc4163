"""Serving operators (include/kda_serving.h): the recurrent step of the gated
delta rule over a pool of states, attention of new tokens over a paged cache,
and the verification of drafted tokens. Thin binding: checks and marshalling.

Lengths, slots and pages stay on the device; the kernels check them and
record what they refuse in ``status`` (an int32 CUDA tensor of one zero, read
with ``kda.query_device_status``).
"""
from __future__ import annotations

import torch

from . import kda as _kda
from ._serving import PagedProblem, check, library, maybe, need, off, refuse, stream

_I32, _BF16, _F32 = torch.int32, torch.bfloat16, torch.float32


def _step(name, q, k, v, g, gates, A_log, dt_bias, cu_seqlens, states, state_index, commit, scale, lower_bound, eps,
          out, status):
    dt = q.dtype
    if q.dim() != 3 or dt not in _kda._DTYPE_CODE:
        raise ValueError(f"q must be [S, H, D] in bfloat16 or float32 (got {dt} {tuple(q.shape)})")
    shape = q.shape
    S, H, D = shape
    dev = q.get_device()
    N = cu_seqlens.numel() - 1
    if states.dim() != 4:
        raise ValueError("states must be [slots, H, D, D]")
    slots = states.shape[0]
    if out is None:
        out = torch.empty_like(q)
    if (dev < 0 or off(q, dt, dev, shape) or off(k, dt, dev, shape) or off(v, dt, dev, shape)
            or off(g, dt, dev, shape) or off(out, dt, dev, shape)):
        refuse((("q", q), ("k", k), ("v", v), ("g", g), ("out", out)), dt, dev, shape)
    if len(gates) == 2:
        gate = (need(gates[0], "erase", shape, dt, dev), need(gates[1], "write", shape, dt, dev))
        flags = _kda.KDA_FLAG_CHANNEL_GATES
    else:
        gate, flags = (need(gates[0], "beta", (S, H), dt, dev),), 0
    p = _kda.KdaProblem(S, N, H, D, _kda._DTYPE_CODE[dt], scale, lower_bound, eps, flags,
                        need(cu_seqlens, "cu_seqlens", (N + 1,), _I32, dev))
    st = getattr(library(), name)(
        p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), *gate, need(A_log, "A_log", (H,), _F32, dev),
        need(dt_bias, "dt_bias", (H, D), _F32, dev), need(states, "states", (slots, H, D, D), _F32, dev), slots,
        maybe(state_index, "state_index", (N,), _I32, dev), maybe(commit, "commit", (N,), _I32, dev), out.data_ptr(),
        maybe(status, "status", (1,), _I32, dev), stream(dev))
    if st:
        check(st, name)
    return out


def kda_step(q, k, v, g, beta, A_log, dt_bias, cu_seqlens, states, *, state_index=None, commit=None,
             scale: float = 1.0, lower_bound: float = -5.0, eps: float = 1e-6, out=None, status=None):
    """The recurrence of ``kda.kda_fwd`` token by token over a pool of states.

    Arguments as for ``kda.kda_fwd``; ``states`` [slots, H, D, D] fp32 is
    updated in place: sequence n continues from slot ``state_index[n]`` (int32;
    n itself when None; negative: an inactive sequence, zero outputs) and
    leaves there the state after its first ``commit[n]`` tokens (int32; all
    when None). Outputs cover every token, so drafted tokens go behind the
    committed ones. Returns o."""
    return _step("kda_step", q, k, v, g, (beta,), A_log, dt_bias, cu_seqlens, states, state_index, commit,
                 scale, lower_bound, eps, out, status)


def gdn2_step(q, k, v, g, erase, write, A_log, dt_bias, cu_seqlens, states, *, state_index=None, commit=None,
              scale: float = 1.0, lower_bound: float = -5.0, eps: float = 1e-6, out=None, status=None):
    """``kda_step`` for GDN-2 (channel-wise erase and write gates)."""
    return _step("kda_gdn2_step", q, k, v, g, (erase, write), A_log, dt_bias, cu_seqlens, states,
                 state_index, commit, scale, lower_bound, eps, out, status)


def verify_drafts(target, draft, draft_tokens, num_drafts, u, noise, *, status=None):
    """Verifies drafted tokens (kda_verify_drafts). target [N, T+1, V] and
    draft [N, T, V] fp32 probabilities (draft None: drafts without a
    distribution), draft_tokens [N, T] int32, num_drafts [N] int32 (None: T),
    u [N, T] uniform and noise [N, V] unit-exponential random numbers. Returns
    (tokens [N, T+1] int32: the accepted drafts, the next token, then -1;
    accepted [N] int32)."""
    if target.dim() != 3 or target.shape[1] < 1:
        raise ValueError("target must be [N, T + 1, V]")
    N, T, V = target.shape[0], target.shape[1] - 1, target.shape[2]
    dev = target.get_device()
    args = (need(target, "target", target.shape, _F32, dev), maybe(draft, "draft", (N, T, V), _F32, dev),
            need(draft_tokens, "draft_tokens", (N, T), _I32, dev), maybe(num_drafts, "num_drafts", (N,), _I32, dev),
            need(u, "u", (N, T), _F32, dev), need(noise, "noise", (N, V), _F32, dev))
    # one allocation for both results
    both = torch.empty(N * (T + 2), dtype=_I32, device=target.device)
    at = both.data_ptr()
    st = library().kda_verify_drafts(N, T, V, *args, at, at + 4 * N * (T + 1),
                                     maybe(status, "status", (1,), _I32, dev), stream(dev))
    if st:
        check(st, "kda_verify_drafts")
    return both[: N * (T + 1)].view(N, T + 1), both[N * (T + 1):]


def _paged(S, Hq, Hkv, D, k_pages, v_pages, page_table, kv_lens, cu_seqlens, scale, dev):
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages must be [pages, page_size, Hkv, D] and page_table [N, max_pages]")
    pages, size = k_pages.shape[0], k_pages.shape[1]
    N, width = page_table.shape
    shape = (pages, size, Hkv, D)
    if dev < 0 or off(k_pages, _BF16, dev, shape) or off(v_pages, _BF16, dev, shape):
        refuse((("k_pages", k_pages), ("v_pages", v_pages)), _BF16, dev, shape)
    return PagedProblem(S, pages, N, Hq, Hkv, D, _kda.KDA_DTYPE_BF16, size, width, scale,
                        need(cu_seqlens, "cu_seqlens", (N + 1,), _I32, dev),
                        need(page_table, "page_table", (N, width), _I32, dev),
                        need(kv_lens, "kv_lens", (N,), _I32, dev))


def paged_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens, *, status=None):
    """Writes the new tokens' k, v [S, Hkv, D] to the end of their sequences in
    the cache (kda_paged_append): kv_lens [N] counts them already."""
    if k.dim() != 3:
        raise ValueError("k must be [S, Hkv, D]")
    shape = k.shape
    S, Hkv, D = shape
    dev = k.get_device()
    p = _paged(S, Hkv, Hkv, D, k_pages, v_pages, page_table, kv_lens, cu_seqlens, 1.0, dev)
    st = library().kda_paged_append(p, need(k, "k", shape, _BF16, dev), need(v, "v", shape, _BF16, dev),
                                    k_pages.data_ptr(), v_pages.data_ptr(), maybe(status, "status", (1,), _I32, dev),
                                    stream(dev))
    if st:
        check(st, "kda_paged_append")


def paged_attention(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, *, scale=None, out=None, workspace=None):
    """Causal attention of the new tokens q [S, Hq, D] over the paged cache
    (kda_paged_attention), whose kv_lens [N] positions end with them. scale:
    D ** -0.5 when None. workspace: a uint8 CUDA buffer of at least
    paged_attention_workspace_bytes, whose head holds the call's status word;
    allocated when None. Returns o [S, Hq, D]."""
    if q.dim() != 3 or k_pages.dim() != 4:
        raise ValueError("q must be [S, Hq, D] and k_pages [pages, page_size, Hkv, D]")
    shape = q.shape
    S, Hq, D = shape
    dev = q.get_device()
    p = _paged(S, Hq, k_pages.shape[2], D, k_pages, v_pages, page_table, kv_lens, cu_seqlens,
               D ** -0.5 if scale is None else scale, dev)
    lib = library()
    if out is None:
        out = torch.empty_like(q)
    size = lib.kda_paged_attention_workspace_bytes(p)
    if workspace is None:
        workspace = torch.empty(max(size, 256), dtype=torch.uint8, device=q.device)
    else:
        _kda._check_buffer(workspace, size, q, "workspace")
    st = lib.kda_paged_attention(p, need(q, "q", shape, _BF16, dev), k_pages.data_ptr(), v_pages.data_ptr(),
                                 need(out, "out", shape, _BF16, dev), workspace.data_ptr(), stream(dev))
    if st:
        check(st, "kda_paged_attention")
    return out


def paged_attention_workspace_bytes(q, k_pages, page_table, kv_lens, cu_seqlens) -> int:
    """Bytes of workspace for paged_attention with these tensors."""
    p = _paged(q.shape[0], q.shape[1], k_pages.shape[2], q.shape[2], k_pages, k_pages, page_table, kv_lens, cu_seqlens,
               1.0, q.get_device())
    return int(library().kda_paged_attention_workspace_bytes(p))
