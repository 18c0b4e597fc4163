/*
 * kda_blocks.h -- C ABI of what attention blocks beside the delta-rule layers
 * need from training to serving: rotary positions, the paged append that
 * rotates on the way, causal attention of packed sequences with its gradient,
 * and the global gradient norm with clipping. Same library (libkda_gb300.so)
 * and the same rules as kda.h and kda_serving.h: the caller owns every
 * buffer, nothing is allocated or synchronised, arguments are checked on the
 * host before any launch, lengths and pages on the device (a bad one is
 * skipped and recorded in `status`), and all work is enqueued on `stream`.
 *
 * Queries, keys and values are [S, heads, D] with the heads of a token side by
 * side and a stride from token to token: slices of a fused projection are
 * taken as they are. Strides are in elements, multiples of 16 bytes.
 */
#ifndef KDA_BLOCKS_H
#define KDA_BLOCKS_H

#include "kda_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions -----------------------------------------------------
 *
 * The first rotary_dim = R channels of every head turn in pairs (a, b): with
 * the angle x = position * frequency of the pair,
 *     a' = magnitude * (a cos x - b sin x),   b' = magnitude * (a sin x + b cos x)
 * pair i being channels (i, i + R/2) or, interleaved, (2i, 2i + 1); channels
 * from R on pass unchanged. Angles are kept as 64-bit fractions of a turn:
 * freqs[i] is the pair's turns per position times 2^64, and a position's angle
 * is the product modulo 2^64, so whole turns drop out exactly however far the
 * position is. inverse: the opposite angles (the gradient of the rotation).
 * Products are fp32, outputs rounded once. */
typedef struct {
  int64_t total_tokens;       /* S */
  int64_t q_stride, k_stride; /* elements from one token to the next */
  int32_t num_seqs;           /* N, with cu_seqlens */
  int32_t num_heads;          /* of q */
  int32_t num_kv_heads;       /* of k; 0: no k */
  int32_t head_dim;           /* D: a multiple of 8, up to 512 */
  int32_t rotary_dim;         /* R: even, 2 .. D */
  int32_t dtype;              /* kda_dtype of q, k and the outputs */
  int32_t interleaved;
  int32_t inverse;
  float magnitude;
  int32_t fresh;              /* outputs that hold nothing yet: 1 q_out, 2 k_out, or both (3) */
  const int64_t* freqs;       /* device [R/2] */
  const int32_t* positions;   /* device [S]; NULL: a token's index in its sequence */
  const int32_t* cu_seqlens;  /* device [N+1], where positions is NULL */
} kda_rotary_problem;

/* q_out [S, Hq, D] and k_out [S, Hkv, D] are contiguous; q_out may be q, and
 * k_out k, where that is contiguous too; they overlap nothing else. Rows of tokens that cu_seqlens puts
 * into no sequence are not written, or, of a fresh output, zeros (recorded in
 * status). One launch. */
kda_status kda_rotary(const kda_rotary_problem* p, const void* q, const void* k,
                      void* q_out, void* k_out, int32_t* status, void* stream);

/* kda_paged_append with rotary positions: keys are rotated by their position
 * in the cache, kv_lens[n] - L + i, on their way there, and the new tokens'
 * queries beside them. r gives strides, rotary_dim, layout, magnitude,
 * freqs and fresh (its other fields are not read, inverse must be 0); v_stride as
 * q_stride. q NULL: keys and values only (q_out NULL then). q_out may be q
 * where that is contiguous; it and the pages overlap nothing else of the call.
 * What kda_paged_append skips is skipped, its row of q_out not written (zeros
 * where that is fresh). */
kda_status kda_paged_append_rotary(const kda_paged_problem* p, const kda_rotary_problem* r, int64_t v_stride,
                                   const void* q, const void* k, const void* v, void* q_out,
                                   void* k_pages, void* v_pages, int32_t* status, void* stream);

/* ---- causal attention of packed sequences -----------------------------------
 *
 * For the tokens cu_seqlens[n] .. cu_seqlens[n+1]-1 of each sequence, token i
 * attends to its sequence's tokens up to itself:
 *     o = softmax(scale * q K^T) V,   lse = log sum exp(scale * q K^T)
 * per query head; heads h * Hq / Hkv .. share key/value head h. bf16, head_dim
 * 64 or 128, Hq a multiple of Hkv, scale > 0. Scores, statistics and sums are
 * fp32; probabilities and, in the backward, the gradient of the scores are
 * rounded to bf16 for the products that they enter. Results do not depend on
 * the order in which the GPU runs things. A value that is not finite may
 * reach tokens of its own sequence that do not see it (zero times it is NaN),
 * never another sequence. */
typedef struct {
  int64_t total_tokens;       /* S */
  int64_t q_stride, k_stride, v_stride;
  int32_t num_seqs;           /* N: 1 .. 65536 */
  int32_t num_heads;          /* Hq, at most 4096 */
  int32_t num_kv_heads;       /* Hkv */
  int32_t head_dim;           /* 64 or 128 */
  int32_t dtype;              /* KDA_DTYPE_BF16 */
  float scale;
  const int32_t* cu_seqlens;  /* device [N+1]: 0 .. S, not decreasing */
} kda_attention_problem;

/* o [S, Hq, D], lse fp32 [Hq, S]; o may be q where that is contiguous. Outputs
 * and workspace overlap nothing else of the call. The call's status word is the head of the
 * workspace (kda_query_device_status): cu_seqlens that decrease or do not
 * reach from 0 to S leave the outputs unwritten. */
size_t kda_attention_fwd_workspace_bytes(const kda_attention_problem* p);
kda_status kda_attention_fwd(const kda_attention_problem* p, const void* q, const void* k, const void* v,
                             void* o, float* lse, void* workspace, void* stream);

/* The same for outputs that hold nothing yet, and with a status of the
 * caller's. fresh: 1 o, 2 lse, or both (3): where cu_seqlens is refused these
 * are filled with NaN. status: int32 on the device, zeroed by the caller, that
 * takes the call's status word instead of the workspace's head (NULL: that). */
kda_status kda_attention_fwd_fresh(const kda_attention_problem* p, const void* q, const void* k, const void* v,
                                   void* o, float* lse, void* workspace, int32_t fresh, int32_t* status, void* stream);

/* Gradients of o in q, k, v from the forward's inputs and outputs and d_o
 * [S, Hq, D]: dq [S, Hq, D], dk, dv [S, Hkv, D], contiguous, as o and d_o.
 * The probabilities are formed again from q, k and lse. */
size_t kda_attention_bwd_workspace_bytes(const kda_attention_problem* p);
kda_status kda_attention_bwd(const kda_attention_problem* p, const void* q, const void* k, const void* v,
                             const void* o, const float* lse, const void* d_o,
                             void* dq, void* dk, void* dv, void* workspace, void* stream);

/* The same for gradients that hold nothing yet (fresh 1; 0: as above), and with
 * a status of the caller's. */
kda_status kda_attention_bwd_fresh(const kda_attention_problem* p, const void* q, const void* k, const void* v,
                                   const void* o, const float* lse, const void* d_o, void* dq, void* dk, void* dv,
                                   void* workspace, int32_t fresh, int32_t* status, void* stream);

/* ---- the global gradient norm, and clipping by it ---------------------------
 *
 *     norm = sqrt(sum of squares over all tensors),
 *     out  = grad * min(1, max_norm / norm)
 * over `num` tensors (arrays on the host) of `sizes` elements, each contiguous
 * in bf16 or fp32. Squares are summed in fp32 over 32 elements and in fp64
 * above, in an order that depends on the sizes and the device only, so the
 * norm neither overflows nor loses small gradients, and is the same every
 * time. A norm that is not finite clips nothing: out = grad, and the norm says
 * so. out[i] may be grads[i] (then nothing is written where nothing is
 * clipped); no two outputs may overlap, nor an output another gradient.
 * norm: fp32 [1] on the device. workspace: kda_grad_norm_workspace_bytes(num)
 * bytes, 16-byte aligned. */
size_t kda_grad_norm_workspace_bytes(int32_t num);
kda_status kda_grad_norm(int32_t num, const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                         float* norm, void* workspace, void* stream);
kda_status kda_clip_grads(int32_t num, const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                          void* const* outs, const int32_t* out_dtypes, double max_norm,
                          float* norm, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_BLOCKS_H */
