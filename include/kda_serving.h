/*
 * kda_serving.h -- C ABI of the operators around kda_fwd / kda_bwd (kda.h)
 * in a stack of delta-rule and attention layers: the recurrent step over a
 * pool of states, the fused norm between blocks, attention of new tokens
 * over a paged cache, and the verification of drafted tokens. Same library
 * (libkda_gb300.so) and the same rules as kda.h: the caller owns every
 * buffer, nothing is allocated or synchronised, tensors are row-major and
 * contiguous, arguments are checked on the host before any launch, and all
 * work is enqueued on `stream` (a cudaStream_t, NULL = legacy default).
 *
 * Device-side checks. Lengths, slots and page numbers live on the device.
 * The kernels check each one that they index by and skip what a bad one
 * names, so no call reads or writes outside the buffers it was given.
 * `status` (optional, one int32 on the device, zeroed by the caller) then
 * holds KDA_ERR_DEVICE_CHECK; kda_query_device_status(status, stream) reads
 * it. The first error stays until the caller zeroes the word again.
 */
#ifndef KDA_SERVING_H
#define KDA_SERVING_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the recurrent gated delta rule ------------------------------------
 *
 * The recurrence of kda_fwd (kda_gdn2_step: of kda_gdn2_fwd) token by token,
 * for decoding: a few tokens per sequence, each sequence continuing from a
 * state in a pool. For sequence n with the tokens cu_seqlens[n] ..
 * cu_seqlens[n+1]-1 (any number, none included) and every head h:
 *     S = states[state_index[n]][h]
 *     for each token t:  S = the state update of kda_fwd;  o_t = S^T qh_t
 *                        after commit[n] tokens: states[state_index[n]][h] = S
 * so the outputs cover every token and the pool keeps the state after the
 * first commit[n]: tokens that may still be refused (drafts) go behind the
 * committed ones and leave no trace. A commit of 0 writes no state.
 *
 *   p           as for kda_fwd (shapes, dtype, scale, gate bound, l2_eps,
 *               cu_seqlens); flags 0, or KDA_FLAG_CHANNEL_GATES for
 *               kda_gdn2_step
 *   q .. beta_raw, erase_raw, write_raw, A_log, dt_bias, o: as for kda_fwd /
 *               kda_gdn2_fwd
 *   states      fp32 [num_slots, H, D, D], rows: key channel (the layout of
 *               h0 / hT), updated in place
 *   state_index int32 [N] on the device; NULL: sequence n uses slot n (then
 *               num_slots >= N). A negative entry is an inactive sequence (a
 *               padded batch entry): its rows of o are zero, no state is
 *               touched. Two sequences of a call must not share a slot.
 *   commit      int32 [N] on the device; NULL: every token. Values above the
 *               sequence's length mean all of it.
 * Refused on the device (sequence skipped, its rows of o not written): a slot
 * >= num_slots, a negative commit, cu_seqlens entries that decrease or leave
 * [0, S]. Sums are fp32 for every dtype; the result does not depend on how
 * tokens are split over calls. One launch. */
kda_status kda_step(const kda_problem* p,
                    const void* q, const void* k, const void* v,
                    const void* g_raw, const void* beta_raw,
                    const float* A_log, const float* dt_bias,
                    float* states, int64_t num_slots, const int32_t* state_index, const int32_t* commit,
                    void* o, int32_t* status, void* stream);

kda_status kda_gdn2_step(const kda_problem* p,
                         const void* q, const void* k, const void* v,
                         const void* g_raw, const void* erase_raw, const void* write_raw,
                         const float* A_log, const float* dt_bias,
                         float* states, int64_t num_slots, const int32_t* state_index, const int32_t* commit,
                         void* o, int32_t* status, void* stream);

/* ---- the norm between blocks --------------------------------------------
 *
 * The norm after a block, its gate, the scaled residual and the norm before
 * the next block, in one pass. Per row of `width` elements (RMS(x) =
 * x / sqrt(mean(x^2) + eps)):
 *     u     = w_post * RMS(y)          (w_post NULL: 1)
 *     u     = u * sigmoid(z)           (z NULL: no gate)
 *     h_out = residual_scale * h + block_scale * u    (h NULL: block_scale * u)
 *     n     = w_pre * RMS(h_out)       (w_pre NULL: no n)
 * With y [S, H, D] seen as S*H rows of D this is the gated output norm of a
 * delta-rule layer (h, w_pre NULL). n is formed from h_out before h_out is
 * rounded to the problem's dtype. rows >= 0, 1 <= width <= 8192; y, z, h,
 * h_out, n in dtype, the weights fp32; fp32 sums. h_out may be h. */
typedef struct {
  int64_t rows;
  int32_t width;
  int32_t dtype;        /* kda_dtype of the [rows, width] tensors */
  float residual_scale;
  float block_scale;
  float eps;            /* inside the square roots, >= 0 */
} kda_norm_problem;

kda_status kda_block_norm_fwd(const kda_norm_problem* p,
                              const void* y, const void* z, const void* h,
                              const float* w_post, const float* w_pre,
                              void* h_out, void* n, void* stream);

/* Gradients of the above from dh_out (NULL: zero) and dn (NULL: zero), with
 * the forward's inputs; everything between is formed again in fp32. dy is
 * always written; dz, dh, dw_post, dw_pre (fp32 [width]) exactly where z, h,
 * w_post, w_pre are given (NULL otherwise). The weight gradients are summed
 * in a fixed order for given sizes. dh may be dh_out, dy may be y (each only
 * as the whole tensor). workspace: kda_block_norm_workspace_bytes(p) bytes,
 * 16-byte aligned (0 without weights: not used then, and may be NULL). */
size_t kda_block_norm_workspace_bytes(const kda_norm_problem* p, int32_t has_w_post, int32_t has_w_pre);
kda_status kda_block_norm_bwd(const kda_norm_problem* p,
                              const void* y, const void* z, const void* h,
                              const float* w_post, const float* w_pre,
                              const void* dh_out, const void* dn,
                              void* dy, void* dz, void* dh, float* dw_post, float* dw_pre,
                              void* workspace, void* stream);

/* ---- verification of drafted tokens -------------------------------------
 *
 * Speculative sampling with the random numbers given. Sequence n has
 * num_drafts[n] drafted tokens x_0, x_1, ...; target row i is the target's
 * distribution after the first i of them, draft row i the distribution that
 * x_i was drawn from. Draft i is accepted while
 *     u[n][i] * draft[n][i][x_i] < target[n][i][x_i]
 * holds for it and every draft before it. After a accepted drafts the next
 * token is drawn from r = max(target[a] - draft[a], 0) if a draft was
 * refused (from target[a] where no entry of that is positive), else from
 * r = target[a], as the entry with the largest r / noise among those with
 * r > 0, the lowest on ties (noise: draws of the unit exponential
 * distribution, so the entry is distributed as r / sum(r)); 0 if no entry of
 * r is positive.
 *   target       fp32 [N, T+1, V]
 *   draft        fp32 [N, T, V]; NULL: the drafts were not drawn (a lookup),
 *                each row is then 1 at the drafted token
 *   draft_tokens int32 [N, T]; one outside [0, V) is refused, and recorded
 *                in status
 *   num_drafts   int32 [N], clamped to [0, T]; NULL: T
 *   u            fp32 [N, T] uniform on [0, 1);  noise fp32 [N, V], > 0
 *   tokens       int32 [N, T+1]: the accepted drafts, the next token, then -1
 *   accepted     int32 [N]
 * T >= 0 (T = 0: plain sampling; draft, draft_tokens, u unused). The
 * probabilities need not sum to one. NaN compares as false: such a draft is
 * refused, such an entry of r does not count. One launch. */
kda_status kda_verify_drafts(int32_t num_seqs, int32_t max_drafts, int32_t vocab,
                             const float* target, const float* draft,
                             const int32_t* draft_tokens, const int32_t* num_drafts,
                             const float* u, const float* noise,
                             int32_t* tokens, int32_t* accepted, int32_t* status, void* stream);

/* ---- attention of new tokens over a paged cache --------------------------
 *
 * The cache holds keys and values in pages: token position t of sequence n is
 * row t % page_size of page page_table[n][t / page_size]. kv_lens[n] counts
 * the cached tokens with the new ones (tokens cu_seqlens[n] ..
 * cu_seqlens[n+1]-1 of the call) at their end: new token i of L sits at
 * position kv_lens[n] - L + i and attends to the positions up to its own,
 *     o = softmax(scale * q K^T) V     per query head; heads h * Hq / Hkv ..
 *                                      share key/value head h.
 * A token whose position is negative (kv_lens[n] < L) sees nothing: o = 0
 * (while one whose scores are all -inf has o = NaN, from 0 / 0).
 * Cache rows past kv_lens[n] are never used, whatever they hold, and a key or
 * value that is not finite reaches the tokens that see it and no other. bf16,
 * head_dim 64 or 128, Hq a multiple of Hkv, page_size a multiple of 8; fp32
 * scores, statistics and sums, probabilities rounded to bf16 for the second
 * product (its fp32 sum over them divides the result). */
typedef struct {
  int64_t total_tokens;       /* S: new tokens of all sequences */
  int64_t num_pages;
  int32_t num_seqs;           /* N >= 1 */
  int32_t num_heads;          /* Hq */
  int32_t num_kv_heads;       /* Hkv */
  int32_t head_dim;           /* 64 or 128 */
  int32_t dtype;              /* KDA_DTYPE_BF16 */
  int32_t page_size;
  int32_t max_pages;          /* columns of page_table */
  float scale;
  const int32_t* cu_seqlens;  /* device [N+1] */
  const int32_t* page_table;  /* device [N, max_pages] */
  const int32_t* kv_lens;     /* device [N] */
} kda_paged_problem;

/* Writes the new tokens' k and v [S, Hkv, D] to their cache rows. A token
 * whose position is negative, past the table, or whose page is outside
 * [0, num_pages), and one that cu_seqlens (where it decreases) puts into no
 * sequence, is skipped and recorded in status. */
kda_status kda_paged_append(const kda_paged_problem* p, const void* k, const void* v,
                            void* k_pages, void* v_pages, int32_t* status, void* stream);

/* q, o: [S, Hq, D]; k_pages, v_pages: [num_pages, page_size, Hkv, D]. The
 * call's status word is the head of workspace (kda_query_device_status):
 * lengths that do not fit S or the table, and pages outside [0, num_pages)
 * within a sequence's length. A kv_lens entry outside the table's reach makes
 * its sequence's rows of o zero, a page outside the pool those rows that look
 * it up (with the others of their tile of 128 rows), and cu_seqlens entries
 * that decrease or leave [0, S] leave o unwritten. */
size_t kda_paged_attention_workspace_bytes(const kda_paged_problem* p);
kda_status kda_paged_attention(const kda_paged_problem* p, const void* q,
                               const void* k_pages, const void* v_pages,
                               void* o, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_SERVING_H */
