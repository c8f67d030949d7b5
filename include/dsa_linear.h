/*
 * libdsa linear attention with a decay for each head.
 *
 * Linear attention keeps a fixed-size state per request and head in place of a cache.
 * This is its form with one fixed decay per head, over the same packed batch of query
 * rows as dsa.h.  It is not the operator of the stack that a DSA layer belongs to: that
 * one's linear layers ("GLM-5.3-Flash-Alis-MLX-4bit", page 3) are KDA, with a gate for
 * each token and channel and a delta rule, and are not computed here.  For the
 * tokens t = 1, 2, .. of a request:
 *
 *   S_t[h] = exp(log_decay[h]) * S_{t-1}[h] + k_t[h]^T v_t[h]      S: fp32 [D_k, D_v]
 *   o_t[h] = scale * q_t[h] S_t[h]
 *
 * dsa_linear_attn computes whole prompts in chunks of 128 tokens, on the tensor
 * cores:
 *
 *   o_i = scale * (e^{ld (i+1)} q_i S + sum_{j <= i} e^{ld (i-j)} (q_i . k_j) v_j)
 *   S'  = e^{ld n} S + sum_j e^{ld (n-1-j)} k_j^T v_j
 *
 * dsa_linear_step is the recurrence itself, for one token of each request.
 * A prompt followed by steps gives what one prompt of all the tokens gives, up
 * to rounding.
 *
 * States: fp32 [n_states, H, D_k, D_v].  Request b uses place state_idx[b] of
 * both state_in and state_out (state_idx NULL: place b).  A negative place marks
 * an unused entry of a padded batch: its rows and states are neither read nor
 * written.  A place >= n_states, and the second and later requests that name
 * the same place, are skipped in the same way and raise DSA_DEVICE_BAD_INDEX.
 * state_in NULL starts from zeros.  state_out may be state_in (updated in
 * place); otherwise the two must not overlap.
 *
 * Precision: q, k, v bf16 (or fp16 with DSA_FLAG_FP16).  The state is held,
 * updated and returned in fp32: in the chunked form each decayed v is split into
 * 16-bit terms that together keep 24 bits (bf16: three) or 22 (fp16: two, scaled for
 * each column and chunk: 22 bits of what is at least 2^-17 of the column's largest
 * decayed v there, 2^-39 of the latter below).  The
 * decayed products (q . k) and the state that a chunk's queries read are rounded
 * to the operands' type for their matrix products (fp16: scaled into its range by
 * powers of two), sums are fp32, and the output is rounded once.  dsa_linear_step
 * computes in fp32 throughout.  Results do not depend on timing.
 *
 * A token's q and k may be anything for the tokens before it, but its v has to be
 * finite: otherwise any output of dsa_linear_attn for its request may be NaN, those of earlier
 * tokens among them (a weight of zero times NaN is NaN).  Rows of other requests, or
 * of none, never reach a request, whatever they hold.
 */
#ifndef DSA_LINEAR_H
#define DSA_LINEAR_H

#include "dsa.h"
#include "dsa_dense.h"   /* DSA_FLAG_FP16 */

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   R         tokens (rows of q, k, v and out)                    0 <= R < 2^31
 *   B         requests                                            1 <= B <= 4096
 *   H         heads                                               1 <= H <= 256
 *   D_k, D_v  head widths, 64 or 128 each
 *   rows_max  >= the most tokens of one request; 0 = not known.  It decides how
 *             a long request is split over the GPU, never the result's meaning.
 *   n_states  places of the state arrays
 *   q_stride, k_stride, v_stride  elements from one token to the next; 0 = packed
 *             (H * D_k, H * D_k, H * D_v).  Multiples of 8, at least the packed width.
 *   scale     multiplies the output
 *   flags     DSA_FLAG_FP16
 *   q, k      [R, H, D_k], v [R, H, D_v]; bases 16-byte aligned
 *   log_decay fp32 [H], natural logarithm of each head's decay, <= 0 (0: nothing is
 *             forgotten; -inf: everything but the last token).  A positive value
 *             counts as 0.
 *   row_offsets  int32 [B+1], as in dsa.h.  dsa_linear_step does not read it: row b
 *             is request b's token, and R must equal B.
 *   state_idx int32 [B] or NULL
 */
typedef struct dsa_linear_problem {
  int32_t R, B, H, D_k, D_v;
  int32_t rows_max, n_states;
  int32_t flags;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  int32_t reserved0;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* log_decay;
  const int32_t* row_offsets;
  const int32_t* state_idx;
} dsa_linear_problem;

/* Workspace bytes of both calls for `p` (host only; 0 if `p` is invalid). */
DSA_API size_t dsa_linear_workspace_size(const dsa_linear_problem* p);

/*
 * Prompts.  Writes out [R, H, D_v] (16-byte aligned; it may not overlap an input)
 * and, if non-NULL, state_out.
 * A request without tokens hands its state on.  Rows outside every request are
 * not written.  ws: at least dsa_linear_workspace_size(p) bytes, 256-byte
 * aligned; its status word is cleared first.  A kernel that clears it, and one, or
 * three where long requests are split; asynchronous, capturable, no host
 * synchronisation.  Calls that may overlap need workspaces of their own.
 */
DSA_API dsa_status dsa_linear_attn(const dsa_linear_problem* p, const float* state_in, float* state_out,
                                   uint16_t* out, void* ws, size_t ws_bytes, void* stream);

/*
 * Single tokens: one for each request (R == B).  Both state_in (or NULL) and
 * state_out as above; state_out must be set.  One kernel (with state_idx, after a
 * memset of the status).
 */
DSA_API dsa_status dsa_linear_step(const dsa_linear_problem* p, const float* state_in, float* state_out,
                                   uint16_t* out, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DSA_LINEAR_H */
