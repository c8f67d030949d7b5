/*
 * libdsa dense attention: softmax attention over every visible position of a
 * packed K/V cache, with grouped heads.
 *
 * The operator of layers that attend to everything they see, for whole prompts,
 * chunks of prompts and single tokens: the same packed batch as dsa_sparse_attn,
 * without a selection, over K and V caches of H_kv heads.  Query head h reads K/V
 * head h / (H_q / H_kv).  A DSA layer, too, attends densely while a row sees no more
 * positions than its top-k ("ds4 PR #964 issue #118", page 2: the full-attention
 * regime at short contexts): this call serves it where its K and V are stored by
 * head, in the widths below.  Over the latent cache of dsa.h (one head of up to 576
 * columns, or FP8 rows), which it refuses, that regime is dsa_sparse_attn with every
 * position selected.
 *
 *   s[r,h,t]  = softmax_scale * q[r,h,:] . k[offsets[b] + t, h / G, :]    t < row_len[r]
 *   out[r,h]  = sum_t softmax_t(s[r,h,:])[t] * v[offsets[b] + t, h / G, :]
 *   lse[r,h]  = log sum_t exp(s[r,h,t])
 *
 * for the rows r of request b.  The mask is each row's own length, as in
 * dsa.h: a causal prompt of n rows over a request of L positions sets
 * row_len = L - n + i + 1 for its row i.  A row that sees nothing (row_len = 0, or
 * every logit -inf) gets zeros and lse = -inf.  Rows before row_offsets[0] or from row_offsets[B]
 * on are not written.
 *
 * Precision: operands bf16 (or fp16 with DSA_FLAG_FP16), products and sums in
 * fp32, softmax statistics in fp32, the softmax weights rounded to the
 * operands' type for their product with V (fp16: those below 2^-21 of a row's largest
 * to multiples of 2^-31 of it), the output rounded once to the
 * operands' type.  Results do not depend on timing.
 *
 * A masked position's k may be anything.  Its v may be anything too where no row of the
 * request sees it (past the request's largest row_len, or another request's): it
 * reaches no output.  A v that some rows of a request see has to be finite, or any
 * output of that request may be NaN, those of rows that mask it among them: a
 * weight of zero times infinity or NaN is NaN.
 */
#ifndef DSA_DENSE_H
#define DSA_DENSE_H

#include "dsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* dsa_dense_problem.flags, dsa_linear_problem.flags */
#define DSA_FLAG_FP16 0x400   /* q, k, v and out are IEEE fp16 instead of bf16 */

/*
 *   R        query rows                                          0 <= R <= 65535
 *   B        requests                                            1 <= B <= 4096
 *   H_q      query heads                                         1 <= H_q <= 128
 *   H_kv     K/V heads, a divisor of H_q
 *   D_k,D_v  head widths: (64, 64), (128, 128) or (192, 128)
 *   L_max    >= max(row_len)
 *   rows_max >= the most query rows of one request; 0 = not known (R is taken).
 *            It decides how the work is split, and bounds the launch: a batch
 *            with more rows in a request raises DSA_DEVICE_CAPACITY, and the
 *            outputs of rows past the launch are then unspecified.
 *   L_total  offsets[B] (rows of k and v)                        L_total <= 2^31 - 256
 *   q_stride, k_stride, v_stride  elements from one row (token) to the next; 0 =
 *            packed (H_q * D_k, H_kv * D_k, H_kv * D_v).  Multiples of 8, at least
 *            the packed width: q, k and v may be views of one fused projection.
 *   q        [R, H_q, D_k], k [L_total, H_kv, D_k], v [L_total, H_kv, D_v];
 *            bases 16-byte aligned
 *   offsets, row_offsets, row_len  as in dsa.h; a row_len outside [0, the
 *            request's length] is clamped to it and raises DSA_DEVICE_BAD_INDEX
 */
typedef struct dsa_dense_problem {
  int32_t R, B, H_q, H_kv, D_k, D_v;
  int32_t L_max, rows_max;
  int64_t L_total;
  int64_t q_stride, k_stride, v_stride;
  float softmax_scale;
  int32_t flags;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* offsets;
  const int32_t* row_offsets;
  const int32_t* row_len;
} dsa_dense_problem;

/* Workspace bytes of dsa_dense_attn for `p` (host only; 0 if `p` is invalid:
 * dsa_last_error_string() says why). */
DSA_API size_t dsa_dense_workspace_size(const dsa_dense_problem* p);

/*
 * Writes out [R, H_q, D_v] (16-byte aligned) and, if non-NULL, lse [R, H_q];
 * neither may overlap an input.
 * ws: at least dsa_dense_workspace_size(p) bytes, 256-byte aligned; the call
 * sets its status word (dsa_read_device_status reads it).  The attention's kernel,
 * where the cache is split over the grid one that joins the parts, and before them
 * one that clears the status where the join does not collect it; asynchronous on
 * `stream`, no host synchronisation, capturable in a CUDA graph.  Calls that
 * may overlap need workspaces of their own.  Host validation failures return
 * non-zero and enqueue nothing.
 */
DSA_API dsa_status dsa_dense_attn(const dsa_dense_problem* p, uint16_t* out, float* lse, void* ws,
                                  size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DSA_DENSE_H */
