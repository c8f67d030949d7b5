/*
 * libdsa norms and rotation: the queries and keys of an attention layer made ready
 * in one pass, each head normed and its position rotated in.
 *
 * For each row r (a token of a packed batch) and head h of q [R, H_q, D_k] and
 * k [R, H_kv, D_k]:
 *
 *   y = x * w / sqrt(mean_d x_d^2 + eps)          where a weight vector is given, else x
 *   angle_i = positions[r] * inv_freq[i]          i < rot / 2
 *   (y_a, y_b) -> (y_a cos angle_i - y_b sin angle_i, y_b cos angle_i + y_a sin angle_i)
 *
 * over the pairs of columns (a, b) of the `rot` columns from rot_first on:
 *   (rot_first + i, rot_first + i + rot / 2), or
 *   (rot_first + 2 i, rot_first + 2 i + 1) with DSA_FLAG_ROPE_ADJACENT.
 * The other columns are normed alone.
 *
 * Precision: sums, norms and the rotation in fp32, one rounding at the end, to the
 * operands' type.  The angle is reduced exactly: inv_freq is held as a 64-bit fraction of
 * a turn, so a position of 10^6 is rotated as exactly as the first one.  Range: a normed head's
 * mean x^2 + eps from 2^-100 to 2^119 (outside, fp32 does not hold the sum of squares, and outputs may be 0 or
 * not finite), and results that the operands' type holds.
 *
 * A row of a negative position is skipped: its outputs are left as they were (padded
 * batches).  A value that is not finite reaches its own head's outputs alone.
 */
#ifndef DSA_ROPE_H
#define DSA_ROPE_H

#include "dsa.h"
#include "dsa_dense.h"   /* DSA_FLAG_FP16 */

#ifdef __cplusplus
extern "C" {
#endif

/* dsa_qk_problem.flags */
#define DSA_FLAG_ROPE_ADJACENT 0x800   /* pairs are adjacent columns, not half the rotated width apart */

/*
 *   R          rows                                                0 <= R <= 65535
 *   B          requests (dsa_kv4_append alone)                     1 <= B <= 4096
 *   H_q, H_kv  heads of q and k                                    0 <= H <= 128; at least 1 where q / k is set
 *   D_k        width of a head: 64, 128, 192 or 256
 *   D_v        width of v's heads (dsa_kv4_append alone)
 *   rot        rotated columns, a multiple of 8 (0: none); rot_first the first of them,
 *              a multiple of 4; rot_first + rot <= D_k
 *   eps        >= 0, finite
 *   flags      DSA_FLAG_FP16 | DSA_FLAG_ROPE_ADJACENT
 *   q_stride, k_stride, v_stride  elements from one row to the next; 0 = packed.
 *              Multiples of 8, at least the packed width: slices of a fused projection.
 *   q, k, v    bf16 (fp16), 16-byte aligned; q or k may be NULL
 *   q_weight, k_weight  [D_k] in the operands' type, 16-byte aligned; NULL: q (k) is not normed
 *   inv_freq   fp64 [rot / 2], radians a position; 8-byte aligned; may be NULL where rot is 0
 *   positions  int32 [R]
 *   row_offsets  int32 [B + 1], rows of each request as in dsa.h (dsa_kv4_append alone)
 */
typedef struct dsa_qk_problem {
  int32_t R, B, H_q, H_kv, D_k, D_v, rot, rot_first;
  float eps;
  int32_t flags;
  int64_t q_stride, k_stride, v_stride;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const double* inv_freq;
  const int32_t* positions;
  const int32_t* row_offsets;
} dsa_qk_problem;

/*
 * Writes q_out [R, H_q, D_k] (where q is set) and k_out [R, H_kv, D_k] (where k is set),
 * 16-byte aligned.  q_out may be q itself and k_out k itself: they are then written in
 * place, with the inputs' strides; otherwise the outputs are packed and overlap no input.
 * One kernel on `stream`, no workspace, no host synchronisation, capturable in a CUDA
 * graph.  Host validation failures return non-zero and enqueue nothing.
 */
DSA_API dsa_status dsa_qk_norm_rope(const dsa_qk_problem* p, uint16_t* q_out, uint16_t* k_out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DSA_ROPE_H */
