/*
 * libdsa 4-bit cache: K and V of attention layers held in 4 bits in pages, with the calls
 * that write it, read it back and attend over it.
 *
 * A pool holds n_pages pages; a page holds page_size positions of one request.  Request
 * b's positions page_size * i .. are in page table[b, i] (pages may be shared between
 * requests).  For each K/V head a page is one block of dsa_kv4_block_bytes() bytes,
 *
 *   K codes   [D_k / 64, page_size, 32]  bytes
 *   V codes   [D_v / 64, page_size, 32]  bytes
 *   K scales  [D_k / 64, page_size]      bf16
 *   V scales  [D_v / 64, page_size]      bf16
 *
 * Each 64 columns of a position are a group with one scale: value = (code - 8) * scale,
 * code 1..15; the code of an even column is the low half of its byte.  Writing x:
 *
 *   scale = max |x| / 7 rounded to 4 significant bits (ties to even; below 2^-126: 0)
 *   code  = x / scale rounded to the nearest whole number (ties to even) + 8
 *
 * 4.25 bits a value, each off by at most half a scale.  A scale of four significant bits
 * times a code of four is exact in bf16 (and in fp16 in its range), so the values that
 * the cache stands for can be multiplied by the tensor cores without another rounding.
 * Scales and codes are those of exact arithmetic, in dsa_rope.h's range: where fp32 cannot tell on which
 * side of a border a normed and rotated key lies, it is computed again in fp64.  A group that
 * holds a value that is not finite has no finite values afterwards.
 */
#ifndef DSA_KV4_H
#define DSA_KV4_H

#include "dsa.h"
#include "dsa_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   n_pages    pages of the pool                         1 <= n_pages < 2^31
 *   page_size  16, 32, 64 or 128 positions
 *   H_kv       K/V heads                                 1 <= H_kv <= 128
 *   D_k, D_v   (64, 64), (128, 128) or (192, 128)
 *   B          requests of the table                     1 <= B <= 4096
 *   table_cols pages that a request's row of the table holds; page_size * table_cols < 2^31 - 256
 *   pages      [n_pages, H_kv, dsa_kv4_block_bytes()], 16-byte aligned
 *   table      int32 [B, table_cols]; entries of positions that a call does not touch may
 *              be anything
 */
typedef struct dsa_kv4_cache {
  int32_t n_pages, page_size, H_kv, D_k, D_v, B, table_cols, reserved0;
  uint8_t* pages;
  const int32_t* table;
} dsa_kv4_cache;

/* Bytes of one page of one K/V head: page_size * (D_k + D_v) * 17 / 32 (host only; 0 for
 * sizes that the cache does not take). */
DSA_API size_t dsa_kv4_block_bytes(int32_t D_k, int32_t D_v, int32_t page_size);

/*
 * Row r of request b goes to position positions[r] of it: its key, normed and rotated as
 * dsa_rope.h describes, and its value, both quantised.  Where p->q is set, q_out gets the
 * rows' queries, normed and rotated (as dsa_qk_norm_rope does it; q_out may be p->q).
 * p->D_k, p->H_kv and p->B are the cache's; p->D_v as well.  Rows of a negative position
 * and rows outside row_offsets are skipped.  A position past the table, or a page outside
 * the pool, is skipped (its query is written all the same) and raises DSA_DEVICE_BAD_INDEX.
 * Positions of one call name different places: what a place holds that two rows are for is
 * not specified.
 * ws: at least 256 bytes, 256-byte aligned; its status word is set by the call
 * (dsa_read_device_status).  One kernel (two from 513 rows on), asynchronous on `stream`, no host
 * synchronisation, capturable in a CUDA graph.  Calls that may overlap need workspaces of
 * their own.  Host validation failures return non-zero and enqueue nothing.
 */
DSA_API dsa_status dsa_kv4_append(const dsa_kv4_cache* c, const dsa_qk_problem* p, uint16_t* q_out, void* ws,
                                  size_t ws_bytes, void* stream);

/*
 * The inverse: k_out [R, H_kv, D_k] and v_out [R, H_kv, D_v] (either may be NULL; 16-byte
 * aligned) get the values that positions[r] of row r's request holds, in bf16, or in fp16 with
 * flags = DSA_FLAG_FP16 (exact in bf16; rounded once in fp16).  row_offsets [B + 1] are the
 * rows of the cache's B requests; R <= 2^31 - 1.  Skipped rows (as above) are left as they
 * were.  In fp16 a value has to be at most 65504, which is a scale up to 9216 (what was written from
 * fp16 without norm and rotation is).  For prompts that attend over a cached prefix with dsa_dense_attn.
 */
DSA_API dsa_status dsa_kv4_read(const dsa_kv4_cache* c, int32_t R, const int32_t* row_offsets, const int32_t* positions,
                                int32_t flags, uint16_t* k_out, uint16_t* v_out, void* ws, size_t ws_bytes, void* stream);

/*
 * Softmax attention over the pages, as dsa_dense.h defines it over a packed cache:
 *
 *   s[r,h,t] = softmax_scale * q[r,h,:] . K[b, t, h / G, :]     t < row_len[r]
 *   out[r,h] = sum_t softmax_t(s[r,h,:])[t] * V[b, t, h / G, :]
 *   lse[r,h] = log sum_t exp(s[r,h,t])
 *
 * with G = H_q / H_kv and K, V the values that the cache stands for.  Row i of a prompt of n
 * rows that ends at position L of its request has row_len = L - n + i + 1.  A row that sees
 * nothing gets zeros and lse = -inf.  Rows outside row_offsets are not written.
 *
 *   R        query rows                                         0 <= R <= 65535
 *   H_q      query heads, a multiple of the cache's H_kv         1 <= H_q <= 128
 *   L_max    >= max(row_len)
 *   rows_max  the most query rows of one request, as far as known; 0 = not known (R is
 *            taken).  It decides which kernel runs (outputs do not depend on it but for rounding)
 *            and with it the workspace: below.
 *   q_stride elements from one row to the next; 0 = packed; a multiple of 8
 *   flags    DSA_FLAG_FP16
 *   q        [R, H_q, D_k], 16-byte aligned
 *   row_offsets  int32 [B + 1] of the cache's B requests, row_len int32 [R].  A row_len outside
 *            [0, min(L_max, page_size * table_cols)] is clamped to it and raises
 *            DSA_DEVICE_BAD_INDEX; so does a page outside the pool, whose positions are
 *            then as if masked.
 *
 * Kernels, by the packed rows of a request, rows_max * G: up to 64 a few rows at a time with the
 * codes as they are, more in tiles of 128 whose K and V are widened to 16 bits, from 2304 on (of
 * which a whole prompt's count half) with the pages widened once into the workspace, where that
 * takes at most 8 GB there: B * L_max positions, whatever the requests' own lengths.  Who has no room for that
 * declares rows_max below 2304 / G (a 2048-row chunk over 10240 positions of 64 heads over 8 then takes 518 us
 * instead of 405).
 * One kernel serves a whole call, so a long chunk and other requests' single tokens are better two calls (31 tokens of up to
 * 32768 positions beside a 2048-row chunk over 10240: 1317 us in one call, 613 in two, 518 where the chunk's call
 * has a cache of its own rows of the table): with the tokens' T rows first, one call with R = T and
 * min(row_offsets, T), one with max(row_offsets, T) and the rows' own L_max and rows_max.
 *
 * Precision: products with K and V are summed in fp32; the softmax statistics are fp32; a softmax
 * weight is rounded once for its product with V, to the operands' type; the output once.  With up to 64
 * packed rows a weight is rounded as its product with V's scale, to fp16: to 11 bits from 2^-20 of the
 * request's largest scale of those 64 columns on, below that by at most 2^-31 of this scale; what a query holds
 * below 2^-25 of its row's largest value is dropped; and the tensor cores cut the addends of a sum of 16
 * products at 2^-16 (K) or 2^-14 (V) of the largest query value, or weight, times scale among them.
 * Results do not depend on timing.  Range: |q| below 2^115; sums over
 * positions of 2^15 |v| below 2^128 (weights are held as up to 2^15 of them).  What lies at positions
 * that no row of a request sees may be anything.  A scale that some rows of a request see has to
 * be finite, or any output of that request may be NaN.  With fp16 queries the kernels of more than 64 packed
 * rows take K and V as dsa_kv4_read gives them in fp16: rounded once, and at most 65504.
 */
typedef struct dsa_kv4_problem {
  int32_t R, H_q, L_max, rows_max;
  float softmax_scale;
  int32_t flags;
  int64_t q_stride;
  const uint16_t* q;
  const int32_t* row_offsets;
  const int32_t* row_len;
} dsa_kv4_problem;

/* Workspace bytes of dsa_kv4_attn (host only; 0 if the problem is invalid:
 * dsa_last_error_string() says why): some megabytes, or with 2304 packed rows or more
 * (see above) B * L_max * H_kv * (D_k + D_v) * 2 bytes beside them. */
DSA_API size_t dsa_kv4_workspace_size(const dsa_kv4_cache* c, const dsa_kv4_problem* p);

/*
 * Writes out [R, H_q, D_v] (16-byte aligned) and, if non-NULL, lse [R, H_q]; neither may
 * overlap an input.  ws: at least dsa_kv4_workspace_size() bytes, 256-byte aligned; the call
 * sets its status word.  Asynchronous on `stream`, no host synchronisation, capturable in a
 * CUDA graph.  Calls that may overlap need workspaces of their own.  Host validation
 * failures return non-zero and enqueue nothing.
 */
DSA_API dsa_status dsa_kv4_attn(const dsa_kv4_cache* c, const dsa_kv4_problem* p, uint16_t* out, float* lse, void* ws,
                                size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DSA_KV4_H */
