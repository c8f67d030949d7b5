// Launchers of the norm, rotation and 4-bit cache kernels (rope.cu, kv4_cache.cu, kv4_attn.cu),
// used by api.cu, and what those units share.
#pragma once

#include "common.cuh"
#include "dense.cuh"
#include "dsa_kv4.h"

namespace dsa {

// What turns a head: dsa_qk_problem with its strides filled in.
struct TurnArgs {
  const uint16_t *q, *k, *v;
  const uint16_t *q_weight, *k_weight;
  const double* inv_freq;
  const int32_t *positions, *row_offsets;
  uint16_t *q_out, *k_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  float eps;
  int R, B, H_q, H_kv, rot, first, adjacent;   // H_q (H_kv) = 0: no q (k)
  int q_runs, k_runs, v_runs;                  // runs of 2^run_log2 heads that a row's q, k and v are cut into
  int run_log2, rows_log2, split;              // rows of a CTA; or CTAs of a row, each `units` runs of it
  int units;
};
// Sets the last ones: `at_once` heads fit a warp, a run has up to `most` (powers of two).
void deal_heads(TurnArgs& t, int at_once, int most, int H_k, int H_v);

struct CacheArgs {
  uint8_t* pages;
  const int32_t* table;
  int n_pages, H_kv, B, cols;
  int ps, ps_log2;
  uint32_t block;      // bytes of one page of one head
};

cudaError_t launch_qk_norm_rope(TurnArgs a, int D, bool f16, cudaStream_t st);
// Whether the next two set the status block for that many rows; they need it cleared where not.
bool kv4_sets_status(int R);
cudaError_t launch_kv4_append(TurnArgs a, const CacheArgs& c, int D_k, int D_v, bool f16, uint32_t* status, cudaStream_t st);
cudaError_t launch_kv4_read(const CacheArgs& c, int R, const int32_t* row_offsets, const int32_t* positions, int D_k, int D_v,
                            bool f16, uint16_t* k_out, uint16_t* v_out, uint32_t* status, cudaStream_t st);

// The attention's workspace: the status block, a word of status bits for each CTA, what the
// join has to know of each CTA's last item, then the parts.
constexpr int kKv4Slots = 304;                 // CTAs that the GPU holds at once
constexpr int kKv4Bits = 64;                   // (words of the status block)
constexpr size_t kKv4DescOffset = 2048;
constexpr size_t kKv4PartsOffset = 16384;
struct Kv4Join {                               // an item that CTA i begins and others end
  int32_t row0, packed, first, head;           // first row and packed rows of the request; first packed row; K/V head
  int32_t parts, pad[3];                       // parts in the workspace, 0: none
};
static_assert(kKv4DescOffset + kKv4Slots * sizeof(Kv4Join) <= kKv4PartsOffset, "workspace map");
static_assert((kKv4Bits + kKv4Slots) * 4 <= kKv4DescOffset, "status words of the CTAs");

// How a call is cut: packed rows of a row block, CTAs, and whether items may be split.
struct Kv4Shape {
  int rows, grid;
  bool join;
};
Kv4Shape kv4_shape(const dsa_kv4_cache& c, const dsa_kv4_problem& p);
// The kernel for many rows (kv4_tile.cu): its problem as dense attention's, how it is cut, its
// workspace and the launch.
struct Kv4Tile {
  DenseShape shape;
  bool copied;           // the pages are widened into the workspace first
  size_t off_ml, off_part, off_gone, off_k, off_v, total;
};
// Packed rows of a request that see a position, on average (half of a whole prompt's), from which on the
// copy pays.  In us, widened by the way and first: a chunk behind 10240 positions of 64 heads over 8, 2048
// packed rows 97 and 91, 4096 166 and 139, 16384 518 and 405; whole prompts of one K/V head to a query head, 2048
// tokens (ragged, 192 wide) 285 and 320, 4096 72 and 70, 8192 135 and 114; eight of 1024 tokens and four query heads
// 74 and 85.  A compromise: at 2048 rows it pays behind a context and costs for whole prompts, and does not for one of 4096.
constexpr int kCopyRows = 2304;
constexpr size_t kCopyBytes = size_t(1) << 33;
dsa_dense_problem kv4_dense(const dsa_kv4_cache& c, const dsa_kv4_problem& p);
Kv4Tile kv4_tile(const dsa_kv4_cache& c, const dsa_kv4_problem& p);
cudaError_t launch_kv4_tile(const dsa_kv4_cache& c, const CacheArgs& ca, const dsa_kv4_problem& p, const Kv4Tile& s,
                            uint16_t* out, float* lse, char* ws, cudaStream_t st, const TestHooks* hooks = nullptr);
// Clears the status block and widens the pages that rows see, request b's positions to rows b * reach on
// of k and v; gone [B], lens [B]: scratch (kv4_cache.cu).
cudaError_t launch_kv4_copy(const CacheArgs& c, int R, int reach, const int32_t* row_offsets, const int32_t* row_len, int D_k,
                            int D_v, bool f16, uint16_t* k, uint16_t* v, int32_t* gone, int32_t* lens, uint32_t* status,
                            cudaStream_t st);
// Whether a call goes to that kernel.
bool kv4_many_rows(const dsa_kv4_cache& c, const dsa_kv4_problem& p);
inline size_t kv4_parts(const Kv4Shape& s) { return s.join ? (size_t)2 * s.grid * s.rows : 0; }
cudaError_t launch_kv4_attn(const dsa_kv4_cache& c, const CacheArgs& ca, const dsa_kv4_problem& p, const Kv4Shape& s,
                            uint16_t* out, float* lse, char* ws, float* ml, float* part, cudaStream_t st,
                            const TestHooks* hooks = nullptr);

#ifdef __CUDACC__
// The request of row `row` (one warp): the last b with row_offsets[b] <= row, or -1.
// Each round narrows the range 32 times: one for up to 31 requests, three for 4096.
__device__ __forceinline__ int find_request(const int32_t* row_offsets, int B, int row, int lane) {
  int base = 0, len = B + 1;
  while (len > 0) {
    const int step = (len + 31) / 32, at = base + (lane + 1) * step - 1;
    const bool le = at < base + len && row_offsets[at] <= row;
    const int n = __popc(__ballot_sync(0xffffffffu, le));
    if (step == 1) {
      base += n;
      break;
    }
    const int end = base + len;
    base += n * step;
    len = min(step, end - base);
  }
  return base >= 1 && base <= B ? base - 1 : -1;
}

// Byte of the pool where position `pos` of request b begins its page for head 0, or -1.
__device__ __forceinline__ int64_t find_page(const CacheArgs& c, int b, int pos) {
  const int col = pos >> c.ps_log2;
  if (b < 0 || col >= c.cols) return -1;
  const int page = c.table[(int64_t)b * c.cols + col];
  if (page < 0 || page >= c.n_pages) return -1;
  return (int64_t)page * c.H_kv * c.block;
}
#endif

}  // namespace dsa
