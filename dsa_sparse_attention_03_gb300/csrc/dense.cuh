// Launcher of the dense attention kernels (dense.cu), used by api.cu.
#pragma once

#include "common.cuh"
#include "dsa_dense.h"

namespace dsa {

// How a problem is cut: row tiles of 128 packed rows per CTA (nw), CTAs along
// the rows (tiles, an upper bound) and parts of the positions (splits); or, without
// splits, the last `tail` items (row tile, K/V head) in `tail_parts` parts each.
struct DenseShape {
  int nw, tiles, splits, tail, tail_parts;
};
// nw: 0, or the row tiles of an item where the caller wants a kernel that has them.
DenseShape dense_shape(const dsa_dense_problem& p, int nw = 0);

// The workspace: the status block with the counter of items, the parts.  Atomics on
// a line slow down every access within 4 KB of it (six requests of 22 rows in all:
// 36 us with the rows just before the workspace, 22 with its parts behind the
// counter, 19 with neither), so the parts start further on and a call whose items
// all have a CTA leaves the counter alone.
constexpr size_t kDensePartsOffset = 4096;
// CTAs that the GPU holds at once.
constexpr int dense_slots(int nw) { return nw == 1 ? 304 : 152; }
// Whether the status block is cleared before the attention kernel.  Not where the cache
// is split and every item has a CTA: the CTAs leave their bits in words from here on
// and the join writes the status (in a graph, one token 14.5 us
// with the clearing kernel, 13.6 without; eager, six requests 20.5 and 19.5).
constexpr int kDenseBits = 64;
static_assert((kDenseBits + dense_slots(1)) * 4 <= kDensePartsOffset, "status words of the CTAs");
inline bool dense_cleared(const dsa_dense_problem& p, const DenseShape& s) {
  return s.splits == 1 || (int64_t)s.tiles * s.splits * p.H_kv > dense_slots(s.nw);
}
// Parts that the launch leaves for its join: O [parts, D_v] in `part`, (m, l) in `ml`.
inline size_t dense_parts(const dsa_dense_problem& p, const DenseShape& s) {
  if (s.splits > 1) return (size_t)p.R * p.H_q * s.splits;
  return s.tail_parts > 1 ? (size_t)s.tail * s.nw * 128 * s.tail_parts : 0;
}
cudaError_t launch_dense(const dsa_dense_problem& p, const DenseShape& s, uint16_t* out, float* lse, float* part,
                         float* ml, uint32_t* status, cudaStream_t st, const TestHooks* hooks = nullptr);

}  // namespace dsa
