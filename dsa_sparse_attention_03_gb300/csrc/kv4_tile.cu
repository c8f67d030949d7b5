// Attention over the 4-bit cache for many rows of a request (dsa_kv4_attn): the dense kernel of
// dense_kernel.cuh with four warps that turn pages into its K and V tiles in the place of
// the copies.
//
// A converting warp's thread holds one position and 64 of its columns at a time: 32 bytes of
// codes and a scale, loaded two chunks ahead, become 128 bytes in the swizzled layout that
// the products read.  A scale has 4 significant bits, so code * scale is exact in the
// operands' type and the products are those of the values that the cache stands for.
#include "dense_kernel.cuh"

namespace dsa {
namespace {

template <int DK, int DV, bool F16>
cudaError_t launch_one(const DenseArgs& a, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DK, DV, 2>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  constexpr int threads = kDenseThreads<2, true>;
  auto kernel = dense_attn_kernel<DK, DV, 2, F16, true>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = item_count(a), slots = dense_slots(2);
  const int64_t grid = items < slots ? items : slots;
  e = launch_pdl(kernel, dim3((unsigned)grid), dim3(threads), smem, st, a);
  if (e != cudaSuccess) return e;
  int64_t rows = 0;
  if (a.splits > 1) rows = (int64_t)a.R * a.H_q;
  if (a.tail_parts > 1) rows = (int64_t)(a.tiles * a.H_kv - a.full) * 2 * kTile;
  if (rows == 0) return cudaSuccess;
  return launch_pdl(dense_join_kernel<DV, F16>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, a, 2 * kTile, (int)grid);
}

template <int DK, int DV>
cudaError_t launch_width(const DenseArgs& a, bool f16, cudaStream_t st) {
  return f16 ? launch_one<DK, DV, true>(a, st) : launch_one<DK, DV, false>(a, st);
}

}  // namespace

dsa_dense_problem kv4_dense(const dsa_kv4_cache& c, const dsa_kv4_problem& p) {
  dsa_dense_problem d;
  std::memset(&d, 0, sizeof d);
  const int64_t held = (int64_t)c.page_size * c.table_cols;
  d.R = p.R; d.B = c.B; d.H_q = p.H_q; d.H_kv = c.H_kv; d.D_k = c.D_k; d.D_v = c.D_v;
  d.L_max = (int)(p.L_max < held ? p.L_max : held);
  d.L_total = (int64_t)d.L_max * c.B;   // (as far as anyone knows here, the requests are of one length)
  d.softmax_scale = p.softmax_scale;
  return d;
}

cudaError_t launch_kv4_tile(const dsa_kv4_cache& c, const CacheArgs& ca, const dsa_kv4_problem& p, const DenseShape& s,
                            uint16_t* out, float* lse, float* part, float* ml, uint32_t* status, cudaStream_t st,
                            const TestHooks* hooks) {
  const dsa_dense_problem d = kv4_dense(c, p);
  DenseArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = p.q; a.row_offsets = p.row_offsets; a.row_len = p.row_len;
  a.out = out; a.lse = lse; a.part = part; a.ml = reinterpret_cast<float2*>(ml);
  a.status = status;
  a.next = status + kBarrierWord;
  a.bits = dense_cleared(d, s) ? nullptr : status + kDenseBits;
  a.q_stride = p.q_stride ? p.q_stride : (int64_t)p.H_q * c.D_k;
  a.wait_ns = hooks ? hooks->wait_ns : kDefaultWaitNs;
  a.test_no_load = hooks ? hooks->tile_no_load : 0;
  a.R = p.R; a.B = c.B; a.H_q = p.H_q; a.H_kv = c.H_kv; a.G = p.H_q / c.H_kv;
  a.splits = s.splits; a.tiles = s.tiles;
  a.tail_parts = s.tail_parts;
  a.full = s.tiles * c.H_kv - s.tail;
  a.scale = p.softmax_scale;
  a.c = (float)(p.softmax_scale * 1.4426950408889634);
  a.kv4 = ca;
  a.reach = d.L_max;
  a.q_tma = kTile % a.G == 0;
  if (a.q_tma) {
    const cudaError_t e = group_map(&a.tq, p.q, p.R, p.H_q, c.D_k, a.q_stride, a.G);
    if (e != cudaSuccess) return e;
  }
  const bool f16 = p.flags & DSA_FLAG_FP16;
  if (c.D_k == 64) return launch_width<64, 64>(a, f16, st);
  if (c.D_k == 128) return launch_width<128, 128>(a, f16, st);
  return launch_width<192, 128>(a, f16, st);
}

}  // namespace dsa
