// Attention over the 4-bit cache for many rows of a request (dsa_kv4_attn), by the dense kernel of
// dense_kernel.cuh in one of two ways.
//
// Few row tiles: the kernel with four warps that turn pages into its K and V tiles in the place of
// the copies.  Their registers come from the softmax warps (192 instead of 224).  The loading warp
// brings a tile's page blocks as they are (two tiles ahead, by bulk copies), and a converting warp's
// thread turns one position and 64 of its columns at a time, 32 bytes of codes and a scale, into 128
// bytes in the swizzled layout that the products read.  The converting warps bound the kernel: a tile of
// 128 positions takes about 1.9 us against 1.75 with a 16-bit cache (16 rows of 64 heads over 8
// and 307200 positions 247 us; eight prompts of up to 2048 tokens, width 192, 285, with a 16-bit
// cache 218).  With the codes loaded into registers, two chunks ahead, a chunk took them 1250
// cycles (357 and 370 us); four chunks ahead were slower still, the code competing for the
// instruction cache.
//
// Many: each K/V tile would be widened once for every pair of row tiles, so kv4_copy_kernel widens
// the pages once into the workspace and the kernel reads that (a 2048-row chunk over 10240
// positions 518 -> 405 us, 14 of them the copy).
//
// A scale has 4 significant bits, so code * scale is exact in bf16 (in fp16 from a scale of 2^-21 on, rounded once
// below) and the products are those of the values that the cache stands for.
#include "dense_kernel.cuh"

namespace dsa {
namespace {

template <int DK, int DV, bool F16, CacheKind Kind>
cudaError_t launch_one(const DenseArgs& a, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DK, DV, 2, Kind>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  auto kernel = dense_attn_kernel<DK, DV, 2, F16, Kind>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = item_count(a), slots = dense_slots(2);
  const int64_t grid = items < slots ? items : slots;
  e = launch_pdl(kernel, dim3((unsigned)grid), dim3(kDenseThreads<2, Kind>), smem, st, a);
  if (e != cudaSuccess) return e;
  int64_t rows = 0;
  if (a.splits > 1) rows = (int64_t)a.R * a.H_q;
  if (a.tail_parts > 1) rows = (int64_t)(a.tiles * a.H_kv - a.full) * 2 * kTile;
  if (rows == 0) return cudaSuccess;
  return launch_pdl(dense_join_kernel<DV, F16>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, a, 2 * kTile, (int)grid);
}

template <int DK, int DV>
cudaError_t launch_width(const DenseArgs& a, bool f16, bool copied, cudaStream_t st) {
  if (copied) return f16 ? launch_one<DK, DV, true, kCopied>(a, st) : launch_one<DK, DV, false, kCopied>(a, st);
  return f16 ? launch_one<DK, DV, true, kPages>(a, st) : launch_one<DK, DV, false, kPages>(a, st);
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

cudaError_t launch_kv4_tile(const dsa_kv4_cache& c, const CacheArgs& ca, const dsa_kv4_problem& p, const Kv4Tile& s,
                            uint16_t* out, float* lse, char* ws, cudaStream_t st, const TestHooks* hooks) {
  const dsa_dense_problem d = kv4_dense(c, p);
  const bool f16 = p.flags & DSA_FLAG_FP16;
  DenseArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = p.q; a.row_offsets = p.row_offsets; a.row_len = p.row_len;
  a.out = out; a.lse = lse;
  a.part = reinterpret_cast<float*>(ws + s.off_part);
  a.ml = reinterpret_cast<float2*>(ws + s.off_ml);
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.next = a.status + kBarrierWord;
  a.bits = s.copied || dense_cleared(d, s.shape) ? nullptr : a.status + kDenseBits;
  a.q_stride = p.q_stride ? p.q_stride : (int64_t)p.H_q * c.D_k;
  a.wait_ns = hooks ? hooks->wait_ns : kDefaultWaitNs;
  a.test_no_load = hooks ? hooks->tile_no_load : 0;
  a.R = p.R; a.B = c.B; a.H_q = p.H_q; a.H_kv = c.H_kv; a.G = p.H_q / c.H_kv;
  a.splits = s.shape.splits; a.tiles = s.shape.tiles;
  a.tail_parts = s.shape.tail_parts;
  a.full = s.shape.tiles * c.H_kv - s.shape.tail;
  a.scale = p.softmax_scale;
  a.c = (float)(p.softmax_scale * 1.4426950408889634);
  a.kv4 = ca;
  a.reach = d.L_max;
  a.q_tma = kTile % a.G == 0;
  if (a.q_tma) {
    const cudaError_t e = group_map(&a.tq, p.q, p.R, p.H_q, c.D_k, a.q_stride, a.G);
    if (e != cudaSuccess) return e;
  }
  if (s.copied) {
    uint16_t *k = reinterpret_cast<uint16_t*>(ws + s.off_k), *v = reinterpret_cast<uint16_t*>(ws + s.off_v);
    int32_t* gone = reinterpret_cast<int32_t*>(ws + s.off_gone);
    a.gone = gone;
    a.L_total = (int)d.L_total;
    cudaError_t e = launch_kv4_copy(ca, p.R, d.L_max, p.row_offsets, p.row_len, c.D_k, c.D_v, f16, k, v, gone, gone + c.B, a.status, st);
    if (e == cudaSuccess) e = chunk_map(&a.tk, k, d.L_total, (int64_t)c.H_kv * c.D_k, (int64_t)c.H_kv * c.D_k);
    if (e == cudaSuccess) e = chunk_map(&a.tv, v, d.L_total, (int64_t)c.H_kv * c.D_v, (int64_t)c.H_kv * c.D_v);
    if (e != cudaSuccess) return e;
  } else if (!a.bits) {
    const cudaError_t e = launch_clear_status(ws, st);
    if (e != cudaSuccess) return e;
  }
  if (c.D_k == 64) return launch_width<64, 64>(a, f16, s.copied, st);
  if (c.D_k == 128) return launch_width<128, 128>(a, f16, s.copied, st);
  return launch_width<192, 128>(a, f16, s.copied, st);
}

Kv4Tile kv4_tile(const dsa_kv4_cache& c, const dsa_kv4_problem& p) {
  const dsa_dense_problem d = kv4_dense(c, p);
  Kv4Tile s;
  s.shape = dense_shape(d, 2);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  size_t off = kDensePartsOffset;
  const size_t parts = dense_parts(d, s.shape);
  s.off_ml = off;
  off = up(off + parts * 8);
  s.off_part = off;
  off = up(off + parts * c.D_v * 4);
  const int64_t most = p.rows_max > 0 && p.rows_max < p.R ? p.rows_max : p.R;
  const size_t positions = (size_t)d.L_total;
  const int64_t packed = most * (p.H_q / c.H_kv), hidden = d.L_max > 0 ? packed * (most < d.L_max ? most : d.L_max) / (2 * (int64_t)d.L_max) : 0;
  s.copied = packed - hidden >= kCopyRows && d.L_max > 0 && positions <= (size_t(1) << 31) - 256 &&
             positions * c.H_kv * (c.D_k + c.D_v) * 2 <= kCopyBytes;
  s.off_gone = s.off_k = s.off_v = off;
  if (s.copied) {
    off = up(off + (size_t)c.B * 8);
    s.off_k = off;
    off = up(off + positions * c.H_kv * c.D_k * 2);
    s.off_v = off;
    off = up(off + positions * c.H_kv * c.D_v * 2);
  }
  s.total = off;
  return s;
}

}  // namespace dsa
