// Launches of dense attention over a packed 16-bit cache (dsa_dense_attn); the kernels, and
// what bounds them, are in dense_kernel.cuh.
#include "dense_kernel.cuh"

namespace dsa {
namespace {

template <int DK, int DV, int NW, bool F16>
cudaError_t launch_one(const DenseArgs& a, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DK, DV, NW, kPacked>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  auto kernel = dense_attn_kernel<DK, DV, NW, F16, kPacked>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = item_count(a), slots = dense_slots(NW);
  const int64_t grid = items < slots ? items : slots;
  e = launch_pdl(kernel, dim3((unsigned)grid), dim3(128 + 128 * NW), smem, st, a);
  if (e != cudaSuccess) return e;
  int64_t rows = 0;
  if (a.splits > 1) rows = (int64_t)a.R * a.H_q;
  if (a.tail_parts > 1) rows = (int64_t)(a.tiles * a.H_kv - a.full) * NW * kTile;
  if (rows == 0) return cudaSuccess;
  return launch_pdl(dense_join_kernel<DV, F16>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, a, NW * kTile, (int)grid);
}

template <int DK, int DV>
cudaError_t launch_width(const DenseArgs& a, int nw, bool f16, cudaStream_t st) {
  if (nw == 1) return f16 ? launch_one<DK, DV, 1, true>(a, st) : launch_one<DK, DV, 1, false>(a, st);
  return f16 ? launch_one<DK, DV, 2, true>(a, st) : launch_one<DK, DV, 2, false>(a, st);
}

}  // namespace

DenseShape dense_shape(const dsa_dense_problem& p, int nw) {
  DenseShape s;
  const int64_t G = p.H_q / p.H_kv;
  // The declared bounds may lie above what the call can hold.
  const int64_t most = p.rows_max > 0 && p.rows_max < p.R ? p.rows_max : p.R;
  const int64_t longest = p.L_max < p.L_total ? p.L_max : p.L_total;
  s.nw = nw ? nw : (most * G <= kTile ? 1 : 2);
  const int64_t per = (int64_t)s.nw * kTile;
  int64_t tiles = p.B * ((most * G + per - 1) / per);
  tiles = tiles < p.R * G / per + p.B ? tiles : p.R * G / per + p.B;
  s.tiles = (int)tiles;
  // Parts per row tile, of at least four K/V tiles (512 rows over 512 positions, 32 heads
  // over 8: 13.6 us in one part, 20.2 in two; 64 rows over 4096: 20.8 in eight, 30.5 in
  // sixteen): the parts' way through memory and the join have to pay.  Single tokens'
  // parts are small: 512 positions in two (9.8 us, 11.0 in one).
  const int64_t items = tiles * p.H_kv, slots = dense_slots(s.nw);
  const int64_t kvt = (longest + kTile - 1) / kTile;
  const int64_t cap = s.nw == 1 && kvt >= 4 && kvt < 8 ? 2 : (kvt / 4 < 64 ? kvt / 4 : 64);
  // Items of one length: one to an SM, or one to a slot where that leaves them eight
  // tiles (one token of 64 heads over 8 and 32768 positions: 35 us in 19 parts, 43 in
  // 38).  So are one request's, and prompts that fill a packed cache; single tokens of
  // several requests may not be, whatever the host knows of a cache laid out by capacity.
  const int64_t full = p.B * longest;
  const bool even = p.B == 1 || (s.nw == 2 && p.L_total <= full && 4 * p.L_total >= 3 * full);
  int64_t splits = 1;
  if (items > 0 && items <= 152 && even) {
    splits = kvt >= 8 * (slots / items) ? slots / items : 152 / items;
  } else if (items > 0 && p.B > 1) {
    // Others, single tokens: eight items per slot, since their lengths differ (32
    // requests of up to 32768 positions: 288 us with two, 268 with four, 258 with eight,
    // 255 with sixteen).  Prompts: two where the row tiles alone leave SMs idle.
    const int64_t each = s.nw == 1 ? 8 : 2;
    if (items < each * slots) splits = (each * slots + items - 1) / items;
    // Finer parts than one a slot only of sixteen tiles, and from 5000 positions on.  The
    // host does not know whether the lengths are alike: parts cost where they are, and
    // where they are not one request is walked when the others are done.  Single tokens
    // of 64 heads over 8, in one part and with this rule (us):
    //   longest                                 4096      5000      6144      8000
    //   64 requests, all of it                158 169   196 207   231 246   301 318
    //   64, spread from 64 on                  74  68    84  76    92  74   113  88
    //   32, one of it and 31 of 100            47  40    57  45    66  41    85  49
    // (one of 32768 and seven of 500: 50, and 69 with parts of 32 tiles; eight of 32768: 179
    // and 166).
    const int64_t wave = slots / items > 1 ? slots / items : 1, fine = kvt >= 40 ? kvt / 16 : 1;
    if (splits > wave && splits > fine) splits = wave > fine ? wave : fine;
  }
  if (splits > cap) splits = cap;
  s.splits = splits < 1 ? 1 : (int)splits;
  // One request whose row tiles all see about as much (a chunk behind a long
  // cache): the last, partly filled wave's items in parts, so that it is shorter
  // (2048 rows over 10240 positions, 512 items: 466 us without, 441 with).
  s.tail = s.tail_parts = 0;
  const int64_t rest = items % slots;
  if (s.splits == 1 && s.nw == 2 && p.B == 1 && items > slots && rest > 0 && rest <= slots / 2 && 2 * (longest - p.R) >= longest) {
    s.tail = (int)rest;
    s.tail_parts = (int)(slots / rest < 4 ? slots / rest : 4);
  }
  return s;
}

cudaError_t launch_dense(const dsa_dense_problem& p, const DenseShape& s, uint16_t* out, float* lse, float* part,
                         float* ml, uint32_t* status, cudaStream_t st, const TestHooks* hooks) {
  DenseArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = p.q; a.offsets = p.offsets; a.row_offsets = p.row_offsets; a.row_len = p.row_len;
  a.out = out; a.lse = lse; a.part = part; a.ml = reinterpret_cast<float2*>(ml);
  a.status = status;
  a.next = status + kBarrierWord;
  a.bits = dense_cleared(p, s) ? nullptr : status + kDenseBits;
  a.q_stride = p.q_stride ? p.q_stride : (int64_t)p.H_q * p.D_k;
  a.wait_ns = hooks ? hooks->wait_ns : kDefaultWaitNs;
  a.test_no_load = hooks ? hooks->tile_no_load : 0;
  a.R = p.R; a.B = p.B; a.H_q = p.H_q; a.H_kv = p.H_kv; a.G = p.H_q / p.H_kv; a.L_total = (int)p.L_total;
  a.splits = s.splits; a.tiles = s.tiles;
  a.tail_parts = s.tail_parts;
  a.full = s.tiles * p.H_kv - s.tail;
  a.scale = p.softmax_scale;
  a.c = (float)(p.softmax_scale * 1.4426950408889634);
  a.q_tma = kTile % a.G == 0;
  if (a.q_tma) {
    const cudaError_t e = group_map(&a.tq, p.q, p.R, p.H_q, p.D_k, a.q_stride, a.G);
    if (e != cudaSuccess) return e;
  }
  if (p.L_total > 0) {   // (an empty cache is never read)
    cudaError_t e = chunk_map(&a.tk, p.k, p.L_total, (int64_t)p.H_kv * p.D_k, p.k_stride ? p.k_stride : (int64_t)p.H_kv * p.D_k);
    if (e == cudaSuccess)
      e = chunk_map(&a.tv, p.v, p.L_total, (int64_t)p.H_kv * p.D_v, p.v_stride ? p.v_stride : (int64_t)p.H_kv * p.D_v);
    if (e != cudaSuccess) return e;
  }
  const bool f16 = p.flags & DSA_FLAG_FP16;
  if (p.D_k == 64) return launch_width<64, 64>(a, s.nw, f16, st);
  if (p.D_k == 128) return launch_width<128, 128>(a, s.nw, f16, st);
  return launch_width<192, 128>(a, s.nw, f16, st);
}

}  // namespace dsa
