// Dense attention over a packed K/V cache with grouped heads (dsa_dense_attn).
//
// Mathematics.  One pass over a row's visible positions in tiles of 128, with a
// running maximum m and sum l per row (base-2 domain, c = scale * log2 e):
//   m' = max(m, max_t s_t),  p_t = 2^(c s_t - c m'),
//   l = l 2^(c m - c m') + sum p_t,   O = O 2^(c m - c m') + P V,
// and out = O / l, lse = scale * m + ln l.  m only has to be near the maximum:
// O and l are rescaled when the maximum has grown by more than 2^8 (p <= 256
// then, exact enough in 16 bits whose precision is relative), which after a
// row's first tiles hardly ever happens.
//
// Rows.  The G = H_q / H_kv query heads of one K/V head and the rows of one
// request are packed into one axis (packed row = row * G + head in group), so a
// tile of 128 packed rows reads each K/V tile once for all of them: whole
// prompts and single tokens of grouped heads run the same kernel.
//
// A CTA takes NW tiles of 128 packed rows (NW = 2 for prompts, 1 where no
// request has more than one tile), one K/V head and a range of K/V tiles:
//   warp 0      producer: K and V tiles by TMA, in 16 KB chunks of 64 columns
//               through one ring, in the order the MMAs use them
//   warps 1..   one per row tile issues its MMAs: S = Q K^T (both operands in shared
//               memory) and O += P V (P in tensor memory, over the S it came from, in
//               two halves, so that the product starts while the second is computed).
//               The tensor core takes few MMAs ahead, so an issuer that waits leaves
//               it idle; with two, the other row tile's go on.
//   warps 4..   softmax, four warps to a row tile: a thread holds one row of S
// Registers are dealt with setmaxnreg: 56 to warps 0-3, 224 (200) to the softmax.
// With two row tiles the tensor core works on one while the other's softmax
// runs; with one, two CTAs share an SM and alternate.
//
// Bounds.  Prompts: the tensor core's rate, 2 (D_k + D_v) flops per visible
// pair and head.  Single tokens: reading K and V once.
//
// Split cache.  Where the row tiles do not fill the grid, each is computed by
// several CTAs over parts of its positions; they leave (m, l, O) in the
// workspace and dense_join_kernel joins them.
//
// V rows past the last position any row of the CTA sees are zeroed in shared
// memory before their MMA: whatever lies there (another request, memory never
// written) has weight zero, and zero times NaN is NaN.
//
// All waits are bounded; on expiry the CTA stops, drains its copies and MMAs and
// frees tensor memory.
#include "dense.cuh"

#include <cstring>

#include "tc.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;

struct DenseArgs {
  CUtensorMap tk, tv;
  const uint16_t* q;
  const int32_t* offsets;
  const int32_t* row_offsets;
  const int32_t* row_len;
  uint16_t* out;
  float* lse;
  float* part;      // [R * H_q, splits, D_v]
  float2* ml;       // [R * H_q, splits]: (c m, l)
  uint32_t* status;
  int64_t q_stride;
  uint64_t wait_ns;
  int R, B, H_q, H_kv, G, L_total, splits, tiles;
  float scale, c;   // c = scale * log2 e
};

struct __align__(16) Shared {
  uint64_t full[16], empty[16];   // ring of chunks
  uint64_t sfull[2], pready[2][2], ofull[2], done[2], turn[2];
  uint32_t tmem;
  int abort;
  int req, tile;                  // request and its tile; req < 0: nothing to do
  int r0, n, o0, len;             // its rows and positions
  int far[2][4];                  // largest length of each warp's rows
};

template <int DK, int DV, int NW>
__host__ __device__ constexpr int ring_slots() {
  constexpr int budget = (NW == 1 ? 113 : 227) * 1024 - 2048;
  constexpr int s = (budget - NW * kTile * DK * 2) / (int)kChunkBytes;
  return s < 16 ? s : 16;
}
template <int DK, int DV, int NW>
__host__ __device__ constexpr size_t smem_bytes() {
  return (size_t)NW * kTile * DK * 2 + (size_t)ring_slots<DK, DV, NW>() * kChunkBytes + sizeof(Shared) + 1024;
}

// Finds the request of this CTA's row tile (warp 0).  Tiles are numbered over
// the requests; the last ones (a causal prompt's longest) come first.
__device__ void locate(const DenseArgs& a, int rows_per_cta, int idx, Shared* sh, int lane) {
  auto bounds = [&](int b, int& r0, int& n) {
    r0 = 0; n = 0;
    if (b >= a.B) return;
    const int x0 = a.B == 1 ? 0 : a.row_offsets[b], x1 = a.B == 1 ? a.R : a.row_offsets[b + 1];
    r0 = min(max(x0, 0), a.R);
    n = max(min(x1, a.R) - r0, 0);
  };
  int total = 0;
  for (int base = 0; base < a.B; base += 32) {
    int r0, n;
    bounds(base + lane, r0, n);
    total += __reduce_add_sync(0xffffffffu, (n * a.G + rows_per_cta - 1) / rows_per_cta);
  }
  if (total > a.tiles && idx == 0 && lane == 0) raise_status(a.status, DSA_DEVICE_CAPACITY);
  if (lane == 0) sh->req = -1;
  __syncwarp();
  const int want = total - 1 - idx;
  if (want < 0) return;
  int run = 0;
  for (int base = 0; base < a.B; base += 32) {
    int r0, n;
    bounds(base + lane, r0, n);
    const int v = (n * a.G + rows_per_cta - 1) / rows_per_cta;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const int first = run + incl - v;
    if (want >= first && want < first + v) {
      const int b = base + lane;
      const int y0 = a.B == 1 ? 0 : a.offsets[b], y1 = a.B == 1 ? a.L_total : a.offsets[b + 1];
      const int o0 = min(max(y0, 0), a.L_total);
      sh->req = b;
      sh->tile = want - first;
      sh->r0 = r0;
      sh->n = n;
      sh->o0 = o0;
      sh->len = max(min(y1, a.L_total) - o0, 0);
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <int DK, int DV, int NW, bool F16>
__global__ void __launch_bounds__(128 + 128 * NW, NW == 1 ? 2 : 1)
    dense_attn_kernel(const __grid_constant__ DenseArgs a) {
  constexpr int NS = ring_slots<DK, DV, NW>();
  constexpr int KC = DK / 64, VC = DV / 64;
  constexpr uint32_t kQBytes = kTile * DK * 2;
  constexpr uint32_t kCols = NW * 256;      // S of each row tile, then O of each
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* Qs = smem;
  unsigned char* ring = smem + NW * kQBytes;
  Shared* sh = reinterpret_cast<Shared*>(ring + NS * kChunkBytes);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  const int h = blockIdx.x % a.H_kv;
  const int split = (blockIdx.x / a.H_kv) % a.splits;
  const int idx = blockIdx.x / a.H_kv / a.splits;

  if (warp == 0) locate(a, NW * kTile, idx, sh, lane);
  __syncthreads();
  if (sh->req < 0) return;

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&sh->full[i]), 1);
      mbar_init(smem_u32(&sh->empty[i]), NW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh->sfull[i]), 1);
      mbar_init(smem_u32(&sh->pready[i][0]), 4);
      mbar_init(smem_u32(&sh->pready[i][1]), 4);
      mbar_init(smem_u32(&sh->ofull[i]), 1);
      mbar_init(smem_u32(&sh->done[i]), 1);
      mbar_init(smem_u32(&sh->turn[i]), 1);
    }
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(&sh->tmem), kCols);

  // Softmax warps: warp w of a tile reads tensor-memory lanes 32 (w % 4).. .
  const int w = (warp >> 2) - 1;                         // row tile of this warp
  const int trow = (warp & 3) * 32 + lane;               // row in the tile
  const int packed = (sh->tile * NW + w) * kTile + trow; // packed row in the request
  const bool valid = warp >= 4 && packed < sh->n * a.G;
  const int row = sh->r0 + (valid ? packed / a.G : 0);
  const int head = h * a.G + (valid ? packed % a.G : 0);
  int len = 0;
  if (warp >= 4) {
    if (valid) {
      const int l = a.row_len[row];
      len = min(max(l, 0), sh->len);
      if (len != l && split == 0) raise_status(a.status, DSA_DEVICE_BAD_INDEX);
    }
    const int m = __reduce_max_sync(0xffffffffu, len);
    if (lane == 0) sh->far[w][warp & 3] = m;
    // Q, K-major and swizzled: 16-byte pieces, consecutive threads along a row.
    const int t0 = (sh->tile * NW + w) * kTile;
    constexpr int P = DK / 8;
    for (int i = tid & 127; i < kTile * P; i += 128) {
      const int r = i / P, x = i % P, pk = t0 + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (pk < sh->n * a.G)
        v = __ldg(reinterpret_cast<const uint4*>(a.q + (int64_t)(sh->r0 + pk / a.G) * a.q_stride +
                                                 (int64_t)(h * a.G + pk % a.G) * DK) + x);
      *reinterpret_cast<uint4*>(Qs + w * kQBytes + (x >> 3) * kChunkBytes + r * 128 + (((x & 7) ^ (r & 7)) << 4)) = v;
    }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0);
  const WaitCtx wc(&sh->abort, a.status, a.wait_ns);

  // K/V tiles of this CTA: [lo, hi); row tile w takes those below its own end.
  int end[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int* f = sh->far[i];
    end[i] = i < NW ? max(max(f[0], f[1]), max(f[2], f[3])) : 0;
  }
  const int kv_end = max(end[0], end[1]);
  const int nt = (kv_end + kTile - 1) / kTile;
  const int lo = (int)((int64_t)nt * split / a.splits);
  const int hi = (int)((int64_t)nt * (split + 1) / a.splits);
  int cnt[2];                               // tiles of each row tile
#pragma unroll
  for (int i = 0; i < 2; ++i) cnt[i] = max(min((end[i] + kTile - 1) / kTile, hi) - lo, 0);
  const int steps = hi - lo;

  if (warp < 4) {
   regs_down<56>();
   if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int n = 0;
      bool ok = true;
      for (int j = lo; j < hi && ok; ++j) {
        for (int c = 0; c < KC + VC; ++c, ++n) {
          const int s = n % NS;
          if (n >= NS && !wait_bar(smem_u32(&sh->empty[s]), (n / NS - 1) & 1, wc)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&sh->full[s]), dst = smem_u32(ring + s * kChunkBytes);
          mbar_expect_tx(bar, kChunkBytes);
          const int y = sh->o0 + j * kTile;
          if (c < KC)
            tma_load_2d(dst, &a.tk, h * DK + c * 64, y, bar);
          else
            tma_load_2d(dst, &a.tv, h * DV + (c - KC) * 64, y, bar);
        }
      }
      for (int i = max(0, n - NS); i < n; ++i)   // (an abort may leave copies in flight)
        drain_bar(smem_u32(&sh->full[i % NS]), (i / NS) & 1, a.wait_ns);
    }
   } else if (warp <= NW) {
    // ------------------------------------------------------------ MMA issuers
    const int i = warp - 1, mine = i ? cnt[1] : cnt[0];
    const uint32_t ids = idesc_16(F16, kTile, kTile, false, false);
    const uint32_t ido = idesc_16(F16, kTile, DV, false, true);
    const uint32_t ido64 = idesc_16(F16, kTile, 64, false, true);
    const uint64_t dq = desc_kmajor(smem_u32(Qs)) + desc_step(i * kQBytes), dr = desc_kmajor(smem_u32(ring));
    const uint64_t dv = desc_mnmajor(smem_u32(ring), kChunkBytes);
    const uint32_t sd = tmem + i * 128, od = tmem + NW * 128 + i * 128;
    auto wait_chunk = [&](int n) { return wait_bar_warp(smem_u32(&sh->full[n % NS]), (n / NS) & 1, wc); };
    // The row tiles take turns at O += P V, S = Q K^T: one's softmax then falls
    // into the other's MMAs, where side by side both would wait and work together.
    auto my_turn = [&](int jj) -> bool {
      return NW == 1 || (i == 0 && jj == 0) || wait_bar_warp(smem_u32(&sh->turn[i]), (jj + i - 1) & 1, wc);
    };
    auto pass_turn = [&]() {
      if (NW == 2 && lane == 0) mbar_arrive(smem_u32(&sh->turn[i ^ 1]));
    };
    // S against K tile jj.
    auto issue_s = [&](int jj) -> bool {
      const int n = jj * (KC + VC);
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        if (!wait_chunk(n + c)) return false;
        tc_fence_after();
        const uint64_t qa = dq + desc_step(c * kChunkBytes), ka = dr + desc_step(((n + c) % NS) * kChunkBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_ss(sd, qa + desc_step(kk * 32), ka + desc_step(kk * 32), ids, c | kk);
      }
      mma_commit(smem_u32(&sh->sfull[i]));
#pragma unroll
      for (int c = 0; c < KC; ++c) mma_commit(smem_u32(&sh->empty[(n + c) % NS]));
      return true;
    };
    // O += P V for V tile jj.
    auto issue_o = [&](int jj) -> bool {
      const int n = jj * (KC + VC) + KC;
#pragma unroll
      for (int c = 0; c < VC; ++c)
        if (!wait_chunk(n + c)) return false;
      const int rows = kv_end - (lo + jj) * kTile;
      if (rows < kTile) {   // the cache's last tile (each row tile's issuer writes the same zeros)
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          uint4* p = reinterpret_cast<uint4*>(ring + ((n + c) % NS) * kChunkBytes + rows * 128);
          for (int x = lane; x < (kTile - rows) * 8; x += 32) p[x] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
      }
      const int s0 = n % NS, s1 = (n + VC - 1) % NS;
#pragma unroll
      for (int half = 0; half < 2; ++half) {           // P comes in two halves of 64 positions
        if (!wait_bar_warp(smem_u32(&sh->pready[i][half]), jj & 1, wc)) return false;
        if (half == 0 && !my_turn(jj)) return false;
        tc_fence_after();
        if (VC == 1 || s1 > s0) {
#pragma unroll
          for (int kk = half * 4; kk < half * 4 + 4; ++kk)
            mma_ts(od, sd + kk * 8, dv + desc_step(s0 * kChunkBytes + kk * 2048), ido, jj | kk);
        } else {   // the tile's second chunk wrapped round the ring
#pragma unroll
          for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int kk = half * 4; kk < half * 4 + 4; ++kk)
              mma_ts(od + c * 64, sd + kk * 8, dv + desc_step((c ? s1 : s0) * kChunkBytes + kk * 2048), ido64, jj | kk);
        }
      }
      if (jj == mine - 1) mma_commit(smem_u32(&sh->ofull[i]));
#pragma unroll
      for (int c = 0; c < VC; ++c) mma_commit(smem_u32(&sh->empty[(n + c) % NS]));
      return true;
    };
    bool ok = mine == 0 || issue_s(0);
    for (int jj = 0; jj < mine && ok; ++jj) {
      ok = issue_o(jj);
      if (ok && jj + 1 < mine) ok = issue_s(jj + 1);
      pass_turn();
    }
    // Tiles past this row tile's last one are given back unread.
    for (int jj = mine; jj < steps && ok; ++jj) {
      for (int n = jj * (KC + VC); n < (jj + 1) * (KC + VC) && ok; ++n) {
        ok = wait_chunk(n);
        if (ok && lane == 0) mbar_arrive(smem_u32(&sh->empty[n % NS]));
      }
      ok = ok && my_turn(jj);
      pass_turn();
    }
    if (mine > 0) {   // every MMA and commit has landed
      mma_commit(smem_u32(&sh->done[i]));
      drain_bar(smem_u32(&sh->done[i]), 0, a.wait_ns);
    }
   }
  } else {
    // ------------------------------------------------------------ softmax
    regs_up<NW == 1 ? 200 : 224>();
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t st = lane_base + w * 128, ot = lane_base + NW * 128 + w * 128;
    const bool any = __any_sync(0xffffffffu, valid);
    const int mylen = valid ? len : kv_end;      // rows of the tile that hold nothing need no mask
    const int mine = w ? cnt[1] : cnt[0];
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int jj = 0; jj < mine; ++jj) {
      if (!(ok = wait_bar_warp(smem_u32(&sh->sfull[w]), jj & 1, wc))) break;
      tc_fence_after();
      if (any) {
        uint32_t v[128];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32(st + x * 32, v + x * 32);
        tmem_wait_ld();
        const int left = mylen - (lo + jj) * kTile;   // columns this row sees
        if (__any_sync(0xffffffffu, left < kTile)) {
#pragma unroll
          for (int x = 0; x < 128; ++x)
            if (x >= left) v[x] = 0xff800000u;
        }
        float t[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) t[x] = __uint_as_float(v[x]);
#pragma unroll
        for (int x = 4; x < 124; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) t[y] = max3(t[y], __uint_as_float(v[x + y]), __uint_as_float(v[x + 4 + y]));
#pragma unroll
        for (int x = 0; x < 4; ++x) t[x] = fmaxf(t[x], __uint_as_float(v[124 + x]));
        const float mn = fmaxf(max3(m, t[0], t[1]), fmaxf(t[2], t[3]));
        if (jj == 0) {
          m = mn;
        } else if (__any_sync(0xffffffffu, (mn - m) * a.c > 8.f)) {
          // S of this tile was issued after O += P V of the previous one, so O is still.
          const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * a.c);
          m = mn;
          l *= f;
#pragma unroll
          for (int x = 0; x < DV; x += 32) {
            uint32_t o[32];
            tmem_ld32(ot + x, o);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            tmem_st32(ot + x, o);
          }
        }
        const float mc = m == -INFINITY ? 0.f : m * a.c;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // P in two halves: the first one's product starts meanwhile
#pragma unroll
          for (int x = half * 64; x < half * 64 + 64; x += 2) {
            const float2 e = fma2(make_float2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), make_float2(a.c, a.c),
                                  make_float2(-mc, -mc));
            const float2 p = make_float2(ex2(e.x), ex2(e.y));
            sum[(x >> 1) & 1] = add2(sum[(x >> 1) & 1], p);
            v[x >> 1] = pack16<F16>(p.x, p.y);
          }
          tmem_st32(st + half * 32, v + half * 32);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->pready[w][half]));
        }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh->pready[w][0]));
          mbar_arrive(smem_u32(&sh->pready[w][1]));
        }
      }
    }
    if (mine > 0 && ok) ok = wait_bar_warp(smem_u32(&sh->ofull[w]), 0, wc);
    tc_fence_after();
    if (ok && any) {
      const int64_t rh = (int64_t)row * a.H_q + head;
      const bool some = mine > 0 && l != 0.f;
      if (a.splits > 1) {
        if (valid) a.ml[rh * a.splits + split] = make_float2(m * a.c, some ? l : 0.f);
        if (__any_sync(0xffffffffu, some)) {
#pragma unroll
          for (int x = 0; x < DV; x += 32) {
            uint32_t o[32];
            tmem_ld32(ot + x, o);
            tmem_wait_ld();
            if (valid && some) {
              uint4* dst = reinterpret_cast<uint4*>(a.part + (rh * a.splits + split) * DV + x);
#pragma unroll
              for (int y = 0; y < 8; ++y) dst[y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            }
          }
        }
      } else {
        // A row of NaN (l is NaN) keeps it; a row that sees nothing gets zeros.
        const bool empty = mine == 0 || l == 0.f;
        const float inv = empty ? 0.f : 1.f / l;
        if (valid && a.lse) a.lse[rh] = empty ? -INFINITY : m * a.scale + logf(l);
#pragma unroll
        for (int x = 0; x < DV; x += 32) {
          uint32_t o[32];
          tmem_ld32(ot + x, o);
          tmem_wait_ld();
          uint32_t q[16];
#pragma unroll
          for (int y = 0; y < 16; ++y)
            q[y] = empty ? 0u : pack16<F16>(__uint_as_float(o[2 * y]) * inv, __uint_as_float(o[2 * y + 1]) * inv);
          if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + rh * DV + x);
#pragma unroll
            for (int y = 0; y < 4; ++y) dst[y] = make_uint4(q[4 * y], q[4 * y + 1], q[4 * y + 2], q[4 * y + 3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kCols);
}

// Joins the parts of each (row, head): one warp each.
template <int DV, bool F16>
__global__ void __launch_bounds__(256) dense_join_kernel(const float* part, const float2* ml, uint16_t* out, float* lse,
                                                         const int32_t* row_offsets, int R, int B, int H_q, int splits) {
  const int lane = threadIdx.x & 31;
  const int64_t rh = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (rh >= (int64_t)R * H_q) return;
  const int row = (int)(rh / H_q);
  pdl_wait();
  if (B > 1 && (row < row_offsets[0] || row >= row_offsets[B])) return;
  float M = -INFINITY;
  for (int i = lane; i < splits; i += 32) {
    const float2 v = ml[rh * splits + i];
    if (v.y != 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  constexpr int E = DV / 32;
  float acc[E] = {}, L = 0.f;
  bool any = false;
  for (int i = 0; i < splits; ++i) {
    const float2 v = ml[rh * splits + i];
    if (v.y == 0.f) continue;
    any = true;
    const float f = ex2(v.x - M);
    L += f * v.y;
    const float* p = part + (rh * splits + i) * DV + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, p[e], acc[e]);
  }
  const float inv = any ? 1.f / L : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(out + rh * DV + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack16<F16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lse && lane == 0) lse[rh] = any ? M * 0.693147180559945309f + logf(L) : -INFINITY;
}

template <int DK, int DV, int NW, bool F16>
cudaError_t launch_one(const DenseArgs& a, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DK, DV, NW>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  auto kernel = dense_attn_kernel<DK, DV, NW, F16>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)a.tiles * a.splits * a.H_kv;
  kernel<<<(unsigned)grid, 128 + 128 * NW, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.R * a.H_q;
  return launch_pdl(dense_join_kernel<DV, F16>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, (const float*)a.part,
                    (const float2*)a.ml, a.out, a.lse, a.row_offsets, a.R, a.B, a.H_q, a.splits);
}

template <int DK, int DV>
cudaError_t launch_width(const DenseArgs& a, int nw, bool f16, cudaStream_t st) {
  if (nw == 1) return f16 ? launch_one<DK, DV, 1, true>(a, st) : launch_one<DK, DV, 1, false>(a, st);
  return f16 ? launch_one<DK, DV, 2, true>(a, st) : launch_one<DK, DV, 2, false>(a, st);
}

}  // namespace

DenseShape dense_shape(const dsa_dense_problem& p) {
  DenseShape s;
  const int64_t G = p.H_q / p.H_kv;
  const int64_t most = p.rows_max > 0 ? p.rows_max : p.R;
  s.nw = most * G <= kTile ? 1 : 2;
  const int64_t per = (int64_t)s.nw * kTile;
  int64_t tiles = p.B * ((most * G + per - 1) / per);
  tiles = tiles < p.R * G / per + p.B ? tiles : p.R * G / per + p.B;
  s.tiles = (int)tiles;
  // Parts per row tile: enough CTAs for two waves of the resident ones, none
  // with less than two K/V tiles.
  const int64_t items = tiles * p.H_kv, slots = s.nw == 1 ? 304 : 152;
  const int64_t kvt = (p.L_max + kTile - 1) / kTile;
  int64_t splits = 1;
  if (items > 0 && items < 2 * slots) splits = p.B == 1 ? slots / items : (2 * slots + items - 1) / items;
  const int64_t cap = kvt / 2 < 64 ? kvt / 2 : 64;
  if (splits > cap) splits = cap;
  s.splits = splits < 1 ? 1 : (int)splits;
  return s;
}

cudaError_t launch_dense(const dsa_dense_problem& p, const DenseShape& s, uint16_t* out, float* lse, float* part,
                         float* ml, uint32_t* status, cudaStream_t st) {
  DenseArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = p.q; a.offsets = p.offsets; a.row_offsets = p.row_offsets; a.row_len = p.row_len;
  a.out = out; a.lse = lse; a.part = part; a.ml = reinterpret_cast<float2*>(ml);
  a.status = status;
  a.q_stride = p.q_stride ? p.q_stride : (int64_t)p.H_q * p.D_k;
  a.wait_ns = kDefaultWaitNs;
  a.R = p.R; a.B = p.B; a.H_q = p.H_q; a.H_kv = p.H_kv; a.G = p.H_q / p.H_kv; a.L_total = (int)p.L_total;
  a.splits = s.splits; a.tiles = s.tiles;
  a.scale = p.softmax_scale;
  a.c = (float)(p.softmax_scale * 1.4426950408889634);
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
