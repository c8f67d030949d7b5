// Dense attention over a packed K/V cache with grouped heads (dsa_dense_attn).
//
// Mathematics.  One pass over a row's visible positions in tiles of 128, with a
// running maximum m and sum l per row (base-2 domain, c = scale * log2 e):
//   m' = max(m, max_t s_t),  p_t = 2^(c s_t - c m'),
//   l = l 2^(c m - c m') + sum p_t,   O = O 2^(c m - c m') + P V,
// and out = O / l, lse = scale * m + ln l.  m only has to be near the maximum:
// O and l are rescaled when the maximum has grown by more than 2^8, which after a
// row's first tiles hardly ever happens.  bf16 holds p as exactly whatever its size.
// fp16 does not: there p is 2^7 times as large (at most 2^15; its range ends at 2^16),
// so that weights down to 2^-21 of the largest keep their 11 bits and smaller ones are off by
// 2^-32 of it.  A tail of 10^5 positions 2^-25 below the peak counts (it vanished without).
//
// Rows.  The G = H_q / H_kv query heads of one K/V head and the rows of one
// request are packed into one axis (packed row = row * G + head in group), so a
// tile of 128 packed rows reads each K/V tile once for all of them: whole
// prompts and single tokens of grouped heads run the same kernel.
//
// An item is NW tiles of 128 packed rows (NW = 2 for prompts, 1 where no request
// has more than one tile), one K/V head and a range of K/V tiles.  CTAs are
// persistent (one per SM with NW = 2, two with NW = 1) and take items from a
// counter, so that an item's loads and first MMAs run under the last one's end:
//   warp 0      producer: Q, and K and V tiles through one ring of 16 KB chunks of
//               64 columns, in the order the MMAs use them, by TMA (the second row
//               tile's Q behind the first K tile: the first one starts meanwhile)
//   warps 1..   one per row tile issues its MMAs: S = Q K^T (both operands in shared
//               memory) and O += P V (P in tensor memory, over the S it came from, in
//               two halves, so that the product starts while the second is computed).
//               The tensor core takes few MMAs ahead, so an issuer that waits leaves
//               it idle; with two, the other row tile's go on.
//   warp 3      scheduler: takes items, finds their request, positions and lengths
//   warps 4..   softmax, four warps to a row tile: a thread holds one row of S
// Registers are dealt with setmaxnreg: 56 to warps 0-3, 224 (200) to the softmax.
// With two row tiles the tensor core works on one while the other's softmax
// runs; with one, two CTAs share an SM and alternate.
//
// Bounds.  Prompts: the tensor core's rate, 2 (D_k + D_v) flops per visible
// pair and head; measured 1.58 PFLOP/s for 16384 tokens of 16 heads over 2
// (693 us, 84% of the cuBLAS burst rate and 93% of the sustained one), where a tile's
// softmax and the hand-overs between it and the MMAs are what the other row tile does
// not cover.  Short prompts: an item's start and end cost about 4 us of loads, fill and
// epilogue, so ragged prompts of up to 2048 tokens and width 192, whose Q leaves
// the ring only 1.6 tiles, reach 1.06 PFLOP/s (234 us).  Two threads to a row of S,
// with its maximum exchanged through shared memory, halve the softmax's work per
// thread but took longer (837 us for the 16384 tokens).  Single tokens: reading K and V
// once; 6.2 TB/s for 32 requests of up to 32768 positions (256 us, 91% of the copy rate).
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
// The softmax weights are held as 2^lift of them.
template <bool F16>
constexpr float kLift = F16 ? 7.f : 0.f;

struct DenseArgs {
  CUtensorMap tq, tk, tv;
  const uint16_t* q;
  const int32_t* offsets;
  const int32_t* row_offsets;
  const int32_t* row_len;
  uint16_t* out;
  float* lse;
  float* part;      // [R * H_q, splits, D_v] (tail: [rows of the tail's tiles, tail_parts, D_v])
  float2* ml;       // the same without D_v: (c m - lift, l)
  uint32_t* status;
  uint32_t* next;   // items taken beyond the grid (zeroed with the status)
  uint32_t* bits;   // status bits of each CTA, joined with the parts; or null: the status is cleared before, and raised
  int64_t q_stride;
  uint64_t wait_ns;
  int R, B, H_q, H_kv, G, L_total, splits, tiles;
  int full, tail_parts;   // tail_parts > 1: items from `full` on come in that many parts
  int test_no_load;       // test hook: arm the first chunk, issue no copy
  int q_tma;        // Q tiles by TMA (the group divides a tile), else by the softmax warps
  float scale, c;   // c = scale * log2 e
};

struct Item {
  int rows, r0, t0, h;   // rows = 0: no more items.  Packed rows and first row of the request; first packed row here
  int o0, len;           // the request's positions
  int split, parts;      // part of the item's positions
  int slot;              // its rows among the tail's, or -1
  int lo, steps;         // K/V tiles of this part
  int cnt[2];            // of them, those each row tile needs
  int kv_end;            // positions past it are seen by no row of the item
};

constexpr int kBlocks = 64;   // request blocks of the lookup table

struct __align__(16) Shared {
  uint64_t full[16], empty[16];   // ring of chunks
  uint64_t sfull[2], pready[2][2], ofull[2], ofree[2], qfull[2], qempty[2], done[2];
  uint64_t ifull[2], ifree[2], inext;   // items
  uint32_t tmem;
  int abort;
  uint32_t bits;                  // status bits, where the join collects them
  volatile int steps[2];          // K/V tiles that each row tile's issuer is through with
  Item item[2];
  int first[kBlocks + 1];         // row tiles before each block of requests
};

template <int DK, int DV, int NW>
__host__ __device__ constexpr int ring_slots() {
  constexpr int budget = (NW == 1 ? 113 : 227) * 1024 - (int)sizeof(Shared);
  constexpr int s = (budget - NW * kTile * DK * 2) / (int)kChunkBytes;
  return s < 16 ? s : 16;
}
template <int DK, int DV, int NW>
__host__ __device__ constexpr size_t smem_bytes() {
  return (size_t)NW * kTile * DK * 2 + (size_t)ring_slots<DK, DV, NW>() * kChunkBytes + sizeof(Shared);
}

__host__ __device__ __forceinline__ uint32_t item_count(const DenseArgs& a) {   // (below 2^31: dense_shape)
  const uint32_t all = (uint32_t)a.tiles * a.splits * a.H_kv;
  return a.tail_parts > 1 ? a.full + (all - a.full) * a.tail_parts : all;
}

// Request b's rows, clamped to the call's.
__device__ __forceinline__ void request_rows(const DenseArgs& a, int b, int& r0, int& n) {
  const int x0 = a.row_offsets[b], x1 = a.row_offsets[b + 1];
  r0 = min(max(x0, 0), a.R);
  n = max(min(x1, a.R) - r0, 0);
}

// Request b's positions, clamped to the call's.
__device__ __forceinline__ void request_cache(const DenseArgs& a, int b, int& o0, int& len) {
  const int y0 = a.offsets[b], y1 = a.offsets[b + 1];
  o0 = min(max(y0, 0), a.L_total);
  len = max(min(y1, a.L_total) - o0, 0);
}

// Up to kBlocks requests, held by the scheduler's lanes (lane, lane + 32): between
// items, dependent loads are what the next one's first MMA waits for.
struct Requests {
  int r0[2], n[2], o0[2], len[2];
  __device__ __forceinline__ void load(const DenseArgs& a, int lane) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      r0[x] = n[x] = o0[x] = len[x] = 0;
      const int b = lane + 32 * x;
      if (a.B > kBlocks || b >= a.B) continue;
      request_rows(a, b, r0[x], n[x]);
      request_cache(a, b, o0[x], len[x]);
    }
  }
};

// Item `idx` (one warp).  Row tiles are numbered over the requests; the last ones
// (a causal prompt's longest) come first, K/V heads and parts vary fastest.
template <int NW>
__device__ void find_item(const DenseArgs& a, uint32_t idx, Shared* sh, Item* it, int lane, const Requests& rq,
                          uint32_t* status) {
  int parts = a.splits, split = 0, slot = -1;
  if (a.tail_parts > 1 && idx >= (uint32_t)a.full) {
    const uint32_t j = idx - a.full, q = j / (uint32_t)a.tail_parts;
    parts = a.tail_parts;
    split = (int)(j - q * parts);
    slot = (int)q * NW * kTile;
    idx = a.full + q;
  }
  const uint32_t hs = idx / (uint32_t)a.H_kv, ts = hs / (uint32_t)a.splits;
  const int h = (int)(idx - hs * a.H_kv);
  if (slot < 0) split = (int)(hs - ts * a.splits);
  const int want = sh->first[kBlocks] - 1 - (int)ts;
  if (want < 0) {
    if (lane == 0) it->rows = 0;
    return;
  }
  // The block of requests, then the request in it.
  const int per = (a.B + kBlocks - 1) / kBlocks;
  const int blk = __popc(__ballot_sync(0xffffffffu, sh->first[lane + 1] <= want)) +
                  __popc(__ballot_sync(0xffffffffu, sh->first[lane + 33] <= want));
  int run = sh->first[blk], r0 = 0, n = 0, tile = 0, o0 = 0, len = 0;
  if (per == 1) {
    tile = want - run;
    r0 = __shfl_sync(0xffffffffu, blk < 32 ? rq.r0[0] : rq.r0[1], blk & 31);
    n = __shfl_sync(0xffffffffu, blk < 32 ? rq.n[0] : rq.n[1], blk & 31);
    o0 = __shfl_sync(0xffffffffu, blk < 32 ? rq.o0[0] : rq.o0[1], blk & 31);
    len = __shfl_sync(0xffffffffu, blk < 32 ? rq.len[0] : rq.len[1], blk & 31);
  } else {
    int b = 0;
    for (int base = blk * per; base < (blk + 1) * per; base += 32) {
      int x0 = 0, xn = 0;
      if (base + lane < (blk + 1) * per && base + lane < a.B) request_rows(a, base + lane, x0, xn);
      const int v = (xn * a.G + NW * kTile - 1) / (NW * kTile);
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const int at = run + incl - v;
      const uint32_t hit = __ballot_sync(0xffffffffu, want >= at && want < at + v);
      run += __shfl_sync(0xffffffffu, incl, 31);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = base + src;
        r0 = __shfl_sync(0xffffffffu, x0, src);
        n = __shfl_sync(0xffffffffu, xn, src);
        tile = want - __shfl_sync(0xffffffffu, at, src);
        break;
      }
    }
    request_cache(a, b, o0, len);
  }
  const int rows = n * a.G, t0 = tile * NW * kTile;
  // The farthest position each row tile sees: at most 128 lengths each, loaded together.
  int end[2] = {0, 0}, l[NW][kTile / 32];
  bool bad = false;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int x0 = t0 + w * kTile, x1 = min(x0 + kTile, rows), first = x0 / a.G + lane;
#pragma unroll
    for (int u = 0; u < kTile / 32; ++u) l[w][u] = (first + 32 * u) * a.G < x1 ? a.row_len[r0 + first + 32 * u] : 0;
  }
#pragma unroll
  for (int w = 0; w < NW; ++w) {
#pragma unroll
    for (int u = 0; u < kTile / 32; ++u) {
      bad |= l[w][u] < 0 || l[w][u] > len;
      end[w] = max(end[w], min(max(l[w][u], 0), len));
    }
    end[w] = __reduce_max_sync(0xffffffffu, end[w]);
  }
  if (bad && split == 0 && h == 0) raise_status(status, DSA_DEVICE_BAD_INDEX);
  if (lane == 0) {
    const int kv_end = max(end[0], end[1]);
    const int nt = (kv_end + kTile - 1) / kTile;
    const int lo = (int)((int64_t)nt * split / parts), hi = (int)((int64_t)nt * (split + 1) / parts);
    it->rows = rows;
    it->r0 = r0;
    it->t0 = t0;
    it->h = h;
    it->o0 = o0;
    it->len = len;
    it->split = split;
    it->parts = parts;
    it->slot = slot;
    it->lo = lo;
    it->steps = hi - lo;
    for (int w = 0; w < 2; ++w) it->cnt[w] = max(min((end[w] + kTile - 1) / kTile, hi) - lo, 0);
    it->kv_end = kv_end;
  }
}

// Lane i of four adjacent ones holds four 16-byte pieces of row i; afterwards piece i of
// the four rows.
__device__ __forceinline__ void exchange4(uint32_t* p, int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & bit) continue;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t &lo = p[4 * k + y], &hi = p[4 * (k | bit) + y];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
        lo = up ? got : lo;
        hi = up ? hi : got;
      }
    }
  }
}

template <int DK, int DV, int NW, bool F16>
__global__ void __launch_bounds__(128 + 128 * NW, NW == 1 ? 2 : 1)
    dense_attn_kernel(const __grid_constant__ DenseArgs a) {
  constexpr int NS = ring_slots<DK, DV, NW>();
  constexpr int KC = DK / 64, VC = DV / 64;
  constexpr uint32_t kQBytes = kTile * DK * 2;
  constexpr uint32_t kCols = NW * 256;      // S of each row tile, then O of each
  constexpr int kReaders = 1 + NW + 4 * NW; // warps that read an item
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* Qs = smem;
  unsigned char* ring = smem + NW * kQBytes;
  Shared* sh = reinterpret_cast<Shared*>(ring + NS * kChunkBytes);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (smem_u32(smem) & 1023) {   // (the swizzle's atoms)
    if (tid == 0) {
      if (a.bits)
        a.bits[blockIdx.x] = DSA_DEVICE_CAPACITY;
      else
        raise_status(a.status, DSA_DEVICE_CAPACITY);
    }
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(sh->full[i]), 1);
      mbar_init(bar(sh->empty[i]), NW);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh->sfull[i]), 1);
      mbar_init(bar(sh->pready[i][0]), 4);
      mbar_init(bar(sh->pready[i][1]), 4);
      mbar_init(bar(sh->ofull[i]), 1);
      mbar_init(bar(sh->ofree[i]), 4);
      mbar_init(bar(sh->qfull[i]), a.q_tma ? 1 : 4);
      mbar_init(bar(sh->qempty[i]), 1);
      mbar_init(bar(sh->done[i]), 1);
      mbar_init(bar(sh->ifull[i]), 1);
      mbar_init(bar(sh->ifree[i]), kReaders);
    }
    mbar_init(bar(sh->inext), 1);
    sh->abort = 0;
    sh->bits = 0;
    sh->steps[0] = sh->steps[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(smem_u32(&sh->tmem), kCols);
  if (a.bits) pdl_wait();   // (the call's first kernel: its inputs may only just be written)
  pdl_trigger();   // (the join, if any, may take its place; it waits for this grid's end)
  // Row tiles before each block of requests: one request to a block, or counted by
  // all threads.
  auto row_tiles = [&](int b) {
    int r0, n;
    request_rows(a, b, r0, n);
    return (n * a.G + NW * kTile - 1) / (NW * kTile);
  };
  if (a.B > kBlocks) {
    const int per = (a.B + kBlocks - 1) / kBlocks;
    if (tid <= kBlocks) sh->first[tid] = 0;
    __syncthreads();
    for (int b = tid; b < a.B; b += blockDim.x) atomicAdd(&sh->first[b / per], row_tiles(b));
    __syncthreads();
  }
  if (warp == 2) {
    int run = 0;
    for (int half = 0; half < 2; ++half) {
      const int blk = half * 32 + lane;
      const int v = a.B > kBlocks ? sh->first[blk] : (blk < a.B ? row_tiles(blk) : 0);
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      sh->first[blk] = run + incl - v;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) sh->first[kBlocks] = run;
  }
  Requests rq;
  if (warp == 3) rq.load(a, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0);
  uint32_t* const status = a.bits ? &sh->bits : a.status;
  const WaitCtx wc(&sh->abort, status, a.wait_ns);
  // Item k of this CTA; whoever has read what it needs gives the slot back.
  auto item_wait = [&](int k) { return wait_bar_warp(bar(sh->ifull[k & 1]), (k >> 1) & 1, wc); };
  auto item_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(sh->ifree[k & 1]));
  };

  if (warp < 4) {
   regs_down<56>();
   if (warp == 3) {
    // ------------------------------------------------------------ scheduler
    pdl_wait();              // (the status block and the counter are cleared)
    // The launch was sized by the declared rows: later tiles come first in the
    // numbering, so those past it are the first requests' and are not computed.
    if (lane == 0 && sh->first[kBlocks] > a.tiles) raise_status(status, DSA_DEVICE_CAPACITY);
    WaitCtx item_wc = wc;   // an item may take long: a thousand times the limit, or until another role gives up
    item_wc.tries *= 1000;
    uint32_t idx;
    const uint32_t items = item_count(a);
    for (int k = 0;; ++k) {
      // Not before the producer nears the end of the last one: an item taken early
      // is one that no idle CTA can take.
      if (k >= 1 && !wait_bar_warp(bar(sh->inext), (k - 1) & 1, item_wc)) break;
      if (k == 0) {
        idx = blockIdx.x;
      } else {
        uint32_t t = 0;
        if (lane == 0 && gridDim.x < items) t = atomicAdd(a.next, 1u);
        idx = gridDim.x + __shfl_sync(0xffffffffu, t, 0);
      }
      if (k >= 2 && !wait_bar_warp(bar(sh->ifree[k & 1]), ((k >> 1) - 1) & 1, wc)) break;
      Item* it = &sh->item[k & 1];
      if (idx < items)
        find_item<NW>(a, idx, sh, it, lane, rq, status);
      else if (lane == 0)
        it->rows = 0;
      __syncwarp();
      const int rows = __shfl_sync(0xffffffffu, it->rows, 0);
      if (lane == 0) mbar_arrive(bar(sh->ifull[k & 1]));
      if (rows == 0) break;
    }
   } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    // K/V tiles before an item's end at which the next one is taken: looking it up takes
    // 2000 to 4000 cycles, and a longer lead takes it from a CTA that would be free (32
    // single tokens 254 us with two, 257 with four, 258 with six; prompts alike).
    constexpr int early = NW == 1 ? 2 : 4;
    int n = 0, nq[2] = {0, 0};   // chunks and Q tiles asked for
    bool ok = true;
    for (int k = 0; ok && item_wait(k); ++k) {
      const Item it = sh->item[k & 1];
      item_done(k);
      if (it.rows == 0) break;
      if (lane == 0) {
        auto load_q = [&](int w) {
          if (!a.q_tma || !ok || (w ? it.cnt[1] : it.cnt[0]) == 0) return;
          int& q = w ? nq[1] : nq[0];
          if (q > 0 && !(ok = wait_bar(bar(sh->qempty[w]), (q - 1) & 1, wc))) return;
          mbar_expect_tx(bar(sh->qfull[w]), kQBytes);
          const int row = it.r0 + (it.t0 + w * kTile) / a.G;
          for (int c = 0; c < KC; ++c)
            tma_load_3d(smem_u32(Qs) + w * kQBytes + c * kChunkBytes, &a.tq, c * 64, it.h * a.G, row, bar(sh->qfull[w]));
          ++q;
        };
        load_q(0);
        if (it.steps == 0) mbar_arrive(bar(sh->inext));
        for (int j = 0; j < it.steps && ok; ++j) {
          if (j == max(it.steps - early, 0)) mbar_arrive(bar(sh->inext));
          for (int c = 0; c < KC + VC; ++c, ++n) {
            if (NW == 2 && j == 0 && c == KC) {   // (row tile 0 starts with what is asked for by now)
              load_q(1);
              if (!ok) break;
            }
            const int s = n % NS;
            if (n >= NS && !(ok = wait_bar(bar(sh->empty[s]), (n / NS - 1) & 1, wc))) break;
            const uint32_t b = bar(sh->full[s]), dst = smem_u32(ring + s * kChunkBytes);
            mbar_expect_tx(b, kChunkBytes);
            const int y = it.o0 + (it.lo + j) * kTile;
            if (a.test_no_load && n == 0) continue;
            if (c < KC)
              tma_load_2d(dst, &a.tk, it.h * DK + c * 64, y, b);
            else
              tma_load_2d(dst, &a.tv, it.h * DV + (c - KC) * 64, y, b);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0);
    }
    if (lane == 0) {   // (an abort may leave copies in flight)
      for (int i = max(0, n - NS); i < n; ++i) drain_bar(bar(sh->full[i % NS]), (i / NS) & 1, a.wait_ns);
      for (int w = 0; w < NW; ++w)
        if (nq[w] > 0) drain_bar(bar(sh->qfull[w]), (nq[w] - 1) & 1, a.wait_ns);
    }
   } else if (warp <= NW) {
    // ------------------------------------------------------------ MMA issuers
    const int i = warp - 1;
    const uint32_t ids = idesc_16(F16, kTile, kTile, false, false);
    const uint32_t ido = idesc_16(F16, kTile, DV, false, true);
    const uint32_t ido64 = idesc_16(F16, kTile, 64, false, true);
    const uint64_t dq = desc_kmajor(smem_u32(Qs)) + desc_step(i * kQBytes), dr = desc_kmajor(smem_u32(ring));
    const uint64_t dv = desc_mnmajor(smem_u32(ring), kChunkBytes);
    const uint32_t sd = tmem + i * 128, od = tmem + NW * 128 + i * 128;
    int n = 0;              // first chunk of the current K/V tile
    int tiles = 0;          // S tiles issued (the softmax's count)
    int used = 0;           // items that had tiles for this row tile
    int turns = 0;          // K/V tiles this issuer is through with
    bool ok = true;
    auto wait_chunk = [&](int m) { return wait_bar_warp(bar(sh->full[m % NS]), (m / NS) & 1, wc); };
    // The row tiles take turns at O += P V, S = Q K^T: one's softmax then falls
    // into the other's MMAs, where side by side both would wait and work together.
    // Tile t waits for the other issuer to be through with tile t - 1 (the second
    // row tile's: with tile t).
    auto my_turn = [&]() -> bool {
      if (NW == 1) return true;
      uint64_t t0 = 0;
      for (uint32_t x = 1; sh->steps[i ^ 1] < turns + i; ++x) {
        if (x % 1024) continue;
        if (!t0) t0 = gtimer();
        if (*wc.abort_flag) return false;
        if (gtimer() - t0 > a.wait_ns) {
          raise_status(status, DSA_DEVICE_TIMEOUT);
          *wc.abort_flag = 1;
          return false;
        }
      }
      return true;
    };
    auto pass_turn = [&]() {
      ++turns;
      if (NW == 2 && lane == 0) sh->steps[i] = turns;
    };
    // S against the K tile whose first chunk is m; `last` of its item.
    auto issue_s = [&](int m, bool last) -> bool {
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        if (!wait_chunk(m + c)) return false;
        tc_fence_after();
        const uint64_t qa = dq + desc_step(c * kChunkBytes), ka = dr + desc_step(((m + c) % NS) * kChunkBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_ss(sd, qa + desc_step(kk * 32), ka + desc_step(kk * 32), ids, c | kk);
      }
      mma_commit(bar(sh->sfull[i]));
#pragma unroll
      for (int c = 0; c < KC; ++c) mma_commit(bar(sh->empty[(m + c) % NS]));
      if (last) mma_commit(bar(sh->qempty[i]));
      return true;
    };
    // O += P V for the item's V tile jj, whose first chunk is m; `rows` of it are seen.
    auto issue_o = [&](int jj, int m, int rows, bool last) -> bool {
#pragma unroll
      for (int c = 0; c < VC; ++c)
        if (!wait_chunk(m + c)) return false;
      if (rows < kTile) {   // the cache's last tile (each row tile's issuer writes the same zeros)
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          uint4* p = reinterpret_cast<uint4*>(ring + ((m + c) % NS) * kChunkBytes + rows * 128);
          for (int x = lane; x < (kTile - rows) * 8; x += 32) p[x] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
      }
      if (jj == 0 && used > 0 && !wait_bar_warp(bar(sh->ofree[i]), (used - 1) & 1, wc)) return false;
      const int s0 = m % NS, s1 = (m + VC - 1) % NS;
#pragma unroll
      for (int half = 0; half < 2; ++half) {           // P comes in two halves of 64 positions
        if (!wait_bar_warp(bar(sh->pready[i][half]), tiles & 1, wc)) return false;
        if (half == 0 && !__all_sync(0xffffffffu, my_turn())) return false;
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
      ++tiles;
      if (last) mma_commit(bar(sh->ofull[i]));
#pragma unroll
      for (int c = 0; c < VC; ++c) mma_commit(bar(sh->empty[(m + c) % NS]));
      return true;
    };
    for (int k = 0; ok && item_wait(k); ++k) {
      const Item& si = sh->item[k & 1];
      const int rows = si.rows, steps = si.steps, mine = i ? si.cnt[1] : si.cnt[0], end = si.kv_end - si.lo * kTile;
      item_done(k);
      if (rows == 0) break;
      if (mine > 0) {
        ok = wait_bar_warp(bar(sh->qfull[i]), used & 1, wc) && issue_s(n, mine == 1);
        for (int jj = 0; jj < mine && ok; ++jj) {
          ok = issue_o(jj, n + KC, end - jj * kTile, jj == mine - 1);
          n += KC + VC;
          if (ok && jj + 1 < mine) ok = issue_s(n, jj + 2 == mine);
          pass_turn();
        }
        ++used;
      }
      // Tiles past this row tile's last one are given back unread.
      for (int jj = mine; jj < steps && ok; ++jj) {
        for (int c = 0; c < KC + VC && ok; ++c, ++n) {
          ok = wait_chunk(n);
          if (ok && lane == 0) mbar_arrive(bar(sh->empty[n % NS]));
        }
        pass_turn();
      }
    }
    mma_commit(bar(sh->done[i]));   // every MMA and commit has landed
    drain_bar(bar(sh->done[i]), 0, a.wait_ns);
   }
  } else {
    // ------------------------------------------------------------ softmax
    regs_up<NW == 1 ? 200 : 224>();
    const int w = (warp >> 2) - 1;                         // row tile of this warp
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t st = lane_base + w * 128, ot = lane_base + NW * 128 + w * 128;
    int tiles = 0, used = 0;                               // S tiles taken; items with tiles
    bool ok = true;
    for (int k = 0; ok && item_wait(k); ++k) {
      const Item& si = sh->item[k & 1];
      const int rows = si.rows, t0 = si.t0 + w * kTile, r0 = si.r0, h = si.h, split = si.split, parts = si.parts, slot = si.slot;
      const int mine = w ? si.cnt[1] : si.cnt[0], lo = si.lo, kv_end = si.kv_end, reach = si.len;
      item_done(k);
      if (rows == 0) break;
      const int packed = t0 + (warp & 3) * 32 + lane;      // packed row in the request
      const bool valid = packed < rows;
      const int row = r0 + (valid ? packed / a.G : 0);
      const int head = h * a.G + (valid ? packed % a.G : 0);
      const bool any = __any_sync(0xffffffffu, valid);
      // Rows of the tile that hold nothing need no mask.
      const int mylen = valid ? min(max(a.row_len[row], 0), reach) : kv_end;
      if (!a.q_tma && mine > 0) {
        // Q, K-major and swizzled: 16-byte pieces, consecutive threads along a row.
        if (used > 0 && !(ok = wait_bar_warp(bar(sh->qempty[w]), (used - 1) & 1, wc))) break;
        constexpr int P = DK / 8;
        for (int x = tid & 127; x < kTile * P; x += 128) {
          const int r = x / P, c = x % P, pk = t0 + r;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (pk < rows)
            v = __ldg(reinterpret_cast<const uint4*>(a.q + (int64_t)(r0 + pk / a.G) * a.q_stride +
                                                     (int64_t)(h * a.G + pk % a.G) * DK) + c);
          *reinterpret_cast<uint4*>(Qs + w * kQBytes + (c >> 3) * kChunkBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->qfull[w]));
      }
      float m = -INFINITY, l = 0.f;
      for (int jj = 0; jj < mine; ++jj, ++tiles) {
        if (!(ok = wait_bar_warp(bar(sh->sfull[w]), tiles & 1, wc))) break;
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
          if (jj == 0) m = mn;
          float mc = m == -INFINITY ? 0.f : fmaf(m, a.c, -kLift<F16>);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          auto weights = [&](int half) {
#pragma unroll
            for (int x = half * 64; x < half * 64 + 64; x += 2) {
              const float2 e = fma2(make_float2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])),
                                    make_float2(a.c, a.c), make_float2(-mc, -mc));
              const float2 p = make_float2(ex2(e.x), ex2(e.y));
              sum[(x >> 1) & 1] = add2(sum[(x >> 1) & 1], p);
              v[x >> 1] = pack16<F16>(p.x, p.y);
            }
          };
          // The first half's weights do not wait for the maximum: it rarely moves the
          // scale.  Where it does, O and l are rescaled and they are computed again.
          weights(0);
          if (__any_sync(0xffffffffu, (mn - m) * a.c > 8.f)) {
            // S of this tile was issued after O += P V of the previous one, so O is still.
            const float f = mn == -INFINITY ? 1.f : ex2((m - mn) * a.c);
            m = mn;
            mc = m == -INFINITY ? 0.f : fmaf(m, a.c, -kLift<F16>);
            l *= f;
#pragma unroll 1
            for (int x = 0; x < DV; x += 32) {
              uint32_t o[32];
              tmem_ld32(ot + x, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st32(ot + x, o);
            }
            tmem_ld32(st, v);
            tmem_ld32(st + 32, v + 32);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 64; ++x)
              if (x >= left) v[x] = 0xff800000u;
            sum[0] = sum[1] = make_float2(0.f, 0.f);
            weights(0);
          }
#pragma unroll
          for (int half = 0; half < 2; ++half) {   // P in two halves: the first one's product starts meanwhile
            if (half) weights(1);
            tmem_st32(st + half * 32, v + half * 32);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sh->pready[w][half]));
          }
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(sh->pready[w][0]));
            mbar_arrive(bar(sh->pready[w][1]));
          }
        }
      }
      if (mine > 0 && ok) ok = wait_bar_warp(bar(sh->ofull[w]), used & 1, wc);
      if (!ok) break;
      tc_fence_after();
      if (any) {
        const int64_t rh = (int64_t)row * a.H_q + head;
        const bool some = mine > 0 && l != 0.f;
        const int64_t at = (slot < 0 ? rh : slot + w * kTile + (packed - t0)) * parts + split;   // its part's place
        // Written as it is into its part, or divided by l: a row of NaN (l is NaN)
        // keeps it, a row that sees nothing gets zeros.
        const float inv = some ? 1.f / l : 0.f;
        const int at_row = valid ? (int)rh : -1;   // (below 2^23: 65535 rows of 128 heads)
        if (valid && parts > 1) a.ml[at] = make_float2(fmaf(m, a.c, -kLift<F16>), some ? l : 0.f);
        if (valid && parts == 1 && a.lse) a.lse[rh] = some ? m * a.scale + logf(F16 ? l * 0x1p-7f : l) : -INFINITY;
        if (parts == 1 || __any_sync(0xffffffffu, some)) {
#pragma unroll 1
          for (int x = 0; x < DV; x += 32) {
            uint32_t o[32];
            tmem_ld32(ot + x, o);
            tmem_wait_ld();
            if (parts > 1) {
              uint4* dst = reinterpret_cast<uint4*>(a.part + at * DV + x);
              if (valid && some)
#pragma unroll
                for (int y = 0; y < 8; ++y) dst[y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            } else {
#pragma unroll
              for (int y = 0; y < 16; ++y)
                o[y] = some ? pack16<F16>(__uint_as_float(o[2 * y]) * inv, __uint_as_float(o[2 * y + 1]) * inv) : 0u;
              // Four lanes exchange their rows' 16-byte pieces, so that a store writes 64
              // bytes of a row: 8 rows to an instruction rather than 32.
              exchange4(o, lane);
              uint16_t* dst = a.out + x + (lane & 3) * 8;
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int to = __shfl_sync(0xffffffffu, at_row, (lane & 28) + y);
                if (to >= 0)
                  *reinterpret_cast<uint4*>(dst + (int64_t)to * DV) = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
              }
            }
          }
        }
      }
      if (mine > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->ofree[w]));
        ++used;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kCols);
  if (tid == 0 && a.bits) a.bits[blockIdx.x] = sh->bits;
}

// Joins the parts of each (row, head): one warp each.  Split calls have parts of
// every (row, head); the tail of others of its own rows (one request).
template <int DV, bool F16>
__global__ void __launch_bounds__(256) dense_join_kernel(const __grid_constant__ DenseArgs a, int row_tile, int ctas) {
  const int lane = threadIdx.x & 31;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  int splits = a.splits;
  int64_t rh = at;
  bool ours = true;
  if (a.tail_parts > 1) {
    splits = a.tail_parts;
    const uint32_t q = (uint32_t)(at / row_tile), id = a.full + q, ts = id / (uint32_t)a.H_kv;
    int r0, n;
    request_rows(a, 0, r0, n);
    const int tiles = (n * a.G + row_tile - 1) / row_tile;   // (numbered from the last one, as the items are)
    const int64_t packed = ((int64_t)tiles - 1 - ts) * row_tile + (at - (int64_t)q * row_tile);
    ours = id < (uint32_t)a.tiles * a.H_kv && packed >= 0 && packed < (int64_t)n * a.G;
    rh = (r0 + packed / a.G) * a.H_q + (int64_t)(id - ts * a.H_kv) * a.G + packed % a.G;
  } else {
    const int64_t row = at / a.H_q;
    ours = row < a.R && row >= a.row_offsets[0] && row < a.row_offsets[a.B];
  }
  pdl_wait();   // (by every thread: whoever waits for this grid's end waits for the parts' too)
  if (a.bits && at == 0) {
    uint32_t bits = 0;
    for (int i = lane; i < ctas; i += 32) bits |= a.bits[i];
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) *a.status = bits;
  }
  if (!ours) return;
  const float2* ml = a.ml + at * splits;
  float M = -INFINITY;
  for (int i = lane; i < splits; i += 32) {
    const float2 v = ml[i];
    if (v.y != 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  constexpr int E = DV / 32;
  float acc[E] = {}, L = 0.f;
  bool any = false;
#pragma unroll 8
  for (int i = 0; i < splits; ++i) {
    const float2 v = ml[i];
    const bool seen = v.y != 0.f;   // (a part that saw nothing has no O)
    any |= seen;
    const float f = seen ? ex2(v.x - M) : 0.f;
    L = fmaf(f, v.y, L);
    const float* p = a.part + (at * splits + i) * DV + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, seen ? p[e] : 0.f, acc[e]);
  }
  const float inv = any ? 1.f / L : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + rh * DV + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack16<F16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (a.lse && lane == 0) a.lse[rh] = any ? M * 0.693147180559945309f + logf(L) : -INFINITY;
}

template <int DK, int DV, int NW, bool F16>
cudaError_t launch_one(const DenseArgs& a, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DK, DV, NW>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  auto kernel = dense_attn_kernel<DK, DV, NW, F16>;
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

DenseShape dense_shape(const dsa_dense_problem& p) {
  DenseShape s;
  const int64_t G = p.H_q / p.H_kv;
  // The declared bounds may lie above what the call can hold.
  const int64_t most = p.rows_max > 0 && p.rows_max < p.R ? p.rows_max : p.R;
  const int64_t longest = p.L_max < p.L_total ? p.L_max : p.L_total;
  s.nw = most * G <= kTile ? 1 : 2;
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
