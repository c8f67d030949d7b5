// Attention over the 4-bit cache, few rows of a request at a time (dsa_kv4_attn).
//
// Mathematics.  K[t] = s_g (u - 8) for the codes u of group g of 64 columns, so
//   q . K[t] = sum_g s_g[t] (sum_d q_d u_d - 8 sum_d q_d),
// and with weights p_t = 2^(c q.K[t] - m):
//   sum_t p_t V[t] = sum_t (p_t s_g[t]) u - 8 sum_t (p_t s_g[t])      for the columns of group g,
// the second part taken off after every 32 positions (a product of the weights with ones).
// The codes go into the products as they are: four bits with zeros around them are the fp16
// number u 2^-24, and four bits higher up u 2^-20, so a pair of codes becomes a pair of operands
// by one AND, without a conversion.  (The tensor core cuts the addends of a sum 24 bits or so below the
// largest exponent, which for these operands is 2^-14's whatever the code: at 2^-14 of the largest weight
// times scale for V, less than its weight's own rounding.  K's codes are shifted up by
// two bits for that: a logit is then off by a tenth, at 1% of the time; lse of one position in
// fp16 1.2e-6 -> 1.4e-7 of its size.)  K's scales are applied to the logits, V's to the weights,
// both in fp32.  A query row is scaled by a power of two to fp16's upper range first (every bit
// of a bf16 query within 2^-25 of the row's largest is kept); the columns whose codes come
// 2^4 too high get a sixteenth of it.  The products are exact, their sums fp32.
//
// Softmax in one pass, base 2: the maximum m only has to be near the row's: O and l are rescaled
// when it has grown by more than 2^8.  For their product with V weights are held times V's scales
// relative to a power of two for each group of 64 columns that leaves these below 2^7, so that fp16
// holds them to 11 bits down to 2^-20 of the largest.  (With one power for both groups, one whose scales were 2^-24 of
// the other's lost bits, and at 2^-32 everything.)  The power follows the scales as they are, before they are multiplied
// by it (V may begin with zeros, and what comes next may have any scale), and it only falls.
//
// What bounds it.  Per position and K/V head (D_k + D_v) 17 / 32 bytes have to be read: 136 for
// 128 + 128, at 45 GB/s for an SM one every 5.7 cycles.  The tensor core has little to do
// (8 to 16 rows), but every code passes through a register: 5 or 6 instructions for 8
// codes, 18 mma.sync for 16 positions, 260 instructions in all with the softmax.  Dequantised tiles in shared
// memory for tcgen05 would cost the same extraction, a store and two reads of 16-bit
// operands; registers are what mma.sync takes and tcgen05 does not.  Measured: one token of 64
// heads over 8 and 307200 positions 62 us, 5.4 TB/s with the start (3.6 us until the first stage is
// there), CTAs that get less of HBM than others and end 6 us after the middle one, and the join with the next
// launch (4.5 us); twice as many positions take another 50, the copy rate.  32 ragged tokens of up to 32768
// positions 81 us in pages of 64 (5.2 TB/s), 85.3 in pages of 16, whose copies are 2 KB each.  One
// token over 4096 positions 10.6 us: a chain of launch, lengths (0.7), the share's place in the batch
// (0.8), table and first pages (1.5), two tiles of 32 positions (1 to 2), the warps' sums and parts
// (1.2), the next launch (0.7) and the join.
//
// A CTA takes 128 positions of one K/V head at a time (a stage: whole page blocks, one bulk
// copy each, through a ring).  Four of its eight warps take a stage, 32 positions each, the other
// four the next one; every warp has its own maximum, sum and O, which are joined when an item
// ends.  Each lane holds 32-bit words of codes in the layout of the products' fragments: rows of K
// are positions, and rows of V columns, so V needs two positions' codes side by side, which is
// how ldmatrix transposes 16-bit units of four codes.  A stage's place in the ring is given back
// before the softmax, with V's codes in registers.
//
// A ninth warp loads.  It shares its scheduler with the others, so its loop over stages is kept
// short (lookups a window of 32 table entries at a time); it also lays out an item's queries for
// the products, which by each warp for itself took registers that spilled.
//
// Work.  Items (request, block of packed rows, K/V head) are laid end to end in stages
// and cut into equal shares, one for each CTA, so ragged requests keep all SMs
// busy to the end.  An item cut by a share's end leaves its parts (m, l, O) in the workspace
// and kv4_join_kernel joins them, always in the same order.
//
// Tried and taken out: pages prefetched into L2 behind the ring (307200 positions 68 -> 71 to 90 us);
// parts of one stage (one token over 4096 positions 14.7 -> 13.0 without: half the warps idled);
// one warp to a row of the join (21 us for 32 parts); pages marked as the first to leave L2 (no change).
//
// All waits are bounded; on expiry the CTA stops and drains its copies.
#include "kv4.cuh"

#include <climits>
#include <cstring>

#include "tc.cuh"

namespace dsa {
namespace {

constexpr int kStage = 128;      // positions
constexpr int kWarps = 8;        // that compute; one more loads
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kBlock = 8;        // packed rows of a product's column block
constexpr int kItems = 3;        // handed over at once
// An item's start and the joining of its warps' sums take a CTA about as long as four stages, and its
// share of the work counts them (32 ragged tokens: 101 us with shares of stages alone, 90 with a cost of two
// stages, 88 with three, 87 with four, 89 with six; width 64: 67, 60, 54, 52, 52).
constexpr int kItemCost = 4;

struct Args {
  CacheArgs c;
  const uint16_t* q;
  const int32_t* row_offsets;
  const int32_t* row_len;
  uint16_t* out;
  float* lse;
  float* part;        // [2 grid, rows, D_v]
  float2* ml;         // [2 grid, rows]: (m, l)
  Kv4Join* join;      // or null: no item is split
  uint32_t* status;
  uint32_t* bits;     // status bits of each CTA, for the join; or null: the status is cleared before, and raised
  int64_t q_stride;
  uint64_t wait_ns;
  int R, H_q, G, L_max, f16;
  int test_no_load;
  float c2;           // softmax_scale * log2 e
  float inv_G;
};

struct Item {
  int row0, packed, first, h;      // packed = 0: no more items
  int len;                         // positions that the request's rows see at most
  int stage, stages;               // the range of stages of this CTA
  int slot;                        // part of the workspace, or -1: the whole item
  // Of each packed row of the block: positions it sees, what a sum of its products is to be multiplied
  // with, and the sums that 8 less in every code makes.
  int see[2 * kBlock];
  float factor[2 * kBlock], less[3][2 * kBlock];
};

struct __align__(16) Shared {
  uint64_t full[8], empty[8];
  uint64_t ifull[kItems], ifree[kItems];
  int abort;
  uint32_t bits;
  uint32_t pages[8];            // pages of each stage that the pool has
  Item item[kItems];
  int64_t units[kWarps + 1];    // of each warp's requests
  float m[kWarps][2 * kBlock], l[kWarps][2 * kBlock];
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from accumulators that two columns share.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// An 8 x 8 block of 16-bit values, lane i holding row i / 4, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void lds2(uint32_t addr, uint32_t& x, uint32_t& y) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds1(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(addr));
  return x;
}
__device__ __forceinline__ float lds_bf16(uint32_t addr) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(addr));
  return __uint_as_float((uint32_t)x << 16);
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A barrier of the computing warps that tells whether any of them says yes.
__device__ __forceinline__ bool consumers_any(bool x) {
  uint32_t y;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, 1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(y) : "r"((uint32_t)x), "n"(32 * kWarps) : "memory");
  return y != 0;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// Request b's rows, clamped to the call's.
__device__ __forceinline__ void request_rows(const Args& a, int b, int& r0, int& n) {
  const int x0 = a.row_offsets[b], x1 = a.row_offsets[b + 1];
  r0 = min(max(x0, 0), a.R);
  n = max(min(x1, a.R) - r0, 0);
}

// Rows and farthest visible position of the request that each lane names (b < B, or none), by a
// whole warp: requests of more than eight rows are read by all lanes together.  Row b's length is
// asked for beside the offsets: of a batch of single tokens it is the one.
__device__ __forceinline__ void request_info(const Args& a, int b, int reach, int lane, int& r0, int& n, int& len, bool& bad) {
  r0 = n = len = 0;
  int guess = 0;
  if (b >= 0 && b < a.c.B) {
    if (b < a.R) guess = a.row_len[b];
    request_rows(a, b, r0, n);
  }
  auto see = [&](int l) {
    bad |= l < 0 || l > reach;
    return min(max(l, 0), reach);
  };
  if (n == 1 && r0 == b)
    len = see(guess);
  else if (n <= 8)
    for (int i = 0; i < n; ++i) len = max(len, see(a.row_len[r0 + i]));
  uint32_t big = __ballot_sync(0xffffffffu, n > 8);
  while (big) {
    const int src = __ffs(big) - 1;
    big &= big - 1;
    const int x0 = __shfl_sync(0xffffffffu, r0, src), xn = __shfl_sync(0xffffffffu, n, src);
    int m = 0;
    for (int i = lane; i < xn; i += 32) m = max(m, see(a.row_len[x0 + i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == src) len = m;
  }
}

// x / y of what hardly ever passes 22 bits, x >= 0, y > 0: by the approximate inverse, off by less than one then.  (The
// divisions of the loading warp stand between the launch and the first load.)
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (x >= 1 << 22 || y >= 1 << 22) return x / y;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"((float)(int)y));
  const int q = (int)((float)(int)x * inv), rest = (int)x - q * (int)y;
  return q + (rest >= (int)y) - (rest < 0);
}
// pk / G (pk below 2^23, and the inverse within 2^-24 of it).
__device__ __forceinline__ int row_of(const Args& a, int pk) {
  const int q = (int)((float)pk * a.inv_G), rest = pk - q * a.G;
  return q + (rest >= a.G) - (rest < 0);
}

__device__ __forceinline__ int blocks_of(const Args& a, int n, int rows) { return (n * a.G + rows - 1) / rows; }
__device__ __forceinline__ int stages_of(int len) { return max((len + kStage - 1) / kStage, 1); }


template <int DK, int DV>
constexpr uint32_t kStageBytes = kStage * (DK + DV) * 17 / 32;
// Beside the ring: the queries of the items, the warps' sums and Shared.
template <int DK, int DV, int NB>
constexpr int kFixedBytes = kItems * NB * kBlock * DK * 2 + kWarps / 2 * kBlock * DV * 4 + (int)sizeof(Shared);
template <int DK, int DV, int NB>
__host__ __device__ constexpr int ring_stages() {
  constexpr int s = ((NB == 1 ? 113 : 227) * 1024 - kFixedBytes<DK, DV, NB>) / (int)kStageBytes<DK, DV>;
  return s < 8 ? s / 2 * 2 : 8;   // (even: a stage's place belongs to one half of the warps)
}
template <int DK, int DV, int NB>
__host__ __device__ constexpr size_t smem_bytes() {
  return (size_t)ring_stages<DK, DV, NB>() * kStageBytes<DK, DV> + kFixedBytes<DK, DV, NB>;
}

template <int DK, int DV, int NB, int PS>
__global__ void __launch_bounds__(kThreads, NB == 1 ? 2 : 1) kv4_attn_kernel(const __grid_constant__ Args a) {
  constexpr int GK = DK / 64, GV = DV / 64, ROWS = NB * kBlock, NS = ring_stages<DK, DV, NB>();
  constexpr uint32_t kBytes = kStageBytes<DK, DV>;
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr uint32_t kQBytes = ROWS * DK * 2;
  unsigned char* qs = smem + NS * kBytes;                            // [items, ROWS, DK]
  float* sums = reinterpret_cast<float*>(qs + kItems * kQBytes);          // [4, 8, DV]
  Shared* sh = reinterpret_cast<Shared*>(sums + kWarps / 2 * kBlock * DV);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  const int reach = (int)min((int64_t)a.L_max, (int64_t)a.c.cols * PS);
  constexpr uint32_t kPage = PS * (DK + DV) * 17 / 32;
  constexpr int npp = kStage / PS;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(sh->full[i]), 1);
      mbar_init(bar(sh->empty[i]), kWarps / 2);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar(sh->ifull[i]), 1);
      mbar_init(bar(sh->ifree[i]), kWarps);
    }
    sh->abort = 0;
    sh->bits = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();      // (the inputs may only just be written; the status block is cleared)
  pdl_trigger();
  // Units (an item's cost, then its stages, at least one) of all requests: each warp adds up those of a run.  Up to
  // 32 requests are the loading warp's lanes (0.2 to 0.4 us less than by all warps: 32 single tokens over 4096 positions
  // 40.0 and 40.4; 33 41.2, 64 63.6, 256 204).
  const int per = (a.c.B + kWarps) / (kWarps + 1);
  const bool few = a.c.B <= 32;
  bool bad = false;
  auto units_of = [&](int n, int len) { return (int64_t)blocks_of(a, n, ROWS) * a.c.H_kv * (kItemCost + stages_of(len)); };
  if (!few) {
    int64_t mine = 0;
    for (int base = 0; base < per; base += 32) {
      int r0, n, len;
      request_info(a, base + lane < per ? warp * per + base + lane : -1, reach, lane, r0, n, len, bad);
      mine += units_of(n, len);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sh->units[warp] = mine;
    __syncthreads();
  }
  uint32_t* const status = a.bits ? &sh->bits : a.status;
  auto raise_bad = [&]() {
    if (__any_sync(0xffffffffu, bad) && blockIdx.x == 0 && lane == 0) raise_status(status, DSA_DEVICE_BAD_INDEX);
  };
  if (!few) raise_bad();
  const WaitCtx wc(&sh->abort, status, a.wait_ns);

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    int base = 0, x = 0, r0 = 0, rows = 0, len = 0;    // 32 requests from `base` on, of which x is the next piece's
    int64_t total = 0, units = 0, incl = 0;            // a lane's request's, and those up to it
    auto add_up = [&]() {
      units = units_of(rows, len);
      incl = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
    };
    if (few) {
      request_info(a, lane, reach, lane, r0, rows, len, bad);
      raise_bad();
      add_up();
      total = __shfl_sync(0xffffffffu, incl, 31);
    } else {
      for (int w = 0; w <= kWarps; ++w) total += sh->units[w];
    }
    // (at least two stages to a share: the two halves of the warps take one each; the first `more`
    // shares have one unit more than the others)
    const int64_t shares = min((total + 1) / 2, (int64_t)gridDim.x);
    const int64_t per_share = shares > 0 ? quotient(total, shares) : 0, more = total - per_share * shares;
    const int64_t lo = per_share * blockIdx.x + min((int64_t)blockIdx.x, more);
    int64_t left = blockIdx.x < shares ? per_share + (blockIdx.x < more) : 0;
    int n = 0, k = 0;             // stages and items handed over
    bool ok = true;
    Kv4Join join = {};
    if (left > 0) {
      // The request where the share begins: its warp's run, then 32 at a time.
      int64_t u = lo;             // units from here to the share's beginning
      if (!few) {
        int w = 0;
        while (u >= sh->units[w]) u -= sh->units[w++];
        base = w * per;
        request_info(a, base + lane, reach, lane, r0, rows, len, bad);
        add_up();
      }
      for (;;) {
        const uint32_t hit = __ballot_sync(0xffffffffu, u < incl);
        if (hit) {
          x = __ffs(hit) - 1;
          u -= __shfl_sync(0xffffffffu, incl - units, x);
          break;
        }
        u -= __shfl_sync(0xffffffffu, incl, 31);
        base += 32;
        request_info(a, base + lane, reach, lane, r0, rows, len, bad);
        add_up();
      }
      int64_t at = lo;            // units before the next piece
      while (left > 0 && ok) {
        if (x == 32) {
          base += 32;
          x = 0;
          request_info(a, base + lane, reach, lane, r0, rows, len, bad);
        }
        const int xr = __shfl_sync(0xffffffffu, r0, x), xn = __shfl_sync(0xffffffffu, rows, x);
        const int xl = __shfl_sync(0xffffffffu, len, x);
        const int st = stages_of(xl);
        if (u >= units_of(xn, xl)) {   // (the request is through, or has no rows)
          u = 0;
          ++x;
          continue;
        }
        const int64_t idx = quotient(u, st + kItemCost);
        const int u0 = (int)(u - idx * (st + kItemCost)), rb = (int)quotient(idx, a.c.H_kv), h = (int)idx - rb * a.c.H_kv;   // (below 2^23: 65535 rows of 128 heads)
        const int take = (int)min((int64_t)(st + kItemCost - u0), left);
        const int s0 = max(u0 - kItemCost, 0), cnt = u0 + take - kItemCost - s0;   // its stages
        const int64_t end = at - u0 + st + kItemCost;                              // the item's last unit and one
        u += take;
        at += take;
        left -= take;
        if (cnt <= 0) continue;   // (nothing but the item's cost)
        const int load = xl > 0 ? cnt : 0;
        const bool whole = cnt == st;
        // What the piece reads first, asked for together.  Pages: 32 entries of the table at a time, the
        // next ones ahead.
        const int ends = (xl + PS - 1) / PS;
        const int32_t* table = a.c.table + (int64_t)(base + x) * a.c.cols;
        auto entry = [&](int i) { return i < ends ? table[i] : -1; };
        int next = entry(s0 * npp + lane);
        const int row = rb * ROWS + lane;
        const bool live = lane < ROWS && row < xn * a.G;
        const int sees = live ? a.row_len[xr + row_of(a, row)] : 0;
        const int i = lane >> 2, j = lane & 3;
        uint4 w[NB][GK][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int pk = rb * ROWS + nb * kBlock + i;
          const bool valid = pk < xn * a.G;
          const int to = valid ? row_of(a, pk) : 0;
          const uint16_t* q = a.q + (int64_t)(xr + to) * a.q_stride + (int64_t)(h * a.G + (valid ? pk - to * a.G : 0)) * DK + 16 * j;
#pragma unroll
          for (int g = 0; g < GK; ++g)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              w[nb][g][y] = valid ? *reinterpret_cast<const uint4*>(q + 64 * g + 8 * y) : make_uint4(0, 0, 0, 0);
        }
        // Stage z of the piece on its way.  A lane holds a page of the 32 / npp stages' from `window` on; the
        // loop over stages has one warp's time beside eight that compute, so it holds little else.
        constexpr int kWindow = 32 / npp;
        const uint8_t* src = nullptr;
        uint32_t have = 0;
        auto issue = [&](int z) {
          const int y = z % kWindow;
          if (y == 0) {
            const int at = (s0 + z) * npp + lane, id = next;
            next = entry(at + 32);
            const bool there = at < ends && id >= 0 && id < a.c.n_pages;
            have = __ballot_sync(0xffffffffu, there);
            if (__any_sync(0xffffffffu, at < ends && at < (s0 + load) * npp && !there) && lane == 0)
              raise_status(status, DSA_DEVICE_BAD_INDEX);
            src = a.c.pages + ((int64_t)id * a.c.H_kv + h) * kPage;
          }
          const uint32_t mask = have >> (y * npp) & ((1u << npp) - 1u);
          const int s = n % NS;
          if (n >= NS && !wait_bar_warp(bar(sh->empty[s]), (n / NS - 1) & 1, wc)) return false;
          if (lane == 0) {
            sh->pages[s] = mask;
            mbar_expect_tx(bar(sh->full[s]), __popc(mask) * kPage);
          }
          __syncwarp();
          if (lane / npp == y && (have >> lane & 1u) && !(a.test_no_load && n == 0))
            bulk_row(smem_u32(smem) + s * kBytes + lane % npp * kPage, src, kPage, bar(sh->full[s]));
          ++n;
          return true;
        };
        if (load > 0 && !(ok = issue(0))) break;
        if (k >= kItems && !(ok = wait_bar_warp(bar(sh->ifree[k % kItems]), (k / kItems - 1) & 1, wc))) break;
        // The item, with its rows' queries as the products take them: scaled to fp16's upper range by a power
        // of two for each row, in the layout of the fragments (lane 4 i + j: row i, columns 16 j ..).
        Item* it = &sh->item[k % kItems];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          auto value = [&](int g, int c) {   // column 64 g + 16 j + c
            const uint4 v = w[nb][g][c >> 3];
            const uint32_t y = (c & 7) < 2 ? v.x : (c & 7) < 4 ? v.y : (c & 7) < 6 ? v.z : v.w;
            const uint16_t z = (uint16_t)(c & 1 ? y >> 16 : y);
            return a.f16 ? to_float<true>(z) : to_float<false>(z);
          };
          uint32_t top = 0;
#pragma unroll
          for (int g = 0; g < GK; ++g)
#pragma unroll
            for (int c = 0; c < 16; ++c) top = max(top, __float_as_uint(value(g, c)) & 0x7f800000u);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // 2^(14 - exponent of the row's largest)
          const float up = top ? __uint_as_float(min((268u << 23) - top, 254u << 23)) : 1.f;
#pragma unroll
          for (int g = 0; g < GK; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int c = 8 * (y >> 1) + 2 * (y & 1);
              const __half2 lo = __floats2half2_rn(value(g, c) * up, value(g, c + 4) * up);
              const __half2 hi = __floats2half2_rn(value(g, c + 1) * (up * 0.0625f), value(g, c + 5) * (up * 0.0625f));
              reinterpret_cast<uint2*>(qs + k % kItems * kQBytes)[((g * NB + nb) * 4 + y) * 32 + lane] =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
              const float2 fl = __half22float2(lo), fh = __half22float2(hi);
              sum += fl.x + fl.y + 16.f * (fh.x + fh.y);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (j == 0) it->less[g][nb * kBlock + i] = -0x1p-19f * sum;
          }
          if (j == 0) it->factor[nb * kBlock + i] = a.c2 * (0x1p22f / up);
        }
        if (lane < ROWS) it->see[lane] = live ? min(max(sees, 0), reach) : xl;
        if (lane == 0) {
          it->row0 = xr;
          it->packed = xn * a.G;
          it->first = rb * ROWS;
          it->h = h;
          it->len = xl;
          it->stage = s0;
          it->stages = load;
          it->slot = whole ? -1 : 2 * (int)blockIdx.x + (s0 == 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->ifull[k % kItems]));
        ++k;
        for (int z = 1; z < load && ok; ++z) ok = issue(z);
        if (!whole && s0 == 0) {  // the item's other parts: as many shares as begin before its end
          const int64_t longer = more * (per_share + 1);
          const int64_t begun = end <= longer ? quotient(end + per_share, per_share + 1) : more + quotient(end - longer + per_share - 1, per_share);
          join = Kv4Join{xr, xn * a.G, rb * ROWS, h, (int)(begun - blockIdx.x), {0, 0, 0}};
        }
      }
    }
    if (ok && k >= kItems) ok = wait_bar_warp(bar(sh->ifree[k % kItems]), (k / kItems - 1) & 1, wc);
    if (lane == 0) {
      if (ok) {
        sh->item[k % kItems].packed = 0;
        mbar_arrive(bar(sh->ifull[k % kItems]));
      }
      if (a.join) a.join[blockIdx.x] = join;
      for (int i = max(0, n - NS); i < n; ++i) drain_bar(bar(sh->full[i % NS]), (i / NS) & 1, a.wait_ns);
    }
  } else {
    // ------------------------------------------------------------ products and softmax
    const int i = lane >> 2, j = lane & 3;
    // Rows i and 8 + i of a fragment are a pair of positions, 2 sigma(i) and the next one, in this
    // order or the other: one load brings both scales, and the first four rows of K that a
    // load takes lie in different banks.
    auto sigma = [](int x) { return x ^ (x >> 1 & 1); };
    const int pair = 2 * sigma(i), ta = pair + (i & 1), tb = pair + (~i & 1);
    const uint32_t sel_a = i & 1 ? 0x3244 : 0x1044, sel_b = i & 1 ? 0x1044 : 0x3244;   // its bf16 scale as fp32
    // Row of V that this lane names for ldmatrix: matrix lane / 8 is rows 0.. or 8.. and half a group's codes.
    const int vr = lane & 7, vrow = 2 * sigma(vr) + ((vr ^ lane >> 3) & 1);
    // The warp's 32 positions of a stage: two tiles, in one page or two.
    constexpr uint32_t kTileCodes = PS == 16 ? kPage : 512, kTileScales = PS == 16 ? kPage : 32;
    const int p0 = 32 * (warp & 3);
    const uint32_t pages = (PS == 16 ? 3u : 1u) << (p0 / PS);
    const uint32_t blk = smem_u32(smem) + p0 / PS * kPage, o = p0 % PS;
    const uint32_t k_at = blk + (o + ta) * 32 + 8 * j;
    const uint32_t s_at = blk + PS * ((DK + DV) / 2) + (o + pair) * 2;
    const uint32_t v_at = blk + PS * (DK / 2) + (o + vrow) * 32 + (lane >> 4) * 16;
    const uint32_t tab = (tb - ta) * 32;
    int n0 = 0;                  // stages of earlier items
    for (int k = 0;; ++k) {
      bool ok = wait_bar_warp(bar(sh->ifull[k % kItems]), (k / kItems) & 1, wc);
      struct {
        int row0, packed, first, h, len, stage, stages, slot;
      } it;
      it.packed = 0;
      const Item& si = sh->item[k % kItems];
      if (ok) it = {si.row0, si.packed, si.first, si.h, si.len, si.stage, si.stages, si.slot};
      const bool last = it.packed == 0;
      float qc[GK][NB][2], factor[NB][2], mm[NB][2], l[NB][2], oo[GV][NB][4][4], vinv[GV];
#pragma unroll
      for (int g = 0; g < GV; ++g) vinv[g] = 0x1p126f;   // (no scale so far)
      int see[NB][2];
      const uint32_t qf = smem_u32(qs) + k % kItems * kQBytes + lane * 8;
      if (!last) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = nb * kBlock + 2 * j + x;
            see[nb][x] = si.see[r];
            factor[nb][x] = si.factor[r];
#pragma unroll
            for (int g = 0; g < GK; ++g) qc[g][nb][x] = si.less[g][r];
            mm[nb][x] = 0.f;
            l[nb][x] = 0.f;
          }
#pragma unroll
        for (int g = 0; g < GV; ++g)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int t = 0; t < 4; ++t) oo[g][nb][t][x] = 0.f;
        int least = see[0][0];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) least = min(least, min(see[nb][0], see[nb][1]));
        least = __reduce_min_sync(0xffffffffu, least);
        bool first = true;         // no positions so far
        // Every other stage is this warp's.
        int pos = it.stage * kStage + p0 + ((n0 ^ (warp >> 2)) & 1) * kStage;   // the warp's first position
        for (int n = n0 + ((n0 ^ (warp >> 2)) & 1); n < n0 + it.stages; n += 2, pos += 2 * kStage) {
          const int s = n % NS;
          if (!(ok = wait_bar_warp(bar(sh->full[s]), (n / NS) & 1, wc))) break;
          const uint32_t have = sh->pages[s] & pages;
          if (pos < it.len && have) {
            const uint32_t ring = s * kBytes;
            float e[2][NB][4], vs[2][GV][2];
#pragma unroll
            for (int g = 0; g < GK; ++g) {
              float acc[2][NB][4];
              uint32_t x[2][2], y[2][2];
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const uint32_t at = ring + k_at + t * kTileCodes + g * PS * 32;
                lds2(at, x[t][0], x[t][1]);
                lds2(at + tab, y[t][0], y[t][1]);
              }
#pragma unroll
              for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  uint32_t b[NB][2];
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) lds2(qf + ((g * NB + nb) * 4 + 2 * w + z) * 256, b[nb][0], b[nb][1]);
#pragma unroll
                  for (int t = 0; t < 2; ++t) {
                    const uint32_t xs = z ? x[t][w] >> 6 : x[t][w] << 2, ys = z ? y[t][w] >> 6 : y[t][w] << 2;
                    const uint32_t a0 = xs & 0x003c003cu, a2 = xs & 0x03c003c0u, a1 = ys & 0x003c003cu, a3 = ys & 0x03c003c0u;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                      if (w + z == 0)
                        mma_f16(acc[t][nb], a0, a1, a2, a3, b[nb][0], b[nb][1], qc[g][nb][0], qc[g][nb][1]);
                      else
                        mma_f16(acc[t][nb], a0, a1, a2, a3, b[nb][0], b[nb][1]);
                    }
                  }
                }
              // Logits in base 2: columns 2 j, 2 j + 1 of positions ta and tb.
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const uint32_t w = lds1(ring + s_at + t * kTileScales + g * PS * 2);
                const float k0 = __uint_as_float(__byte_perm(w, 0, sel_a)), k1 = __uint_as_float(__byte_perm(w, 0, sel_b));
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                  for (int z = 0; z < 4; ++z)
                    e[t][nb][z] = g == 0 ? (z < 2 ? k0 : k1) * acc[t][nb][z] : fmaf(z < 2 ? k0 : k1, acc[t][nb][z], e[t][nb][z]);
              }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) e[t][nb][x] = fmaf(e[t][nb][x], factor[nb][x & 1], -mm[nb][x & 1]);
#pragma unroll
              for (int g = 0; g < GV; ++g) {
                const uint32_t w = lds1(ring + s_at + t * kTileScales + (GK + g) * PS * 2);
                vs[t][g][0] = __uint_as_float(__byte_perm(w, 0, sel_a));
                vs[t][g][1] = __uint_as_float(__byte_perm(w, 0, sel_b));
              }
            }
            // V's codes, after which the stage's place is given back: it is loaded again under the rest.
            uint32_t v[2][GV][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int g = 0; g < GV; ++g)
                ldsm_x4_t(ring + v_at + t * kTileCodes + g * PS * 32, v[t][g][0], v[t][g][1], v[t][g][2], v[t][g][3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sh->empty[s]));
            if (pos + 32 > least || have != pages) {
              // Positions that a row does not see, or whose page the pool does not have.
#pragma unroll
              for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int at = have >> ((p0 + 16 * t) / PS) & 1u ? pos + 16 * t + (x ? tb : ta) : INT_MAX;
#pragma unroll
                  for (int g = 0; g < GV; ++g)
                    if (at >= it.len) vs[t][g][x] = 0.f;   // (what lies there may be anything)
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) {
                    if (at >= see[nb][0]) e[t][nb][2 * x] = -INFINITY;
                    if (at >= see[nb][1]) e[t][nb][2 * x + 1] = -INFINITY;
                  }
                }
            }
            float top = -INFINITY, big[GV], most = 0.f;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) top = max3(max3(e[t][nb][0], e[t][nb][1], top), e[t][nb][2], e[t][nb][3]);
#pragma unroll
            for (int g = 0; g < GV; ++g) {
              big[g] = max3(vs[0][g][0], vs[0][g][1], fmaxf(vs[1][g][0], vs[1][g][1]));
              most = fmaxf(most, big[g] * vinv[g]);
            }
            if (__any_sync(0xffffffffu, first || top > 8.f || most > 128.f)) {
              // A row's maximum has grown by more than 2^8, or a scale is above all so far.
              float vf[GV];
#pragma unroll
              for (int g = 0; g < GV; ++g) {
                const uint32_t x = __reduce_max_sync(0xffffffffu, __float_as_uint(big[g])) >> 23;   // 2^(x - 127) <= it
                const float from = vinv[g], to = fminf(from, __uint_as_float(min(260u - x, 253u) << 23));   // 2^6 of its inverse, about
                // What O is to be multiplied with: to / from, or nothing where that is below 2^-126.
                vf[g] = __uint_as_float((uint32_t)max(__float_as_int(to) - __float_as_int(from) + (127 << 23), 0));
                vinv[g] = to;
              }
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                float f[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  float m = max3(e[0][nb][y], e[0][nb][y + 2], fmaxf(e[1][nb][y], e[1][nb][y + 2]));
#pragma unroll
                  for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
                  // (a row that sees none of the first positions sees none of this item's)
                  m = first ? (m == -INFINITY ? 0.f : m) : fmaxf(m, 0.f);
                  f[y] = first ? 1.f : ex2(-m);
                  mm[nb][y] += m;
                  l[nb][y] *= f[y];
#pragma unroll
                  for (int t = 0; t < 2; ++t) {
                    e[t][nb][y] -= m;
                    e[t][nb][y + 2] -= m;
                  }
                }
                if (!first)
#pragma unroll
                  for (int g = 0; g < GV; ++g)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                      for (int t = 0; t < 4; ++t) oo[g][nb][t][y] *= f[y & 1] * vf[g];
              }
              first = false;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int g = 0; g < GV; ++g) {
                vs[t][g][0] *= vinv[g];
                vs[t][g][1] *= vinv[g];
              }
            float sp[GV][NB][4];       // sums of the weights that go to the groups of V
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  e[t][nb][x] = ex2(e[t][nb][x]);
                  l[nb][x & 1] += e[t][nb][x];
                }
#pragma unroll
              for (int g = 0; g < GV; ++g) {
                uint32_t b0[NB], b1[NB];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  b0[nb] = transposed(half2_bits(e[t][nb][0] * vs[t][g][0], e[t][nb][1] * vs[t][g][0]));
                  b1[nb] = transposed(half2_bits(e[t][nb][2] * vs[t][g][1], e[t][nb][3] * vs[t][g][1]));
                  if (t == 0)
                    mma_f16(sp[g][nb], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, b0[nb], b1[nb], 0.f, 0.f);
                  else
                    mma_f16(sp[g][nb], 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u, b0[nb], b1[nb]);
                }
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                  for (int z = 0; z < 2; ++z) {
                    const uint32_t x = v[t][g][2 * w] >> (8 * z), y = v[t][g][2 * w + 1] >> (8 * z);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                      mma_f16(oo[g][nb][2 * w + z], x & 0x000f000fu, x & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u, b0[nb],
                              b1[nb]);
                  }
              }
            }
            // The 8 less in every code, at once: a sum that grew with it would lose its low bits (one token over 307200
            // positions in fp16 9.3e-4 off, 3.5e-4 this way at the same time; by a product with -8 before each other
            // one 3.4e-4, 66 us instead of 62).
#pragma unroll
            for (int g = 0; g < GV; ++g)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    oo[g][nb][w][x] = fmaf(sp[g][nb][x & 1], x < 2 ? -0x1p-21f : -0x1p-17f, oo[g][nb][w][x]);
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(sh->empty[s]));
          }
        }
        n0 += it.stages;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->ifree[k % kItems]));   // (the item and its queries are read)
        // The warps' sums are joined.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) l[nb][x] += __shfl_xor_sync(0xffffffffu, l[nb][x], z);
            if (i == 0) {
              sh->m[warp][nb * kBlock + 2 * j + x] = mm[nb][x];
              sh->l[warp][nb * kBlock + 2 * j + x] = l[nb][x];
            }
          }
      }
      if (consumers_any(!ok || last)) break;
      float back[GV];
#pragma unroll
      for (int g = 0; g < GV; ++g) back[g] = __uint_as_float((254u << 23) - __float_as_uint(vinv[g]));   // 1 / vinv
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        // The common maximum and sum of row lane % 8, over the warps lane / 8 and 4 + lane / 8.
        const int r = nb * kBlock + (lane & 7), wa = lane >> 3, wb = wa + 4;
        const float la = sh->l[wa][r], lb = sh->l[wb][r], ma = la != 0.f ? sh->m[wa][r] : -INFINITY,
                    mb = lb != 0.f ? sh->m[wb][r] : -INFINITY;
        float most = fmaxf(ma, mb);
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 8));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
        float all = (la != 0.f ? ex2(ma - most) * la : 0.f) + (lb != 0.f ? ex2(mb - most) * lb : 0.f);
        all += __shfl_xor_sync(0xffffffffu, all, 8);
        all += __shfl_xor_sync(0xffffffffu, all, 16);
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float to = __shfl_sync(0xffffffffu, most, 2 * j + x);
          f[x] = l[nb][x] != 0.f ? ex2(mm[nb][x] - to) : 0.f;
        }
        const float m = __shfl_sync(0xffffffffu, most, warp), sum = __shfl_sync(0xffffffffu, all, warp);   // the row that this warp writes
        const bool any = sum != 0.f;
        // Columns 64 g + 32 w + 4 i .. of rows 2 j and 2 j + 1, in the common scale.
        float4 v[GV][2][2];
#pragma unroll
        for (int g = 0; g < GV; ++g)
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float4& y = v[g][w][x];
              const float fb = f[x] * back[g];
              y.x = oo[g][nb][2 * w][x] * 0x1p24f * fb;
              y.y = oo[g][nb][2 * w][x + 2] * 0x1p20f * fb;
              y.z = oo[g][nb][2 * w + 1][x] * 0x1p24f * fb;
              y.w = oo[g][nb][2 * w + 1][x + 2] * 0x1p20f * fb;
              if (l[nb][x] == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        // The upper four warps hand theirs to the lower four, lane to lane; these lay down
        // rows of DV floats in pieces of four, their order turned by the row (no two of eight
        // lanes that store together share banks), and each warp adds up one row.
        float4* mine = reinterpret_cast<float4*>(sums) + (warp & 3) * GV * 4 * 32;
        if (warp >= 4) {
#pragma unroll
          for (int g = 0; g < GV; ++g)
#pragma unroll
            for (int w = 0; w < 4; ++w) mine[(g * 4 + w) * 32 + lane] = v[g][w >> 1][w & 1];
        }
        consumers_sync();
        if (warp < 4) {
#pragma unroll
          for (int g = 0; g < GV; ++g)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float4 y = mine[(g * 4 + w) * 32 + lane];
              float4& x = v[g][w >> 1][w & 1];
              x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
            }
          __syncwarp();
#pragma unroll
          for (int g = 0; g < GV; ++g)
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int x = 0; x < 2; ++x) mine[(2 * j + x) * (DV / 4) + ((16 * g + 8 * w + i) ^ 2 * j)] = v[g][w][x];
        }
        consumers_sync();
        const int pk = it.first + nb * kBlock + warp;
        if (pk < it.packed && lane < DV / 4) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float4 y = reinterpret_cast<const float4*>(sums)[(w * kBlock + warp) * (DV / 4) + (lane ^ (warp & 6))];
            v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
          }
          if (it.slot < 0) {
            const int to = row_of(a, pk);
            const int64_t rh = (int64_t)(it.row0 + to) * a.H_q + it.h * a.G + pk - to * a.G;
            const float inv = any ? 1.f / sum : 0.f;
            auto pack = [&](float x, float y) { return a.f16 ? pack16<true>(x, y) : pack16<false>(x, y); };
            *reinterpret_cast<uint2*>(a.out + rh * DV + 4 * lane) =
                any ? make_uint2(pack(v.x * inv, v.y * inv), pack(v.z * inv, v.w * inv)) : make_uint2(0, 0);
            if (a.lse && lane == 0) a.lse[rh] = any ? (m + log2f(sum)) * 0.693147180559945309f : -INFINITY;
          } else {
            const int64_t at = (int64_t)it.slot * ROWS + nb * kBlock + warp;
            reinterpret_cast<float4*>(a.part + at * DV)[lane] = v;
            if (lane == 0) a.ml[at] = make_float2(m, any ? sum : 0.f);
          }
        }
        if (nb + 1 < NB) consumers_sync();
      }
    }
  }
  __syncthreads();
  if (tid == 0 && a.bits) a.bits[blockIdx.x] = sh->bits;
}

// Joins the parts of the items that CTA i of the attention began and others ended: four warps to
// a row, each a quarter of the parts with up to ten of them in flight (one warp to a row walked
// its parts at one load's latency each: 21 us for 32 parts; with eight in flight 307200 positions
// took 0.7 us longer, with twelve one token over 4096 0.5).
constexpr int kJoinRows = 2;   // of a CTA
constexpr int kJoinLoads = 10;

template <int DV, bool F16>
__global__ void __launch_bounds__(128 * kJoinRows) kv4_join_kernel(const __grid_constant__ Args a, int rows, int ctas) {
  constexpr int E = DV / 32;
  __shared__ float2 ml[kJoinRows][4];
  __shared__ float sums[kJoinRows][4][DV];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp & 3, per = rows / kJoinRows;
  const int i = blockIdx.x / per, r = (blockIdx.x - i * per) * kJoinRows + (warp >> 2);
  pdl_wait();   // (by every thread: whoever waits for this grid's end waits for the parts' too)
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    uint32_t bits = 0;
    for (int x = lane; x < ctas; x += 32) bits |= a.bits[x];
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) *a.status = bits;
  }
  auto slot = [&](int x) { return (x == 0 ? 2 * i + 1 : 2 * (i + x)) * rows + r; };
  const Kv4Join jn = a.join[i];
  // (asked for beside the item, whether it has that many parts or not)
  const float2 early = i + w + 4 * lane < ctas ? a.ml[slot(w + 4 * lane)] : make_float2(0.f, 0.f);
  const int pk = jn.first + r;
  if (jn.parts == 0) return;
  float M = -INFINITY, L = 0.f, acc[E] = {};
  if (pk < jn.packed) {
    // The first of its parts, under way while the maxima are compared.
    float v[kJoinLoads][E];
    auto load = [&](int first, int n) {
#pragma unroll
      for (int z = 0; z < kJoinLoads; ++z) {
        const float* p = a.part + (int64_t)slot(first + 4 * min(z, n - 1)) * DV + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) v[z][e] = p[e];
      }
    };
    if (w < jn.parts) load(w, (jn.parts - w + 3) / 4);
    for (int x = w + 4 * lane; x < jn.parts; x += 128) {
      const float2 v = x < 128 ? early : a.ml[slot(x)];
      if (v.y != 0.f) M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int base = w; base < jn.parts; base += 128) {
      const int x = base + 4 * lane;
      float f = 0.f;
      if (x < jn.parts) {
        const float2 v = x < 128 ? early : a.ml[slot(x)];
        f = v.y != 0.f ? ex2(v.x - M) : 0.f;   // (a part that saw nothing counts nothing)
        L = fmaf(f, v.y, L);
      }
      const int n = min((jn.parts - base + 3) / 4, 32);
      for (int y = 0; y < n; y += kJoinLoads) {
        if (base != w || y > 0) load(base + 4 * y, n - y);
#pragma unroll
        for (int z = 0; z < kJoinLoads; ++z) {
          const float g = __shfl_sync(0xffffffffu, f, (y + z) & 31);
          if (y + z < n)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(g, v[z][e], acc[e]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) ml[warp >> 2][w] = make_float2(M, L);
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp >> 2][w][lane * E + e] = acc[e];
  }
  __syncthreads();
  if (w != 0 || pk >= jn.packed) return;
  M = -INFINITY;
  bool any = false;
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (ml[warp >> 2][x].y != 0.f) {
      M = fmaxf(M, ml[warp >> 2][x].x);
      any = true;
    }
  L = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const float2 v = ml[warp >> 2][x];
    const float f = v.y != 0.f ? ex2(v.x - M) : 0.f;
    L = fmaf(f, v.y, L);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, sums[warp >> 2][x][lane * E + e], acc[e]);
  }
  const float inv = any ? 1.f / L : 0.f;
  const int to = row_of(a, pk);
  const int64_t rh = (int64_t)(jn.row0 + to) * a.H_q + jn.head * a.G + pk - to * a.G;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + rh * DV + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = any ? pack16<F16>(acc[2 * e] * inv, acc[2 * e + 1] * inv) : 0u;
  if (a.lse && lane == 0) a.lse[rh] = any ? (M + log2f(L)) * 0.693147180559945309f : -INFINITY;
}

template <int DK, int DV, int NB, int PS>
cudaError_t launch_one(const Args& a, int grid, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DK, DV, NB>();
  static_assert(smem <= 232448 && ring_stages<DK, DV, NB>() >= 2, "shared memory of one CTA");
  auto kernel = kv4_attn_kernel<DK, DV, NB, PS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), smem, st, a);
  if (e != cudaSuccess || !a.join) return e;
  const dim3 joins((unsigned)(grid * NB * kBlock / kJoinRows)), threads(128 * kJoinRows);
  return a.f16 ? launch_pdl(kv4_join_kernel<DV, true>, joins, threads, 0, st, a, NB * kBlock, grid)
               : launch_pdl(kv4_join_kernel<DV, false>, joins, threads, 0, st, a, NB * kBlock, grid);
}

template <int DK, int DV, int NB>
cudaError_t launch_page(const Args& a, int grid, cudaStream_t st) {
  switch (a.c.ps) {
    case 16: return launch_one<DK, DV, NB, 16>(a, grid, st);
    case 32: return launch_one<DK, DV, NB, 32>(a, grid, st);
    case 64: return launch_one<DK, DV, NB, 64>(a, grid, st);
    default: return launch_one<DK, DV, NB, 128>(a, grid, st);
  }
}

template <int DK, int DV>
cudaError_t launch_width(const Args& a, int rows, int grid, cudaStream_t st) {
  return rows == kBlock ? launch_page<DK, DV, 1>(a, grid, st) : launch_page<DK, DV, 2>(a, grid, st);
}

}  // namespace

// 64 packed rows, four passes here and half a tile there, in us: one request of 16384 positions 30 and 38, of 307200 319
// and 244, 32 ragged ones 447 and 514; of width 64, 336 and 368.
bool kv4_many_rows(const dsa_kv4_cache& c, const dsa_kv4_problem& p) {
  const int64_t most = p.rows_max > 0 && p.rows_max < p.R ? p.rows_max : p.R;
  return most * (p.H_q / c.H_kv) > 64;
}

Kv4Shape kv4_shape(const dsa_kv4_cache& c, const dsa_kv4_problem& p) {
  Kv4Shape s;
  const int64_t G = p.H_q / c.H_kv, most = p.rows_max > 0 && p.rows_max < p.R ? p.rows_max : p.R;
  const int64_t held = (int64_t)c.page_size * c.table_cols, longest = p.L_max < held ? p.L_max : held;
  s.rows = most * G <= kBlock ? kBlock : 2 * kBlock;
  // No more CTAs than there can be stages.
  int64_t blocks = c.B * ((most * G + s.rows - 1) / s.rows);
  if (blocks > p.R * G / s.rows + c.B) blocks = p.R * G / s.rows + c.B;
  const int64_t stages = longest > kStage ? (longest + kStage - 1) / kStage : 1;
  const int64_t slots = s.rows == kBlock ? kKv4Slots : kKv4Slots / 2;
  const int64_t items = blocks * c.H_kv;
  s.grid = (int)(items >= slots || items * stages >= slots ? slots : items * stages);
  if (s.grid < 1) s.grid = 1;
  s.join = stages > 1;
  return s;
}

cudaError_t launch_kv4_attn(const dsa_kv4_cache& c, const CacheArgs& ca, const dsa_kv4_problem& p, const Kv4Shape& s,
                            uint16_t* out, float* lse, char* ws, float* ml, float* part, cudaStream_t st,
                            const TestHooks* hooks) {
  Args a;
  std::memset(&a, 0, sizeof a);
  a.c = ca;
  a.q = p.q; a.row_offsets = p.row_offsets; a.row_len = p.row_len;
  a.out = out; a.lse = lse; a.part = part; a.ml = reinterpret_cast<float2*>(ml);
  a.status = reinterpret_cast<uint32_t*>(ws);
  if (s.join) {
    a.join = reinterpret_cast<Kv4Join*>(ws + kKv4DescOffset);
    a.bits = a.status + kKv4Bits;
  }
  a.q_stride = p.q_stride ? p.q_stride : (int64_t)p.H_q * c.D_k;
  a.wait_ns = hooks ? hooks->wait_ns : kDefaultWaitNs;
  a.test_no_load = hooks ? hooks->tile_no_load : 0;
  a.R = p.R; a.H_q = p.H_q; a.G = p.H_q / c.H_kv; a.L_max = p.L_max;
  a.inv_G = 1.f / (float)a.G;
  a.c2 = (float)(p.softmax_scale * 1.4426950408889634);
  a.f16 = (p.flags & DSA_FLAG_FP16) != 0;
  if (c.D_k == 64) return launch_width<64, 64>(a, s.rows, s.grid, st);
  if (c.D_k == 128) return launch_width<128, 128>(a, s.rows, s.grid, st);
  return launch_width<192, 128>(a, s.rows, s.grid, st);
}

}  // namespace dsa
