// Linear attention over whole prompts, in chunks of 128 tokens (dsa_linear_attn).
//
// Mathematics.  With lambda = e^{ld} the decay of a head, H the state before a
// chunk of n tokens and i, j tokens of the chunk:
//
//   S_ij = q_i . k_j                              128 x 128 x D_k
//   P_ij = scale * lambda^(i-j) S_ij  (j <= i)
//   O    = diag(scale * lambda^(i+1)) Q H + P V   two products into one accumulator
//   H'   = lambda^n H + sum_j lambda^(n-1-j) k_j^T v_j
//
// Every power has an exponent >= 0, so nothing overflows whatever the decay.
//
// The state stays in fp32 registers, transposed: a thread holds the D_k values of
// one column of H (one dv).  Per chunk the tensor core adds
//   dH^T = (V diag(lambda^(n-1-j)))^T K
// whose A operand is written into tensor memory: the decayed v, split into 16-bit
// terms that add up to its fp32 value (bf16 three terms, fp16 two after a
// power-of-two scaling per column), so the state loses nothing to the operands' 8
// or 11 bits.  Q H reads H rounded to the operands' type, as P V reads P (fp16: each
// column of H and row of P scaled by a power of two into range).
//
// A CTA takes one head of one request, or of one segment of a long request, and
// walks its chunks.  Five warpgroups, so that the chunks' steps overlap:
//   warp 0        producer: Q, K, V tiles by TMA, two chunks in flight
//   warp 1        issues S = Q K^T, O = Q H, O += P V
//   warp 2        issues dH^T
//   warps 4-11    "rows": two threads per token hold its row of S, P and O, one the
//                 32-column blocks 0 and 2, the other 1 and 3
//   warp 3        stores the output tiles by TMA, through the shared memory of
//                 their own Q tile, which no MMA reads by then
//   warps 12-15   "decay": they write the decayed V, a quarter chunk (32 tokens) at a
//                 time into two buffers in turn; in a request's last chunk they
//                 first zero the K and V rows behind the last token (another
//                 request's: weight zero times NaN is NaN)
//   warps 16-19   "state": a thread holds one column of H
// Registers are dealt to the groups with setmaxnreg (40 + 3 x 88 + 176 of 5 x 96).
//
// The groups' code together has to fit the instruction cache: unrolling the loops
// over column blocks cost more than they saved (65536 tokens: 432 us unrolled, 357
// rolled), as did out-of-place copies of the waits and of the MMA operands.
//
// Bound: reading q, k, v and writing out once.  With every SM at work a chunk of
// 96 + 32 KB takes about 5600 cycles, 6.1 TB/s: 12 ragged prompts of 32 heads take
// 106 us against 86 us for their bytes, the rest being the longest prompt's walk (fp16
// 119 us: a second pass over S and one over V for the largest values).
// Where requests and heads do not fill the GPU, long requests are split into
// segments: a first launch computes each segment's own end state (K and V only), a
// scan adds them up to each segment's start, and a second launch walks the segments
// side by side.  65536 tokens of 16 heads, launches back to back on three sets of inputs in
// turn: 244 us in nine segments, 1146 us in one walk (258 us as one call among others;
// 159 us for its bytes, 238 with K and V read twice).  With each segment's CTA adding up
// the states before it, one warpgroup's loads at a time, instead of the scan, 4096 tokens of
// 16 heads that go on from a state took almost twice as long (63 us, with the scan 33, both
// with inputs in L2; 37 on inputs in turn).
#include "linear.cuh"

#include <algorithm>
#include <cstring>

#include "linear_protocol.h"
#include "tc.cuh"

namespace dsa {
namespace {

constexpr int kC = 128;            // tokens of a chunk
constexpr int kThreads = 640;
constexpr int kQuarter = 32;       // tokens of the decayed V in one buffer
constexpr int kStages = ChunkPipe<false>::stages;        // of Q, K and V; the state launch, without Q,
constexpr int kStateStages = ChunkPipe<true>::stages;    // has room for three

// Tensor-memory columns.
constexpr uint32_t kColS = 0, kColO = 128, kColH = 256, kColV = 384;

struct ChunkParams {
  CUtensorMap tq, tk, tv, to;
  LinearArgs a;
};

struct __align__(16) Shared {
  uint64_t q_full[kStages], kv_full[kStateStages], q_empty[kStages], kv_empty[kStateStages];
  uint64_t o_staged[ChunkPipe<false>::o_tiles];
  uint64_t s_ready, qh_ready, h_ready, p_ready, o_ready, o_free, tail, done1, done2;
  uint64_t dh_ready[2], dh_free[2];
  uint64_t v_ready[4], v_free[4], pair[4];
  uint32_t tmem;
  int abort;
  int place, scratch;              // (here: the next four, 16-byte aligned, were loaded as one and spilled)
  int req, seg, nseg, first;       // request, its segment, its segments, their first index; req < 0: nothing
  int t0, n;                       // tokens of the segment
  __align__(16) float pw[2 * kC + 4];            // pw[128 + e] = lambda^e for e = 0 .. 128, 0 for e < 0
  float column[32];                // lambda^(31-y)
  unsigned char mx[2][128];        // fp16: exponent fields of the two halves' largest weight of each row
  unsigned char cs[2][128];        // fp16: scale of each column of H as Q H read it (a power of two's exponent field)
  unsigned char vs[ChunkPipe<true>::scale_slots][128];   // fp16: the same of each column of the decayed V
};

template <int DK, int DV>
__host__ __device__ constexpr uint32_t stage_bytes() {
  return ((DK > DV ? DK : DV) / 64 + DK / 64 + DV / 64) * kChunkBytes;   // Q (later O), K, V
}
template <int DK, int DV>
__host__ __device__ constexpr size_t smem_bytes() {
  return kStages * stage_bytes<DK, DV>() + DV * DK * 2 + sizeof(Shared);
}

// Request b's first token, tokens and segments, clamped to the call's.
__device__ __forceinline__ void request(const LinearArgs& a, int b, int& t0, int& n, int& v) {
  const int x0 = a.row_offsets[b], x1 = a.row_offsets[b + 1];
  t0 = min(max(x0, 0), a.R);
  n = max(min(x1, a.R) - t0, 0);
  v = n > a.seg_len ? (n - 1) / a.seg_len + 1 : 1;
}

__device__ __forceinline__ void take_segment(const LinearArgs& a, Shared* sh, int b, int s, int first, int t0, int n, int v) {
  const int skip = s * a.seg_len;   // (below n)
  sh->req = b;
  sh->seg = s;
  sh->nseg = v;
  sh->first = first;
  sh->t0 = t0 + skip;
  sh->n = v == 1 ? n : min(n - skip, a.seg_len);
}

// Segment `idx` of the call (the whole CTA; the result is there after its next
// __syncthreads).  Split requests' segments come first, so that only these need end
// states; up to 32 requests from the longest on, so that the longest walks start first.
__device__ void locate(const LinearArgs& a, int idx, Shared* sh) {
  int* sums = reinterpret_cast<int*>(sh->pw);   // (the table is filled later)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sh->req = -1;
  __syncthreads();
  if (a.B <= 32) {
    if (warp > 0) return;
    int t0 = 0, n = -1, v = 0;
    if (lane < a.B) request(a, lane, t0, n, v);
    int first = 0;
    for (int o = 0; o < a.B; ++o) {
      const int on = __shfl_sync(0xffffffffu, n, o), ov = __shfl_sync(0xffffffffu, v, o);
      if (on > n || (on == n && o < lane)) first += ov;
    }
    if (idx >= first && idx < first + v) take_segment(a, sh, lane, idx - first, first, t0, n, v);
    return;
  }
  if (a.R <= a.seg_len) {   // no request is split
    if (tid == 0 && idx < a.B) {
      int t0, n, v;
      request(a, idx, t0, n, v);
      take_segment(a, sh, idx, 0, idx, t0, n, v);
    }
    return;
  }
  // A thread counts some adjacent requests' segments, those of split requests and the
  // others; the one whose range holds idx looks for it there.
  const int per = (a.B + kThreads - 1) / kThreads;
  int mine[2] = {0, 0}, incl[2], first[2] = {0, 0}, split = 0;
  for (int b = tid * per; b < min((tid + 1) * per, a.B); ++b) {
    int t0, n, v;
    request(a, b, t0, n, v);
    if (v == 1)
      ++mine[1];
    else
      mine[0] += v;
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    incl[x] = mine[x];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl[x], o);
      if (lane >= o) incl[x] += t;
    }
    if (lane == 31) sums[warp * 2 + x] = incl[x];
  }
  __syncthreads();
  for (int w = 0; w < kThreads / 32; ++w) {
    split += sums[w * 2];
    if (w < warp) {
      first[0] += sums[w * 2];
      first[1] += sums[w * 2 + 1];
    }
  }
  const bool one = idx >= split;
  int at = one ? split + first[1] + incl[1] - mine[1] : first[0] + incl[0] - mine[0];
  if (idx < at || idx >= at + (one ? mine[1] : mine[0])) return;
  for (int b = tid * per; b < min((tid + 1) * per, a.B); ++b) {
    int t0, n, v;
    request(a, b, t0, n, v);
    if ((v == 1) != one) continue;
    if (idx < at + v) {
      take_segment(a, sh, b, idx - at, at, t0, n, v);
      return;
    }
    at += v;
  }
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}

// 16 lanes x 16 columns in the shape of four 8 x 8 blocks of 16-bit pairs: thread t
// holds column 4 i + t % 4 of lanes t / 4 (v[2 i]) and t / 4 + 8 (v[2 i + 1]).
__device__ __forceinline__ void tmem_st_16x128_x4(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ float exponent_value(unsigned char e) { return __uint_as_float((uint32_t)e << 23); }
__device__ __forceinline__ unsigned char exponent_field(float x) { return (unsigned char)(__float_as_uint(x) >> 23); }

// The two values of a packed pair, widened.
template <bool F16>
__device__ __forceinline__ float2 widen(uint32_t p) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&p));
  return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}

// The power of two that takes m >= 0 into [2^14, 2^15), and its inverse: values of
// which m is the largest then fit fp16.  Rounded to it, those below 2^-28 of m (fp16 is
// normal from 2^-14 on) are off by 2^-39 m; split into two terms, those from 2^-17 of m on
// keep 22 bits and those below are off by 2^-39 m.  1 where m is 0, below 2^-112 or not
// finite.
__device__ __forceinline__ float half_range(float m, float* back) {
  const uint32_t e = (__float_as_uint(m) >> 23) & 255u;
  if (e < 15 || e > 252) {
    *back = 1.f;
    return 1.f;
  }
  *back = __uint_as_float((e - 14) << 23);
  return __uint_as_float((268u - e) << 23);
}

// STATE: the first launch of a split call, the segments' end states alone.
template <int DK, int DV, bool F16, bool STATE>
__global__ void __launch_bounds__(kThreads, 1) linear_chunk_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int KC = DK / 64, VC = DV / 64, QC = KC > VC ? KC : VC;
  constexpr uint32_t kStage = stage_bytes<DK, DV>();
  constexpr int kTerms = F16 ? 2 : 3;
  using Pipe = ChunkPipe<STATE>;
  const LinearArgs& a = p.a;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = smem_raw;   // (1024-byte aligned: checked below)
  unsigned char* Hb = smem + kStages * kStage;     // H in the operands' type, D_v rows of D_k, K-major
  Shared* sh = reinterpret_cast<Shared*>(Hb + DV * DK * 2);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int h = blockIdx.x % a.H;

  if (smem_u32(smem_raw) & 1023) {
    if (tid == 0) raise_status(a.status, DSA_DEVICE_CAPACITY);
    return;
  }
  locate(a, blockIdx.x / a.H, sh);
  __syncthreads();
  // Each launch starts under the one before it (the clearing of the status block, or
  // the state launch); its state warps wait for that one's end, as does whoever
  // touches the status block and every CTA before it leaves.
  if (STATE) pdl_trigger();
  if (sh->req < 0 || (STATE && sh->seg >= sh->nseg - 1)) {   // (nothing here; no segment follows)
    pdl_wait();
    return;
  }
  if (sh->nseg > 1 && sh->first + sh->nseg > a.split_segs) {   // (offsets that overlap: more than the workspace holds)
    pdl_wait();
    if (tid == 0) raise_status(a.status, DSA_DEVICE_CAPACITY);
    return;
  }
  const int place = state_place(a, sh->req, &sh->scratch, h == 0 && sh->seg == 0);
  if (place < 0) {
    pdl_wait();
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sh->q_full[i]), 1);
      mbar_init(smem_u32(&sh->q_empty[i]), 1);
    }
    for (int i = 0; i < kStateStages; ++i) {
      mbar_init(smem_u32(&sh->kv_full[i]), 1);
      mbar_init(smem_u32(&sh->kv_empty[i]), Pipe::kv_releases);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sh->v_ready[i]), DV / 32);
      mbar_init(smem_u32(&sh->v_free[i]), 1);
    }
    mbar_init(smem_u32(&sh->s_ready), 1);
    for (int i = 0; i < ChunkPipe<false>::o_tiles; ++i) mbar_init(smem_u32(&sh->o_staged[i]), 8);
    mbar_init(smem_u32(&sh->qh_ready), 1);
    mbar_init(smem_u32(&sh->h_ready), DV / 32);
    mbar_init(smem_u32(&sh->p_ready), 8);
    mbar_init(smem_u32(&sh->o_ready), 1);
    mbar_init(smem_u32(&sh->o_free), 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh->dh_ready[i]), 1);
      mbar_init(smem_u32(&sh->dh_free[i]), DV / 32);
    }
    mbar_init(smem_u32(&sh->tail), DV / 32);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&sh->pair[i]), 2);
    mbar_init(smem_u32(&sh->done1), 1);
    mbar_init(smem_u32(&sh->done2), 1);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc(smem_u32(&sh->tmem), 512);
  const float ld2 = log2_decay(a.log_decay[h]);
  for (int i = tid; i <= 2 * kC; i += kThreads) sh->pw[i] = i < kC ? 0.f : exp2f(ld2 * (float)(i - kC));
  if (tid < 32) sh->column[tid] = exp2f(ld2 * (float)(31 - tid));
  const float* pw = sh->pw + kC;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0);
  const WaitCtx wc(&sh->abort, a.status, a.wait_ns);

  const int n = sh->n, t0 = sh->t0, seg = sh->seg, nseg = sh->nseg;
  const int all = (n + kC - 1) / kC;
  // The state launch walks a segment (whole chunks) from its end: dH of its chunk c
  // counts with lambda^(128 c), and where that is 0 in fp32 (below 2^-150) the walk
  // ends.  It leaves the segments' first tokens in the L2 cache, where the second
  // launch begins.
  const int chunks = STATE ? min(all, (int)fminf(151.f / (fabsf(ld2) * kC), 1e9f) + 2) : all;
  auto token = [&](int c) { return t0 + (STATE ? all - 1 - c : c) * kC; };   // first token of chunk c
  const int last_n = n - (chunks - 1) * kC;               // tokens of the last chunk
  const bool ragged = chunks > 0 && last_n < kC;
  const bool final_state = STATE || (seg == nseg - 1 && a.state_out);
  const int deltas = final_state ? chunks : chunks - 1;   // chunks whose dH is needed
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  // Buffers of the decayed V: two, each used twice a chunk; in the state launch four
  // (it has no S), used once.
  auto v_col = [&](int b) -> uint32_t { return b < 2 ? kColV + b * 64 : kColS + (b - 2) * 64; };
  // dH^T likewise: one accumulator, or two in turn (the second in O's place).
  auto dh_col = [&](int c) -> uint32_t { return Pipe::dh(c) ? kColO : kColH; };
  const uint32_t k_off = STATE ? 0 : QC * kChunkBytes;   // K in a stage, behind Q
  const uint32_t stride = STATE ? (KC + VC) * kChunkBytes : kStage;
  static_assert(kStateStages * (KC + VC) * kChunkBytes <= kStages * kStage, "the state launch's stages");
  constexpr int stages = Pipe::stages;
  auto stage = [&](int c) { return smem + Pipe::stage(c) * stride; };
  auto phase = [&](int c) { return Pipe::stage_phase(c); };
  const int quad = warp & 3;

  if (warp < 4) {
    regs_down<40>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        int c = 0;
        bool q_last = false;   // chunk c's Q tile was asked for
        for (; c < chunks; ++c) {
          const int s = Pipe::stage(c), y = token(c);
          const uint32_t q = smem_u32(stage(c)), k = q + k_off, v = k + KC * kChunkBytes;
          if (c >= stages && !wait_bar(bar(sh->kv_empty[s]), phase(c - stages), wc)) break;
          mbar_expect_tx(bar(sh->kv_full[s]), (KC + VC) * kChunkBytes);
          if (a.test_no_load && c == 0) continue;
          for (int x = 0; x < KC; ++x) tma_load_2d(k + x * kChunkBytes, &p.tk, h * DK + x * 64, y, bar(sh->kv_full[s]));
          for (int x = 0; x < VC; ++x) tma_load_2d(v + x * kChunkBytes, &p.tv, h * DV + x * 64, y, bar(sh->kv_full[s]));
          if (STATE) continue;
          if (c >= stages && !wait_bar(bar(sh->q_empty[s]), phase(c - stages), wc)) {
            ++c;
            q_last = true;     // (its K and V were asked for, its Q was not)
            break;
          }
          mbar_expect_tx(bar(sh->q_full[s]), KC * kChunkBytes);
          for (int x = 0; x < KC; ++x) tma_load_2d(q + x * kChunkBytes, &p.tq, h * DK + x * 64, y, bar(sh->q_full[s]));
        }
        for (int i = max(0, c - stages); i < c; ++i) {   // (an abort may leave copies in flight)
          drain_bar(bar(sh->kv_full[i % stages]), phase(i), a.wait_ns);
          if (!STATE && !(q_last && i == c - 1) && !(a.test_no_load && i == 0)) drain_bar(bar(sh->q_full[i % stages]), phase(i), a.wait_ns);
        }
      }
    } else if (warp == 1 && !STATE) {
      // ---------------------------------------------------------- S, Q H, P V
      const uint32_t id_s = idesc_16(F16, kC, kC, false, false);
      const uint32_t id_h = idesc_16(F16, kC, DV, false, false);
      const uint32_t id_o = idesc_16(F16, kC, DV, false, true);
      const uint64_t dh = desc_kmajor(smem_u32(Hb));
      for (int c = 0; c < chunks; ++c) {
        const int s = Pipe::stage(c);
        const uint32_t q = smem_u32(stage(c)), k = q + k_off, v = k + KC * kChunkBytes;
        const uint64_t dq = desc_kmajor(q), dk = desc_kmajor(k), dv = desc_mnmajor(v, kChunkBytes);
        if (!wait_bar_warp(bar(sh->kv_full[s]), phase(c), wc)) break;
        if (!wait_bar_warp(bar(sh->q_full[s]), phase(c), wc)) break;
        tc_fence_after();
        {
#pragma unroll
          for (int x = 0; x < KC * 4; ++x) {
            const uint32_t at = (x >> 2) * kChunkBytes + (x & 3) * 32;
            mma_ss(tmem + kColS, dq + desc_step(at), dk + desc_step(at), id_s, x);
          }
          mma_commit(bar(sh->s_ready));
        }
        if (!wait_bar_warp(bar(sh->h_ready), c & 1, wc)) break;
        if (c > 0 && !wait_bar_warp(bar(sh->o_free), (c - 1) & 1, wc)) break;
        tc_fence_after();
        {
#pragma unroll
          for (int x = 0; x < KC * 4; ++x)
            mma_ss(tmem + kColO, dq + desc_step((x >> 2) * kChunkBytes + (x & 3) * 32),
                   dh + desc_step((x >> 2) * (DV * 128) + (x & 3) * 32), id_h, x);
          mma_commit(bar(sh->qh_ready));
        }
        if (ragged && c == chunks - 1 && !wait_bar_warp(bar(sh->tail), 0, wc)) break;
        if (!wait_bar_warp(bar(sh->p_ready), c & 1, wc)) break;
        tc_fence_after();
        {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            mma_ts(tmem + kColO, tmem + kColS + (x >> 1) * 32 + (x & 1) * 8, dv + desc_step(x * 2048), id_o, 1);
          mma_commit(bar(sh->o_ready));
          mma_commit(bar(sh->kv_empty[s]));
        }
      }
      if (chunks > 0) {
        mma_commit(bar(sh->done1));
        drain_bar(bar(sh->done1), 0, a.wait_ns);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- dH^T
      // (the decayed V of a chunk is ready only after its K has landed)
      const uint32_t id_d = idesc_16(F16, kC, DK, false, true);
      bool ok = true;
      for (int c = 0; c < deltas && ok; ++c) {
        const uint64_t dk = desc_mnmajor(smem_u32(stage(c)) + k_off, kChunkBytes);
        if (ragged && c == chunks - 1 && !(ok = wait_bar_warp(bar(sh->tail), 0, wc))) break;
        const int db = Pipe::dh(c);
        if (c >= Pipe::dh_bufs && !(ok = wait_bar_warp(bar(sh->dh_free[db]), Pipe::dh_phase(c - Pipe::dh_bufs), wc))) break;
#pragma unroll 1
        for (int g = 0; g < 4 && ok; ++g) {
          const int b = Pipe::v(g);
          if (!(ok = wait_bar_warp(bar(sh->v_ready[b]), Pipe::v_phase(c, g), wc))) break;
          const uint32_t va = tmem + v_col(b);
          tc_fence_after();
          {
#pragma unroll
            for (int t = kTerms - 1; t >= 0; --t)    // the smallest terms first: the sum stays small meanwhile
#pragma unroll
              for (int x = 0; x < 2; ++x)
                mma_ts(tmem + dh_col(c), va + t * 16 + x * 8,
                       dk + desc_step((g * 2 + x) * 2048), id_d, g | (kTerms - 1 - t) | x);
            mma_commit(bar(sh->v_free[b]));
            if (g == 3) {
              mma_commit(bar(sh->dh_ready[db]));
              mma_commit(bar(sh->kv_empty[Pipe::stage(c)]));
            }
          }
        }
      }
      if (deltas > 0) {
        mma_commit(bar(sh->done2));
        drain_bar(bar(sh->done2), 0, a.wait_ns);
      }
    } else if (warp == 3 && !STATE) {
      // ---------------------------------------------------------- output tiles
      if (lane == 0) {
        for (int c = 0; c < chunks - (ragged ? 1 : 0); ++c) {
          if (!wait_bar(bar(sh->o_staged[Pipe::stage(c)]), phase(c), wc)) break;
          for (int x = 0; x < VC; ++x)
            tma_store_2d(&p.to, h * DV + x * 64, t0 + c * kC, smem_u32(stage(c) + x * kChunkBytes));
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          mbar_arrive(bar(sh->q_empty[Pipe::stage(c)]));
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      }
    }
  } else if (warp < 16) {
   regs_down<88>();
   if (warp < 12 && !STATE) {
    // ------------------------------------------------------------ rows
    const int half = (warp >> 2) - 1;   // this thread's blocks of 32 columns: half, half + 2
    const int i = quad * 32 + lane;     // token of the chunk
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const float reach = F16 ? pw[i + 1] : pw[i + 1] * a.scale;
    uint32_t turn = 0;                  // (fp16)
    auto pair_sync = [&]() -> bool {    // the rows' two warps meet
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh->pair[quad]));
      const bool r = wait_bar_warp(bar(sh->pair[quad]), turn, wc);
      turn ^= 1;
      return r;
    };
    for (int c = 0; c < chunks; ++c) {
      if (!wait_bar_warp(bar(sh->s_ready), c & 1, wc)) break;
      tc_fence_after();
      // The weights of a block of S, over it: S_ij lambda^(i-j) times f0.
      auto weigh = [&](int x, uint32_t* s, float f0) {
        if (x < quad) {
          // Every column lies before the row: lambda^(i-j) = lambda^(i-e) lambda^(e-j)
          // with e the block's last column, one power per thread, one per column.
          const float f = f0 * pw[i - (x * 32 + 31)];
          const float4* w = reinterpret_cast<const float4*>(sh->column);
#pragma unroll
          for (int y = 0; y < 32; y += 4) {
            const float4 e = w[y >> 2];
            const float2 u = mul2(mul2(make_float2(__uint_as_float(s[y]), __uint_as_float(s[y + 1])), make_float2(f, f)), make_float2(e.x, e.y));
            const float2 v = mul2(mul2(make_float2(__uint_as_float(s[y + 2]), __uint_as_float(s[y + 3])), make_float2(f, f)), make_float2(e.z, e.w));
            s[y] = __float_as_uint(u.x);
            s[y + 1] = __float_as_uint(u.y);
            s[y + 2] = __float_as_uint(v.x);
            s[y + 3] = __float_as_uint(v.y);
          }
        } else {
          // The diagonal's block (the table is 0 where the column lies behind the row;
          // what S holds there may be anything, so it is also replaced).
          const float* w = pw + lane;
#pragma unroll
          for (int y = 0; y < 32; ++y) s[y] = __float_as_uint((y <= lane ? __uint_as_float(s[y]) : 0.f) * (f0 * w[-y]));
        }
      };
      // fp16: the weights go back over S in fp32, and the row is brought into fp16's range
      // by the largest of them.  (By the largest of S, an early key that a fast head has
      // forgotten would push the weights that count out of it.)  The scale waits for the output.
      float pf = 1.f, pback = 1.f;
      if (F16) {
        float mx = 0.f;
#pragma unroll 1
        for (int x = half; x <= quad; x += 2) {
          uint32_t s[32];
          tmem_ld32(lanes + kColS + x * 32, s);
          tmem_wait_ld();
          weigh(x, s, 1.f);
#pragma unroll
          for (int y = 0; y < 32; y += 2) mx = max3(mx, fabsf(__uint_as_float(s[y])), fabsf(__uint_as_float(s[y + 1])));
          tmem_st32(lanes + kColS + x * 32, s);
        }
        tmem_wait_st();
        sh->mx[half][i] = exponent_field(mx);
        if (!pair_sync()) break;
        pf = half_range(exponent_value(max(sh->mx[0][i], sh->mx[1][i])), &pback);
        pback *= a.scale;
      }
      // (Rolled loops: the groups' code has to fit the instruction cache together.)
#pragma unroll 1
      for (int x = half; x < 4; x += 2) {   // P of a block goes over the first half of its S
        uint32_t s[32];
        if (x <= quad) {
          tmem_ld32(lanes + kColS + x * 32, s);
          tmem_wait_ld();
          if (!F16) weigh(x, s, a.scale);
#pragma unroll
          for (int y = 0; y < 32; y += 2)
            s[y >> 1] = pack16<F16>(__uint_as_float(s[y]) * pf, __uint_as_float(s[y + 1]) * pf);
        } else {
#pragma unroll
          for (int y = 0; y < 16; ++y) s[y] = 0;
        }
        tmem_st16(lanes + kColS + x * 32, s);
      }
      if (!wait_bar_warp(bar(sh->qh_ready), c & 1, wc)) break;
      tc_fence_after();
      const float f = reach * pf;
#pragma unroll 1
      for (int x = half * 32; x < DV; x += 64) {
        uint32_t o[32];
        tmem_ld32(lanes + kColO + x, o);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; y += 2) {
          float2 g = make_float2(f, f);
          if (F16) g = mul2(g, make_float2(exponent_value(sh->cs[c & 1][x + y]), exponent_value(sh->cs[c & 1][x + y + 1])));
          g = mul2(g, make_float2(__uint_as_float(o[y]), __uint_as_float(o[y + 1])));
          o[y] = __float_as_uint(g.x);
          o[y + 1] = __float_as_uint(g.y);
        }
        tmem_st32(lanes + kColO + x, o);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh->p_ready));
      if (!wait_bar_warp(bar(sh->o_ready), c & 1, wc)) break;
      tc_fence_after();
      // A whole chunk leaves by TMA through the shared memory of its Q tile; a
      // request's last rows are stored one by one.
      const bool whole = !(ragged && c == chunks - 1);
      unsigned char* tile = stage(c);
      uint16_t* dst = a.out + ((int64_t)(t0 + c * kC + i) * a.H + h) * DV;
#pragma unroll 1
      for (int x = half * 32; x < DV; x += 64) {
        uint32_t o[32];
        tmem_ld32(lanes + kColO + x, o);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; y += 2)
          o[y >> 1] = pack16<F16>(__uint_as_float(o[y]) * pback, __uint_as_float(o[y + 1]) * pback);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint4 w = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          if (whole)
            *reinterpret_cast<uint4*>(tile + (x >> 6) * kChunkBytes + i * 128 + (((((x & 63) >> 3) + y) ^ (i & 7)) << 4)) = w;
          else if (i < last_n)
            reinterpret_cast<uint4*>(dst + x)[y] = w;
        }
      }
      tc_fence_before();
      if (whole) fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(sh->o_free));
        if (whole) mbar_arrive(bar(sh->o_staged[Pipe::stage(c)]));
      }
    }
   } else if ((STATE || warp >= 12) && quad * 32 < DV) {
    // ------------------------------------------------------------ decay
    // Quarter g of chunk c is task 4 c + g.  The state launch has no rows: there the
    // row warps share the tasks.
    const int groups = STATE ? 3 : 1, group = STATE ? (warp >> 2) - 1 : 0;
    const int d = quad * 32 + lane;                    // column of V
    // V is read in 8 x 8 blocks transposed (ldmatrix): a thread holds, of every 8
    // tokens, two adjacent ones (2 (lane % 4) and the next) of four columns, lane / 4
    // + 0, 8, 16, 24, and stores them in the matching tensor-memory shape.
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int at_row = ((lane >> 4) << 3) + (lane & 7), at_piece = (lane >> 3) & 1;   // this lane's row address
    bool ok = true;
    for (int c = 0; c < chunks && ok; ++c) {
      const bool short_chunk = ragged && c == chunks - 1;
      if (c >= deltas && !short_chunk) break;
      const int g0 = (group + 3 * groups - 4 * c % groups) % groups;   // this group's first quarter of the chunk
      if (!(ok = wait_bar_warp(bar(sh->kv_full[Pipe::stage(c)]), phase(c), wc))) break;
      unsigned char* kv = stage(c) + k_off;   // the K chunks, then the V chunks
      if (short_chunk) {
        // Zeros in K and V behind the last token.
        for (int x = 0; x < KC + VC; ++x) {
          uint4* w = reinterpret_cast<uint4*>(kv + x * kChunkBytes + last_n * 128);
          for (int i = d; i < (kC - last_n) * 8; i += DV) w[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->tail));
        if (c >= deltas || !(ok = wait_bar_warp(bar(sh->tail), 0, wc))) break;   // (they read the zeros below)
      }
      const int m = short_chunk ? last_n : kC;
      // Columns quad * 32 ..: four 16-byte pieces of a row of one V chunk.
      const uint32_t v = smem_u32(kv) + (KC + (quad >> 1)) * kChunkBytes;
      auto blocks = [&](int j, int hh, uint32_t* r) {   // tokens j .. j + 15, columns 16 hh ..
        const int row = j + at_row, piece = (quad & 1) * 4 + hh * 2 + at_piece;
        ldsm_x4_t(v + row * 128 + ((piece ^ (row & 7)) << 4), r[0], r[1], r[2], r[3]);
      };
      const float* fade = pw + m - 1;          // fade[-j] = lambda^(m-1-j), 0 behind the last token
      float vf[4] = {1.f, 1.f, 1.f, 1.f};
      float vback[4];
      if (F16) {
        // The columns of the decayed V brought into fp16's range.  (Of V as it is, an early
        // token that a fast head has forgotten would push those that count out of it.)
        float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int j = 0; j < kC; j += 16) {
          float2 fd[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int at = j + 8 * y + 2 * (lane & 3);
            fd[y] = make_float2(fade[-at], fade[-at - 1]);
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t r[4];
            blocks(j, hh, r);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 x = mul2(widen<F16>(r[y]), fd[y >> 1]);
              mx[hh * 2 + (y & 1)] = max3(mx[hh * 2 + (y & 1)], fabsf(x.x), fabsf(x.y));
            }
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], 1));
          mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], 2));
          vf[y] = half_range(mx[y], &vback[y]);
        }
      }
#pragma unroll 1
      for (int g = g0; g < 4; g += groups) {
        const int b = Pipe::v(g);
        if (!Pipe::v_first(c, g) && !(ok = wait_bar_warp(bar(sh->v_free[b]), Pipe::v_phase_before(c, g), wc))) break;
        tc_fence_after();
        if (F16 && g == 0 && (lane & 3) == 0) {
#pragma unroll
          for (int y = 0; y < 4; ++y) sh->vs[Pipe::scale(c)][quad * 32 + (lane >> 2) + 8 * y] = exponent_field(vback[y]);
        }
        float2 fd[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int j = g * kQuarter + 8 * y + 2 * (lane & 3);
          fd[y] = make_float2(fade[-j], fade[-j - 1]);
        }
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {       // 16 columns at a time
          uint32_t r[8], w[kTerms][8];
          blocks(g * kQuarter, hh, r);
          blocks(g * kQuarter + 16, hh, r + 4);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            float2 x = mul2(widen<F16>(r[y]), fd[y >> 1]);
            if (F16) x = mul2(x, make_float2(vf[hh * 2 + (y & 1)], vf[hh * 2 + (y & 1)]));
#pragma unroll
            for (int t = 0; t < kTerms; ++t) {
              w[t][y] = pack16<F16>(x.x, x.y);
              if (t + 1 < kTerms) x = fma2(widen<F16>(w[t][y]), make_float2(-1.f, -1.f), x);
            }
          }
#pragma unroll
          for (int t = 0; t < kTerms; ++t) tmem_st_16x128_x4(lanes + ((uint32_t)(hh * 16) << 16) + v_col(b) + t * 16, w[t]);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->v_ready[b]));
      }
    }
   }
  } else {
    // ------------------------------------------------------------ state
    regs_up<176>();
    if (quad * 32 < DV) {
    const int d = quad * 32 + lane;                    // column of H
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int64_t head = (int64_t)DK * DV;
    float H[DK];
#pragma unroll
    for (int x = 0; x < DK; ++x) H[x] = 0.f;
    auto load = [&](const float* src) {
#pragma unroll
      for (int x = 0; x < DK; ++x) H[x] = src[x * DV + d];
    };
    auto store = [&](float* dst) {
#pragma unroll
      for (int x = 0; x < DK; ++x) dst[x * DV + d] = H[x];
    };
    float* ends = a.seg_state + ((int64_t)sh->first * a.H + h) * head;   // [segment] of this request, H heads apart
    pdl_wait();
    if (!STATE) {
      // Segment s of a split request starts from what the scan left for it.
      const float* start = a.state_in ? a.state_in + ((int64_t)place * a.H + h) * head : nullptr;
      if (nseg > 1) start = ends + (int64_t)(seg > 0 ? seg - 1 : nseg - 1) * a.H * head;
      if (start && (seg > 0 || a.state_in)) load(start);
    }
    // lambda^128: rounded to fp32 it would be off the same way with every chunk (a head
    // that remembers 4096 tokens by 30 times that), so the walk takes its two fp32
    // neighbours in the proportion that keeps their product on the true power.
    // e^y = (e^(y / 8192))^8192, by a short series and 13 squarings in 64 bits.
    const float y128 = fminf(a.log_decay[h], 0.f) * kC;
    const double r = (double)fmaxf(y128, -110.f) * (1.0 / 8192);   // |r| < 0.0135: the series is good to 2^-52
    double decay = 1.0 + r * (1.0 + r * (1.0 / 2) * (1.0 + r * (1.0 / 3) * (1.0 + r * (1.0 / 4) * (1.0 + r * (1.0 / 5) * (1.0 + r * (1.0 / 6))))));
#pragma unroll 1
    for (int x = 0; x < 13; ++x) decay *= decay;
    if (y128 < -104.f) decay = 0.0;                           // (below fp32's range)
    float below = pw[kC], above = below, part = 0.f, turn = 0.f;
    if (pw[kC] <= 1.f) {                                      // (not NaN)
      below = __double2float_rd(decay);
      above = __double2float_ru(decay);
      if (above > below) part = (float)((decay - (double)below) / ((double)above - (double)below));
    }
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      if (!STATE) {
        // H in the operands' type, once Q H of the chunk before has read the last one.
        if (c > 0 && !(ok = wait_bar_warp(bar(sh->qh_ready), (c - 1) & 1, wc))) break;
        {
          float hf = 1.f;
          if (F16) {
            float mx = 0.f, back;
#pragma unroll
            for (int x = 0; x < DK; ++x) mx = fmaxf(mx, fabsf(H[x]));
            hf = half_range(mx, &back);
            sh->cs[c & 1][d] = exponent_field(back);
          }
#pragma unroll
          for (int x = 0; x < DK; x += 8) {
            uint4 w;
            w.x = pack16<F16>(H[x] * hf, H[x + 1] * hf);
            w.y = pack16<F16>(H[x + 2] * hf, H[x + 3] * hf);
            w.z = pack16<F16>(H[x + 4] * hf, H[x + 5] * hf);
            w.w = pack16<F16>(H[x + 6] * hf, H[x + 7] * hf);
            *reinterpret_cast<uint4*>(Hb + (x >> 6) * (DV * 128) + d * 128 + ((((x >> 3) & 7) ^ (d & 7)) << 4)) = w;
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->h_ready));
      }
      if (c >= deltas) break;
      if (!(ok = wait_bar_warp(bar(sh->dh_ready[Pipe::dh(c)]), Pipe::dh_phase(c), wc))) break;
      tc_fence_after();
      {
        // Forwards, H = lambda^n H + dH; backwards, H = H + lambda^(128 c) dH.
        float f;
        if (STATE) {
          f = exp2f(fmaxf(ld2 * (float)(c * kC), -300.f));
        } else if (ragged && c == chunks - 1) {
          f = pw[last_n];
        } else {
          turn += part;
          f = turn >= 1.f ? above : below;
          if (turn >= 1.f) turn -= 1.f;
        }
        const float vback = F16 ? exponent_value(sh->vs[Pipe::scale(c)][d]) : 1.f;
        const float2 f2 = STATE ? make_float2(f * vback, f * vback) : make_float2(f, f);
#pragma unroll
        for (int x = 0; x < DK; x += 16) {
          uint32_t e[16];
          tmem_ld16(lanes + dh_col(c) + x, e);
          tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            float2 g = make_float2(__uint_as_float(e[y]), __uint_as_float(e[y + 1]));
            const float2 o = make_float2(H[x + y], H[x + y + 1]);
            if (F16 && !STATE) g = mul2(g, make_float2(vback, vback));
            const float2 r = STATE ? fma2(f2, g, o) : fma2(f2, o, g);
            H[x + y] = r.x;
            H[x + y + 1] = r.y;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh->dh_free[Pipe::dh(c)]));
    }
    if (ok && final_state)
      store(STATE ? ends + (int64_t)seg * a.H * head : a.state_out + ((int64_t)place * a.H + h) * head);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// Between the two launches of a split call.  E_s the end state that segment s has on
// its own, each segment starts with
//   P_0 = the request's state,  P_{s+1} = lambda^seg_len P_s + E_s.
// P_{s+1} is written over E_s, and P_0 behind them (state_out may be state_in).  One CTA
// for 256 elements of a split request's head: a thread walks the segments with one
// element, 16 loads in flight.  Bound by latency: 9.4 MB of nine segments of 16 heads are
// in L2 (a CTA for each segment, of which the first works: 20 us more in CTAs that leave).
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads) linear_scan_kernel(const LinearArgs a) {
  __shared__ int req, segs, first, scratch, sums[kScanThreads / 32][2];
  const int head = a.D_k * a.D_v, parts = head / kScanThreads;
  const int part = blockIdx.x % parts, h = blockIdx.x / parts % a.H, k = blockIdx.x / parts / a.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  // The k-th split request in the order of the segments (locate).
  if (tid == 0) req = -1;
  __syncthreads();
  if (a.B <= 32) {
    if (warp == 0) {
      int t0, n = -1, v = 0;
      if (lane < a.B) request(a, lane, t0, n, v);
      int rank = 0, at = 0;
      for (int o = 0; o < a.B; ++o) {
        const int on = __shfl_sync(0xffffffffu, n, o), ov = __shfl_sync(0xffffffffu, v, o);
        if (on > n || (on == n && o < lane)) {
          ++rank;
          at += ov;
        }
      }
      if (rank == k && v > 1) req = lane, segs = v, first = at;
    }
  } else {
    const int per = (a.B + kScanThreads - 1) / kScanThreads;
    int mine[2] = {0, 0}, incl[2];   // split requests, their segments
    for (int b = tid * per; b < min((tid + 1) * per, a.B); ++b) {
      int t0, n, v;
      request(a, b, t0, n, v);
      if (v > 1) ++mine[0], mine[1] += v;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      incl[x] = mine[x];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl[x], o);
        if (lane >= o) incl[x] += t;
      }
      if (lane == 31) sums[warp][x] = incl[x];
    }
    __syncthreads();
    int rank = incl[0] - mine[0], at = incl[1] - mine[1];
    for (int w = 0; w < warp; ++w) rank += sums[w][0], at += sums[w][1];
    for (int b = tid * per; b < min((tid + 1) * per, a.B); ++b) {
      int t0, n, v;
      request(a, b, t0, n, v);
      if (v == 1) continue;
      if (rank == k) req = b, segs = v, first = at;
      ++rank, at += v;
    }
  }
  __syncthreads();
  const float f = exp2f(fmaxf(log2_decay(a.log_decay[h]) * (float)a.seg_len, -300.f));
  const int place = req >= 0 && first + segs <= a.split_segs ? state_place(a, req, &scratch, false) : -1;
  pdl_wait();
  if (place < 0) return;
  const int64_t step = (int64_t)a.H * head;
  float* p = a.seg_state + ((int64_t)first * a.H + h) * head + part * kScanThreads + tid;
  float x = 0.f;
  if (a.state_in) p[(segs - 1) * step] = x = a.state_in[((int64_t)place * a.H + h) * head + part * kScanThreads + tid];
  if (f == 0.f) return;              // (whatever the states before hold)
  for (int s = 0; s < segs - 1; s += 16) {
    float e[16];
#pragma unroll
    for (int y = 0; y < 16; ++y) e[y] = s + y < segs - 1 ? p[(s + y) * step] : 0.f;
#pragma unroll
    for (int y = 0; y < 16; ++y)
      if (s + y < segs - 1) p[(s + y) * step] = x = fmaf(f, x, e[y]);
  }
}

template <int DK, int DV, bool F16>
cudaError_t launch_one(ChunkParams& p, bool split, cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DK, DV>();
  static_assert(smem <= 232448, "shared memory of one CTA");
  const unsigned grid = (unsigned)p.a.segs * (unsigned)p.a.H;
  cudaError_t e;
  if (split) {
    auto states = linear_chunk_kernel<DK, DV, F16, true>;
    if ((e = cudaFuncSetAttribute(states, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
    const unsigned heads = (unsigned)p.a.split_segs * (unsigned)p.a.H;
    if ((e = launch_pdl(states, dim3(heads), dim3(kThreads), smem, st, p)) != cudaSuccess) return e;
    const unsigned requests = (unsigned)std::min(p.a.B, p.a.R / p.a.seg_len);   // that are split, at most
    if ((e = launch_pdl(linear_scan_kernel, dim3(requests * p.a.H * (DK * DV / kScanThreads)), dim3(kScanThreads), 0, st, p.a)) !=
        cudaSuccess)
      return e;
  }
  auto kernel = linear_chunk_kernel<DK, DV, F16, false>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, st, p);
}

template <int DK, int DV>
cudaError_t launch_width(ChunkParams& p, bool f16, bool split, cudaStream_t st) {
  return f16 ? launch_one<DK, DV, true>(p, split, st) : launch_one<DK, DV, false>(p, split, st);
}

}  // namespace

// One walk over a request's n chunks takes about 7 + 2.4 n us.  Split into segments of m
// chunks, the states' launch, the scan and the outputs' launch take about 19 + 4.2 m, if
// the segments fill SMs that would idle.  Measured (width 128, bf16, launches back to back on
// three sets of inputs in turn; us), one walk and segments:
//   tokens x heads   65536 x 16   4096 x 16   4096 x 32   1024 x 16   4096 x 64   512 x 16
//                    1146  244     80   37     85   55     26   22     85   92     16   20
// Where requests and heads alone fill the GPU, only a request that is still walked when
// the others are done is split: n above 1.5 times the chunks of each SM if the work were
// level, in which a request counts its tokens and 3.5 chunks (3 for its start and end, half
// a one for its last, partly filled one).  One request and 100 of 200 tokens:
//   tokens x heads   4096 x 16  8192 x 16  24576 x 32  12288 x 16  16384 x 16  24576 x 16
//   n / level           0.56       1.06       1.30        1.51        1.91        2.60
//                     143  198   177  215   486  490    249  228    321  238    464  262
int linear_seg_len(const dsa_linear_problem& p) {
  constexpr int kWhole = INT32_MAX - 127;
  const int64_t longest = p.rows_max > 0 && p.rows_max < p.R ? p.rows_max : p.R;
  const double n = (double)((longest + 127) / 128);
  int64_t segs = 152 / p.H - (p.B - 1);            // segments that find an SM each
  if (segs < 2) {
    const double even = ((double)p.R / kC + 3.5 * p.B) * p.H / 152;   // chunks of each SM if the work were level
    if (n <= 1.5 * even) return kWhole;
    segs = 152 / p.H > 0 ? 152 / p.H : 1;
  }
  const int64_t len = ((p.R + segs - 1) / segs + 127) / 128 * 128;
  return 2.4 * n > 12.0 + 4.2 * (double)(len / 128) ? (int)len : kWhole;
}

int64_t linear_segs(const dsa_linear_problem& p, int seg_len) { return (int64_t)p.R / seg_len + p.B; }

cudaError_t launch_linear(const LinearArgs& a, bool f16, bool split, cudaStream_t st) {
  ChunkParams p;
  std::memset(&p, 0, sizeof p);
  p.a = a;
  if (a.R > 0) {   // (no tokens: only states are handed on)
    cudaError_t e = chunk_map(&p.tq, a.q, a.R, (int64_t)a.H * a.D_k, a.q_stride);
    if (e == cudaSuccess) e = chunk_map(&p.tk, a.k, a.R, (int64_t)a.H * a.D_k, a.k_stride);
    if (e == cudaSuccess) e = chunk_map(&p.tv, a.v, a.R, (int64_t)a.H * a.D_v, a.v_stride);
    if (e == cudaSuccess) e = chunk_map(&p.to, a.out, a.R, (int64_t)a.H * a.D_v, (int64_t)a.H * a.D_v);
    if (e != cudaSuccess) return e;
  }
  if (a.D_k == 64) return a.D_v == 64 ? launch_width<64, 64>(p, f16, split, st) : launch_width<64, 128>(p, f16, split, st);
  return a.D_v == 64 ? launch_width<128, 64>(p, f16, split, st) : launch_width<128, 128>(p, f16, split, st);
}

}  // namespace dsa
