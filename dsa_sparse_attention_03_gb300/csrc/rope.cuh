// Norm and rotation of one head's row, shared by rope.cu and kv4_cache.cu.
//
// D / 8 lanes hold a head: two vectors of four columns each, so that a rotated pair
// lies in one lane whatever the pairing.  With halves rot / 2 apart the vectors of lane
// j are columns 4 j.. of either half; with adjacent pairs they are eight columns in a
// row.  Columns that do not rotate follow, four at a time, over the remaining lanes.
#pragma once

#include "kv4.cuh"
#include "tc.cuh"

namespace dsa {

// Lanes that a head takes (a power of two; the first D / 8 of them hold columns).
template <int D>
constexpr int kHeadLanes = D == 64 ? 8 : (D == 128 ? 16 : 32);

// Sum over the head's lanes.
template <int D>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = kHeadLanes<D> / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// inv_freq in turns a position, as a 64-bit fraction: position times it, modulo 2^64, is the
// angle's fraction of a turn without any loss, whatever the position.  In whole numbers (the
// fp64 unit does two operations a cycle and SM: 9601 rows took 104 us for it): inv_freq is
// M 2^E, and 1 / (2 pi) is C 2^-66 within 2^-67, so the fraction is M C 2^(E - 2) modulo 2^64.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  const uint64_t u = (uint64_t)__double_as_longlong(inv_freq);
  const int e = (int)(u >> 52 & 0x7ff);
  const uint64_t m = (u & 0xfffffffffffffull) | (e ? 1ull << 52 : 0), C = 0xa2f9836e4e44152aull;   // 2^66 / (2 pi)
  const uint64_t hi = __umul64hi(m, C), lo = m * C;
  const int right = 1077 - (e ? e : 1);   // 2 - E
  uint64_t f = 0;
  if (right >= 64)
    f = right < 128 ? hi >> (right - 64) : 0;
  else if (right > 0)
    f = hi << (64 - right) | lo >> right;
  else if (right > -64)
    f = lo << -right;
  return u >> 63 ? 0 - f : f;
}

// (cos, sin) of `fraction` 2^-64 turns: quarter turns exactly, the rest, at most an eighth, by the Taylor
// series up to y^9 and y^10 (what is left out is below 2^-25), off by at most 4 * 2^-24 in all.
__device__ __forceinline__ float2 cos_sin(uint64_t fraction) {
  const uint32_t p = (uint32_t)(fraction >> 32), q = (p + 0x20000000u) >> 30;
  const float y = (float)(int32_t)(p - (q << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float z = y * y;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f), c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  s = fmaf(z, s, 8.3333333e-3f);
  c = fmaf(z, c, -1.3888889e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  c = fmaf(z, c, 4.1666667e-2f);
  s = fmaf(z * y, s, y);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float a = q & 1 ? s : c, b = q & 1 ? c : s;                           // cos, sin up to their signs
  return make_float2((q + 1) & 2 ? -a : a, q & 2 ? -b : b);
}
// The same in fp64 by the series up to y^17 and y^16, below 2^-50 off (a library function's code is longer, and this is
// code that an SM runs once).
__device__ __forceinline__ double2 cos_sin_exactly(uint64_t fraction) {
  const uint32_t q = (uint32_t)((fraction + (1ull << 61)) >> 62);
  const double y = (double)(int64_t)(fraction - ((uint64_t)q << 62)) * 3.40612158008655459e-19;   // 2 pi / 2^64
  const double z = -y * y;
  // (over (2 i + 1)! and (2 i)!)
  constexpr double over[9] = {1.0, 1.0 / 2, 1.0 / 24, 1.0 / 720, 1.0 / 40320, 1.0 / 3628800, 1.0 / 479001600, 1.0 / 87178291200.0,
                              1.0 / 20922789888000.0};
  double s = over[8] / 17, c = over[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    s = fma(z, s, over[i] / (2 * i + 1));
    c = fma(z, c, over[i]);
  }
  s *= y;
  const double a = q & 1 ? s : c, b = q & 1 ? c : s;
  return make_double2((q + 1) & 2 ? -a : a, q & 2 ? -b : b);
}

struct HeadLane {
  int a, b;      // first columns of the two vectors, or -1: the lane holds none
  int f;         // first of its four frequencies, or -1: the lane's columns do not rotate
};
template <int D>
__device__ __forceinline__ HeadLane head_lane(const TurnArgs& t, int j) {
  HeadLane l = {-1, -1, -1};
  if (j >= D / 8) return l;
  if (8 * j < t.rot) {
    l.f = 4 * j;
    l.a = t.first + (t.adjacent ? 8 * j : 4 * j);
    l.b = t.adjacent ? l.a + 4 : l.a + t.rot / 2;
  } else {
    const int u = 8 * j - t.rot;     // columns that do not rotate, before this lane's
    l.a = u < t.first ? u : u + t.rot;
    l.b = u + 4 < t.first ? u + 4 : u + 4 + t.rot;
  }
  return l;
}

template <bool F16>
__device__ __forceinline__ void unpack4(uint2 w, float* x) {
  x[0] = to_float<F16>((uint16_t)w.x);
  x[1] = to_float<F16>((uint16_t)(w.x >> 16));
  x[2] = to_float<F16>((uint16_t)w.y);
  x[3] = to_float<F16>((uint16_t)(w.y >> 16));
}

__device__ __forceinline__ uint2 load4(const uint16_t* row, int col) {
  return col < 0 ? make_uint2(0, 0) : *reinterpret_cast<const uint2*>(row + col);
}

// The angles' cos and sin of a CTA's rows, worked out once for all heads and columns.
constexpr int kTurnRows = 8, kTurnThreads = 256;
typedef float2 RowTurns[kTurnRows][128];
__device__ __forceinline__ void row_turns(const TurnArgs& t, RowTurns& cs, int row0) {
  for (int i = threadIdx.x >> 6; i >> t.rows_log2 == 0 && row0 + i < t.R; i += kTurnThreads / 64)
    for (int f = threadIdx.x & 63; f < t.rot / 2; f += 64)
      cs[i][f] = cos_sin(turn_fraction(t.inv_freq[f]) * (uint64_t)(int64_t)t.positions[row0 + i]);
}
// The units (a run of heads, a row of the CTA's) that this CTA's warps share: run u >> rows_log2 of row
// u & mask, so that each warp gets runs of every kind.
__device__ __forceinline__ void cta_units(const TurnArgs& t, int runs, int& row0, int& u0, int& u1) {
  row0 = blockIdx.x << t.rows_log2;
  u0 = blockIdx.y * t.units;
  u1 = min(u0 + t.units, runs << t.rows_log2);
}
__device__ __forceinline__ void run_heads(const TurnArgs& t, int n, int run, int& h0, int& h1) {
  h0 = run << t.run_log2;
  h1 = min(h0 + (1 << t.run_log2), n);
}

// What a lane keeps of its columns: cos and sin of its frequencies, the norm's weights.
struct LaneTurn {
  float2 cs[4];
  float w[8];
};
template <bool F16>
__device__ __forceinline__ LaneTurn lane_turn(const float2* cs, const uint16_t* weight, const HeadLane& l) {
  LaneTurn x;
  if (l.f >= 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x.cs[i] = cs[l.f + i];
  }
  if (weight) {
    unpack4<F16>(load4(weight, l.a), x.w);
    unpack4<F16>(load4(weight, l.b), x.w + 4);
  }
  return x;
}

// The head's eight columns of this lane, x[0..3] from l.a and x[4..7] from l.b, normed and rotated in
// place.  By whole warps; `norm` is the same for all heads of a warp.
template <int D>
__device__ __forceinline__ void turn_head(const TurnArgs& t, bool norm, const HeadLane& l, const LaneTurn& y, float* x) {
  if (norm) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
    const float r = rsqrtf(fmaf(head_sum<D>(sum), 1.f / D, t.eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r * y.w[i];
  }
  if (l.f < 0) return;
  auto pair = [&](int i, int a, int b) {
    const float u = x[a], v = x[b];
    x[a] = u * y.cs[i].x - v * y.cs[i].y;
    x[b] = v * y.cs[i].x + u * y.cs[i].y;
  };
  if (t.adjacent) {
#pragma unroll
    for (int i = 0; i < 4; ++i) pair(i, 2 * i, 2 * i + 1);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) pair(i, i, i + 4);
  }
}

// Heads h0 .. h1 - 1 of one row, by one warp, 32 / kHeadLanes at a time: `src` to `dst`, which may be the
// same.  Loads of four rounds are under way together.
template <int D, bool F16>
__device__ __forceinline__ void turn_row(const TurnArgs& t, const uint16_t* weight, const float2* cs, const uint16_t* src,
                                         uint16_t* dst, int h0, int h1, int lane) {
  constexpr int L = kHeadLanes<D>, S = 32 / L, U = 4;
  const int sub = lane / L;
  const HeadLane l = head_lane<D>(t, lane % L);
  LaneTurn y;
  for (int base = h0; base < h1; base += U * S) {
    uint2 v[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = base + u * S + sub;
      const uint16_t* p = src + (int64_t)h * D;
      v[u][0] = h < h1 ? load4(p, l.a) : make_uint2(0, 0);
      v[u][1] = h < h1 ? load4(p, l.b) : make_uint2(0, 0);
    }
    if (base == h0) y = lane_turn<F16>(cs, weight, l);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * S >= h1) break;
      const int h = base + u * S + sub;
      float x[8];
      unpack4<F16>(v[u][0], x);
      unpack4<F16>(v[u][1], x + 4);
      turn_head<D>(t, weight != nullptr, l, y, x);
      if (h < h1 && l.a >= 0) {
        uint16_t* p = dst + (int64_t)h * D;
        *reinterpret_cast<uint2*>(p + l.a) = make_uint2(pack16<F16>(x[0], x[1]), pack16<F16>(x[2], x[3]));
        *reinterpret_cast<uint2*>(p + l.b) = make_uint2(pack16<F16>(x[4], x[5]), pack16<F16>(x[6], x[7]));
      }
    }
  }
}

}  // namespace dsa
