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
// angle's fraction of a turn without any loss, whatever the position.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
  return (uint64_t)((t - floor(t)) * 18446744073709551616.0);
}

// (cos, sin) of pos * inv_freq.  The angle is in half turns within [-1, 1), off by at most
// 2^-25 from the conversion.
__device__ __forceinline__ float2 turn(uint64_t fraction, int pos) {
  const uint64_t phase = fraction * (uint64_t)(int64_t)pos;
  float2 cs;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &cs.y, &cs.x);
  return cs;
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

// The head's eight columns of this lane, x[0..3] from l.a and x[4..7] from l.b, normed and
// rotated in place.  cs: cos and sin of the lane's four frequencies.  Returns through `off`, where
// wanted, what each value's error is relative to: its own and its partner's magnitudes
// before the rotation; 0 for values that come as they are (see kv4_cache.cu).
template <int D, bool F16, bool Off>
__device__ __forceinline__ void turn_head(const TurnArgs& t, const uint16_t* weight, const HeadLane& l, const float2* cs,
                                          float* x, float* off) {
  // A warp may hold heads of q and of k, of which one alone is normed: all its lanes sum.
  float sum = 0.f;
  if (t.q_weight || t.k_weight) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
    sum = head_sum<D>(sum);
  }
  if (weight) {
    const float r = rsqrtf(fmaf(sum, 1.f / D, t.eps));
    float w[8];
    unpack4<F16>(load4(weight, l.a), w);
    unpack4<F16>(load4(weight, l.b), w + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
  }
  if (Off) {
#pragma unroll
    for (int i = 0; i < 8; ++i) off[i] = weight ? fabsf(x[i]) : 0.f;
  }
  if (l.f < 0) return;
  auto pair = [&](int i, int a, int b) {
    const float u = x[a], v = x[b];
    x[a] = u * cs[i].x - v * cs[i].y;
    x[b] = v * cs[i].x + u * cs[i].y;
    if (Off) off[a] = off[b] = fabsf(u) + fabsf(v);
  };
  if (t.adjacent) {
#pragma unroll
    for (int i = 0; i < 4; ++i) pair(i, 2 * i, 2 * i + 1);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) pair(i, i, i + 4);
  }
}

}  // namespace dsa
