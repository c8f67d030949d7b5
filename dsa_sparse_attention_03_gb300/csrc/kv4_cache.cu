// The 4-bit cache written (dsa_kv4_append) and read back (dsa_kv4_read).
//
// Append.  Keys are normed and rotated (rope.cuh), then each 64 columns of K and V are
// quantised: scale = max |x| / 7 to four significant bits, code = x / scale to the nearest
// whole number.  Four significant bits are rounded to the nearest, not up: the largest
// value is then at most 7.44 scales, still nearest to 7.  A CTA takes one row and some of its
// heads of q, k and v, a head 8 to 32 lanes; K goes through shared memory once, from lanes
// that hold rotated pairs to lanes that hold eight columns in a row, one 32-bit word of codes.
//
// Borders.  A key that was normed or rotated is off by some 2^-20 in fp32, so near the border
// between two codes (or two scales) fp32 cannot tell which one exact arithmetic gives.  Each
// value carries a bound of its error; where a border lies within it, the value is computed
// again in fp64 (about one head in 600).  What the cache holds then does not depend on how
// sums were ordered.  Values that are neither normed nor rotated are quantised exactly: x has at
// most 11 significant bits and a scale 4, so the fp32 quotient is a half only where the real
// one is.
//
// Read.  code * scale, one 32-bit word of codes to 16 bytes; in bf16 by packed products
// that are exact.
//
// Both move each byte once and are bound by HBM, or by latency for few rows.
#include "rope.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
// A normed and rotated value's error in fp32, relative to its own and its partner's
// magnitudes: in units of 2^-24, the sum of squares over a head 13 (8 in a lane, 5 between
// lanes) and its mean and eps 2, of which the root halves to 7.5, the root 4 (2 ulp), two
// products 2, sine or cosine 4 (the angle's conversion and 2 ulp), the rotation 2: 19.5.
constexpr float kTurnErr = 20.f * 0x1p-24f;

// x >= 0 to four significant bits, ties to even; below 2^-126: 0.
__device__ __forceinline__ float four_bits(float x) {
  if (x < 0x1p-126f) return x >= 0x1.fp-127f ? 0x1p-126f : 0.f;
  const uint32_t u = __float_as_uint(x);
  if (u >= 0x7f800000u) return __uint_as_float(0x7fc00000u);   // (a group that is not finite)
  return __uint_as_float((u + 0x7ffffu + ((u >> 20) & 1u)) & ~0xfffffu);
}
__device__ __forceinline__ double four_bits(double x) {
  if (x < 0x1p-126) return x >= 0x1.fp-127 ? 0x1p-126 : 0.0;
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  if (u >= 0x7ff0000000000000ull) return __longlong_as_double(0x7ff8000000000000ll);
  return __longlong_as_double((long long)((u + 0xffffffffffffull + ((u >> 49) & 1ull)) & ~0x1ffffffffffffull));
}

// Eight columns from 8 * j on of the head `x` points at, normed and rotated in fp64: those of
// `mask`.  By a whole warp (the sum of squares takes all the head's lanes).
template <int D, bool F16>
__device__ __noinline__ void turn_exactly(const TurnArgs& t, const uint16_t* x, int pos, int j, uint32_t mask, double* y) {
  double r = 1.0;
  if (t.k_weight) {
    double s = 0.0;
    if (x && j < D / 8)
      for (int i = 0; i < 8; ++i) {
        const double v = to_float<F16>(x[8 * j + i]);
        s = fma(v, v, s);
      }
    for (int o = kHeadLanes<D> / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    r = 1.0 / sqrt(s / D + (double)t.eps);
  }
  if (!x || j >= D / 8) mask = 0;
  auto at = [&](int d) {
    const double v = to_float<F16>(x[d]);
    return t.k_weight ? v * r * (double)to_float<F16>(t.k_weight[d]) : v;
  };
  for (int i = 0; i < 8; ++i) {
    if (!(mask >> i & 1u)) continue;
    const int d = 8 * j + i, c = d - t.first;
    double v = at(d);
    if (c >= 0 && c < t.rot) {
      const int half = t.rot / 2;
      const bool second = t.adjacent ? c & 1 : c >= half;
      const int f = t.adjacent ? c >> 1 : (second ? c - half : c);
      const double p = at(t.adjacent ? t.first + (c ^ 1) : t.first + (second ? c - half : c + half));
      double sn, cs;
      sincospi((double)(int64_t)(turn_fraction(t.inv_freq[f]) * (uint64_t)(int64_t)pos) * 0x1p-63, &sn, &cs);
      v = second ? v * cs + p * sn : v * cs - p * sn;
    }
    y[i] = v;
  }
}

// Eight columns of a head to a word of codes and their group's scale.  `off`: bounds of x's
// errors (all 0: exact).  `head`, `pos`: what turn_exactly needs, head null where the lane
// has none.  Whole warp; a group is eight adjacent lanes.
template <int D, bool F16, bool Turned>
__device__ __forceinline__ uint32_t quantise(const TurnArgs& t, const float* x, const float* off, const uint16_t* head,
                                             int pos, int j, float* scale_out) {
  uint32_t top = 0;   // (as bits: a NaN is then above all)
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float amax = __uint_as_float(top);
  float scale = four_bits(__fdiv_rn(amax, 7.f));
  uint32_t near = 0;   // columns next to a border
  bool wide = false;   // the scale itself may be another one
  if (Turned) {
    float e = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) e = fmaxf(e, off[i]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, o));
    e *= kTurnErr;
    // (2^-22: the quotient's own rounding)
    wide = e > 0.f && four_bits((amax - e) * (1.f - 0x1p-22f) / 7.f) != four_bits((amax + e) * (1.f + 0x1p-22f) / 7.f);
    if (!(scale == scale)) wide = false;
  }
  const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
  int code[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = scale > 0.f ? __fdiv_rn(x[i], scale) : 0.f;
    const float n = rintf(q);
    code[i] = (int)n;
    // (2^-21: the quotient's rounding, at most 2^-22, and what off * inv itself is off by)
    if (Turned && off[i] > 0.f && fabsf(q - n) > 0.5f - 0x1p-21f - off[i] * kTurnErr * inv) near |= 1u << i;
  }
  if (Turned && __any_sync(0xffffffffu, near | (uint32_t)wide)) {
    double y[8];
    turn_exactly<D, F16>(t, head, pos, j, wide ? 0xffu : near, y);
    double s = scale;
    double m = 0.0;
    if (wide && head && j < D / 8)
      for (int i = 0; i < 8; ++i) m = fmax(m, fabs(y[i]));
    for (int o = 4; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (wide) {
      s = four_bits(m / 7.0);
      scale = (float)s;
      near = 0xffu;
    }
    if (head && j < D / 8)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (near >> i & 1u) code[i] = s > 0.0 ? (int)rint(y[i] / s) : 0;
  }
  *scale_out = scale;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= ((uint32_t)(code[i] + 8) & 15u) << (4 * i);
  return word;
}

template <int DK, int DV, bool F16>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const TurnArgs t, const CacheArgs c, uint32_t* status) {
  constexpr int L = kHeadLanes<DK>, S = kThreads / L;
  __shared__ float2 cs[128];
  __shared__ __align__(16) float2 ys[S][DK];      // a key's values and their error bounds
  const int tid = threadIdx.x, lane = tid & 31, j = tid % L, slot = tid / L;
  const int row = blockIdx.x / t.chunks, chunk = blockIdx.x - row * t.chunks;
  const int tasks = t.H_q + 2 * c.H_kv;           // heads of q, then of k, then of v
  const int x0 = (int)((int64_t)tasks * chunk / t.chunks), x1 = (int)((int64_t)tasks * (chunk + 1) / t.chunks);
  const HeadLane l = head_lane<DK>(t, j);
  pdl_trigger();
  const int pos = t.positions[row];
  const int b = find_request(t.row_offsets, t.B, row, lane);
  if (pos < 0 || b < 0) return;
  const int64_t page = find_page(c, b, pos);
  const int place = pos & (c.ps - 1);
  if (page < 0 && chunk == 0 && tid == 0) {
    pdl_wait();                                   // (the status block is cleared)
    raise_status(status, DSA_DEVICE_BAD_INDEX);
  }
  if (tid < t.rot / 2) cs[tid] = turn(turn_fraction(t.inv_freq[tid]), pos);
  __syncthreads();
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = l.f >= 0 ? cs[l.f + i] : make_float2(1.f, 0.f);
  for (int base = x0; base < x1; base += S) {
    const int x = base + slot;
    const bool is_q = x < t.H_q, is_k = !is_q && x < t.H_q + c.H_kv, live = x < x1;
    // Heads of q and k.
    if (base < t.H_q + c.H_kv) {                  // (the same for a whole CTA)
      const int h = is_q ? x : x - t.H_q;
      const uint16_t* src = is_q ? t.q + row * t.q_stride + (int64_t)h * DK : t.k + row * t.k_stride + (int64_t)h * DK;
      const bool mine = live && (is_q || is_k);
      float y[8], off[8];
      unpack4<F16>(mine ? load4(src, l.a) : make_uint2(0, 0), y);
      unpack4<F16>(mine ? load4(src, l.b) : make_uint2(0, 0), y + 4);
      turn_head<DK, F16, true>(t, is_q ? t.q_weight : t.k_weight, l, f, y, off);
      if (mine && is_q && l.a >= 0) {
        uint16_t* p = t.q_out + row * t.q_out_stride + (int64_t)h * DK;
        *reinterpret_cast<uint2*>(p + l.a) = make_uint2(pack16<F16>(y[0], y[1]), pack16<F16>(y[2], y[3]));
        *reinterpret_cast<uint2*>(p + l.b) = make_uint2(pack16<F16>(y[4], y[5]), pack16<F16>(y[6], y[7]));
      }
      if (l.a >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ys[slot][l.a + i] = make_float2(y[i], off[i]);
          ys[slot][l.b + i] = make_float2(y[4 + i], off[4 + i]);
        }
      }
      __syncwarp();
      float off8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 v = j < DK / 8 ? ys[slot][8 * j + i] : make_float2(0.f, 0.f);
        y[i] = is_k ? v.x : 0.f;
        off8[i] = is_k ? v.y : 0.f;
      }
      __syncwarp();
      float scale;
      const uint32_t word = quantise<DK, F16, true>(t, y, off8, live && is_k ? src : nullptr, pos, j, &scale);
      if (live && is_k && page >= 0 && j < DK / 8) {
        uint8_t* p = c.pages + page + (int64_t)h * c.block;
        const uint32_t at = (j >> 3) * c.ps + place;
        *reinterpret_cast<uint32_t*>(p + at * 32 + (j & 7) * 4) = word;
        if ((j & 7) == 0)
          *reinterpret_cast<uint16_t*>(p + c.ps * ((DK + DV) / 2) + at * 2) = (uint16_t)(__float_as_uint(scale) >> 16);
      }
    }
    // Heads of v: eight columns to a lane.
    if (base + S > t.H_q + c.H_kv) {              // (the same for a whole CTA)
      const int h = x - t.H_q - c.H_kv;
      const bool mine = live && h >= 0 && j < DV / 8;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (mine) w = *reinterpret_cast<const uint4*>(t.v + row * t.v_stride + (int64_t)h * DV + 8 * j);
      float y[8], scale;
      unpack4<F16>(make_uint2(w.x, w.y), y);
      unpack4<F16>(make_uint2(w.z, w.w), y + 4);
      const uint32_t word = quantise<DV, F16, false>(t, y, nullptr, nullptr, 0, j, &scale);
      if (mine && page >= 0) {
        uint8_t* p = c.pages + page + (int64_t)h * c.block;
        const uint32_t at = (j >> 3) * c.ps + place;
        *reinterpret_cast<uint32_t*>(p + c.ps * (DK / 2) + at * 32 + (j & 7) * 4) = word;
        if ((j & 7) == 0)
          *reinterpret_cast<uint16_t*>(p + c.ps * ((DK + DV) / 2 + DK / 32) + at * 2) = (uint16_t)(__float_as_uint(scale) >> 16);
      }
    }
  }
}

// Eight codes times their scale, in 16 bits.
template <bool F16>
__device__ __forceinline__ uint4 dequantise(uint32_t w, uint16_t scale) {
  uint32_t o[4];
  if (F16) {
    const float s = __uint_as_float((uint32_t)scale << 16);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack16<true>((float)((int)(w >> (8 * i) & 15u) - 8) * s, (float)((int)(w >> (8 * i + 4) & 15u) - 8) * s);
  } else {
    const __nv_bfloat162 s = __halves2bfloat162(__ushort_as_bfloat16(scale), __ushort_as_bfloat16(scale));
    const __nv_bfloat162 zero = __floats2bfloat162_rn(-136.f, -136.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = w >> (8 * i);
      uint32_t u = (b & 15u) | ((b & 0xf0u) << 12) | 0x43004300u;   // 128 + code, twice
      const __nv_bfloat162 v = __hmul2(__hadd2(*reinterpret_cast<__nv_bfloat162*>(&u), zero), s);
      o[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int kReadRows = 16;   // rows of a CTA

template <int DK, int DV, bool F16>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const CacheArgs c, int R, const int32_t* row_offsets, const int32_t* positions, uint16_t* k_out,
                    uint16_t* v_out, uint32_t* status) {
  __shared__ int64_t pages[kReadRows];
  __shared__ int places[kReadRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row0 = (int64_t)blockIdx.x * kReadRows;
  pdl_trigger();
  for (int i = warp; i < kReadRows; i += kThreads / 32) {
    const int64_t row = row0 + i;
    int64_t page = -1;
    int pos = -1;
    if (row < R) {
      pos = positions[row];
      const int b = find_request(row_offsets, c.B, (int)row, lane);
      if (pos >= 0 && b >= 0) {
        page = find_page(c, b, pos);
        if (page < 0 && lane == 0) {
          pdl_wait();
          raise_status(status, DSA_DEVICE_BAD_INDEX);
        }
      }
    }
    if (lane == 0) {
      pages[i] = page;
      places[i] = pos & (c.ps - 1);
    }
  }
  __syncthreads();
  constexpr int WK = DK / 8, WV = DV / 8;      // words of a head
  auto half = [&](uint16_t* out, int W, uint32_t codes, uint32_t scales) {
    const int per = c.H_kv * W;
    for (int x = tid; x < kReadRows * per; x += kThreads) {
      const int i = x / per, y = x - i * per, h = y / W, j = y - h * W;
      const int64_t page = pages[i];
      if (page < 0) continue;
      const uint8_t* p = c.pages + page + (int64_t)h * c.block;
      const uint32_t at = (j >> 3) * c.ps + places[i];
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p + codes + at * 32 + (j & 7) * 4);
      const uint16_t s = *reinterpret_cast<const uint16_t*>(p + scales + at * 2);
      *reinterpret_cast<uint4*>(out + ((row0 + i) * per + y) * 8) = dequantise<F16>(w, s);
    }
  };
  if (k_out) half(k_out, WK, 0, c.ps * ((DK + DV) / 2));
  if (v_out) half(v_out, WV, c.ps * (DK / 2), c.ps * ((DK + DV) / 2 + DK / 32));
}

template <int DK, int DV>
cudaError_t launch_append_width(TurnArgs t, const CacheArgs& c, bool f16, uint32_t* status, cudaStream_t st) {
  constexpr int S = kThreads / kHeadLanes<DK>;
  // CTAs to a row: heads one after the other where the rows fill the GPU, else spread.
  const int tasks = t.H_q + 2 * c.H_kv, most = (tasks + S - 1) / S;
  t.chunks = 1;
  while (t.chunks < most && (int64_t)t.R * t.chunks < 608) ++t.chunks;
  const dim3 grid((unsigned)((int64_t)t.R * t.chunks));
  return f16 ? launch_pdl(kv4_append_kernel<DK, DV, true>, grid, dim3(kThreads), 0, st, t, c, status)
             : launch_pdl(kv4_append_kernel<DK, DV, false>, grid, dim3(kThreads), 0, st, t, c, status);
}

template <int DK, int DV>
cudaError_t launch_read_width(const CacheArgs& c, int R, const int32_t* row_offsets, const int32_t* positions, bool f16,
                              uint16_t* k_out, uint16_t* v_out, uint32_t* status, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)R + kReadRows - 1) / kReadRows));
  return f16 ? launch_pdl(kv4_read_kernel<DK, DV, true>, grid, dim3(kThreads), 0, st, c, R, row_offsets, positions, k_out, v_out, status)
             : launch_pdl(kv4_read_kernel<DK, DV, false>, grid, dim3(kThreads), 0, st, c, R, row_offsets, positions, k_out, v_out, status);
}

}  // namespace

cudaError_t launch_kv4_append(TurnArgs a, const CacheArgs& c, int D_k, int D_v, bool f16, uint32_t* status, cudaStream_t st) {
  (void)D_v;
  if (D_k == 64) return launch_append_width<64, 64>(a, c, f16, status, st);
  if (D_k == 128) return launch_append_width<128, 128>(a, c, f16, status, st);
  return launch_append_width<192, 128>(a, c, f16, status, st);
}

cudaError_t launch_kv4_read(const CacheArgs& c, int R, const int32_t* row_offsets, const int32_t* positions, int D_k, int D_v,
                            bool f16, uint16_t* k_out, uint16_t* v_out, uint32_t* status, cudaStream_t st) {
  (void)D_v;
  if (D_k == 64) return launch_read_width<64, 64>(c, R, row_offsets, positions, f16, k_out, v_out, status, st);
  if (D_k == 128) return launch_read_width<128, 128>(c, R, row_offsets, positions, f16, k_out, v_out, status, st);
  return launch_read_width<192, 128>(c, R, row_offsets, positions, f16, k_out, v_out, status, st);
}

}  // namespace dsa
