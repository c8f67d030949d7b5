// The 4-bit cache written (dsa_kv4_append) and read back (dsa_kv4_read).
//
// Append.  Keys are normed and rotated (rope.cuh), then each 64 columns of K and V are
// quantised: scale = max |x| / 7 to four significant bits, code = x / scale to the nearest
// whole number.  Four significant bits are rounded to the nearest, not up: the largest
// value is then at most 7.44 scales, still nearest to 7.  A CTA takes up to eight rows, its warps
// runs of a row's heads of q, k and v; a head takes 8 to 32 lanes.  A key is quantised in the
// layout in which it is rotated (two vectors of four columns a lane, 16 bits of codes each).
//
// Borders.  A key that was normed or rotated is off by some 2^-20 in fp32, so near the border
// between two codes (or two scales) fp32 cannot tell which one exact arithmetic gives.  Each
// head has a bound of its values' errors; where a border lies within it (one head in 200), each value's own
// bound is looked at, and where that leaves it open (one head in 500) the value is computed again in
// fp64, after the warp's run of heads, so that the common path keeps its registers.  What the
// cache holds then does not depend on how sums were ordered.  Values
// that are neither normed nor rotated are quantised exactly: x has at most 11 significant bits
// and a scale 4, so a quotient is a half or well off one.
//
// Read.  code * scale, 8 bytes of codes of a lane to 32 bytes of values, by packed products that
// are exact in bf16 (kv4_widen.cuh).
//
// Both move each byte once.  Measured: 9601 rows of 8 + 8 heads of 128 appended in 32 us (1.6 TB/s:
// 22.6 million warp instructions, 62% of the issue slots; the quantising of keys, some 230 instructions
// for two heads, is most of it; 5 us are the last heads computed again), a prefix of 10240 positions read in 12.8 us
// (4.1 TB/s, in fp16 as well; a wave of CTAs that look up, load and write in step), 8000 positions of 64 heads of 192 + 128 in 71 us
// (5.9 TB/s).  Prefetching the rows into L2 at the start gained 1 us.
#include "kv4_widen.cuh"
#include "rope.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
// A normed and rotated value's error in fp32, relative to its own and its partner's
// magnitudes: in units of 2^-24, the sum of squares over a head 13 (8 in a lane, 5 between
// lanes) and its mean and eps 2, of which the root halves to 7.5, the root 4 (2 ulp), two
// products 2, sine or cosine 4, the rotation 2: 19.5.
constexpr float kTurnErr = 20.f * 0x1p-24f;

// max / 7 to four significant bits, ties to even; below 2^-126: 0.  From the product with the rounded
// 1 / 7, whose first four bits may be one too few; on which side of the border above them max / 7
// lies is then told exactly, by seven times the border (five significant bits).  `exact`: the same
// maximum, or what fp64 makes of it (the four bits may then also be one too many, just below max / 7's
// own: no border lies between).
template <typename T>
__device__ __forceinline__ float group_scale(float top, T exact) {
  const uint32_t base = __float_as_uint(top * (1.f / 7.f)) & ~0xfffffu;
  const T border = 7.f * __uint_as_float(base | 0x80000u);
  const bool up = exact > border || (exact == border && (base >> 20 & 1u));
  float scale = __uint_as_float(up ? base + 0x100000u : base);
  if (top < 0x1.cp-124f) scale = exact >= T(0x1.b2p-124) ? 0x1p-126f : 0.f;  // 7, and 7 * 31 / 32, times 2^-126
  return top <= 3.4028234e38f ? scale : __uint_as_float(0x7fc00000u);        // (a group that is not finite)
}

// A code, x / scale to the nearest whole number and 8, in the low bits of 12582920 + x / scale (1.5 * 2^23 + 8:
// fp32 there holds whole numbers, and the sum is rounded to the nearest, ties to even).
constexpr float kCode = 12582920.f;
__device__ __forceinline__ float code(float x, float inv) { return fmaf(x, inv, kCode); }
// The same for x of at most 11 significant bits and a scale of four, ties included: the quotient lies on a
// half or at least 2^-13 off one, so x times the rounded inverse, itself rounded to multiples of 2^-14
// (768 is 1.5 * 2^9), is a half exactly where it has to be.
__device__ __forceinline__ float code_exactly(float x, float inv) { return __fadd_rn(fmaf(x, inv, 768.f), kCode - 768.f); }

// Codes of four columns, 16 bits (with what lies above them).
__device__ __forceinline__ uint32_t pack_codes(const float* c) {
  return __float_as_uint(c[0]) - 0x4b400000u + ((__float_as_uint(c[1]) - 0x4b400000u) << 4) +
         ((__float_as_uint(c[2]) - 0x4b400000u) << 8) + ((__float_as_uint(c[3]) - 0x4b400000u) << 12);
}

// The scale's inverse within 2^-23 of it (scales are at most 2^126); 0 where there is none.
__device__ __forceinline__ float inverse(float scale) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(scale));
  return scale > 0.f ? y : 0.f;
}

// The larger; a NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ double max_nan(double a, double b) { return fmax(a, b); }

// Largest of the lanes' values for each group of 64 columns: va of the group that holds l.a, vb of l.b's.
// Returned are this lane's two groups' (x: l.a's, y: l.b's) and the head's.
template <int D, typename T>
__device__ __forceinline__ T group_max(const HeadLane& l, T va, T vb, T& x, T& y) {
  T all = 0;
#pragma unroll
  for (int g = 0; g < D / 64; ++g) {
    const bool a = l.a >= 0 && l.a / 64 == g, b = l.b >= 0 && l.b / 64 == g;
    T m = max_nan(a ? va : T(0), b ? vb : T(0));
#pragma unroll
    for (int o = kHeadLanes<D> / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (a) x = m;
    if (b) y = m;
    all = max_nan(all, m);
  }
  return all;
}

// A key's eight columns of this lane, four from l.a and four from l.b: their codes, 16 bits each, and
// their groups' scales.
struct Held {
  uint32_t codes[2];
  float scale[2];
};

// Whether fp32 leaves a scale open: the border above its four bits lies within the errors.  Below 2^-126 it is the one from which
// on a scale is 2^-126: 31 / 32 of that, 0x7c0000.
__device__ __forceinline__ bool open_scale(float top, float e) {
  const float m = top * (1.f / 7.f), border = __uint_as_float(max((__float_as_uint(m) & ~0xfffffu) | 0x80000u, 0x7c0000u));
  return fabsf(m - border) <= fmaf(m, 0x1p-22f, e * (1.f / 7.f));   // (2^-22: the product's own rounding)
}
// A bound of the errors of a head's values, of which `all` is the largest.  A pair's magnitudes before the rotation add up
// to at most twice the larger one after it.  No bound where a value is NaN: the other groups' are looked at one by one.
__device__ __forceinline__ float head_error(float all) { return fminf(2.f * kTurnErr * all, INFINITY); }
// A quotient nearer to a half than that may be rounded wrongly (2^-18: its own and the inverse's
// roundings, of at most 7.5, and the bound's).
__device__ __forceinline__ float open_code(float e, float inv) { return 0.5f - 0x1p-18f - e * inv; }

// Whether the 64 columns that hold column d have any that is normed or rotated: the others come as they are,
// and their scale is exact (one bf16 maximum in sixteen lies on a border).
__device__ __forceinline__ bool group_turned(const TurnArgs& t, int d) {
  const int g = d & ~63;
  return t.k_weight || (t.rot > 0 && t.first < g + 64 && t.first + t.rot > g);
}

// Column d of the head at `x`, normed by the factor r and rotated, in fp64.
template <bool F16>
__device__ __noinline__ double turned_exactly(const TurnArgs& t, const uint16_t* x, double r, int pos, int d) {
  auto value = [&](int d) {
    const double v = to_float<F16>(x[d]);
    return t.k_weight ? v * (double)to_float<F16>(t.k_weight[d]) : v;
  };
  const int c = d - t.first;
  if (c < 0 || c >= t.rot) return value(d) * r;
  const int half = t.rot / 2;
  const bool second = t.adjacent ? c & 1 : c >= half;
  const int f = t.adjacent ? c >> 1 : (second ? c - half : c);
  const double v = value(d), p = value(t.first + (t.adjacent ? c ^ 1 : (second ? c - half : c + half)));
  const double2 cs = cos_sin_exactly(turn_fraction(t.inv_freq[f]) * (uint64_t)(int64_t)pos);
  return (second ? v * cs.x + p * cs.y : v * cs.x - p * cs.y) * r;
}

// The same with what fp32 leaves open computed in fp64 from the head at `x` (null: the lane has none):
// the largest values of a group whose scale is open, then the columns next to a border.  Whole warp.
// It runs seldom, so its time is that of its code's way into the SM and of a chain of fp64 operations, two a cycle
// and SM: as few of them as may be, and no division, square root or library function (with those a head
// took 7 us, and 9601 rows 35).
template <int D, bool F16>
__device__ __noinline__ Held hold_exactly(const TurnArgs& t, const float2* cs, const uint16_t* x, int pos, int lane) {
  const HeadLane l = head_lane<D>(t, lane % kHeadLanes<D>);
  const bool live = x && l.a >= 0, turned = t.k_weight || l.f >= 0;
  float y[8];
  unpack4<F16>(live ? load4(x, l.a) : make_uint2(0, 0), y);
  unpack4<F16>(live ? load4(x, l.b) : make_uint2(0, 0), y + 4);
  double r = 1.0;
  if (t.k_weight) {
    // (squares of 11 bits are exact in fp32, or below 2^-126 off by less than 2^-50 of the mean in its range, and so is
    // what each sum is off by: low holds these)
    float high = 0.f, low = 0.f;
    auto add = [&](float x) {
      const float sum = high + x, part = sum - high;
      low += (high - (sum - part)) + (x - part);
      high = sum;
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) add(y[i] * y[i]);
#pragma unroll
    for (int o = kHeadLanes<D> / 2; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, high, o);
      low += __shfl_xor_sync(0xffffffffu, low, o);
      add(x);
    }
    const double s = fma((double)high + (double)low, 1.0 / D, (double)t.eps);   // (D = 192: 1 / D is off by 2^-54 of it)
    // s r^2 = 1 - e: r / sqrt(1 - e) by the binomial series, 1 + e / 2 + 3 e^2 / 8, and e is below 2^-21.
    r = (double)rsqrtf((float)s);
    const double e = fma(-s * r, r, 1.0);
    r = fma(r * e, fma(0.375, e, 0.5), r);
  }
  turn_head<D>(t, t.k_weight != nullptr, l, lane_turn<F16>(cs, t.k_weight, l), y);
  auto four = [&](const float* v) { return max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3]))); };
  float top[2] = {0.f, 0.f}, scale[2];
  const float all = group_max<D>(l, four(y), four(y + 4), top[0], top[1]);
  const bool exact = !t.k_weight && t.rot == 0;
  const float e = exact ? 0.f : head_error(all);
  double most[2] = {0.0, 0.0}, most_of[2] = {0.0, 0.0};
  bool open[2];
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    scale[v] = group_scale(top[v], top[v]);
    open[v] = scale[v] == scale[v] && group_turned(t, v ? l.b : l.a) && open_scale(top[v], e);
  }
  if (__any_sync(0xffffffffu, open[0] || open[1])) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const int v = i >> 2;
      if ((v ? open[1] : open[0]) && live && fabsf(y[i]) >= (v ? top[1] : top[0]) - 2.f * e) {
        const double x0 = fabs(turned_exactly<F16>(t, x, r, pos, (v ? l.b : l.a) + (i & 3)));
        most[v] = fmax(most[v], x0);
      }
    }
    // (an open group is open for all its lanes)
    group_max<D>(l, most[0], most[1], most_of[0], most_of[1]);
#pragma unroll
    for (int v = 0; v < 2; ++v)
      if (open[v]) scale[v] = group_scale(top[v], most_of[v]);
  }
  Held h;
  uint32_t left = 0;                                 // columns next to a border
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float inv = inverse(scale[v]), border = open_code(e, inv);
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = y[4 * v + i];
      c[i] = turned ? code(x0, inv) : code_exactly(x0, inv);
      if (turned && live && fabsf(fmaf(x0, inv, kCode - c[i])) > border && scale[v] > 0.f) left |= 1u << (4 * v + i);
    }
    h.codes[v] = pack_codes(c) & 0xffffu;
    h.scale[v] = scale[v];
  }
  while (__any_sync(0xffffffffu, left)) {
    if (left) {
      // fp32's code is at most one off: what it leaves of the value, against half a scale.
      const int i = __ffs(left) - 1, at = 4 * (i & 3);
      left &= left - 1;
      const uint32_t codes = i < 4 ? h.codes[0] : h.codes[1];
      const int k = (int)(codes >> at & 15u) - 8;
      const float sc = i < 4 ? scale[0] : scale[1];
      const double half = 0.5 * (double)sc;
      const double rest = fma((double)-k, (double)sc, turned_exactly<F16>(t, x, r, pos, (i < 4 ? l.a : l.b) + (i & 3)));
      const int up = (rest > half || (rest == half && (k & 1))) - (rest < -half || (rest == -half && (k & 1)));
      if (i < 4) h.codes[0] += up << at;
      else h.codes[1] += up << at;
    }
  }
  return h;
}

// The same in fp32; false where that leaves something open.  x: normed and rotated.  Whole warp.
template <int D>
__device__ __forceinline__ bool hold_key(const TurnArgs& t, const float* x, const HeadLane& l, Held& h) {
  auto four = [&](const float* v) { return max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3]))); };
  float top[2] = {0.f, 0.f};
  const float all = group_max<D>(l, four(x), four(x + 4), top[0], top[1]);
  // (columns that are neither normed nor rotated come as they are)
  const bool exact = !t.k_weight && t.rot == 0, turned = t.k_weight || l.f >= 0;
  const float e = exact ? 0.f : head_error(all);
  bool open = false;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float scale = group_scale(top[v], top[v]), inv = inverse(scale);
    open |= group_turned(t, v ? l.b : l.a) && open_scale(top[v], e);
    float c[4], d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = code(x[4 * v + i], inv);
      d[i] = fabsf(fmaf(x[4 * v + i], inv, kCode - c[i]));
    }
    if (turned) {
      open |= max3(d[0], d[1], fmaxf(d[2], d[3])) > open_code(e, inv);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = code_exactly(x[4 * v + i], inv);
    }
    h.codes[v] = pack_codes(c);
    h.scale[v] = scale;
  }
  return !open;
}

// What hold_key leaves open with a bound for the whole head, looked at with each value's own: 19.5 units times
// the magnitudes of its pair before the rotation, which add up to at most sqrt 2 times those after it.
template <int D>
__device__ __noinline__ bool still_open(const TurnArgs& t, float4 xa, float4 xb, HeadLane l, float2 scale) {
  const float x[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
  auto four = [&](const float* v) { return max_nan(max_nan(fabsf(v[0]), fabsf(v[1])), max_nan(fabsf(v[2]), fabsf(v[3]))); };
  float own[8], top[2] = {0.f, 0.f}, e[2] = {0.f, 0.f};
  const bool turned = t.k_weight || l.f >= 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float pair = fabsf(x[i]) + fabsf(t.adjacent ? x[i ^ 1] : x[i ^ 4]);
    own[i] = l.f >= 0 ? 1.42f * kTurnErr * pair : (turned ? kTurnErr * fabsf(x[i]) : 0.f);
  }
  group_max<D>(l, four(x), four(x + 4), top[0], top[1]);
  group_max<D>(l, four(own), four(own + 4), e[0], e[1]);
  bool open = false;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float inv = inverse(v ? scale.y : scale.x);
    open |= group_turned(t, v ? l.b : l.a) && top[v] > 0.f && open_scale(top[v], e[v]);   // (nothing in it: no scale)
    if (!turned) continue;
#pragma unroll
    for (int i = 4 * v; i < 4 * v + 4; ++i) open |= fabsf(fmaf(x[i], inv, kCode - code(x[i], inv))) > open_code(own[i], inv);
  }
  return open;
}

// A lane's part of a key into its head's block.
template <int DK, int DV>
__device__ __forceinline__ void put_key(const CacheArgs& c, uint8_t* to, int place, const HeadLane& l, const Held& held) {
  const uint32_t ta = (l.a >> 6) * c.ps + place, tb = (l.b >> 6) * c.ps + place, scales = c.ps * ((DK + DV) / 2);
  *reinterpret_cast<uint16_t*>(to + ta * 32 + (l.a & 63) / 2) = (uint16_t)held.codes[0];
  *reinterpret_cast<uint16_t*>(to + tb * 32 + (l.b & 63) / 2) = (uint16_t)held.codes[1];
  if ((l.a & 63) == 0) *reinterpret_cast<uint16_t*>(to + scales + ta * 2) = (uint16_t)(__float_as_uint(held.scale[0]) >> 16);
  if ((l.b & 63) == 0) *reinterpret_cast<uint16_t*>(to + scales + tb * 2) = (uint16_t)(__float_as_uint(held.scale[1]) >> 16);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Few rows: the status block is not cleared by a launch before, but set by one more CTA, which looks every row's
// page up for itself.  us in a graph, by a launch before and by that CTA (called from the host: a launch less, 1.4 us for
// reads): append of 32 rows 5.1 and 3.8, of 512 requests' tokens 10.1 and 9.7, of 1024 14.4 and 13.5, of 2048 17.1
// and 21.9; read of 32 rows 3.2 and 2.7, of 512 rows of eight requests 3.4 and 2.9, of 512 requests 3.4 and 4.1 (from the
// host 7.3 and 6.0), of 1024 4.2 and 7.4.
constexpr int kOwnRows = 512;
__device__ __forceinline__ void set_status(const CacheArgs& c, int R, const int32_t* row_offsets, const int32_t* positions,
                                           uint32_t* status) {
  bool bad = false;
  for (int row = threadIdx.x; row < R; row += kThreads) {
    const int pos = positions[row];
    int before = 0, n = c.B + 1;                     // offsets that are no greater than the row, among n from there on
    while (pos >= 0 && n > 0) {
      const int half = n >> 1;
      if (row_offsets[before + half] <= row) {
        before += half + 1;
        n -= half + 1;
      } else {
        n = half;
      }
    }
    bad |= pos >= 0 && before >= 1 && before <= c.B && find_page(c, before - 1, pos) < 0;
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x < 64) status[threadIdx.x] = any && threadIdx.x == 0 ? DSA_DEVICE_BAD_INDEX : 0;
}

// A run of one row's keys into its page, by one warp.
template <int DK, int DV, bool F16>
__device__ __forceinline__ void append_keys(const TurnArgs& t, const CacheArgs& c, const float2* cs, int64_t page, int row,
                                            int run, int lane) {
  const int pos = t.positions[row], place = pos & (c.ps - 1);
  constexpr int L = kHeadLanes<DK>, S = 32 / L;
  int h0, h1;
  run_heads(t, c.H_kv, run, h0, h1);
  const int sub = lane / L;
  const HeadLane l = head_lane<DK>(t, lane % L);
  const uint16_t* src = t.k + row * t.k_stride + (h0 + sub) * DK;
  uint8_t* dst = c.pages + page + (uint32_t)(h0 + sub) * c.block;
  const LaneTurn turns = lane_turn<F16>(cs, t.k_weight, l);
  const int rounds = (h1 - h0 + S - 1) / S;     // (at most 8)
  uint32_t opens = 0;          // rounds that fp32 left open
  for (int first = 0; first < rounds; first += 4) {
    uint2 v[4][2];             // (four rounds' loads under way together)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const bool live = h0 + (first + y) * S + sub < h1;
      v[y][0] = live ? load4(src + (first + y) * S * DK, l.a) : make_uint2(0, 0);
      v[y][1] = live ? load4(src + (first + y) * S * DK, l.b) : make_uint2(0, 0);
    }
#pragma unroll 1
    for (int n = first; n < min(first + 4, rounds); ++n) {
      const bool live = h0 + n * S + sub < h1 && l.a >= 0;
      float x[8];
      unpack4<F16>(v[0][0], x);
      unpack4<F16>(v[0][1], x + 4);
#pragma unroll
      for (int y = 1; y < 4; ++y) {
        v[y - 1][0] = v[y][0];
        v[y - 1][1] = v[y][1];
      }
      turn_head<DK>(t, t.k_weight != nullptr, l, turns, x);
      Held held;
      if (__any_sync(0xffffffffu, !hold_key<DK>(t, x, l, held) && live) &&
          __any_sync(0xffffffffu, still_open<DK>(t, make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7]), l,
                                                 make_float2(held.scale[0], held.scale[1])) && live))
        opens |= 1u << n;
      if (live) put_key<DK, DV>(c, dst + n * S * c.block, place, l, held);
    }
  }
  for (; opens; opens &= opens - 1) {
    const int n = __ffs(opens) - 1;
    const bool live = h0 + n * S + sub < h1 && l.a >= 0;
    const Held held = hold_exactly<DK, F16>(t, cs, live ? src + n * S * DK : nullptr, pos, lane);
    if (live) put_key<DK, DV>(c, dst + n * S * c.block, place, l, held);
  }
}

// A run of one row's values: eight columns to a lane, eight lanes to a group.
template <int DK, int DV, bool F16>
__device__ __forceinline__ void append_values(const TurnArgs& t, const CacheArgs& c, int64_t page, int row, int run, int lane) {
  const int place = t.positions[row] & (c.ps - 1);
  constexpr int L = DV / 8, S = 32 / L, U = 4;
  int h0, h1;
  run_heads(t, c.H_kv, run, h0, h1);
  const int sub = lane / L, j = lane % L;
  const uint32_t at = (j >> 3) * c.ps + place;
  const uint16_t* src = t.v + row * t.v_stride + (h0 + sub) * DV + 8 * j;
  uint8_t* dst = c.pages + page + (uint32_t)(h0 + sub) * c.block;
  const uint32_t to = c.ps * (DK / 2) + at * 32 + (j & 7) * 4, scales = c.ps * ((DK + DV) / 2 + DK / 32) + at * 2;
  for (int base = h0; base < h1; base += U * S) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (base + u * S + sub < h1) v[u] = *reinterpret_cast<const uint4*>(src + u * S * DV);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (base + u * S >= h1) break;
      float x[8];
      unpack4<F16>(make_uint2(v[u].x, v[u].y), x);
      unpack4<F16>(make_uint2(v[u].z, v[u].w), x + 4);
      float top = max_nan(max_nan(max_nan(fabsf(x[0]), fabsf(x[1])), max_nan(fabsf(x[2]), fabsf(x[3]))),
                          max_nan(max_nan(fabsf(x[4]), fabsf(x[5])), max_nan(fabsf(x[6]), fabsf(x[7]))));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = group_scale(top, top), inv = inverse(scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = code_exactly(x[i], inv);
      if (base + u * S + sub < h1) {
        *reinterpret_cast<uint32_t*>(dst + to) = pack_codes(x) + (pack_codes(x + 4) << 16);
        if ((j & 7) == 0) *reinterpret_cast<uint16_t*>(dst + scales) = (uint16_t)(__float_as_uint(scale) >> 16);
      }
      dst += S * c.block;
    }
    src += U * S * DV;
  }
}

template <int DK, int DV, bool F16>
__global__ void __launch_bounds__(kTurnThreads, 4)
    kv4_append_kernel(const __grid_constant__ TurnArgs t, const __grid_constant__ CacheArgs c, bool own, uint32_t* status) {
  __shared__ RowTurns cs;
  __shared__ int64_t pages[kTurnRows];             // a row's page; -1: outside the pool, -2: the row is skipped
  __shared__ int next;                             // unit that the next warp to be through takes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, runs = t.q_runs + t.k_runs + t.v_runs;
  int row0, u0, u1;
  cta_units(t, runs, row0, u0, u1);
  if (own) pdl_wait();                             // (else the launch that clears the status has waited)
  pdl_trigger();
  if (own && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) set_status(c, t.R, t.row_offsets, t.positions, status);
    return;
  }
  // The rows' keys and values on their way to L2 while pages and angles are looked up.
  for (int i = warp; i >> t.rows_log2 == 0 && row0 + i < t.R; i += kTurnThreads / 32) {
    const uint16_t *k = t.k + (row0 + i) * t.k_stride, *v = t.v + (row0 + i) * t.v_stride;
    for (int x = lane; x < c.H_kv * (DK / 64); x += 32) prefetch_l2(k + 64 * x);
    for (int x = lane; x < c.H_kv * (DV / 64); x += 32) prefetch_l2(v + 64 * x);
  }
  if (threadIdx.x == 0) next = u0 + kTurnThreads / 32;
  if (warp >> t.rows_log2 == 0) {
    int64_t page = -2;
    if (row0 + warp < t.R) {
      const int pos = t.positions[row0 + warp], b = find_request(t.row_offsets, t.B, row0 + warp, lane);
      if (pos >= 0 && b >= 0) page = find_page(c, b, pos);
    }
    if (lane == 0) {
      pages[warp] = page;
      if (page == -1 && u0 == 0 && !own) {
        pdl_wait();                                // (the status block is cleared)
        raise_status(status, DSA_DEVICE_BAD_INDEX);
      }
    }
  }
  row_turns(t, cs, row0);
  __syncthreads();
  // Keys come before values, and a warp that has to look at a head again leaves the rest to the others.
  for (int u = u0 + warp; u < u1; u = __shfl_sync(0xffffffffu, lane == 0 ? atomicAdd(&next, 1) : 0, 0)) {
    const int run = u >> t.rows_log2, i = u - (run << t.rows_log2), row = row0 + i;
    const int64_t page = pages[i];
    if (page == -2) continue;
    if (run < t.q_runs) {
      int h0, h1;
      run_heads(t, t.H_q, run, h0, h1);
      turn_row<DK, F16>(t, t.q_weight, cs[i], t.q + row * t.q_stride, t.q_out + row * t.q_out_stride, h0, h1, lane);
    } else if (page >= 0) {
      if (run < t.q_runs + t.k_runs)
        append_keys<DK, DV, F16>(t, c, cs[i], page, row, run - t.q_runs, lane);
      else
        append_values<DK, DV, F16>(t, c, page, row, run - t.q_runs - t.k_runs, lane);
    }
  }
  if (threadIdx.x == 0) pdl_wait();                // (whoever waits for this grid's end waits for its predecessors' too)
}

// 32 bytes; in halves where the caller's buffer is aligned to 16 alone.
__device__ __forceinline__ void store8(uint16_t* p, const uint32_t* v) {
  if (reinterpret_cast<uintptr_t>(p) & 31) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}

template <int N>
struct Width {
  static constexpr int value = N;
};

// A row is read in rounds: 32 lanes of 16 columns each (8 bytes of codes, 32 of values), the keys' rounds, then
// the values'.
template <int D>
__device__ __forceinline__ int read_rounds(int heads) { return (heads * (D / 16) + 31) / 32; }

// Four rounds from `first` on of one row, by one warp, their loads under way together.  page: the byte of
// the pool where it begins (-1: nothing is read or written; -2: zeros are written).  ko, vo: the row's places.
template <int DK, int DV, bool F16>
__device__ __forceinline__ void read_row(const CacheArgs& c, int64_t page, uint32_t place, uint16_t* ko, uint16_t* vo, int nk, int nv,
                                         int first, int lane) {
  if (page == -1) return;
  const uint8_t* p = c.pages + page;
  uint2 w[4];
  uint32_t s[4];
  uint16_t* to[4];
  auto look = [&](auto width, int round, uint32_t codes, uint32_t scales, uint16_t* out, int u) {
    constexpr int N = decltype(width)::value / 16;        // pieces of a head
    const uint32_t x = round * 32 + lane, h = x / N, j = x - h * N;
    if (h >= (uint32_t)c.H_kv) return;
    to[u] = out + x * 16;
    if (page < 0) return;
    const uint32_t blk = h * c.block, n = (j >> 2) * c.ps + place;
    w[u] = *reinterpret_cast<const uint2*>(p + (blk + codes + n * 32 + (j & 3) * 8));
    s[u] = *reinterpret_cast<const uint16_t*>(p + (blk + scales + n * 2));
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    w[u] = make_uint2(0, 0);
    s[u] = 0;
    to[u] = nullptr;
    const int round = first + u;
    if (round < nk)
      look(Width<DK>(), round, 0, c.ps * ((DK + DV) / 2), ko, u);
    else if (round < nk + nv)
      look(Width<DV>(), round - nk, c.ps * (DK / 2), c.ps * ((DK + DV) / 2 + DK / 32), vo, u);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t o[8];
    widen8<F16>(w[u].x, s[u], o);
    widen8<F16>(w[u].y, s[u], o + 4);
    if (to[u]) store8(to[u], o);
  }
}

constexpr int kReadRows = 16;   // rows of a CTA, at most

template <int DK, int DV, bool F16>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const CacheArgs c, int R, int rows, const int32_t* row_offsets, const int32_t* positions, uint16_t* k_out,
                    uint16_t* v_out, bool own, uint32_t* status) {
  __shared__ int64_t pages[kReadRows];
  __shared__ int places[kReadRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * rows;
  if (own) pdl_wait();                               // (else the launch that clears the status has waited)
  pdl_trigger();
  if (own && blockIdx.x == gridDim.x - 1) {
    set_status(c, R, row_offsets, positions, status);
    return;
  }
  // (a warp's two rows are looked up together)
  constexpr int kWarps = kThreads / 32, kOfWarp = kReadRows / kWarps;
  int pos[kOfWarp], b[kOfWarp];
#pragma unroll
  for (int u = 0; u < kOfWarp; ++u) {
    const int i = warp + u * kWarps;
    pos[u] = i < rows && row0 + i < R ? positions[row0 + i] : -1;
  }
#pragma unroll
  for (int u = 0; u < kOfWarp; ++u) b[u] = pos[u] >= 0 ? find_request(row_offsets, c.B, (int)row0 + warp + u * kWarps, lane) : -1;
#pragma unroll
  for (int u = 0; u < kOfWarp; ++u) {
    const int i = warp + u * kWarps;
    const bool asked = pos[u] >= 0 && b[u] >= 0;
    const int64_t page = asked ? find_page(c, b[u], pos[u]) : -1;
    if (asked && page < 0 && lane == 0 && !own) {
      pdl_wait();
      raise_status(status, DSA_DEVICE_BAD_INDEX);
    }
    if (lane == 0 && i < rows) {
      pages[i] = page;
      places[i] = pos[u] & (c.ps - 1);
    }
  }
  __syncthreads();
  const int nk = k_out ? read_rounds<DK>(c.H_kv) : 0, nv = v_out ? read_rounds<DV>(c.H_kv) : 0;
  int i = warp, first = 0;                           // (four rounds of every row, then the next)
  for (;;) {
    while (i >= rows) {
      i -= rows;
      first += 4;
    }
    if (first >= nk + nv) break;
    read_row<DK, DV, F16>(c, pages[i], places[i], k_out + (row0 + i) * c.H_kv * DK, v_out + (row0 + i) * c.H_kv * DV, nk, nv, first,
                          lane);
    i += kThreads / 32;
  }
  if (threadIdx.x == 0) pdl_wait();                  // (whoever waits for this grid's end waits for its predecessors' too)
}

// Clears the status block (64 words) and counts how far each request's rows see: a CTA to a request.
__global__ void __launch_bounds__(kThreads)
    kv4_lens_kernel(int R, int reach, const int32_t* row_offsets, const int32_t* row_len, int32_t* gone, int32_t* lens,
                    uint32_t* status) {
  __shared__ int most[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, r0 = min(max(row_offsets[b], 0), R), r1 = min(row_offsets[b + 1], R);
  if (b == 0 && threadIdx.x < 64) status[threadIdx.x] = 0;
  int m = 0;
  for (int r = r0 + threadIdx.x; r < r1; r += kThreads) m = max(m, min(row_len[r], reach));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) m = max(m, most[w]);
    lens[b] = m;
    gone[b] = 0;
  }
}

// Sixteen positions of a request, which lie in one page, to the copy.
template <int DK, int DV, bool F16>
__global__ void __launch_bounds__(kThreads, 4)
    kv4_copy_kernel(const CacheArgs c, int reach, int blocks, uint16_t* k, uint16_t* v, int32_t* gone, const int32_t* lens,
                    uint32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x / blocks, pos = (blockIdx.x - b * blocks) * 16;
  pdl_wait();
  pdl_trigger();
  const int n = min(lens[b] - pos, 16);
  if (n <= 0) return;
  int64_t page = find_page(c, b, pos);
  if (page < 0) {
    if (threadIdx.x == 0) {
      raise_status(status, DSA_DEVICE_BAD_INDEX);
      gone[b] = 1;
    }
    page = -2;
  }
  const int64_t row0 = (int64_t)b * reach + pos;
  const int nk = read_rounds<DK>(c.H_kv), nv = read_rounds<DV>(c.H_kv);
  for (int i = warp; i < n; i += kThreads / 32)
    for (int first = 0; first < nk + nv; first += 4)
      read_row<DK, DV, F16>(c, page, (pos + i) & (c.ps - 1), k + (row0 + i) * c.H_kv * DK, v + (row0 + i) * c.H_kv * DV, nk, nv,
                            first, lane);
}

template <int DK, int DV>
cudaError_t launch_append_width(TurnArgs t, const CacheArgs& c, bool f16, uint32_t* status, cudaStream_t st) {
  deal_heads(t, 32 / kHeadLanes<DK>, 8, c.H_kv, c.H_kv);
  const bool own = t.R <= kOwnRows;
  const dim3 grid((unsigned)(((t.R + (1 << t.rows_log2) - 1) >> t.rows_log2) + own), (unsigned)t.split);
  return f16 ? launch_pdl(kv4_append_kernel<DK, DV, true>, grid, dim3(kTurnThreads), 0, st, t, c, own, status)
             : launch_pdl(kv4_append_kernel<DK, DV, false>, grid, dim3(kTurnThreads), 0, st, t, c, own, status);
}

template <int DK, int DV>
cudaError_t launch_read_width(const CacheArgs& c, int R, const int32_t* row_offsets, const int32_t* positions, bool f16,
                              uint16_t* k_out, uint16_t* v_out, uint32_t* status, cudaStream_t st) {
  // Rows to a CTA: up to sixteen where that leaves two CTAs an SM or more.
  int rows = 1;
  while (rows < kReadRows && R / (2 * rows) >= 304) rows *= 2;
  const bool own = R <= kOwnRows;
  const dim3 grid((unsigned)(((int64_t)R + rows - 1) / rows + own));
  return f16 ? launch_pdl(kv4_read_kernel<DK, DV, true>, grid, dim3(kThreads), 0, st, c, R, rows, row_offsets, positions, k_out,
                          v_out, own, status)
             : launch_pdl(kv4_read_kernel<DK, DV, false>, grid, dim3(kThreads), 0, st, c, R, rows, row_offsets, positions, k_out,
                          v_out, own, status);
}

template <int DK, int DV>
cudaError_t launch_copy_width(const CacheArgs& c, int reach, bool f16, uint16_t* k, uint16_t* v, int32_t* gone,
                              const int32_t* lens, uint32_t* status, cudaStream_t st) {
  const int blocks = (reach + 15) / 16;
  const dim3 grid((unsigned)(c.B * blocks));
  return f16 ? launch_pdl(kv4_copy_kernel<DK, DV, true>, grid, dim3(kThreads), 0, st, c, reach, blocks, k, v, gone, lens, status)
             : launch_pdl(kv4_copy_kernel<DK, DV, false>, grid, dim3(kThreads), 0, st, c, reach, blocks, k, v, gone, lens, status);
}

}  // namespace

bool kv4_sets_status(int R) { return R > 0 && R <= kOwnRows; }

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

cudaError_t launch_kv4_copy(const CacheArgs& c, int R, int reach, const int32_t* row_offsets, const int32_t* row_len, int D_k,
                            int D_v, bool f16, uint16_t* k, uint16_t* v, int32_t* gone, int32_t* lens, uint32_t* status,
                            cudaStream_t st) {
  (void)D_v;
  const cudaError_t e = launch_pdl(kv4_lens_kernel, dim3((unsigned)c.B), dim3(kThreads), 0, st, R, reach, row_offsets, row_len,
                                   gone, lens, status);
  if (e != cudaSuccess) return e;
  if (D_k == 64) return launch_copy_width<64, 64>(c, reach, f16, k, v, gone, lens, status, st);
  if (D_k == 128) return launch_copy_width<128, 128>(c, reach, f16, k, v, gone, lens, status, st);
  return launch_copy_width<192, 128>(c, reach, f16, k, v, gone, lens, status, st);
}

}  // namespace dsa
