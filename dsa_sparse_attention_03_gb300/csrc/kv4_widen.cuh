// 4-bit codes to 16 bits, shared by kv4_cache.cu and the dense kernel's widening warps.
#pragma once

#include "tc.cuh"

namespace dsa {

// Eight 4-bit codes times their scale (bf16 bits) in 16 bits, in order.  bf16: 128 + code by byte
// permutations, then one packed multiply-add, (128 + code) s - 136 s: exact, since 136 s has 8
// significant bits; a scale from 2^120 on, where 136 s would leave the range, is taken 2^-8 of and the
// values 2^8 times.  fp16: 1024 + code, minus 1032, times s: the last step alone may round.  A scale below
// 2^-21, whose four bits fp16 does not hold, is taken 2^14 times, and the exact values 2^-14 of (below 2^-35 the
// scale is rounded after all, and the values are 0).
template <bool F16>
__device__ __forceinline__ void widen8(uint32_t w, uint32_t scale, uint32_t* o) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
  const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);   // codes 0..3, 4..7
  constexpr uint32_t top = F16 ? 0x64646464u : 0x43434343u;
  uint32_t u[4] = {__byte_perm(lo, top, 0x4140), __byte_perm(lo, top, 0x4342), __byte_perm(hi, top, 0x4140),
                   __byte_perm(hi, top, 0x4342)};
  if (F16) {
    const bool tiny = scale < 0x3500u;
    const float s = __uint_as_float((tiny ? scale + 0x700u : scale) << 16);
    const __half2 s2 = __floats2half2_rn(s, s), zero = __floats2half2_rn(-1032.f, -1032.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __hmul2(__hadd2(*reinterpret_cast<__half2*>(&u[i]), zero), s2);
      o[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    if (tiny) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 v = __hmul2(*reinterpret_cast<__half2*>(&o[i]), __floats2half2_rn(0x1p-14f, 0x1p-14f));
        o[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
  } else {
    const bool huge = scale >= 0x7b80u && scale < 0x7f80u;
    uint32_t sb = (huge ? scale - 0x400u : scale) * 0x10001u;
    const __nv_bfloat162 s2 = *reinterpret_cast<__nv_bfloat162*>(&sb);
    const __nv_bfloat162 zero = __hmul2(s2, __floats2bfloat162_rn(-136.f, -136.f));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 v = __hfma2(*reinterpret_cast<__nv_bfloat162*>(&u[i]), s2, zero);
      if (huge) v = __hmul2(v, __floats2bfloat162_rn(256.f, 256.f));
      o[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}

}  // namespace dsa
