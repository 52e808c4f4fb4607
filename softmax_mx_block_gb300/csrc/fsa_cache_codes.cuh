// fsa_cache_codes.cuh -- rows of values as rows of the cache: 4-bit codes and block scales, and
// the exchanges between the order of a row's elements and that of its bytes in the cache
// (fsa_cache.h).  Shared by the kernels that write and read the cache (fsa_cache.cu) and the one
// that rotates keys on their way into it (fsa_append_rope.cu).
#pragma once
#include "fsa_cache.h"
#include "fsa_mx.cuh"

namespace fsa {

// Cut to 12 fraction bits: a quotient that was raised by 2^-21 to 2^-19 of it becomes a tie
// again where it was one (see below).
__device__ __forceinline__ float cut12(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFFF800u); }

// 8 consecutive elements of a row, D/8 lanes a row: their codes, element 0 in the lowest
// nibble, and their block's scale byte.  The block's maximum is taken on the bf16 patterns
// (as integers they are ordered as their magnitudes, Inf and NaN above all).
//
// Quotients without a division: amax / 6 and x / s are rounded to a few bits next, to the
// nearest with ties to even.  bf16 has 8 significant bits, E4M3 4 and 6 is 3 * 2, so a
// quotient is a tie or at least 2^-10 of it away from one.  The product with a reciprocal
// raised by 2^-20 lies above the quotient by 2^-21 to 2^-19 of it; cut to 12 fraction bits, a
// tie is that tie and the others stay on their side.  (The same bytes as the divisions of
// fsa_mx_quantize for every pair of a bf16 value and a scale.)
template <int CF>
__device__ __forceinline__ uint32_t quantise8(uint4 u, uint32_t& sb) {
  constexpr uint32_t MAG = 0x7FFF7FFFu;
  uint32_t m = __vmaxu2(__vimax3_u16x2(u.x & MAG, u.y & MAG, u.z & MAG), u.w & MAG);
  m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));           // 16 elements
  if constexpr (CF == CF_MX) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));    // 32
  m = max(m & 0xFFFFu, m >> 16);
  const bool finite = m < 0x7F80u;
  float mul;
  if constexpr (CF == CF_MX) {
    sb = finite ? (uint32_t)max((int)(m >> 7) - 2, 0) : 0xFFu;   // exponent of amax, less 2 (zero and subnormal: 0)
    mul = __uint_as_float((254u - min(sb, 254u)) << 23);
    if (!finite) return 0u;
  } else {
    sb = finite ? cvt_e4m3x2(cut12(__uint_as_float(m << 16) * (0.16666667163372039795f * (1.0f + 0x1p-20f))), 0.f) & 0xFFu : 0x7Fu;
    const float s = e4m3_to_f32(sb);
    if (!(s > 0.0f)) return 0u;                                  // zero or NaN
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(mul) : "f"(s));
    mul *= 1.0f + 0x1p-20f;
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16) * mul;
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u) * mul;
    if constexpr (CF == CF_NV) {
      x[2 * e] = cut12(x[2 * e]);
      x[2 * e + 1] = cut12(x[2 * e + 1]);
    }
  }
  return cvt_e2m1x8(x);
}

// The exchanges between the two orders of a row's codes.  lane = l of a row of L = D/8 lanes
// (`row`: its first lane); plain word l: elements 8l .. 8l + 7; cache word l: bytes 4l .. 4l + 3.
// K cache word l = t*(L/4) + w has elements 16s + 4t .. + 3 of s = 2w, 2w + 1: half t%2 of plain
// words 2s + t/2.  V cache word l = g*(L/8) + i has elements 16s + 2g, + 1 of s = 4i .. 4i + 3: byte
// g%4 of plain words 2s + g/4.
template <int L>
__device__ __forceinline__ uint32_t k_to_cache(uint32_t plain, int row, int l) {
  const int t = l / (L / 4), w = l % (L / 4);
  const uint32_t a = __shfl_sync(0xFFFFFFFFu, plain, row + 4 * w + t / 2);
  const uint32_t b = __shfl_sync(0xFFFFFFFFu, plain, row + 4 * w + 2 + t / 2);
  return __byte_perm(a, b, t & 1 ? 0x7632 : 0x5410);
}
template <int L>
__device__ __forceinline__ uint32_t k_from_cache(uint32_t cache, int row, int l) {
  const int s = l / 2, t = 2 * (l & 1);
  const uint32_t a = __shfl_sync(0xFFFFFFFFu, cache, row + t * (L / 4) + s / 2);
  const uint32_t b = __shfl_sync(0xFFFFFFFFu, cache, row + (t + 1) * (L / 4) + s / 2);
  return __byte_perm(a, b, s & 1 ? 0x7632 : 0x5410);
}
template <int L>
__device__ __forceinline__ uint32_t v_to_cache(uint32_t plain, int row, int l) {
  const int g = l / (L / 8), i = l % (L / 8);
  uint32_t w[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) w[x] = __shfl_sync(0xFFFFFFFFu, plain, row + 8 * i + 2 * x + g / 4);
  const uint32_t pick = (g & 3) * 0x11 + 0x40;                   // byte g%4 of the first, then of the second
  return __byte_perm(__byte_perm(w[0], w[1], pick), __byte_perm(w[2], w[3], pick), 0x5410);
}
template <int L>
__device__ __forceinline__ uint32_t v_from_cache(uint32_t cache, int row, int l) {
  const int s = l / 2, g = 4 * (l & 1);
  uint32_t w[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) w[x] = __shfl_sync(0xFFFFFFFFu, cache, row + (g + x) * (L / 8) + s / 4);
  const uint32_t pick = (s & 3) * 0x11 + 0x40;
  return __byte_perm(__byte_perm(w[0], w[1], pick), __byte_perm(w[2], w[3], pick), 0x5410);
}

}  // namespace fsa
