// fsa_cache.cu -- writing the paged 4-bit K/V cache and reading it back.
//
// Both kernels are bound by memory: append reads 2 bytes and writes 0.53 (E2M1) or 0.56
// (NVFP4) bytes an element, read the other way round.  A warp takes a run of UNIT tokens of
// a kv head within a group (a contiguous piece of a page), so that page and addresses are
// worked out once for 2 * 1024 elements, all of whose loads go out together.  On the bf16
// side a lane holds 8 consecutive elements (16 bytes), D/8 lanes a row; on the cache's side
// one word of a row.  The two orders (fsa_cache.h) differ, so the code words cross the lanes
// in between: a K word is two halves of two lanes' words, a V word four bytes of four.  The rounding is that of fsa_mx_quantize.
//
// Measured (one GB300): reading 128K tokens of 8 kv heads back 104 us for 688 MB (6.6 TB/s,
// 0.97 of the copy bandwidth); four prompts of up to 4096 tokens written and read back 25.7 us
// for 118 MB of unavoidable bytes, two kernels that at this size are bound by their
// instructions (2.7 and 3.0 a cycle) as much as by memory; a step of 128 single tokens written
// and read back 4.1 us, two launches.
#include "fsa_cache.h"
#include "fsa_mx.cuh"

namespace fsa {
namespace {

constexpr int CIO_WARPS = 4;
template <int D>
constexpr int UNIT = 1024 / D;     // tokens of a warp: 8 or 16

// A warp's rows r0 <= r < r1 of the group that begins at pos: rows r - shift of its tensor,
// counted from the first position asked for.
struct Group {
  int64_t pos, shift;
  int r0, r1;
};

// Unit ui of the sequence, counted from the one that holds its first position; false if none
// of its rows is asked for.  `first`, `count`: the positions asked for.
template <int U>
__device__ __forceinline__ bool find_rows(int64_t first, int64_t count, int ui, Group& g) {
  const int64_t at = ((first > 0 ? first : 0) / U + ui) * U;      // the unit's first position
  g.pos = at & ~15ll;
  const int u0 = (int)(at - g.pos);
  g.shift = first - g.pos;
  g.r0 = (int)max((int64_t)u0, g.shift);
  g.r1 = (int)max((int64_t)0, min((int64_t)(u0 + U), g.shift + count));
  return g.r0 < g.r1;
}
// Its group in the pool, or null.
__device__ __forceinline__ uint8_t* find_page(const CacheIo& a, int b, int h, int64_t pos, int group_bytes) {
  const int64_t pi = pos >> a.c.page_shift;
  if (pi >= a.max_pages) return nullptr;
  const int page = a.table[(int64_t)b * a.max_pages + pi];
  if (page < 0 || page >= a.c.num_pages) {
    if (a.status && (threadIdx.x & 31) == 0) atomicExch(a.status, -1);       // FSA_ERR_INVALID_ARG
    return nullptr;
  }
  const int inside = (int)(pos & ((1 << a.c.page_shift) - 1)) / 16;
  return a.c.pages + page * a.c.page_bytes + (((int64_t)h << (a.c.page_shift - 4)) + inside) * group_bytes;
}

// Which of the launch's units this warp has: units of a sequence, then heads, fastest last.
__device__ __forceinline__ bool my_item(const CacheIo& a, int units, int& b, int& ui, int& h) {
  const uint32_t item = blockIdx.x * CIO_WARPS + threadIdx.x / 32;
  const uint32_t rest = item / (uint32_t)a.c.Hkv;
  h = (int)(item - rest * a.c.Hkv);
  b = (int)(rest / (uint32_t)units);
  ui = (int)(rest - (uint32_t)b * units);
  return b < a.B;
}

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

template <int D, int CF>
__global__ void __launch_bounds__(CIO_WARPS * 32) cache_append_kernel(const CacheIo a, int units) {
  using Gr = CacheGroup<D, CF>;
  constexpr int L = D / 8, ROWS = 32 / L, BATCH = UNIT<D> / ROWS;      // rows at a time, times
  constexpr int PER = CF == CF_MX ? 4 : 2;                       // lanes of a block
  griddep_launch();
  griddep_wait();
  int b, ui, h;
  if (!my_item(a, units, b, ui, h)) return;
  const int fresh = a.which ? min(max(a.which[b], 0), a.S) : a.S;
  // positions below 0 are dropped: the first of them is 0 then, and row 0 is `skip`
  const int64_t first = (int64_t)a.lens[b] - fresh, skip = first < 0 ? -first : 0;
  Group g;
  if (!find_rows<UNIT<D>>(first + skip, fresh - skip, ui, g)) return;
  const int lane = threadIdx.x & 31, l = lane % L, row = lane - l;
  const int r = g.r0 / UNIT<D> * UNIT<D> + lane / L;             // this lane's row the first time, ROWS on each time
  const uint16_t* ksrc = a.k + b * a.ks.b + h * a.ks.h + (skip - g.shift + r) * a.ks.s + 8 * l;
  const uint16_t* vsrc = a.v + b * a.vs.b + h * a.vs.h + (skip - g.shift + r) * a.vs.s + 8 * l;
  uint4 ku[BATCH], vu[BATCH];
#pragma unroll
  for (int x = 0; x < BATCH; ++x) {
    const bool in = r + x * ROWS >= g.r0 && r + x * ROWS < g.r1;
    ku[x] = in ? *reinterpret_cast<const uint4*>(ksrc) : make_uint4(0u, 0u, 0u, 0u);
    vu[x] = in ? *reinterpret_cast<const uint4*>(vsrc) : make_uint4(0u, 0u, 0u, 0u);
    ksrc += ROWS * a.ks.s;
    vsrc += ROWS * a.vs.s;
  }
  uint8_t* const at = find_page(a, b, h, g.pos, Gr::BYTES);      // while they are on their way
  if (!at) return;
  uint8_t* const codes = at + r * (D / 2) + 4 * l;
  uint8_t* const scales = at + Gr::KS + r * Gr::SB + l / PER;
#pragma unroll
  for (int x = 0; x < BATCH; ++x) {
    if (r - lane / L + x * ROWS >= g.r1 || r - lane / L + (x + 1) * ROWS <= g.r0) continue;      // a single token: one of these has it
    uint32_t ksb, vsb;
    const uint32_t kw = k_to_cache<L>(quantise8<CF>(ku[x], ksb), row, l);
    const uint32_t vw = v_to_cache<L>(quantise8<CF>(vu[x], vsb), row, l);
    if (r + x * ROWS >= g.r0 && r + x * ROWS < g.r1) {
      *reinterpret_cast<uint32_t*>(codes + x * ROWS * (D / 2) + Gr::K) = kw;
      *reinterpret_cast<uint32_t*>(codes + x * ROWS * (D / 2) + Gr::V) = vw;
      if (l % PER == 0) {
        scales[x * ROWS * Gr::SB] = (uint8_t)ksb;
        scales[x * ROWS * Gr::SB + Gr::VS - Gr::KS] = (uint8_t)vsb;
      }
    }
  }
}

// The 8 values of a plain word under a scale, as bf16: exact, at most 6 significant bits
__device__ __forceinline__ uint4 values8(uint32_t codes, float s) {
  uint32_t h[4], v[4];
  cvt_e2m1x8_f16(codes, h);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}" : "=f"(lo), "=f"(hi) : "r"(h[e]));
    v[e] = cvt_bf16x2(__fmul_rn(lo, s), __fmul_rn(hi, s));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
template <int CF>
__device__ __forceinline__ float scale_value(uint32_t sb) {
  if constexpr (CF == CF_MX) {
    float f, unused;
    e8m0x2_f32(sb, f, unused);
    return f;
  } else {
    return e4m3_to_f32(sb);
  }
}

template <int D, int CF>
__global__ void __launch_bounds__(CIO_WARPS * 32) cache_read_kernel(const CacheIo a, int units) {
  using Gr = CacheGroup<D, CF>;
  constexpr int L = D / 8, ROWS = 32 / L, BATCH = UNIT<D> / ROWS;
  constexpr int PER = CF == CF_MX ? 4 : 2;
  griddep_launch();
  griddep_wait();
  int b, ui, h;
  if (!my_item(a, units, b, ui, h)) return;
  const int64_t start = a.which ? a.which[b] : 0, skip = start < 0 ? -start : 0;
  Group g;
  if (!find_rows<UNIT<D>>(start + skip, min((int64_t)a.S, (int64_t)a.lens[b] - start) - skip, ui, g)) return;
  const uint8_t* const at = find_page(a, b, h, g.pos, Gr::BYTES);
  const int lane = threadIdx.x & 31, l = lane % L, row = lane - l;
  const int r = g.r0 / UNIT<D> * UNIT<D> + lane / L;             // this lane's row the first time, ROWS on each time
  const uint8_t* const codes = at + r * (D / 2) + 4 * l;
  const uint8_t* const scales = at + Gr::KS + r * Gr::SB + l / PER;
  uint32_t kw[BATCH], vw[BATCH], ks[BATCH], vs[BATCH];
#pragma unroll
  for (int x = 0; x < BATCH; ++x) {
    kw[x] = vw[x] = ks[x] = vs[x] = 0;
    if (at) {
      kw[x] = *reinterpret_cast<const uint32_t*>(codes + x * ROWS * (D / 2) + Gr::K);
      vw[x] = *reinterpret_cast<const uint32_t*>(codes + x * ROWS * (D / 2) + Gr::V);
      ks[x] = scales[x * ROWS * Gr::SB];
      vs[x] = scales[x * ROWS * Gr::SB + Gr::VS - Gr::KS];
    }
  }
  uint16_t* kdst = a.k + b * a.ks.b + h * a.ks.h + (skip - g.shift + r) * a.ks.s + 8 * l;
  uint16_t* vdst = a.v + b * a.vs.b + h * a.vs.h + (skip - g.shift + r) * a.vs.s + 8 * l;
#pragma unroll
  for (int x = 0; x < BATCH; ++x) {
    if (r - lane / L + x * ROWS < g.r1 && r - lane / L + (x + 1) * ROWS > g.r0) {
      const bool in = r + x * ROWS >= g.r0 && r + x * ROWS < g.r1;
      const uint4 k = values8(k_from_cache<L>(kw[x], row, l), scale_value<CF>(ks[x]));
      const uint4 v = values8(v_from_cache<L>(vw[x], row, l), scale_value<CF>(vs[x]));
      if (in && a.k) *reinterpret_cast<uint4*>(kdst) = k;
      if (in && a.v) *reinterpret_cast<uint4*>(vdst) = v;
    }
    kdst += ROWS * a.ks.s;
    vdst += ROWS * a.vs.s;
  }
}

// units that S consecutive tokens can touch
int units_of(const CacheIo& a) {
  const int u = 1024 / a.c.D;
  return (int)(((int64_t)a.S + u - 2) / u + 1);
}
unsigned blocks_of(const CacheIo& a) {
  return (unsigned)(((int64_t)a.B * units_of(a) * a.c.Hkv + CIO_WARPS - 1) / CIO_WARPS);
}

}  // namespace

cudaError_t launch_cache_append(const CacheIo& a, cudaStream_t st) {
  const unsigned grid = blocks_of(a);
  const int units = units_of(a);
  if (a.c.D == 128) {
    if (a.c.cf == CF_MX) return launch_early(cache_append_kernel<128, CF_MX>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
    else return launch_early(cache_append_kernel<128, CF_NV>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
  } else {
    if (a.c.cf == CF_MX) return launch_early(cache_append_kernel<64, CF_MX>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
    else return launch_early(cache_append_kernel<64, CF_NV>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
  }
}

cudaError_t launch_cache_read(const CacheIo& a, cudaStream_t st) {
  const unsigned grid = blocks_of(a);
  const int units = units_of(a);
  if (a.c.D == 128) {
    if (a.c.cf == CF_MX) return launch_early(cache_read_kernel<128, CF_MX>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
    else return launch_early(cache_read_kernel<128, CF_NV>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
  } else {
    if (a.c.cf == CF_MX) return launch_early(cache_read_kernel<64, CF_MX>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
    else return launch_early(cache_read_kernel<64, CF_NV>, dim3(grid), CIO_WARPS * 32, 0, st, a, units);
  }
}

}  // namespace fsa
