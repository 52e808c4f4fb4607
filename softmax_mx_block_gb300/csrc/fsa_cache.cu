// fsa_cache.cu -- writing the paged 4-bit K/V cache and reading it back.
//
// Both kernels are bound by memory: append reads 2 bytes and writes 0.53 (E2M1) or
// 0.56 (NVFP4) bytes an element, read the other way round.  D/8 lanes take one token
// of one kv head, its K row and its V row; a thread's 8 elements of a row are the ones
// whose codes are 4 consecutive bytes of the cache's row order (fsa_cache.h), so the
// codes move as whole words and the bf16 pieces of a warp fill whole 32-byte sectors.
// The rounding is that of fsa_mx_quantize, bit for bit.
#include "fsa_cache.h"
#include "fsa_mx.cuh"

namespace fsa {
namespace {

constexpr int CIO_THREADS = 256;

// The place of a sequence's token in the pool (its group's first byte), or null.  A page
// number outside the pool sets the status word.
__device__ __forceinline__ uint8_t* group_of(const CacheIo& a, int b, int64_t at, int h, int group_bytes) {
  const int64_t pi = at >> a.c.page_shift;
  if (at < 0 || pi >= a.max_pages) return nullptr;
  const int page = a.table[(int64_t)b * a.max_pages + pi];
  if (page < 0 || page >= a.c.num_pages) {
    if (a.status) atomicExch(a.status, -1);       // FSA_ERR_INVALID_ARG
    return nullptr;
  }
  const int inside = (int)(at & ((1 << a.c.page_shift) - 1));
  const int64_t groups = 1 << (a.c.page_shift - 4);
  return a.c.pages + page * a.c.page_bytes + (h * groups + inside / 16) * group_bytes;
}

// max over the lanes that differ in the given lane bits
template <int FROM, int TO>
__device__ __forceinline__ float lanes_max(float x, uint32_t mask) {
#pragma unroll
  for (int m = FROM; m < TO; m *= 2) x = fmaxf(x, __shfl_xor_sync(mask, x, m));
  return x;
}

// NaN-keeping magnitude: NaN and Inf become Inf, so that fmaxf passes them on
__device__ __forceinline__ float magnitude(float x) {
  const float a = fabsf(x);
  return a <= 3.4e38f ? a : __uint_as_float(0x7F800000u);
}

// The scale byte of a block and the code byte of a pair of its elements.
template <int CF>
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  if constexpr (CF == CF_MX) return block_scale_byte(amax, 2);
  else return nvfp4_scale_byte(amax, amax > 3.4e38f);
}
template <int CF>
__device__ __forceinline__ uint32_t code_byte(float lo, float hi, uint32_t sb) {
  if constexpr (CF == CF_MX) {
    const float mul = pow2_neg((int)sb - 127);
    return sb == 0xFFu ? 0u : cvt_e2m1x2(__fmul_rn(lo, mul), __fmul_rn(hi, mul));
  } else {
    const float s = e4m3_to_f32(sb);
    return s > 0.0f ? cvt_e2m1x2(__fdiv_rn(lo, s), __fdiv_rn(hi, s)) : 0u;
  }
}

template <int D, int CF>
__global__ void __launch_bounds__(CIO_THREADS) cache_append_kernel(const CacheIo a) {
  using Gr = CacheGroup<D, CF>;
  constexpr int L = D / 8, C = D / 32;            // lanes of a row; 4-byte words of a K chunk (of a t)
  const int lane = threadIdx.x % L;
  const uint32_t mask = (uint32_t)((1ull << L) - 1) << (threadIdx.x % 32 / L * L);
  const int64_t row = ((int64_t)blockIdx.x * CIO_THREADS + threadIdx.x) / L;
  const int64_t rows = (int64_t)a.B * a.S * a.c.Hkv;
  if (row >= rows) return;
  const int h = (int)(row % a.c.Hkv);
  const int64_t tokn = row / a.c.Hkv;
  const int b = (int)(tokn / a.S), s = (int)(tokn % a.S);
  const int fresh = a.which ? min(max(a.which[b], 0), a.S) : a.S;
  if (s >= fresh) return;
  const int64_t at = (int64_t)a.lens[b] - fresh + s;
  uint8_t* const grp = group_of(a, b, at, h, Gr::BYTES);
  if (!grp) return;
  const int r = (int)(at & 15);
  const uint16_t* ksrc = a.k + b * a.ks.b + s * a.ks.s + h * a.ks.h;
  const uint16_t* vsrc = a.v + b * a.vs.b + s * a.vs.s + h * a.vs.h;

  // K: lane = t*C + sp holds elements 16s' + 4t .. + 3 of the steps s' = 2sp, 2sp + 1
  const int t = lane / C, sp = lane % C;
  uint2 ku[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) ku[i] = *reinterpret_cast<const uint2*>(ksrc + 16 * (2 * sp + i) + 4 * t);
  // V: lane = g*(L/8) + ih holds elements 16i + 2g, + 1 of i = 4ih .. 4ih + 3
  constexpr int IH = L / 8;
  const int g = lane / IH, ih = lane % IH;
  uint32_t vu[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) vu[i] = *reinterpret_cast<const uint32_t*>(vsrc + 16 * (4 * ih + i) + 2 * g);

  {
    float x[8], m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = bf16_to_f32(ku[i].x & 0xFFFF); x[4 * i + 1] = bf16_to_f32(ku[i].x >> 16);
      x[4 * i + 2] = bf16_to_f32(ku[i].y & 0xFFFF); x[4 * i + 3] = bf16_to_f32(ku[i].y >> 16);
      m[i] = fmaxf(fmaxf(magnitude(x[4 * i]), magnitude(x[4 * i + 1])), fmaxf(magnitude(x[4 * i + 2]), magnitude(x[4 * i + 3])));
    }
    if (CF == CF_MX) m[0] = m[1] = fmaxf(m[0], m[1]);           // both steps lie in one block of 32
    uint32_t sb[2], w = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = (CF == CF_MX && i == 1) ? m[0] : lanes_max<C, L>(m[i], mask);   // over the t
      sb[i] = scale_byte<CF>(m[i]);
      w |= (code_byte<CF>(x[4 * i], x[4 * i + 1], sb[i]) | code_byte<CF>(x[4 * i + 2], x[4 * i + 3], sb[i]) << 8) << (16 * i);
    }
    *reinterpret_cast<uint32_t*>(grp + Gr::K + r * (D / 2) + 4 * lane) = w;
    if (t == 0) {
      if (CF == CF_MX) grp[Gr::KS + r * Gr::SB + sp] = (uint8_t)sb[0];
      else *reinterpret_cast<uint16_t*>(grp + Gr::KS + r * Gr::SB + 2 * sp) = (uint16_t)(sb[0] | sb[1] << 8);
    }
  }
  {
    float x[8], m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_to_f32(vu[i] & 0xFFFF); x[2 * i + 1] = bf16_to_f32(vu[i] >> 16);
      m[i] = fmaxf(magnitude(x[2 * i]), magnitude(x[2 * i + 1]));
    }
    if (CF == CF_MX) { m[0] = m[1] = fmaxf(m[0], m[1]); m[2] = m[3] = fmaxf(m[2], m[3]); }
    uint32_t sb[4], w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = (CF == CF_MX && (i & 1)) ? m[i - 1] : lanes_max<IH, L>(m[i], mask);   // over the g
      sb[i] = scale_byte<CF>(m[i]);
      w |= code_byte<CF>(x[2 * i], x[2 * i + 1], sb[i]) << (8 * i);
    }
    *reinterpret_cast<uint32_t*>(grp + Gr::V + r * (D / 2) + 4 * lane) = w;
    if (g == 0) {
      if (CF == CF_MX) *reinterpret_cast<uint16_t*>(grp + Gr::VS + r * Gr::SB + 2 * ih) = (uint16_t)(sb[0] | sb[2] << 8);
      else *reinterpret_cast<uint32_t*>(grp + Gr::VS + r * Gr::SB + 4 * ih) = sb[0] | sb[1] << 8 | sb[2] << 16 | sb[3] << 24;
    }
  }
}

// value pair (bf16x2) of a code byte under a scale: exact, at most 6 significant bits
__device__ __forceinline__ uint32_t value_pair(uint32_t h2, float s) {
  float lo, hi;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}" : "=f"(lo), "=f"(hi) : "r"(h2));
  return cvt_bf16x2(__fmul_rn(lo, s), __fmul_rn(hi, s));
}
template <int CF>
__device__ __forceinline__ float scale_value(uint32_t sb) {
  if constexpr (CF == CF_MX) return sb == 0xFFu ? __uint_as_float(0x7FC00000u) : sb ? __uint_as_float(sb << 23) : __uint_as_float(0x00400000u);
  else return e4m3_to_f32(sb);
}

template <int D, int CF>
__global__ void __launch_bounds__(CIO_THREADS) cache_read_kernel(const CacheIo a) {
  using Gr = CacheGroup<D, CF>;
  constexpr int L = D / 8, C = D / 32, IH = L / 8;
  const int lane = threadIdx.x % L;
  const int64_t row = ((int64_t)blockIdx.x * CIO_THREADS + threadIdx.x) / L;
  const int64_t rows = (int64_t)a.B * a.S * a.c.Hkv;
  if (row >= rows) return;
  const int h = (int)(row % a.c.Hkv);
  const int64_t tokn = row / a.c.Hkv;
  const int b = (int)(tokn / a.S), s = (int)(tokn % a.S);
  const int64_t at = (int64_t)(a.which ? a.which[b] : 0) + s;
  if (at < 0 || at >= a.lens[b]) return;
  const uint8_t* const grp = group_of(a, b, at, h, Gr::BYTES);
  const int r = (int)(at & 15);
  if (a.k) {
    const int t = lane / C, sp = lane % C;
    uint32_t w = 0, h2[4];
    float sc[2] = {0.f, 0.f};
    if (grp) {
      w = *reinterpret_cast<const uint32_t*>(grp + Gr::K + r * (D / 2) + 4 * lane);
      if (CF == CF_MX) sc[0] = sc[1] = scale_value<CF>(grp[Gr::KS + r * Gr::SB + sp]);
      else {
        const uint32_t u = *reinterpret_cast<const uint16_t*>(grp + Gr::KS + r * Gr::SB + 2 * sp);
        sc[0] = scale_value<CF>(u & 0xFF); sc[1] = scale_value<CF>(u >> 8);
      }
    }
    cvt_e2m1x8_f16(w, h2);
    uint16_t* dst = a.k + b * a.ks.b + s * a.ks.s + h * a.ks.h;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint2*>(dst + 16 * (2 * sp + i) + 4 * t) = make_uint2(value_pair(h2[2 * i], sc[i]), value_pair(h2[2 * i + 1], sc[i]));
  }
  if (a.v) {
    const int g = lane / IH, ih = lane % IH;
    uint32_t w = 0, h2[4];
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
    if (grp) {
      w = *reinterpret_cast<const uint32_t*>(grp + Gr::V + r * (D / 2) + 4 * lane);
      if (CF == CF_MX) {
        const uint32_t u = *reinterpret_cast<const uint16_t*>(grp + Gr::VS + r * Gr::SB + 2 * ih);
        sc[0] = sc[1] = scale_value<CF>(u & 0xFF); sc[2] = sc[3] = scale_value<CF>(u >> 8);
      } else {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(grp + Gr::VS + r * Gr::SB + 4 * ih);
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = scale_value<CF>((u >> (8 * i)) & 0xFF);
      }
    }
    cvt_e2m1x8_f16(w, h2);
    uint16_t* dst = a.v + b * a.vs.b + s * a.vs.s + h * a.vs.h;
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(dst + 16 * (4 * ih + i) + 2 * g) = value_pair(h2[i], sc[i]);
  }
}

int64_t blocks_of(const CacheIo& a) {
  return ((int64_t)a.B * a.S * a.c.Hkv * (a.c.D / 8) + CIO_THREADS - 1) / CIO_THREADS;
}

}  // namespace

cudaError_t launch_cache_append(const CacheIo& a, cudaStream_t st) {
  const unsigned grid = (unsigned)blocks_of(a);
  if (a.c.D == 128) {
    if (a.c.cf == CF_MX) cache_append_kernel<128, CF_MX><<<grid, CIO_THREADS, 0, st>>>(a);
    else cache_append_kernel<128, CF_NV><<<grid, CIO_THREADS, 0, st>>>(a);
  } else {
    if (a.c.cf == CF_MX) cache_append_kernel<64, CF_MX><<<grid, CIO_THREADS, 0, st>>>(a);
    else cache_append_kernel<64, CF_NV><<<grid, CIO_THREADS, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheIo& a, cudaStream_t st) {
  const unsigned grid = (unsigned)blocks_of(a);
  if (a.c.D == 128) {
    if (a.c.cf == CF_MX) cache_read_kernel<128, CF_MX><<<grid, CIO_THREADS, 0, st>>>(a);
    else cache_read_kernel<128, CF_NV><<<grid, CIO_THREADS, 0, st>>>(a);
  } else {
    if (a.c.cf == CF_MX) cache_read_kernel<64, CF_MX><<<grid, CIO_THREADS, 0, st>>>(a);
    else cache_read_kernel<64, CF_NV><<<grid, CIO_THREADS, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace fsa
