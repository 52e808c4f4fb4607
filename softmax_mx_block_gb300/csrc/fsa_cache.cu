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
#include "fsa_cache_codes.cuh"

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
