// fsa_cache_attn.cu -- attention of few query rows over the paged 4-bit cache
// (decode steps, guessed tokens, prompt chunks).
//
//   o = softmax(scale q K^T) V  over the keys a row sees, K and V the values the cache
//   stands for (codes times block scales), q as given, sums in fp32.
//
// What bounds it: the cache is read once, 1.06 (E2M1) or 1.125 (NVFP4) bytes per pair of
// K and V elements.  A kv head has only G x Sq query rows (often 8 or fewer), so a 128-row
// tcgen05 tile would be nearly all padding, and V's scales run along D while its product
// runs along the keys, which the block-scaled instructions cannot take.  So each warp works
// on its own keys with m16n8k16 products whose m is the keys (S^T = K Q^T) and then
// D (O^T = V^T P^T), n the query rows ("columns" here: 8 or 16 a pass).
//
//   - The codes go to the products unscaled: E2M1 to f16 is exact in one instruction a
//     pair.  K's scales multiply the fp32 sums of each block; V's scales multiply the
//     probabilities before they are rounded to f16 (11 bits).  Q as f16 with a power of
//     two per row is exact down to 2^-28 of the row's maximum.
//   - The f16 probabilities get a shift R, the running maximum exponent of V's scales, so
//     that p * scale stays below 2^15; 2^28 below that they are still exact to 11 bits.
//     The running maximum M of the scores is raised only when a score beats it by more
//     than 2^4 (then the sums are rescaled), so most tiles need no reduction over lanes.
//     Both offsets multiply numerator and denominator alike and cancel.
//   - Work is split evenly over the warps of one CTA per SM: all (sequence, kv head, 32-key
//     tile) triples in one list, a contiguous share each.  A warp's share of a sequence
//     that others share too is a partial result (maximum, sum, unnormalised rows); the
//     warps of a CTA join theirs in shared memory, and a second kernel joins the CTAs'.
//     The lengths are read on the device, so a captured call follows them.
//   - Each warp has a ring of its own: one bulk copy per page part and tile, an mbarrier a
//     stage.  No warp waits for another before the end.
#include "fsa_cache.h"
#include "fsa_ptx.cuh"

namespace fsa {
namespace {

constexpr int NWC = 12;             // warps of a CTA
constexpr int STG = 3;              // stages of a warp's ring
constexpr int TILE = 32;            // keys of a tile
constexpr float M_NONE = -1e30f;    // maximum of no keys
constexpr float LAZY = 4.0f;        // log2 of how far a score may beat M

template <int D, int CF, int NT>
struct Cfg {
  using Gr = CacheGroup<D, CF>;
  static constexpr int STAGE = 2 * Gr::BYTES;
  static constexpr int COLS = 8 * NT;
  static constexpr int PART = COLS * (D + 2);        // floats of a partial result: rows, maxima, sums
  static constexpr int RING = NWC * STG * STAGE;
  static constexpr int JOIN = NWC * PART * 4;
  static constexpr int SMEM = 1024 + NWC * 32 * 8 + (RING > JOIN ? RING : JOIN);
};

// ---------------------------------------------------------------- the work list
// "Virtual sequence" vb = b * CT + ct: the ct-th pass of columns of sequence b.
struct Span {
  int qlen, len, kmax, tiles;   // rows, keys, keys that some column sees, tiles (0: no rows)
};
__device__ __forceinline__ Span span_of(const CacheAttnArgs& p, int vb, int cols) {
  Span s;
  const int b = p.CT == 1 ? vb : vb / p.CT, ct = vb - b * p.CT;
  s.qlen = p.q_lens ? min(max(p.q_lens[b], 0), p.Sq) : p.Sq;
  s.len = (int)min((int64_t)max(p.lens[b], 0), (int64_t)p.max_pages << p.c.page_shift);
  const int c0 = ct * cols;
  if (c0 >= s.qlen * p.G) { s.kmax = s.tiles = 0; return s; }
  const int last = min(s.qlen - 1, (c0 + cols - 1) / p.G);
  s.kmax = p.causal ? max(0, s.len - s.qlen + last + 1) : s.len;
  s.tiles = max(1, (s.kmax + TILE - 1) / TILE);      // a tile for rows that see nothing: they are written
  return s;
}

// Keys that column c of virtual sequence (b, ct) sees (0 for none and for padding).
__device__ __forceinline__ int limit_of(const CacheAttnArgs& p, const Span& s, int col) {
  const int i = col / p.G;
  if (i >= s.qlen) return 0;
  return p.causal ? max(0, s.len - s.qlen + i + 1) : s.len;
}

__device__ __forceinline__ float e8m0_shifted(uint32_t w, int j) {     // 2^(byte j - 127); 0xFF: Inf, 0: 0
  return __uint_as_float(((w >> (8 * j)) << 23) & 0x7F800000u);
}

// scale factors of one row's blocks (NB = D/32 or D/16 of them)
template <int D, int CF>
__device__ __forceinline__ void load_scales(const uint8_t* at, float* f) {
  if constexpr (CF == CF_MX) {
    const uint32_t w = D == 128 ? *reinterpret_cast<const uint32_t*>(at) : *reinterpret_cast<const uint16_t*>(at);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) f[j] = e8m0_shifted(w, j);
  } else {
    uint32_t w[2];
    if constexpr (D == 128) {
      const uint2 u = *reinterpret_cast<const uint2*>(at);
      w[0] = u.x; w[1] = u.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(at);
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {               // pairs of E4M3
      uint32_t h2;
      asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}"
          : "=r"(h2) : "r"(j & 1 ? w[j / 2] >> 16 : w[j / 2]));
      asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}"
          : "=f"(f[2 * j]), "=f"(f[2 * j + 1]) : "r"(h2));
    }
  }
}

// One warp's running state for one (sequence, kv head, pass of columns).  A thread holds,
// of n-tile n, columns 8n + 2t and + 1 and, of m-tile i, dims 16i + 2g and + 1.
template <int D, int NT>
struct Acc {
  float o[D / 16][NT][4];   // [dim 16i+2g: col 2t, 2t+1; dim 16i+2g+1: col 2t, 2t+1]
  float l[NT][2];           // this thread's part of the row sums
  float m[NT][2];           // running maximum (log2 units), the same in all g
  float r;                  // exponent offset of V's scales
  float vtop;               // 2^(r + 3): a larger scale raises r
};

template <int D, int NT>
__device__ __forceinline__ void reset(Acc<D, NT>& a) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) a.o[i][n][e] = 0.f;
    a.l[n][0] = a.l[n][1] = 0.f;
    a.m[n][0] = a.m[n][1] = M_NONE;
  }
  a.r = -80.f;
  a.vtop = 0.f;
}

// One tile of 32 keys from shared memory.  first: position of the tile's first key.
template <int D, int CF, int NT, bool MASK>
__device__ __forceinline__ void tile_step(const uint8_t* st, const uint2 (&q)[D / 16][NT], const float (&cq)[NT][2],
                                          const int (&lim)[NT][2], int first, uint32_t bad, Acc<D, NT>& a) {
  using Gr = CacheGroup<D, CF>;
  constexpr int NB = CF == CF_MX ? D / 32 : D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tok = (g >> 1) + 4 * (g & 1);            // the key of S^T row g (and 8 more for row g + 8)
  float s[2][NT][4];
  float vs[2][2][NB];
  float vmax = 0.f;
#pragma unroll
  for (int gr = 0; gr < 2; ++gr) {
    const uint8_t* base = st + gr * Gr::BYTES;
    float f0[NB], f1[NB];
    load_scales<D, CF>(base + Gr::KS + tok * Gr::SB, f0);
    load_scales<D, CF>(base + Gr::KS + (tok + 8) * Gr::SB, f1);
    uint32_t w0[D / 32], w1[D / 32];
    const uint8_t* kr = base + Gr::K + tok * (D / 2) + t * (D / 8);
    if constexpr (D == 128) {
      const uint4 u0 = *reinterpret_cast<const uint4*>(kr), u1 = *reinterpret_cast<const uint4*>(kr + 4 * D);
      w0[0] = u0.x; w0[1] = u0.y; w0[2] = u0.z; w0[3] = u0.w;
      w1[0] = u1.x; w1[1] = u1.y; w1[2] = u1.z; w1[3] = u1.w;
    } else {
      const uint2 u0 = *reinterpret_cast<const uint2*>(kr), u1 = *reinterpret_cast<const uint2*>(kr + 4 * D);
      w0[0] = u0.x; w0[1] = u0.y;
      w1[0] = u1.x; w1[1] = u1.y;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[gr][n][e] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      uint32_t r0[4], r1[4];
      cvt_e2m1x8_f16(w0[j], r0);
      cvt_e2m1x8_f16(w1[j], r1);
      const uint32_t lo[4] = {r0[0], r1[0], r0[1], r1[1]}, hi[4] = {r0[2], r1[2], r0[3], r1[3]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16_16816(c, lo, q[2 * j][n].x, q[2 * j][n].y);
        if constexpr (CF == CF_NV) {
#pragma unroll
          for (int e = 0; e < 4; ++e) { s[gr][n][e] = fmaf(c[e], e < 2 ? f0[2 * j] : f1[2 * j], s[gr][n][e]); c[e] = 0.f; }
        }
        mma_f16_16816(c, hi, q[2 * j + 1][n].x, q[2 * j + 1][n].y);
        constexpr int S = CF == CF_NV ? 2 : 1;
#pragma unroll
        for (int e = 0; e < 4; ++e) s[gr][n][e] = fmaf(c[e], e < 2 ? f0[S * j + S - 1] : f1[S * j + S - 1], s[gr][n][e]);
      }
    }
    load_scales<D, CF>(base + Gr::VS + tok * Gr::SB, vs[gr][0]);
    load_scales<D, CF>(base + Gr::VS + (tok + 8) * Gr::SB, vs[gr][1]);
    if (MASK) {
      const int k0 = first + 16 * gr + tok, k1 = k0 + 8;
      const bool gone = (bad >> gr) & 1;
      bool seen0 = false, seen1 = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (gone || k0 >= lim[n][e]) s[gr][n][e] = -INFINITY; else seen0 = true;
          if (gone || k1 >= lim[n][e]) s[gr][n][2 + e] = -INFINITY; else seen1 = true;
        }
      // a key that none of this thread's columns sees has no part in R either
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (!seen0) vs[gr][0][j] = 0.f;
        if (!seen1) vs[gr][1][j] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) vmax = fmaxf(vmax, fmaxf(vs[gr][0][j], vs[gr][1][j]));
  }

  // raise the running maxima where a score or a scale asks for it
  bool raise = vmax > a.vtop;
  float top[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[n][e] = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e])) * cq[n][e];
      raise |= top[n][e] > a.m[n][e] + LAZY;
    }
  if (__any_sync(0xFFFFFFFFu, raise)) {
    float v = 0.f;                                     // the largest finite scale (Inf stands for NaN blocks)
#pragma unroll
    for (int gr = 0; gr < 2; ++gr)
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (vs[gr][0][j] <= 3.4e38f) v = fmaxf(v, vs[gr][0][j]);
        if (vs[gr][1][j] <= 3.4e38f) v = fmaxf(v, vs[gr][1][j]);
      }
#pragma unroll
    for (int x = 1; x < 32; x *= 2) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, x));
    float r = a.r;
    if (v > a.vtop) {
      r = fmaxf((float)((int)(__float_as_uint(v) >> 23) - 126), -80.f);     // 2^r > v
      a.vtop = r > 123.f ? 3.4e38f : exp2f(r + 3.f);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = top[n][e];
#pragma unroll
        for (int x = 4; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
        m = fmaxf(a.m[n][e], m);
        const float f = exp2f((a.m[n][e] + a.r) - (m + r));
        a.m[n][e] = m;
        a.l[n][e] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) { a.o[i][n][e] *= f; a.o[i][n][2 + e] *= f; }
      }
    a.r = r;
  }

  // probabilities, and the products with V
  float off[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) off[n][e] = 8.f - a.r - a.m[n][e];
#pragma unroll
  for (int gr = 0; gr < 2; ++gr) {
    const uint8_t* base = st + gr * Gr::BYTES;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = ex2_approx(fmaf(s[gr][n][e], cq[n][e & 1], off[n][e & 1]));
        s[gr][n][e] = x;
        a.l[n][e & 1] += x;
      }
    // V rows of the keys t, 4 + t, 8 + t, 12 + t, interleaved so that a pair of f16 is one
    // dim of two keys
    const uint8_t* vr = base + Gr::V + t * (D / 2) + g * (D / 16);
    uint32_t x[2][2][D / 64], y[2][2][D / 64];     // [][half][word]: x low nibbles (dim 2g), y high (2g + 1)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t wa[D / 64], wb[D / 64];
      const uint8_t* ra = vr + hf * 4 * D;
      if constexpr (D == 128) {
        const uint2 ua = *reinterpret_cast<const uint2*>(ra), ub = *reinterpret_cast<const uint2*>(ra + 2 * D);
        wa[0] = ua.x; wa[1] = ua.y; wb[0] = ub.x; wb[1] = ub.y;
      } else {
        wa[0] = *reinterpret_cast<const uint32_t*>(ra);
        wb[0] = *reinterpret_cast<const uint32_t*>(ra + 2 * D);
      }
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        x[0][hf][k] = (wa[k] & 0x0F0F0F0Fu) | ((wb[k] << 4) & 0xF0F0F0F0u);
        y[0][hf][k] = ((wa[k] >> 4) & 0x0F0F0F0Fu) | (wb[k] & 0xF0F0F0F0u);
      }
    }
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      uint32_t xa[4], xb[4], ya[4], yb[4];
      cvt_e2m1x8_f16(x[0][0][k], xa);
      cvt_e2m1x8_f16(x[0][1][k], xb);
      cvt_e2m1x8_f16(y[0][0][k], ya);
      cvt_e2m1x8_f16(y[0][1][k], yb);
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int i = 4 * k + ii;
        constexpr int PER = CF == CF_MX ? 2 : 1;      // m-tiles of a scale block
        const int blk = i / PER;
        const uint32_t va[4] = {xa[ii], ya[ii], xb[ii], yb[ii]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p0 = s[gr][n][0] * vs[gr][0][blk], p1 = s[gr][n][1] * vs[gr][0][blk];
          float p2 = s[gr][n][2] * vs[gr][1][blk], p3 = s[gr][n][3] * vs[gr][1][blk];
          if (MASK) {                                  // 0 times a masked key's NaN scale
            const int k0 = first + 16 * gr + tok, k1 = k0 + 8;
            if (k0 >= lim[n][0]) p0 = 0.f;
            if (k0 >= lim[n][1]) p1 = 0.f;
            if (k1 >= lim[n][0]) p2 = 0.f;
            if (k1 >= lim[n][1]) p3 = 0.f;
          }
          const uint32_t b0 = transpose_8x8(cvt_f16x2(p0, p1)), b1 = transpose_8x8(cvt_f16x2(p2, p3));
          mma_f16_16816(a.o[i][n], va, b0, b1);
        }
      }
    }
  }
}

// ------------------------------------------------------------------- a warp's ring
// Page numbers of a piece, 32 at a time in the lanes' registers.
struct Pages {
  const int32_t* row;
  int base, mine, n;
};
__device__ __forceinline__ void pages_at(Pages& pg, int i) {
  pg.base = i;
  const int at = i + (threadIdx.x & 31);
  pg.mine = at < pg.n ? pg.row[at] : -1;
}
__device__ __forceinline__ int page_of(Pages& pg, int i) {
  if (i >= pg.base + 32) pages_at(pg, i);
  return __shfl_sync(0xFFFFFFFFu, pg.mine, i - pg.base);
}

template <int D, int CF, int NT>
__global__ void __launch_bounds__(NWC * 32, 1) cache_attn_kernel(const CacheAttnArgs p) {
  using C = Cfg<D, CF, NT>;
  using Gr = CacheGroup<D, CF>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);                  // [NWC][STG]
  int* flag = reinterpret_cast<int*>(smem + 512);                      // abort
  int* final_seg = reinterpret_cast<int*>(smem + 576);                 // [NWC]
  int64_t* wsum = reinterpret_cast<int64_t*>(smem + 640);              // [NWC + 1]
  int64_t* pre = reinterpret_cast<int64_t*>(smem + 1024);              // [NWC * 32]
  uint8_t* ring = smem + 1024 + NWC * 32 * 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const AbortCtl ac{flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) *flag = 0;
  if (threadIdx.x < NWC * STG) mbar_init(&bars[threadIdx.x], 1);
  fence_mbar_init();

  // the list's length and its prefix sums: a chunk of virtual sequences per thread
  const int VB = p.B * p.CT;
  const int chunk = (VB + NWC * 32 - 1) / (NWC * 32);
  int64_t mine = 0;
  for (int vb = threadIdx.x * chunk; vb < min(VB, (int)(threadIdx.x + 1) * chunk); ++vb)
    mine += (int64_t)span_of(p, vb, C::COLS).tiles * p.c.Hkv;
  int64_t inc = mine;
#pragma unroll
  for (int x = 1; x < 32; x *= 2) {
    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, inc, x);
    if (lane >= x) inc += up;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NWC; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  pre[threadIdx.x] = before + inc - mine;
  __syncthreads();

  // shares: as few warps of each CTA as give every one of them a tile, so small calls
  // spread over the SMs and no share between two others is empty
  const int wpc = (int)max((int64_t)1, min((int64_t)NWC, (total + gridDim.x - 1) / gridDim.x));
  const int NW = (int)min(total, (int64_t)gridDim.x * wpc);
  const int W = blockIdx.x * wpc + warp, slot = blockIdx.x * NWC + warp;
  const bool works = warp < wpc && W < NW;
  int64_t lo = works ? total * W / NW : 0;
  const int64_t hi = works ? total * (W + 1) / NW : 0;
  int4 start = make_int4(-1, 0, 0, 0);
  int seg_open = -1;                                   // the piece that the loop leaves in `a`
  Acc<D, NT> a;
  float cq[NT][2];
  int lim[NT][2];
  Span sp;
  int vb = 0, hkv = 0, tile = 0;
  uint64_t* bar = bars + warp * STG;
  uint8_t* mem = ring + warp * STG * C::STAGE;
  uint32_t phase = 0;                                  // bit s: the phase to wait for next on stage s
  int stage_in = 0, stage_out = 0;

  if (lo < hi) {
    int j = 0;                                         // the last thread whose chunk begins at or before lo
    for (int x = 256; x; x >>= 1)
      if (j + x < NWC * 32 && pre[j + x] <= lo) j += x;
    int64_t acc = pre[j];
    for (vb = j * chunk;; ++vb) {
      sp = span_of(p, vb, C::COLS);
      const int64_t n = (int64_t)sp.tiles * p.c.Hkv;
      if (lo < acc + n) break;
      acc += n;
    }
    hkv = (int)((lo - acc) / sp.tiles);
    tile = (int)((lo - acc) % sp.tiles);
  }

  bool ok = true;
  while (lo < hi && ok) {
    const int b = p.CT == 1 ? vb : vb / p.CT, c0 = (vb - b * p.CT) * C::COLS;
    const int t0 = tile, t1 = (int)min((int64_t)sp.tiles, t0 + (hi - lo));
    const int seg = vb * p.c.Hkv + hkv;
    const int tend = min(t1, (sp.kmax + TILE - 1) / TILE);

    // pages and first copies
    Pages pg{p.table + (int64_t)b * p.max_pages, 0, 0, p.max_pages};
    pages_at(pg, (t0 * TILE) >> p.c.page_shift);
    uint32_t bads = 0;                                  // 2 bits a stage: groups without a page
    auto issue = [&](int tl) {
      const int s = stage_in;
      stage_in = stage_in + 1 == STG ? 0 : stage_in + 1;
      const int pos = tl * TILE;
      const int groups = min(2, (sp.kmax - pos + 15) / 16);
      uint32_t bad = 0, bytes = 0;
      const uint8_t* src[2] = {nullptr, nullptr};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k >= groups) continue;
        const int at = pos + 16 * k;
        const int page = page_of(pg, at >> p.c.page_shift);
        if (page < 0 || page >= p.c.num_pages) {
          bad |= 1u << k;
        } else {
          const int inside = at & ((1 << p.c.page_shift) - 1);
          src[k] = p.c.pages + page * p.c.page_bytes + ((int64_t)(hkv << (p.c.page_shift - 4)) + inside / 16) * Gr::BYTES;
          bytes += Gr::BYTES;
        }
      }
      bads = (bads & ~(3u << (2 * s))) | bad << (2 * s);
      if (lane == 0) {
        if (bad && p.status) atomicExch(p.status, -1);  // FSA_ERR_INVALID_ARG
        mbar_expect_tx(&bar[s], bytes);
        if (src[0] && src[1] == src[0] + Gr::BYTES) {
          bulk_load(mem + s * C::STAGE, src[0], 2 * Gr::BYTES, &bar[s]);
        } else {
          if (src[0]) bulk_load(mem + s * C::STAGE, src[0], Gr::BYTES, &bar[s]);
          if (src[1]) bulk_load(mem + s * C::STAGE + Gr::BYTES, src[1], Gr::BYTES, &bar[s]);
        }
      }
    };
    int issued = t0;
    for (; issued < min(tend, t0 + STG); ++issued) issue(issued);

    // this piece's columns: q as f16 fragments, its factor, its last key
    reset(a);
    uint2 q[D / 16][NT];
    int min_lim = 0x7FFFFFFF;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = c0 + 8 * n + g;                  // fragment columns: g
      const int i = col / p.G;
      const bool live = i < sp.qlen;
      const uint16_t* src = p.q + b * p.qs.b + i * p.qs.s + (int64_t)(hkv * p.G + col - i * p.G) * p.qs.h + 4 * t;
      uint2 u[D / 16];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        u[k] = live ? *reinterpret_cast<const uint2*>(src + 16 * k) : make_uint2(0u, 0u);
        top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(u[k].x << 16)), fabsf(__uint_as_float(u[k].x & 0xFFFF0000u))),
                               fmaxf(fabsf(__uint_as_float(u[k].y << 16)), fabsf(__uint_as_float(u[k].y & 0xFFFF0000u)))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int e = (int)(__float_as_uint(top) >> 23) - 127;                 // floor(log2 top)
      const int up = e == 128 || top == 0.f ? 0 : min(max(4 - e, -126), 126);
      const float f = __uint_as_float((uint32_t)(up + 127) << 23) * p.q_sign;
      const float back = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][n].x = cvt_f16x2(__uint_as_float(u[k].x << 16) * f, __uint_as_float(u[k].x & 0xFFFF0000u) * f);
        q[k][n].y = cvt_f16x2(__uint_as_float(u[k].y << 16) * f, __uint_as_float(u[k].y & 0xFFFF0000u) * f);
      }
      // accumulator columns: 2t, 2t + 1
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        cq[n][c] = p.scale_log2 * __shfl_sync(0xFFFFFFFFu, back, 4 * (2 * t + c));
        lim[n][c] = limit_of(p, sp, c0 + 8 * n + 2 * t + c);
      }
    }
    min_lim = limit_of(p, sp, c0);                      // the first column sees the fewest keys

    for (int tl = t0; tl < tend; ++tl) {
      const int s = stage_out;
      if (!mbar_wait(&bar[s], (phase >> s) & 1, ac)) { ok = false; break; }
      phase ^= 1u << s;
      stage_out = stage_out + 1 == STG ? 0 : stage_out + 1;
      const uint32_t bad = (bads >> (2 * s)) & 3;
      if (bad == 0 && (tl + 1) * TILE <= min_lim) tile_step<D, CF, NT, false>(mem + s * C::STAGE, q, cq, lim, tl * TILE, 0, a);
      else tile_step<D, CF, NT, true>(mem + s * C::STAGE, q, cq, lim, tl * TILE, bad, a);
      __syncwarp();
      if (issued < tend) { issue(issued); ++issued; }
    }
    if (!ok) {                                          // give up: the copies in flight end first
      for (int k = 0; k < STG; ++k) {
        const int s = stage_out;
        if (stage_out == stage_in && k) break;
        mbar_drain(&bar[s], (phase >> s) & 1, ac);
        stage_out = stage_out + 1 == STG ? 0 : stage_out + 1;
      }
      break;
    }

    // row sums over the lanes that share a column
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x *= 2) a.l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, a.l[n][e], x);

    lo += t1 - t0;
    if (t0 == 0 && t1 == sp.tiles) {                    // all of it: write the rows
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = c0 + 8 * n + 2 * t + e, i = col / p.G;
          if (i >= sp.qlen) continue;
          const int h = hkv * p.G + col - i * p.G;
          const bool none = lim[n][e] == 0;
          const float inv = none ? 0.f : 1.0f / a.l[n][e];
          const int64_t at = b * p.os.b + i * p.os.s + h * p.os.h + 2 * g;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const float x = none ? 0.f : a.o[k][n][e] * inv, y = none ? 0.f : a.o[k][n][2 + e] * inv;
            if (p.out_bf16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at + 16 * k) = cvt_bf16x2(x, y);
            else *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at + 16 * k) = make_float2(x, y);
          }
          if (p.lse && g == 0)
            p.lse[((int64_t)b * p.Sq + i) * p.H + h] =
                none ? -INFINITY : (a.m[n][e] + a.r - 8.f + log2f(a.l[n][e])) * 0.69314718055994530942f;
        }
    } else if (lo < hi) {                               // the end of a segment that began before this warp
      float* part = p.partials + (int64_t)(2 * slot) * C::PART;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 8 * n + 2 * t + e;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            *reinterpret_cast<float2*>(part + col * D + 16 * k + 2 * g) = make_float2(a.o[k][n][e], a.o[k][n][2 + e]);
          if (g == 0) {
            part[C::COLS * D + col] = a.m[n][e] + a.r - 8.f;
            part[C::COLS * (D + 1) + col] = a.l[n][e];
          }
        }
    } else {
      seg_open = seg;
    }
    if (t0 == 0 && t1 < sp.tiles) {                     // it goes on: where it ends
      const int64_t end = lo + (sp.tiles - t1) - 1;     // its last tile in the list
      int64_t w = (end * NW + NW - 1) / total;          // near it: the warp with first <= end < first of the next
      if (w >= NW) w = NW - 1;
      while (w > 0 && total * w / NW > end) --w;
      while (w + 1 < NW && total * (w + 1) / NW <= end) ++w;
      start = make_int4(seg, (int)w, total * (w + 1) / NW > end + 1, wpc);   // .z: that warp goes on to others
    }
    tile = 0;
    if (lo < hi && t1 == sp.tiles && ++hkv == p.c.Hkv) {
      hkv = 0;
      do { sp = span_of(p, ++vb, C::COLS); } while (sp.tiles == 0);
    }
  }
  if (lane == 0) p.starts[slot] = start;

  // join the CTA's open pieces
  __syncthreads();
  float* parts = reinterpret_cast<float*>(ring);
  if (lane == 0) final_seg[warp] = ok ? seg_open : -1;
  if (ok && seg_open >= 0) {
    float* part = parts + warp * C::PART;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * n + 2 * t + e;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          *reinterpret_cast<float2*>(part + col * D + 16 * k + 2 * g) = make_float2(a.o[k][n][e], a.o[k][n][2 + e]);
        if (g == 0) {
          part[C::COLS * D + col] = a.m[n][e] + a.r - 8.f;
          part[C::COLS * (D + 1) + col] = a.l[n][e];
        }
      }
  }
  __syncthreads();
  for (int w = 0; w < NWC;) {
    const int seg = final_seg[w];
    int end = w + 1;
    while (end < NWC && final_seg[end] == seg) ++end;
    if (seg >= 0) {
      float* dst = p.partials + (int64_t)(2 * (blockIdx.x * NWC + w) + 1) * C::PART;
      for (int x = threadIdx.x; x < C::COLS * D; x += NWC * 32) {
        const int col = x / D;
        float m = M_NONE * 2.f;
        for (int k = w; k < end; ++k) m = fmaxf(m, parts[k * C::PART + C::COLS * D + col]);
        float o = 0.f, l = 0.f;
        for (int k = w; k < end; ++k) {
          const float* pk = parts + k * C::PART;
          const float f = exp2f(pk[C::COLS * D + col] - m);
          o = fmaf(f, pk[x], o);
          l = fmaf(f, pk[C::COLS * (D + 1) + col], l);
        }
        dst[x] = o;
        if (x % D == 0) {
          dst[C::COLS * D + col] = m;
          dst[C::COLS * (D + 1) + col] = l;
        }
      }
    }
    w = end;
  }
}

// Joins the partial results of the segments that several warps share: a block takes the
// one that begins in its warp, if it goes on.  Its parts: that warp's own (joined over its
// CTA), one for each later CTA, and the last warp's, which has one of its own when it
// goes on to another segment.
template <int D, int NT>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheAttnArgs p) {
  constexpr int COLS = 8 * NT, PART = COLS * (D + 2);
  const int4 st = p.starts[blockIdx.x];
  if (st.x < 0) return;
  const int vb = st.x / p.c.Hkv, hkv = st.x - vb * p.c.Hkv;
  const int b = p.CT == 1 ? vb : vb / p.CT, c0 = (vb - b * p.CT) * COLS;
  const Span sp = span_of(p, vb, COLS);
  const int last = st.y, wpc = st.w, first_cta = blockIdx.x / NWC, last_cta = last / wpc;
  // parts k = 0 .. n-1
  const bool tail_own = st.z != 0;                       // the last warp's part is its leading one
  const int ctas = last_cta - first_cta;                 // CTAs after the first
  const bool last_joined = ctas > 0 && (last_cta * wpc < last || !tail_own);
  const int n = 1 + max(0, ctas - 1) + (last_joined ? 1 : 0) + (tail_own ? 1 : 0);
  auto slot = [&](int k) -> const float* {
    int64_t s;
    if (k == 0) s = 2 * (int64_t)blockIdx.x + 1;
    else if (tail_own && k == n - 1) s = 2 * ((int64_t)last_cta * NWC + last % wpc);
    else s = 2 * (int64_t)(first_cta + k) * NWC + 1;
    return p.partials + s * PART;
  };
  for (int x = threadIdx.x; x < COLS * D / 2; x += 256) {
    const int c = x / (D / 2), d = 2 * (x % (D / 2));
    const int col = c0 + c, i = col / p.G;
    if (i >= sp.qlen) continue;
    float m = M_NONE * 2.f;
    for (int k = 0; k < n; ++k) m = fmaxf(m, slot(k)[COLS * D + c]);
    float o0 = 0.f, o1 = 0.f, l = 0.f;
    for (int k = 0; k < n; ++k) {
      const float* pk = slot(k);
      const float f = exp2f(pk[COLS * D + c] - m);
      const float2 o = *reinterpret_cast<const float2*>(pk + c * D + d);
      o0 = fmaf(f, o.x, o0);
      o1 = fmaf(f, o.y, o1);
      l = fmaf(f, pk[COLS * (D + 1) + c], l);
    }
    const int h = hkv * p.G + col - i * p.G;
    const bool none = limit_of(p, sp, col) == 0;
    const float inv = none ? 0.f : 1.0f / l;
    o0 = none ? 0.f : o0 * inv;
    o1 = none ? 0.f : o1 * inv;
    const int64_t at = b * p.os.b + i * p.os.s + h * p.os.h + d;
    if (p.out_bf16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at) = cvt_bf16x2(o0, o1);
    else *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(o0, o1);
    if (p.lse && d == 0)
      p.lse[((int64_t)b * p.Sq + i) * p.H + h] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  }
}

template <int D, int CF, int NT>
cudaError_t launch(const CacheAttnArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<D, CF, NT>;
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<D, CF, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  cache_attn_kernel<D, CF, NT><<<sms, NWC * 32, C::SMEM, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cache_join_kernel<D, NT><<<sms * NWC, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

int cache_attn_ntiles(int cols) { return cols <= 8 ? 1 : 2; }

size_t cache_attn_workspace(int nt, int D, int sms, size_t* starts_at) {
  const size_t parts = (size_t)2 * sms * NWC * 8 * nt * (D + 2) * sizeof(float);
  if (starts_at) *starts_at = parts;
  return parts + (size_t)sms * NWC * sizeof(int4);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int nt, int sms, cudaStream_t st) {
  if (a.c.D == 128) {
    if (a.c.cf == CF_MX) return nt == 1 ? launch<128, CF_MX, 1>(a, sms, st) : launch<128, CF_MX, 2>(a, sms, st);
    return nt == 1 ? launch<128, CF_NV, 1>(a, sms, st) : launch<128, CF_NV, 2>(a, sms, st);
  }
  if (a.c.cf == CF_MX) return nt == 1 ? launch<64, CF_MX, 1>(a, sms, st) : launch<64, CF_MX, 2>(a, sms, st);
  return nt == 1 ? launch<64, CF_NV, 1>(a, sms, st) : launch<64, CF_NV, 2>(a, sms, st);
}

}  // namespace fsa
