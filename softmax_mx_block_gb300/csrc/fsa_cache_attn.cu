// fsa_cache_attn.cu -- attention of few query rows over the paged 4-bit cache
// (decode steps, guessed tokens, short prompt chunks).
//
//   o = softmax(scale q K^T) V  over the keys a row sees, K and V the values the cache
//   stands for (codes times block scales), q as given, sums in fp32.
//
// What bounds it: the cache is read once, 1.06 (E2M1) or 1.125 (NVFP4) bytes per pair of
// K and V elements, as long as a kv head has no more than 16 query rows (G x Sq); it is read and
// converted again for each 16 more.  V's scales run along D while its product runs along the
// keys, which the block-scaled tcgen05 instructions cannot take, and q would have to be split
// or quantised for them; the f16 ones would need the codes converted into shared memory.  So
// each warp works on its own keys with m16n8k16 products whose m is the keys (S^T = K Q^T) and
// then D (O^T = V^T P^T), n the query rows ("columns" here: 8 or 16 a pass), the codes converted
// in registers.
//
//   - E2M1 to f16 is exact in one instruction a pair.  An E8M0 scale of K multiplies the fp32
//     sum of its block; an E4M3 one multiplies the codes (6 bits: exact in f16).  V's scales
//     multiply the probabilities: E8M0 in fp32 before they are rounded to f16, E4M3 as f16
//     after (a second rounding).  Q as f16 with a power of two per row is exact down to 2^-18
//     of the row's maximum and off by at most 2^-29 of it below.
//   - A tile's scales are unpacked once, a token a lane, through shared memory: every lane of
//     a quad needs the same ones (13% of the arithmetic pipe with E8M0, 22% with E4M3).
//   - The f16 probabilities carry 2^(8 - r), r the running maximum exponent of V's scales,
//     so that p * scale stays below 2^15.  With E8M0 scales r spans fp32's whole range: what of
//     it exceeds 2^40 divides the unpacked scales instead, so that no weight down to 2^-94 of the
//     largest is flushed from the sum.  The rows of a pass share r while they see the same keys;
//     in the last tiles, where they do not, each has its own.  The running maximum m of the raw
//     scores is raised only when a score beats it by more than 2^4 in the softmax (then the
//     sums are rescaled), so most tiles need one vote and no reduction over lanes.
//   - Work is split evenly over the warps of one CTA per SM: all (sequence, kv head, 32-key
//     tile) triples in one list, a contiguous share each, a segment's start weighing as
//     three tiles (64 ragged sequences: 59 us at none, 36.2 at two, 35.6 at three, 36.5 at four).
//     A warp's share of a segment that others share too is a partial result (maximum, sum,
//     unnormalised rows); the warps of a CTA join theirs in shared memory, and a second
//     kernel, launched early, joins the CTAs'.  The lengths are read on the device, so a
//     captured call follows them.  Short tables take a kernel of a CTA a segment instead.
//   - Each warp has a ring of its own: one bulk copy per page part and tile, an mbarrier a
//     stage, the lane that looked the page up copies it.  No warp waits for another before
//     the end.  Two stages: 24 tiles in flight an SM cover the latency, and a third cost 3%.
//     12 warps of 168 registers: 8 were 5 to 7% slower, 10 (uneven over the four schedulers)
//     10%, 14 and 16 12% (more spills: with 12 the E2M1 instance of 128 dims and 8 columns spills 76
//     bytes, the NVFP4 one 24; those of 64 dims and 16 columns 48 and 44; of 128 dims and 16 columns,
//     8 warps of 255, the E2M1 one 116; the others none).
//
// Measured (one GB300, copies at 6.79 TB/s): 8 sequences of 128K tokens, 8 kv heads, 4 query
// heads each: E2M1 199 us, 5.74 TB/s of cache, NVFP4 221 us, 5.47 TB/s; one sequence 35.7 us
// for 143 MB.  Of that 1.4 us go until the list is summed, 0.6 until a warp has its place in it,
// 1.7 until its first copies are on their way; the warps of a CTA end 2.8 us before its slowest
// on average, its join takes 1.3, the second kernel 3.  Counters at the large sizes: 265 (E2M1) and
// 295 (NVFP4) warp instructions for 16 keys of a kv head, 2.5 and 2.4 a cycle of 4.
#include <atomic>
#include "fsa_cache.h"
#include "fsa_ptx.cuh"

namespace fsa {
namespace {

// warps of a CTA, by the registers that a warp's columns take
template <int D, int NT>
__host__ __device__ constexpr int cta_warps() { return NT == 1 || D == 64 ? 12 : 8; }
constexpr int TILE = 32;            // keys of a tile
constexpr int EXTRA = 3;            // what a segment's start costs a warp, in tiles
constexpr float S_NONE = -3e38f;    // maximum of no keys (raw scores)
constexpr float LAZY = 4.0f;        // log2 of how far a score may beat M

template <int D, int CF, int NT>
struct Cfg {
  using Gr = CacheGroup<D, CF>;
  static constexpr int NWC = cta_warps<D, NT>();
  static constexpr int STAGE = 2 * Gr::BYTES;
  static constexpr int COLS = 8 * NT;
  static constexpr int PART = COLS * (D + 6);        // floats of a partial result (put_part)
  static constexpr int STG = 2;                      // stages of a warp's ring
  static constexpr int RING = NWC * STG * STAGE;
  static constexpr int JOIN = NWC * PART * 4;
  static constexpr int SCALES = TILE * Gr::SB * 8;   // unpacked scales of a tile: a word each for K and for V
  static constexpr int SMEM = 1024 + NWC * 32 * 8 + NWC * SCALES + JOIN + (RING > JOIN ? RING : JOIN);
};

// ---------------------------------------------------------------- the work list
// "Virtual sequence" vb = b * CT + ct: the ct-th pass of columns of sequence b.
// The units of all virtual sequences together fit an int (the host sees to it).
struct Span {
  int qlen, len, kmax, tiles;   // rows, keys, keys that some column sees, tiles (0: no rows)
  __device__ __forceinline__ int units() const { return tiles ? tiles + EXTRA : 0; }
};
// row i of a column i * G + its head: col / G
__device__ __forceinline__ int row_of(const CacheAttnArgs& p, int col) {
  return p.g_mul ? (int)__umulhi((uint32_t)col, p.g_mul) : p.G == 1 ? col : col / p.G;
}
__device__ __forceinline__ Span span_of(const CacheAttnArgs& p, int vb, int cols) {
  Span s;
  const int b = p.CT == 1 ? vb : vb / p.CT, ct = vb - b * p.CT;
  s.qlen = p.q_lens ? min(max(p.q_lens[b], 0), p.Sq) : p.Sq;
  s.len = (int)min((int64_t)max(p.lens[b], 0), (int64_t)p.max_pages << p.c.page_shift);
  const int c0 = ct * cols;
  if (c0 >= s.qlen * p.G) { s.kmax = s.tiles = 0; return s; }
  const int last = min(s.qlen - 1, row_of(p, c0 + cols - 1));
  s.kmax = p.causal ? max(0, s.len - s.qlen + last + 1) : s.len;
  s.tiles = max(1, (s.kmax + TILE - 1) / TILE);      // a tile for rows that see nothing: they are written
  return s;
}

// `total` units over n warps: the first `more` of them take base + 1, the others base.
struct Shares {
  int base, more;
  __device__ __forceinline__ Shares(int total, int n) {
    base = n > 0 ? (int)((uint32_t)total / (uint32_t)n) : 0;
    more = total - base * n;
  }
  __device__ __forceinline__ int first(int w) const { return base * w + min(w, more); }
  __device__ __forceinline__ int of(int unit) const {          // the warp that has it
    const int cut = (base + 1) * more;
    return unit < cut ? (int)((uint32_t)unit / (uint32_t)(base + 1)) : more + (int)((uint32_t)(unit - cut) / (uint32_t)base);
  }
};

// Keys that column c of virtual sequence (b, ct) sees (0 for none and for padding).
__device__ __forceinline__ int limit_of(const CacheAttnArgs& p, const Span& s, int col) {
  const int i = row_of(p, col);
  if (i >= s.qlen) return 0;
  return p.causal ? max(0, s.len - s.qlen + i + 1) : s.len;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t low_twice(uint32_t x) { return __byte_perm(x, x, 0x1010); }
__device__ __forceinline__ uint32_t high_twice(uint32_t x) { return __byte_perm(x, x, 0x3232); }
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two_bytes) {     // the low two bytes, exact
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(two_bytes));
  return r;
}

// The part of the offset r that the probabilities and their sum carry, and the part that divides
// V's scales.  2^40: p goes down to 2^(8 - 40 - 94), fp32's end, and from the least r, -80, a sum is
// brought to the highest by one factor, 2^-120.
constexpr int R_CAP = 40;
template <class R>
__device__ __forceinline__ R p_offset(R r) { return r < (R)R_CAP ? r : (R)R_CAP; }
// 1 over the part that divides V's scales
__device__ __forceinline__ float excess(int r) { return __uint_as_float((uint32_t)(127 + p_offset(r) - r) << 23); }

// One warp's running state for one (sequence, kv head, pass of columns).  A thread holds,
// of n-tile n, columns 8n + 2t and + 1 and, of m-tile i, dims 16i + 2g and + 1.
template <int D, int CF, int NT>
struct Acc {
  // the offset of V's scales: p carries 2^(8 - r), 2^r above the scales seen, so that p times
  // a scale fits f16 (E4M3's range is narrow: there r starts at 0)
  static constexpr int R_MIN = CF == CF_MX ? -80 : 0;
  float o[D / 16][NT][4];   // [dim 16i+2g: col 2t, 2t+1; dim 16i+2g+1: col 2t, 2t+1]
  float l[NT][2];           // this thread's part of the row sums
  float m[NT][2];           // running maximum of the raw scores, the same in all g
  float top[NT][2];         // a raw score above this raises m
  float cq[NT][2];          // what a raw score was multiplied by (log2 units); last set by finish
  int r;                    // o holds exp2((s - m) cq + 8 - r) times values, l the same with p_offset(r)
  float shift;              // 8 - p_offset(r)
  uint32_t vtop;            // highest scale byte that r allows, as the high bytes of two halves
  // The columns' offsets: r, but for rows of which some do not see some keys of the last tiles.
  // There each column goes by the keys it sees, so that a value behind a row does not take
  // bits from it.
  int rc[NT][2];

  static __device__ __forceinline__ int offset(int x) { return CF == CF_MX ? p_offset(x) : x; }     // (E4M3's r: 0 to 9)
  __device__ __forceinline__ void set_r(int x) {
    r = x;
    shift = 8.f - (float)offset(x);
    vtop = (uint32_t)allowed(x) * 0x01000100u | 0x00FF00FFu;
  }
  static __device__ __forceinline__ int allowed(int x) { return CF == CF_MX ? min(x + 3 + 127, 254) : min((x + 10) * 8 - 1, 0x7E); }
  // the offset to go on with from x when a scale byte v comes: 2^r > scale
  static __device__ __forceinline__ int raised(int x, int v) {
    return v > allowed(x) ? max(R_MIN, CF == CF_MX ? v - 126 : (v >> 3) - 6) : x;
  }
  __device__ __forceinline__ void set_m(int n, int e, float x, float c) {
    m[n][e] = x;
    top[n][e] = x + fminf(LAZY / c, 3.4e38f);   // (finite from no keys on: scores of fp32's top quarter raise m)
  }
  __device__ __forceinline__ void reset(const float (&f)[NT][2]) {
    set_r(R_MIN);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] = 0.f;
        set_m(n, e, S_NONE, f[n][e]);
      }
    }
  }
  // After the last tile: the sums over all lanes.
  __device__ __forceinline__ void finish(const float (&f)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[n][e] += __shfl_xor_sync(0xFFFFFFFFu, l[n][e], x);
        cq[n][e] = f[n][e];
      }
  }
};

// The scales of a tile as the products take them, a token a lane: E8M0 as fp32, E4M3 as f16
// twice in a word.  Every lane of a quad needs the same ones, so they are unpacked once.
// Layout: 16-byte (or SB-word) pieces [K pieces][32 tokens], then V's.  Returns V's scale
// bytes.
template <int D, int CF>
struct TileScales {
  static constexpr int SB = CacheGroup<D, CF>::SB;
  static constexpr int PW = SB < 4 ? SB : 4, PIECES = SB / PW;         // words of a piece, pieces of a row
  static constexpr int BYTE_WORDS = SB == 8 ? 2 : 1;
  uint32_t v[BYTE_WORDS];                                              // V's bytes of this lane's token

  static __device__ __forceinline__ void unpack(const uint32_t* w, uint32_t* dst) {
    uint32_t f[SB];
#pragma unroll
    for (int x = 0; x < SB; x += 2) {
      const uint32_t two = w[x / 4] >> (8 * (x % 4));
      if constexpr (CF == CF_MX) {
        float a, b;
        e8m0x2_f32(two, a, b);
        f[x] = __float_as_uint(a);
        f[x + 1] = __float_as_uint(b);
      } else {
        const uint32_t h = e4m3x2_f16(two);
        f[x] = low_twice(h);
        f[x + 1] = high_twice(h);
      }
    }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      if constexpr (PW == 4) *reinterpret_cast<uint4*>(dst + (q * TILE + lane) * 4) = make_uint4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
      else *reinterpret_cast<uint2*>(dst + lane * 2) = make_uint2(f[0], f[1]);
    }
  }
  static __device__ __forceinline__ void bytes(const uint8_t* at, uint32_t* w) {
    if constexpr (SB == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(at);
      w[0] = u.x; w[1] = u.y;
    } else if constexpr (SB == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(at);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(at);
    }
  }
  __device__ __forceinline__ TileScales(const uint8_t* st, uint32_t* dst) {
    using Gr = CacheGroup<D, CF>;
    const int lane = threadIdx.x & 31;
    const uint8_t* const grp = st + (lane >> 4) * Gr::BYTES + (lane & 15) * SB;
    uint32_t k[BYTE_WORDS];
    bytes(grp + Gr::KS, k);
    bytes(grp + Gr::VS, v);
    unpack(k, dst);
    unpack(v, dst + TILE * SB);
  }
  // V's scales of this lane's token times 2^e, -88 <= e <= 88 (all lanes together)
  static __device__ __forceinline__ void shift_v(uint32_t* dst, int e) {
    const float f = __uint_as_float((uint32_t)(127 + e) << 23);
    uint32_t w[SB];
    const int lane = threadIdx.x & 31;
    __syncwarp();
    row(dst, lane, w);
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
#pragma unroll
      for (int x = 0; x < PW; ++x) dst[(q * TILE + lane) * PW + x] = __float_as_uint(__uint_as_float(w[q * PW + x]) * f);
    __syncwarp();
  }
  // a row's scales: word x of token tok, of K (from = sc) or V (from = sc + TILE * SB)
  static __device__ __forceinline__ void row(const uint32_t* from, int tok, uint32_t* f) {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      if constexpr (PW == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(from + (q * TILE + tok) * 4);
        f[4 * q] = u.x; f[4 * q + 1] = u.y; f[4 * q + 2] = u.z; f[4 * q + 3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(from + tok * 2);
        f[0] = u.x; f[1] = u.y;
      }
    }
  }
};

// NG groups of 16 keys of a tile, from group g0 on, in shared memory.  sc: the tile's unpacked
// scales; vs: V's scale bytes of this lane's token (0 for a token that no column sees);
// first: position of the tile's first key; bad: groups without a page.  MASK 1: some column
// does not see some key, but those with rows see the same ones; 2: they do not, and each has an
// offset of its own.
template <int D, int CF, int NT, int NG, int MASK>
__device__ __forceinline__ void tile_step(const uint8_t* st, uint32_t* sc, const uint32_t (&vs)[TileScales<D, CF>::BYTE_WORDS], int g0,
                                          const uint2 (&q)[D / 16][NT], const float (&cq)[NT][2],
                                          const int (&lim)[NT][2], int first, uint32_t bad, Acc<D, CF, NT>& a) {
  using Gr = CacheGroup<D, CF>;
  using Ts = TileScales<D, CF>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // the key of S^T row g (and 8 more for row g + 8): 0 5 1 6 2 7 3 4.  Rows 2t and 2t + 1 are
  // keys of different parity, so the two rows that a quarter of the warp loads lie in
  // different banks; and the four even rows, which V's loads take together, are keys 0 to 3.
  const int tok = g & 1 ? 4 + (((g >> 1) + 1) & 3) : g >> 1;
  float s[NG][NT][4];
#pragma unroll
  for (int gr = 0; gr < NG; ++gr) {
    const uint8_t* base = st + (g0 + gr) * Gr::BYTES;
    uint32_t ks[2][Gr::SB];
    Ts::row(sc, 16 * (g0 + gr) + tok, ks[0]);
    Ts::row(sc, 16 * (g0 + gr) + tok + 8, ks[1]);
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
      if constexpr (CF == CF_NV) {                   // code times E4M3 scale: 6 bits, exact in f16
        const uint32_t f0l = ks[0][2 * j], f0h = ks[0][2 * j + 1], f1l = ks[1][2 * j], f1h = ks[1][2 * j + 1];
        r0[0] = hmul2(r0[0], f0l); r0[1] = hmul2(r0[1], f0l); r0[2] = hmul2(r0[2], f0h); r0[3] = hmul2(r0[3], f0h);
        r1[0] = hmul2(r1[0], f1l); r1[1] = hmul2(r1[1], f1l); r1[2] = hmul2(r1[2], f1h); r1[3] = hmul2(r1[3], f1h);
      }
      const uint32_t lo[4] = {r0[0], r1[0], r0[1], r1[1]}, hi[4] = {r0[2], r1[2], r0[3], r1[3]};
      if constexpr (CF == CF_NV) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16_16816(s[gr][n], lo, q[2 * j][n].x, q[2 * j][n].y);
          mma_f16_16816(s[gr][n], hi, q[2 * j + 1][n].x, q[2 * j + 1][n].y);
        }
      } else {                                       // the E8M0 scale has fp32's range: on the block's sum
        const float f0 = __uint_as_float(ks[0][j]), f1 = __uint_as_float(ks[1][j]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float c[4];
          mma_f16_16816_zero(c, lo, q[2 * j][n].x, q[2 * j][n].y);
          mma_f16_16816(c, hi, q[2 * j + 1][n].x, q[2 * j + 1][n].y);
          s[gr][n][0] = fmaf(c[0], f0, s[gr][n][0]);
          s[gr][n][1] = fmaf(c[1], f0, s[gr][n][1]);
          s[gr][n][2] = fmaf(c[2], f1, s[gr][n][2]);
          s[gr][n][3] = fmaf(c[3], f1, s[gr][n][3]);
        }
      }
    }
  }

  uint32_t seen[NG][NT][2];                           // MASK: all ones in the halves (columns) that see the row
  if (MASK) {
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const int k0 = first + 16 * (g0 + gr) + tok, k1 = k0 + 8;
      const bool gone = (bad >> (g0 + gr)) & 1;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        seen[gr][n][0] = gone ? 0u : (k0 < lim[n][0] ? 0xFFFFu : 0u) | (k0 < lim[n][1] ? 0xFFFF0000u : 0u);
        seen[gr][n][1] = gone ? 0u : (k1 < lim[n][0] ? 0xFFFFu : 0u) | (k1 < lim[n][1] ? 0xFFFF0000u : 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(seen[gr][n][e >> 1] & (e & 1 ? 0xFFFF0000u : 0xFFFFu))) s[gr][n][e] = -INFINITY;
      }
    }
  }

  // raise the running maxima where a score or a scale asks for it
  uint32_t vm = a.vtop;                              // with this token's scale bytes in the high bytes of the halves
#pragma unroll
  for (int x = 0; x < Ts::BYTE_WORDS; ++x) vm = __vimax3_u16x2(vm, vs[x], vs[x] << 8);
  bool raise = vm != a.vtop;
  float top[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[n][e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
      if (NG == 2) top[n][e] = fmaxf(top[n][e], fmaxf(s[NG - 1][n][e], s[NG - 1][n][2 + e]));
      raise |= top[n][e] > a.top[n][e];
    }
  if (__any_sync(0xFFFFFFFFu, raise)) {
    constexpr uint32_t NAN_BYTE = CF == CF_MX ? 0xFF : 0x7F;
    uint32_t v = 0;
#pragma unroll
    for (int x = 0; x < Gr::SB; ++x) {
      const uint32_t byte = (vs[x / 4] >> (8 * (x % 4))) & 0xFF;
      if (byte != NAN_BYTE) v = max(v, byte);
    }
    int dr, dl;                                      // the offset's change, for the rows and for the sums
    if constexpr (MASK < 2) {
      const int r_old = a.r;
      a.set_r(a.raised(r_old, (int)__reduce_max_sync(0xFFFFFFFFu, v)));
      dr = r_old - a.r;
      dl = a.offset(r_old) - a.offset(a.r);
      if constexpr (CF == CF_MX) {                   // this tile's scales are divided by what r_old had over the cap
        if (dr != dl) Ts::shift_v(sc + TILE * Gr::SB, dr - dl);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (MASK == 2) {
          int mine = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {              // the columns of the lanes t = c
            const int last = __shfl_sync(0xFFFFFFFFu, lim[n][e], c);
            const int most = (int)__reduce_max_sync(0xFFFFFFFFu, first + lane < last ? v : 0u);
            if (t == c) mine = most;
          }
          const int r_old = a.rc[n][e];
          a.rc[n][e] = a.raised(r_old, mine);
          dr = r_old - a.rc[n][e];
          dl = a.offset(r_old) - a.offset(a.rc[n][e]);
        }
        const float fr = (float)dr, fl = (float)dl;
        float m = top[n][e];
#pragma unroll
        for (int x = 4; x < 32; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
        m = fmaxf(a.m[n][e], m);
        const float f = exp2f(fmaf(a.m[n][e] - m, cq[n][e], fr));
        if (CF == CF_MX && dr != dl) a.l[n][e] *= exp2f(fmaf(a.m[n][e] - m, cq[n][e], fl));     // (r over the cap)
        else a.l[n][e] *= f;
        a.set_m(n, e, m, cq[n][e]);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) { a.o[i][n][e] *= f; a.o[i][n][2 + e] *= f; }
      }
  }

  // probabilities (the difference first: its error is relative to it, however large the scores),
  // and the products with V
#pragma unroll
  for (int gr = 0; gr < NG; ++gr) {
    const uint8_t* base = st + (g0 + gr) * Gr::BYTES;
    float x4[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x4[n][e] = ex2_approx(fmaf(s[gr][n][e] - a.m[n][e & 1], cq[n][e & 1], MASK == 2 ? 8.f - (float)a.offset(a.rc[n][e & 1]) : a.shift));
        a.l[n][e & 1] += x4[n][e];
      }
    // E8M0 scales multiply in fp32 and the product is rounded; E4M3 ones multiply p as f16
    uint32_t p[NT][2], vf[2][Gr::SB];
    Ts::row(sc + TILE * Gr::SB, 16 * (g0 + gr) + tok, vf[0]);
    Ts::row(sc + TILE * Gr::SB, 16 * (g0 + gr) + tok + 8, vf[1]);
    if constexpr (CF == CF_NV) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        p[n][0] = cvt_f16x2(x4[n][0], x4[n][1]);     // row g: columns 2t, 2t + 1
        p[n][1] = cvt_f16x2(x4[n][2], x4[n][3]);     // row g + 8
      }
    }
    // V rows of the keys of S^T rows 2t, 2t + 1 and 8 more, interleaved so that a pair of f16
    // is one dim of two keys
    const uint8_t* vr = base + Gr::V + t * (D / 2) + g * (D / 16);
    const uint8_t* vr1 = base + Gr::V + (4 + ((t + 1) & 3)) * (D / 2) + g * (D / 16);
    uint32_t x[2][D / 64], y[2][D / 64];             // [half][word]: x low nibbles (dim 2g), y high (2g + 1)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t wa[D / 64], wb[D / 64];
      const uint8_t *ra = vr + hf * 4 * D, *rb = vr1 + hf * 4 * D;
      if constexpr (D == 128) {
        const uint2 ua = *reinterpret_cast<const uint2*>(ra), ub = *reinterpret_cast<const uint2*>(rb);
        wa[0] = ua.x; wa[1] = ua.y; wb[0] = ub.x; wb[1] = ub.y;
      } else {
        wa[0] = *reinterpret_cast<const uint32_t*>(ra);
        wb[0] = *reinterpret_cast<const uint32_t*>(rb);
      }
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        x[hf][k] = (wa[k] & 0x0F0F0F0Fu) | ((wb[k] << 4) & 0xF0F0F0F0u);
        y[hf][k] = ((wa[k] >> 4) & 0x0F0F0F0Fu) | (wb[k] & 0xF0F0F0F0u);
      }
    }
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      uint32_t xa[4], xb[4], ya[4], yb[4];
      cvt_e2m1x8_f16(x[0][k], xa);
      cvt_e2m1x8_f16(x[1][k], xb);
      cvt_e2m1x8_f16(y[0][k], ya);
      cvt_e2m1x8_f16(y[1][k], yb);
      uint32_t b0[NT], b1[NT];
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int i = 4 * k + ii;
        const uint32_t va[4] = {xa[ii], ya[ii], xb[ii], yb[ii]};
        if (CF == CF_NV || (ii & 1) == 0) {           // a new block: 16 or 32 dims
          const int blk = CF == CF_MX ? i / 2 : i;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t p0, p1;
            if constexpr (CF == CF_NV) {
              p0 = hmul2(p[n][0], vf[0][blk]);
              p1 = hmul2(p[n][1], vf[1][blk]);
            } else {
              float va0 = __uint_as_float(vf[0][blk]), vb0 = va0, va1 = __uint_as_float(vf[1][blk]), vb1 = va1;
              if constexpr (MASK == 2) {              // divided by what the columns' offsets have over the cap
                const float fa = excess(a.rc[n][0]), fb = excess(a.rc[n][1]);
                va0 *= fa; va1 *= fa;
                vb0 *= fb; vb1 *= fb;
              }
              p0 = cvt_f16x2(x4[n][0] * va0, x4[n][1] * vb0);
              p1 = cvt_f16x2(x4[n][2] * va1, x4[n][3] * vb1);
            }
            if (MASK) { p0 &= seen[gr][n][0]; p1 &= seen[gr][n][1]; }   // 0 times a masked key's NaN scale
            b0[n] = transpose_8x8(p0);
            b1[n] = transpose_8x8(p1);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_f16_16816(a.o[i][n], va, b0[n], b1[n]);
      }
    }
  }
}

// ------------------------------------------------------------------------ results
// What a row's sums say: its maximum raw score, the sum of exp2((s - m) cq + 8 - p_offset(r)) over its
// keys, and the two numbers that go with them.
struct Sum {
  float m, l, r, cq;
};
// One finished row: where it goes, and what its sums say.
struct Row {
  int64_t at, lse_at;
  float inv, lse;
  bool none;               // no key: zeros (none by the lengths, or none on a page of the pool: nothing was summed)
  __device__ __forceinline__ Row(const CacheAttnArgs& p, int b, int hkv, int col, const Span& s, const Sum& sum) {
    const int i = row_of(p, col), h = hkv * p.G + col - i * p.G;
    at = b * p.os.b + i * p.os.s + h * p.os.h;
    lse_at = ((int64_t)b * p.Sq + i) * p.H + h;
    none = limit_of(p, s, col) == 0 || sum.l == 0.f;
    inv = exp2f(sum.r - p_offset(sum.r)) / sum.l;
    lse = none ? -INFINITY : fmaf(sum.m, sum.cq, p_offset(sum.r) - 8.f + log2f(sum.l)) * 0.69314718055994530942f;
  }
  __device__ __forceinline__ void put(const CacheAttnArgs& p, int d, float2 o) const {
    o.x = none ? 0.f : o.x * inv;
    o.y = none ? 0.f : o.y * inv;
    if (p.out_bf16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at + d) = cvt_bf16x2(o.x, o.y);
    else *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at + d) = o;
  }
  __device__ __forceinline__ void put_lse(const CacheAttnArgs& p) const {
    if (p.lse) p.lse[lse_at] = lse;
  }
};

// A partial result: the unnormalised rows [COLS][D + 4] (4 more, so that the lanes of a quad,
// two columns apart, store to different banks; r and cq are in the first two of them), their
// maxima, their sums.  The maxima are raw scores: in log2 units and with r in them, scores far
// from zero would swallow r and the differences between parts.
template <int D, int COLS>
__device__ __forceinline__ void put_sum(float* part, int col, const Sum& s) {
  *reinterpret_cast<float2*>(part + col * (D + 4) + D) = make_float2(s.r, s.cq);
  part[COLS * (D + 4) + col] = s.m;
  part[COLS * (D + 5) + col] = s.l;
}
template <int D, int COLS>
__device__ __forceinline__ Sum get_sum(const float* part, int col) {
  const float2 f = *reinterpret_cast<const float2*>(part + col * (D + 4) + D);
  return {part[COLS * (D + 4) + col], part[COLS * (D + 5) + col], f.x, f.y};
}
// What a part's rows and its sum count in a join to maximum m and offset r: nothing if it saw no key.
struct PartWeight {
  float o, l;
  __device__ __forceinline__ PartWeight(const Sum& s, float m, float r) {
    o = s.l == 0.f ? 0.f : exp2f(fmaf(s.m - m, s.cq, s.r - r));
    l = s.l == 0.f ? 0.f : exp2f(fmaf(s.m - m, s.cq, p_offset(s.r) - p_offset(r)));
  }
};
template <int D, int CF, int NT>
__device__ __forceinline__ void put_part(float* part, const Acc<D, CF, NT>& a) {
  constexpr int COLS = 8 * NT, DP = D + 4;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = 8 * n + 2 * t + e;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        *reinterpret_cast<float2*>(part + col * DP + 16 * k + 2 * g) = make_float2(a.o[k][n][e], a.o[k][n][2 + e]);
      if (g == 0) put_sum<D, COLS>(part, col, Sum{a.m[n][e], a.l[n][e], (float)a.rc[n][e], a.cq[n][e]});
    }
}

// ---------------------------------------------------------------------- a warp's work
// A warp's ring of stages, and where it stands in it.
struct Ring {
  uint64_t* bar;
  uint8_t* mem;
  uint32_t* scales;        // of the tile at work
  uint32_t phase;          // bit s: the phase to wait for next on stage s
  int in, out;
};

// The tiles [t0, t1) of one segment: (sequence b, kv head, columns c0 ..).  Leaves the
// running state in `a`; false if a wait ran out.
template <int D, int CF, int NT>
__device__ __forceinline__ bool run_piece(const CacheAttnArgs& p, const Span& sp, int b, int hkv, int c0, int t0, int t1,
                                          Ring& r, const AbortCtl& ac, Acc<D, CF, NT>& a) {
  using C = Cfg<D, CF, NT>;
  using Gr = CacheGroup<D, CF>;
  constexpr int STG = C::STG;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  bool ok = true;
  // What a raw score of a column is multiplied by (log2 units): beside `a` until the end for 8
  // columns, in it for 16 (us beside / in it: 8 sequences of 128K E2M1 keys 199 / 204, 8 of 32K NVFP4 keys
  // with 16 columns 94 / 89; the others within 3%).
  float own[NT][2];
  float (&cq)[NT][2] = NT == 1 ? own : a.cq;
  int lim[NT][2];                                       // how many keys it sees
  const int tend = min(t1, (sp.kmax + TILE - 1) / TILE);
  // q's rows, on their way while the pages are looked up
  uint2 u[NT][D / 16];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = c0 + 8 * n + g;                   // fragment columns: g
    const int i = row_of(p, col);
    const uint16_t* src = p.q + b * p.qs.b + i * p.qs.s + (int64_t)(hkv * p.G + col - i * p.G) * p.qs.h + 4 * t;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      u[n][k] = i < sp.qlen ? *reinterpret_cast<const uint2*>(src + 16 * k) : make_uint2(0u, 0u);
  }

  // Pages of 32 tiles at a time, a tile a lane; the lane that has a tile copies it.
  const uint8_t* const head = p.c.pages + ((int64_t)hkv << (p.c.page_shift - 4)) * Gr::BYTES;
  const int32_t* const row = p.table + (int64_t)b * p.max_pages;
  int batch = 0, page0 = 0, page1 = 0;
  uint32_t bad0 = 0, bad1 = 0, bads = 0;              // tiles of the batch, and (2 bits each) stages, with groups without a page
  auto look_up = [&](int first) {
    batch = first;
    const int pos = (first + lane) * TILE;
    const bool in0 = first + lane < tend, in1 = in0 && pos + 16 < sp.kmax;
    const int i0 = pos >> p.c.page_shift, i1 = (pos + 16) >> p.c.page_shift;
    page0 = in0 ? row[i0] : -1;
    page1 = !in1 ? -1 : i1 == i0 ? page0 : row[i1];
    if ((uint32_t)page0 >= (uint32_t)p.c.num_pages) page0 = -1;
    if ((uint32_t)page1 >= (uint32_t)p.c.num_pages) page1 = -1;
    bad0 = __ballot_sync(0xFFFFFFFFu, in0 && page0 < 0);
    bad1 = __ballot_sync(0xFFFFFFFFu, in1 && page1 < 0);
    if ((bad0 | bad1) && lane == 0 && p.status) atomicExch(p.status, -1);    // FSA_ERR_INVALID_ARG
  };
  auto issue = [&](int tl) {
    const int s = r.in, at = tl - batch;
    r.in = s + 1 == STG ? 0 : s + 1;
    if (bad0 | bad1 | bads) bads = (bads & ~(3u << (2 * s))) | ((bad0 >> at & 1) | (bad1 >> at & 1) << 1) << (2 * s);
    if (lane == at) {
      const int inside = ((tl * TILE) & ((1 << p.c.page_shift) - 1)) / 16;
      const uint8_t* const src = head + page0 * p.c.page_bytes + inside * Gr::BYTES;
      uint8_t* const dst = r.mem + s * C::STAGE;
      mbar_expect_tx(&r.bar[s], (page0 >= 0 ? Gr::BYTES : 0) + (page1 >= 0 ? Gr::BYTES : 0));
      if (p.c.page_shift > 4 && page0 >= 0 && page1 == page0) {
        bulk_load(dst, src, 2 * Gr::BYTES, &r.bar[s]);
      } else {                                        // 16 tokens a page, or a single group left
        if (page0 >= 0) bulk_load(dst, src, Gr::BYTES, &r.bar[s]);
        if (page1 >= 0) bulk_load(dst + Gr::BYTES, head + page1 * p.c.page_bytes + (p.c.page_shift > 4 ? (inside + 1) * Gr::BYTES : 0), Gr::BYTES, &r.bar[s]);
      }
    }
  };
  if (t0 < tend) look_up(t0);
  int issued = t0;
  for (; issued < min(tend, t0 + STG); ++issued) issue(issued);

  // this piece's columns: q as f16 fragments, its factor, its last key
  uint2 q[D / 16][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(u[n][k].x << 16)), fabsf(__uint_as_float(u[n][k].x & 0xFFFF0000u))),
                             fmaxf(fabsf(__uint_as_float(u[n][k].y << 16)), fabsf(__uint_as_float(u[n][k].y & 0xFFFF0000u)))));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int e = (int)(__float_as_uint(top) >> 23) - 127;                 // floor(log2 top)
    const int up = e == 128 || top == 0.f ? 0 : min(max(4 - e, -126), 126);
    // (a row with an infinity becomes NaN as a whole, as its softmax is, even if all scores were
    // -inf: a sum of 0 then says that no key was seen)
    const float f = e == 128 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(up + 127) << 23) * p.q_sign;
    const float back = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      q[k][n].x = cvt_f16x2(__uint_as_float(u[n][k].x << 16) * f, __uint_as_float(u[n][k].x & 0xFFFF0000u) * f);
      q[k][n].y = cvt_f16x2(__uint_as_float(u[n][k].y << 16) * f, __uint_as_float(u[n][k].y & 0xFFFF0000u) * f);
    }
    // accumulator columns: 2t, 2t + 1
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      cq[n][c] = fmaxf(p.scale_log2 * __shfl_sync(0xFFFFFFFFu, back, 4 * (2 * t + c)), 1.4e-45f);   // (0 times -inf is NaN)
      lim[n][c] = limit_of(p, sp, c0 + 8 * n + 2 * t + c);
    }
  }
  a.reset(cq);
  const int min_lim = limit_of(p, sp, c0);            // the first column sees the fewest keys

  // the tiles that all columns see alike, and those behind some row (their rows' own tokens)
  const int alike = min_lim == sp.kmax ? tend : min(tend, min_lim / TILE);
  uint32_t bad = 0;
  const uint8_t* at = nullptr;
  auto arrived = [&] {
    const int s = r.out;
    if (!mbar_wait(&r.bar[s], (r.phase >> s) & 1, ac)) return false;
    r.phase ^= 1u << s;
    r.out = r.out + 1 == STG ? 0 : r.out + 1;
    bad = (bads >> (2 * s)) & 3;
    at = r.mem + s * C::STAGE;
    return true;
  };
  auto unseen = [&](int tl, TileScales<D, CF>& ts) {      // no part in the offset of V's scales
    if (tl * TILE + lane >= sp.kmax || (bad >> (lane >> 4) & 1)) {
#pragma unroll
      for (int x = 0; x < TileScales<D, CF>::BYTE_WORDS; ++x) ts.v[x] = 0;
    }
  };
  auto go_on = [&] {
    __syncwarp();
    if (issued < tend) {
      if (issued - batch == 32) look_up(issued);
      issue(issued++);
    }
  };
  int tl = t0;
  for (; tl < alike; ++tl) {
    ok = arrived();
    if (!ok) break;
    TileScales<D, CF> ts(at, r.scales);
    if (CF == CF_MX && a.shift == 8.f - R_CAP) ts.shift_v(r.scales + TILE * Gr::SB, R_CAP - a.r);
    __syncwarp();
    if (bad == 0 && (tl + 1) * TILE <= min_lim) {
      tile_step<D, CF, NT, 2, 0>(at, r.scales, ts.v, 0, q, cq, lim, tl * TILE, 0, a);
    } else {
      unseen(tl, ts);
#pragma unroll 1
      for (int gr = 0; gr < 2 && tl * TILE + 16 * gr < sp.kmax; ++gr)
        tile_step<D, CF, NT, 1, 1>(at, r.scales, ts.v, gr, q, cq, lim, tl * TILE, bad, a);
    }
    go_on();
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) a.rc[n][0] = a.rc[n][1] = a.r;
  for (; ok && tl < tend; ++tl) {
    ok = arrived();
    if (!ok) break;
    TileScales<D, CF> ts(at, r.scales);
    __syncwarp();
    unseen(tl, ts);
#pragma unroll 1
    for (int gr = 0; gr < 2 && tl * TILE + 16 * gr < sp.kmax; ++gr)
      tile_step<D, CF, NT, 1, 2>(at, r.scales, ts.v, gr, q, cq, lim, tl * TILE, bad, a);
    go_on();
  }
  if (!ok) {                                            // give up: the copies in flight end first
    for (int k = 0; k < STG; ++k) {
      const int s = r.out;
      if (r.out == r.in && k) break;
      mbar_drain(&r.bar[s], (r.phase >> s) & 1, ac);
      r.out = s + 1 == STG ? 0 : s + 1;
    }
    return false;
  }
  a.finish(cq);
  return true;
}

// The rows of a segment from one warp's state.
template <int D, int CF, int NT>
__device__ __forceinline__ void put_rows(const CacheAttnArgs& p, const Span& sp, int b, int hkv, int c0, const Acc<D, CF, NT>& a) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int col = c0 + 8 * n + 2 * t + e;
      if (col >= sp.qlen * p.G) continue;
      const Row row(p, b, hkv, col, sp, Sum{a.m[n][e], a.l[n][e], (float)a.rc[n][e], a.cq[n][e]});
#pragma unroll
      for (int k = 0; k < D / 16; ++k) row.put(p, 16 * k + 2 * g, make_float2(a.o[k][n][e], a.o[k][n][2 + e]));
      if (g == 0) row.put_lse(p);
    }
}

// One column of n <= 16 parts joined by half a warp: a lane weighs part `lane`, and has dims
// 4 (16x + lane) .. + 3 of the sum.  Both halves run it together, on columns of their own.
template <int D, int COLS>
struct Column {
  static constexpr int DP = D + 4;
  Sum s;
  float4 o[D / 64];
  template <class Part>
  __device__ __forceinline__ Column(Part part, int n, int col) {
    const int lane = threadIdx.x & 15;
    s = get_sum<D, COLS>(part(min(lane, n - 1)), col);
    if (lane >= n) s.l = 0.f;
    float m = s.l == 0.f ? -INFINITY : s.m, r = s.l == 0.f ? -INFINITY : s.r;
#pragma unroll
    for (int x = 1; x < 16; x *= 2) {
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
      r = fmaxf(r, __shfl_xor_sync(0xFFFFFFFFu, r, x));
    }
    const PartWeight w(s, m, r);
    s.m = m;
    s.r = r;
    s.l *= w.l;
#pragma unroll
    for (int x = 1; x < 16; x *= 2) s.l += __shfl_xor_sync(0xFFFFFFFFu, s.l, x);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float* const pk = part(k) + col * DP + 4 * lane;
      const float f = __shfl_sync(0xFFFFFFFFu, w.o, k, 16);
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(pk + 64 * x);
        o[x].x = fmaf(f, v.x, o[x].x);
        o[x].y = fmaf(f, v.y, o[x].y);
        o[x].z = fmaf(f, v.z, o[x].z);
        o[x].w = fmaf(f, v.w, o[x].w);
      }
    }
  }
  __device__ __forceinline__ void put_row(const CacheAttnArgs& p, const Span& sp, int b, int hkv, int col) const {
    const int lane = threadIdx.x & 15;
    const Row row(p, b, hkv, col, sp, s);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
      row.put(p, 64 * x + 4 * lane, make_float2(o[x].x, o[x].y));
      row.put(p, 64 * x + 4 * lane + 2, make_float2(o[x].z, o[x].w));
    }
    if (lane == 0) row.put_lse(p);
  }
  __device__ __forceinline__ void put_part(float* part, int col) const {
    const int lane = threadIdx.x & 15;
#pragma unroll
    for (int x = 0; x < D / 64; ++x) *reinterpret_cast<float4*>(part + col * DP + 64 * x + 4 * lane) = o[x];
    if (lane == 0) put_sum<D, COLS>(part, col, s);
  }
};

// Short segments: a CTA of 4 warps each, three CTAs an SM; no list, no second kernel.  Block x
// is segment x.
constexpr int WHOLE_WARPS = 4;
template <int D, int CF, int NT>
struct WholeCfg {
  using C = Cfg<D, CF, NT>;
  static constexpr int RING = WHOLE_WARPS * C::STG * C::STAGE, JOIN = WHOLE_WARPS * C::PART * 4;
  static constexpr int SMEM = 1024 + WHOLE_WARPS * C::SCALES + (RING > JOIN ? RING : JOIN);
  static constexpr int CTAS = NT == 2 && D == 128 ? 2 : 3;
};
template <int D, int CF, int NT>
__global__ void __launch_bounds__(WHOLE_WARPS * 32, WholeCfg<D, CF, NT>::CTAS) cache_attn_whole_kernel(const CacheAttnArgs p) {
  using C = Cfg<D, CF, NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int STG = C::STG;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem);
  int* const flag = reinterpret_cast<int*>(smem + 512);
  uint32_t* const scales = reinterpret_cast<uint32_t*>(smem + 1024);
  uint8_t* const ring = smem + 1024 + WHOLE_WARPS * C::SCALES;
  const int warp = threadIdx.x >> 5;
  const AbortCtl ac{flag, p.status, p.timeout_ns};
  griddep_launch();
  if (threadIdx.x == 0) *flag = 0;
  if (threadIdx.x < WHOLE_WARPS * STG) mbar_init(&bars[threadIdx.x], 1);
  fence_mbar_init();
  griddep_wait();                                       // before any tensor is read
  const int vb = blockIdx.x / p.c.Hkv, hkv = blockIdx.x - vb * p.c.Hkv;
  const int b = p.CT == 1 ? vb : vb / p.CT, c0 = (vb - b * p.CT) * C::COLS;
  const Span sp = span_of(p, vb, C::COLS);
  if (sp.tiles == 0) return;
  __syncthreads();
  Ring r{bars + warp * STG, ring + warp * STG * C::STAGE, scales + warp * C::SCALES / 4, 0, 0, 0};
  Acc<D, CF, NT> a;
  const int n = min(WHOLE_WARPS, sp.tiles), t0 = sp.tiles * warp / n, t1 = sp.tiles * (warp + 1) / n;
  bool ok = true;
  if (warp < n) ok = run_piece<D, CF, NT>(p, sp, b, hkv, c0, t0, t1, r, ac, a);
  if (n == 1) {
    if (warp == 0 && ok) put_rows<D, CF, NT>(p, sp, b, hkv, c0, a);
    return;
  }
  __syncthreads();                                      // every ring is done with
  float* const parts = reinterpret_cast<float*>(ring);
  if (warp < n && ok) put_part<D, CF, NT>(parts + warp * C::PART, a);
  __syncthreads();
  if (lds_vol(flag)) return;                            // a wait ran out: the status word says so
  const int cols = min(C::COLS, sp.qlen * p.G - c0), half = (threadIdx.x >> 4) & 1;
  for (int first = 2 * warp; first < cols; first += 2 * WHOLE_WARPS) {
    const Column<D, C::COLS> sum([&](int k) { return parts + k * C::PART; }, n, first + half);
    if (first + half < cols) sum.put_row(p, sp, b, hkv, c0 + first + half);
  }
}

template <int D, int CF, int NT>
__global__ void __launch_bounds__(cta_warps<D, NT>() * 32, 1) cache_attn_kernel(const CacheAttnArgs p) {
  using C = Cfg<D, CF, NT>;
  constexpr int NWC = C::NWC, STG = C::STG;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);                  // [NWC][STG]
  int* flag = reinterpret_cast<int*>(smem + 512);                      // abort
  int* wsum = reinterpret_cast<int*>(smem + 576);              // [NWC]
  int2* ends = reinterpret_cast<int2*>(smem + 520);                    // x: the first open piece begins, y: tiles behind the last
  int4* pieces = reinterpret_cast<int4*>(smem + 704);                  // [NWC] segments of the leading and the open piece; its qlen, len
  int* pre = reinterpret_cast<int*>(smem + 1024);              // [NWC * 32]
  uint32_t* scales = reinterpret_cast<uint32_t*>(smem + 1024 + NWC * 32 * 8);
  float* leads = reinterpret_cast<float*>(smem + 1024 + NWC * 32 * 8 + NWC * C::SCALES);  // [NWC] parts
  uint8_t* ring = smem + 1024 + NWC * 32 * 8 + NWC * C::SCALES + C::JOIN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AbortCtl ac{flag, p.status, p.timeout_ns};

  griddep_launch();
  if (threadIdx.x == 0) *flag = 0;
  if (threadIdx.x < NWC * STG) mbar_init(&bars[threadIdx.x], 1);
  fence_mbar_init();
  griddep_wait();                                       // before any tensor is read

  // the list's length and its prefix sums.  Up to 4 virtual sequences a lane, every warp does
  // it by itself (no barrier, and the loads of a lane go out together); beyond, the CTA
  // shares the work, a chunk a thread.
  const int VB = p.B * p.CT;
  const bool small = VB <= 128;
  const int chunk = small ? (VB + 31) / 32 : (VB + NWC * 32 - 1) / (NWC * 32);
  const int who = small ? lane : threadIdx.x;
  int mine = 0, before = 0, total = 0;
  if (small) {
    int n[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) n[x] = x < chunk && who * chunk + x < VB ? span_of(p, who * chunk + x, C::COLS).units() : 0;
    mine = (n[0] + n[1] + n[2] + n[3]) * p.c.Hkv;
  } else {
    for (int vb = who * chunk; vb < min(VB, (who + 1) * chunk); ++vb)
      mine += span_of(p, vb, C::COLS).units() * p.c.Hkv;
  }
  int inc = mine;
#pragma unroll
  for (int x = 1; x < 32; x *= 2) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, inc, x);
    if (lane >= x) inc += up;
  }
  if (small) {
    total = __shfl_sync(0xFFFFFFFFu, inc, 31);
  } else {
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NWC; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    pre[threadIdx.x] = before + inc - mine;
  }
  __syncthreads();

  // shares: as few warps of each CTA as give every one of them a tile, so small calls
  // spread over the SMs and no share between two others is empty
  const int wpc = total >= (int)gridDim.x * NWC ? NWC : max(1, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  const int NW = min(total, (int)gridDim.x * wpc);
  const Shares sh(total, NW);
  const int W = blockIdx.x * wpc + warp;
  const bool works = warp < wpc && W < NW;
  float* const entering = p.partials + (int64_t)(2 * blockIdx.x) * C::PART;   // the CTA's part of a segment begun before it
  int lo = works ? sh.first(W) : 0;
  const int hi = works ? sh.first(W + 1) : 0;
  // A warp's leading piece is the end of a segment that began before it, its open piece
  // the one that the loop leaves in `a`, of a segment that others share; -1: none.
  int seg_lead = -1, seg_open = -1;
  bool open_begins = false;                            // the open piece is its segment's first
  int open_rest = 0;                                   // tiles of its segment behind it
  Acc<D, CF, NT> a;
  Span sp;
  int vb = 0, hkv = 0, unit = 0;
  Ring r{bars + warp * STG, ring + warp * STG * C::STAGE, scales + warp * C::SCALES / 4, 0, 0, 0};

  if (lo < hi) {
    int j = 0;                                         // the last chunk that begins at or before lo
    int acc;
    if (small) {
      j = 31 - __clz(__ballot_sync(0xFFFFFFFFu, inc - mine <= lo));
      acc = __shfl_sync(0xFFFFFFFFu, inc - mine, j);
    } else {
      for (int x = 256; x; x >>= 1)
        if (j + x < NWC * 32 && pre[j + x] <= lo) j += x;
      acc = pre[j];
    }
    for (vb = j * chunk;; ++vb) {
      sp = span_of(p, vb, C::COLS);
      const int n = sp.units() * p.c.Hkv;
      if (lo < acc + n) break;
      acc += n;
    }
    hkv = (int)((uint32_t)(lo - acc) / (uint32_t)sp.units());
    unit = lo - acc - hkv * sp.units();
  }

  bool ok = true;
  while (lo < hi && ok) {
    const int b = p.CT == 1 ? vb : vb / p.CT, c0 = (vb - b * p.CT) * C::COLS;
    const int unit1 = min(sp.units(), unit + (hi - lo));
    const int t0 = max(0, unit - EXTRA), t1 = max(0, unit1 - EXTRA);
    const int seg = vb * p.c.Hkv + hkv;
    lo += unit1 - unit;
    unit = 0;
    auto next = [&] {                                   // the segment after this one
      if (lo < hi && ++hkv == p.c.Hkv) {
        hkv = 0;
        do { sp = span_of(p, ++vb, C::COLS); } while (sp.tiles == 0);
      }
    };
    if (t0 == t1) { next(); continue; }                 // none of its tiles

    ok = run_piece<D, CF, NT>(p, sp, b, hkv, c0, t0, t1, r, ac, a);
    if (!ok) break;
    if (t0 == 0 && t1 == sp.tiles) {                    // all of it: write the rows
      put_rows<D, CF, NT>(p, sp, b, hkv, c0, a);
    } else if (lo < hi) {                               // the end of a segment that began before this warp
      seg_lead = seg;
      put_part<D, CF, NT>(warp == 0 ? entering : leads + warp * C::PART, a);
    } else {
      seg_open = seg;
      open_begins = t0 == 0;
      open_rest = sp.tiles - t1;
    }
    next();
  }

  // Join the pieces of each segment that the CTA's warps share, a column half a warp.  A segment
  // that began and ends in this CTA is written; one that came from the CTA before, or goes
  // on to the next, is a part for the second kernel.
  __syncthreads();                                      // every ring is done with
  float* parts = reinterpret_cast<float*>(ring);
  const int active = max(1, min(wpc, NW - (int)blockIdx.x * wpc));     // warps of this CTA that have a share
  if (!ok) seg_lead = seg_open = -1;
  if (lane == 0) {
    pieces[warp] = make_int4(seg_lead, seg_open, sp.qlen, sp.len);
    if (warp == 0) ends->x = open_begins;
    if (warp == active - 1) ends->y = open_rest;
  }
  if (seg_open >= 0) put_part<D, CF, NT>(parts + warp * C::PART, a);
  __syncthreads();
  int4 start = make_int4(-1, 0, 0, 0);
  for (int w0 = 0, w1, turn = 0; w0 < active; w0 = w1) {
    const int4 pc = pieces[w0];
    w1 = w0 + 1;
    if (pc.y < 0) continue;
    while (w1 < active && pieces[w1].y == pc.y) ++w1;
    const bool lead = w1 < active && pieces[w1].x == pc.y;
    const int n = w1 - w0 + (lead ? 1 : 0);
    // whether it began in this CTA is known to its first warp, where it ends to its last
    const bool begins = w0 > 0 || ends->x != 0;
    const int rest = lead || w1 < active ? 0 : ends->y;
    if (begins && rest > 0) start = make_int4(pc.y, sh.of(sh.first(blockIdx.x * wpc + w1) + rest - 1) / wpc, pc.z, pc.w);
    const int vs = pc.y / p.c.Hkv, hs = pc.y - vs * p.c.Hkv;
    const int b = p.CT == 1 ? vs : vs / p.CT, c0 = (vs - b * p.CT) * C::COLS;
    const Span sg{pc.z, pc.w, 0, 0};
    const int cols = min(C::COLS, sg.qlen * p.G - c0), half = lane >> 4;
    int first = warp - turn;                            // pairs of columns of all segments in turn
    if (first < 0) first += NWC;
    turn = (turn + (cols + 1) / 2) % NWC;
    for (first *= 2; first < cols; first += 2 * NWC) {
      const int col = first + half;                     // (COLS is even: column `cols` lies in the parts)
      const Column<D, C::COLS> sum([&](int k) { return w0 + k < w1 ? parts + (w0 + k) * C::PART : leads + w1 * C::PART; }, n, col);
      if (col >= cols) continue;
      if (begins && rest == 0) sum.put_row(p, sg, b, hs, c0 + col);
      else sum.put_part(begins ? p.partials + (int64_t)(2 * blockIdx.x + 1) * C::PART : entering, col);
    }
  }
  if (threadIdx.x == 0) p.starts[blockIdx.x] = start;
}

// Joins the parts of the segments that several CTAs share.  Block (c, y) takes the one that
// begins in CTA c and goes on, columns of the y-th quarter: CTA c's second part and the
// first part of each later CTA up to the last.
constexpr int JOIN_THREADS = 128, JOIN_Y = 4, JOIN_AHEAD = 16;
template <int D, int NT>
__global__ void __launch_bounds__(JOIN_THREADS) cache_join_kernel(const CacheAttnArgs p) {
  constexpr int COLS = 8 * NT, DP = D + 4, PART = COLS * (D + 6), CY = COLS / JOIN_Y, PER = CY * D / 2 / JOIN_THREADS + (CY * D / 2 < JOIN_THREADS);
  extern __shared__ Sum part_sums[];                     // [parts][CY]; l is then the weight of a part's rows
  __shared__ Sum sums[CY];
  griddep_launch();
  griddep_wait();                                        // the first kernel's results are complete
  const int4 st = p.starts[blockIdx.x];                  // segment, last CTA, its rows, its keys
  if (st.x < 0) return;
  const int lane = threadIdx.x & 31;
  const int vb = st.x / p.c.Hkv, hkv = st.x - vb * p.c.Hkv;
  const int b = p.CT == 1 ? vb : vb / p.CT, first = blockIdx.y * CY, c0 = (vb - b * p.CT) * COLS + first;
  const int n = st.y - (int)blockIdx.x + 1;
  const Span sp{st.z, st.w, 0, 0};
  if (c0 >= sp.qlen * p.G) return;
  const float* const parts = p.partials + (int64_t)2 * blockIdx.x * PART;
  auto part = [&](int k) { return parts + (k == 0 ? (int64_t)PART : (int64_t)2 * k * PART); };
  // the first parts' rows set out together with all maxima and sums
  float2 v[PER][JOIN_AHEAD];
#pragma unroll
  for (int y = 0; y < PER; ++y) {
    const int x = threadIdx.x + y * JOIN_THREADS, c = x / (D / 2), d = 2 * (x % (D / 2));
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k)
      if (k < n && c < CY) v[y][k] = *reinterpret_cast<const float2*>(part(k) + (first + c) * DP + d);
  }
  for (int x = threadIdx.x; x < n * CY; x += JOIN_THREADS) part_sums[x] = get_sum<D, COLS>(part(x / CY), first + x % CY);
  __syncthreads();
  if (threadIdx.x < CY * 32) {                           // a warp a column
    const int c = threadIdx.x / 32;
    float m = -INFINITY, r = -INFINITY, l = 0.f;
    for (int k = lane; k < n; k += 32) {
      const Sum s = part_sums[k * CY + c];
      m = fmaxf(m, s.l == 0.f ? -INFINITY : s.m);
      r = fmaxf(r, s.l == 0.f ? -INFINITY : s.r);
    }
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
      r = fmaxf(r, __shfl_xor_sync(0xFFFFFFFFu, r, x));
    }
    for (int k = lane; k < n; k += 32) {
      const Sum s = part_sums[k * CY + c];
      const PartWeight f(s, m, r);
      part_sums[k * CY + c].l = f.o;
      l = fmaf(f.l, s.l, l);
    }
#pragma unroll
    for (int x = 1; x < 32; x *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    if (lane == 0) sums[c] = Sum{m, l, r, part_sums[c].cq};
  }
  __syncthreads();
#pragma unroll
  for (int y = 0; y < PER; ++y) {
    const int x = threadIdx.x + y * JOIN_THREADS, c = x / (D / 2), d = 2 * (x % (D / 2));
    if (c >= CY || c0 + c >= sp.qlen * p.G) continue;
    float2 o = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k)
      if (k < n) {
        const float f = part_sums[k * CY + c].l;
        o.x = fmaf(f, v[y][k].x, o.x);
        o.y = fmaf(f, v[y][k].y, o.y);
      }
#pragma unroll 8
    for (int k = JOIN_AHEAD; k < n; ++k) {
      const float f = part_sums[k * CY + c].l;
      const float2 u = *reinterpret_cast<const float2*>(part(k) + (first + c) * DP + d);
      o.x = fmaf(f, u.x, o.x);
      o.y = fmaf(f, u.y, o.y);
    }
    const Row row(p, b, hkv, c0 + c, sp, sums[c]);
    row.put(p, d, o);
    if (d == 0) row.put_lse(p);
  }
}

// Which kernel: a CTA for each segment where none is longer than 28 tiles and there are at most
// 8 an SM, else the list split evenly.  (The table's width bounds a segment's tiles; the
// lengths are on the device.)  Measured, list / whole, us, 8 kv heads of 128 dims, E2M1:
//   1 sequence of 100, 760, 890, 1020, 1500 keys: 8.9 / 4.2, 9.3 / 8.7, 9.5 / 9.5, 9.7 / 10.3, 9.9 / 13.5
//   64 sequences of 100, 890, 1500 keys: 13.2 / 8.8, 25.0 / 23.0, 32.9 / 32.4
//   152 sequences (8 segments an SM) of 100, 890, 1 to 890: 17.6 / 14.1, 43.7 / 40.3, 20.0 / 20.5
//   256 sequences of 100, 1 to 100, 1 to 890: 21.0 / 21.8, 18.1 / 19.2, 27.1 / 32.1
// and 2 kv heads of 64 dims, 7 query heads each, 2 rows, NVFP4:
//   1 sequence of 100, 760, 890, 1020, 1500 keys: 8.6 / 4.9, 9.3 / 9.2, 10.6 / 10.0, 10.0 / 10.8, 12.8 / 14.0
//   64 sequences of 100, 890, 1500 keys: 11.4 / 6.3, 15.0 / 13.0, 16.4 / 18.4
//   152 sequences of 100, 890, 1 to 890: 14.5 / 6.9, 20.2 / 14.6, 14.1 / 12.0
// The rule goes by what the host knows: one short sequence in a wide table takes the list.
bool whole_segments(const Cache& c, int B, int CT, int max_pages, int sms) {
  const int64_t tiles = (((int64_t)max_pages << c.page_shift) + TILE - 1) / TILE;
  return tiles <= 28 && (int64_t)B * CT * c.Hkv <= 8 * (int64_t)sms;
}

// Opt in to the kernel's shared memory, once a device.
template <class K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& devices) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (devices.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) devices.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int D, int CF, int NT>
cudaError_t launch(const CacheAttnArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<D, CF, NT>;
  cudaError_t e;
  static std::atomic<uint64_t> whole_ready{0}, list_ready{0};
  if (whole_segments(a.c, a.B, a.CT, a.max_pages, sms)) {
    constexpr int smem = WholeCfg<D, CF, NT>::SMEM;
    e = allow_smem(cache_attn_whole_kernel<D, CF, NT>, smem, whole_ready);
    if (e != cudaSuccess) return e;
    return launch_early(cache_attn_whole_kernel<D, CF, NT>, dim3(a.B * a.CT * a.c.Hkv), WHOLE_WARPS * 32, smem, st, a);
  }
  e = allow_smem(cache_attn_kernel<D, CF, NT>, C::SMEM, list_ready);
  if (e != cudaSuccess) return e;
  e = launch_early(cache_attn_kernel<D, CF, NT>, dim3(sms), C::NWC * 32, C::SMEM, st, a);
  if (e != cudaSuccess) return e;
  return launch_early(cache_join_kernel<D, NT>, dim3(sms, JOIN_Y), JOIN_THREADS,
                      (size_t)(sms + 2) * (C::COLS / JOIN_Y) * sizeof(Sum), st, a);
}

}  // namespace

int cache_attn_ntiles(int cols) { return cols <= 8 ? 1 : 2; }

// parts of the CTAs, two each; where segments begin that go on
size_t cache_attn_workspace(const Cache& c, int B, int H, int Sq, int max_pages, int sms, size_t* starts_at) {
  const int cols = Sq * (H / c.Hkv), nt = cache_attn_ntiles(cols);
  *starts_at = (size_t)2 * sms * 8 * nt * (c.D + 6) * sizeof(float);
  if (whole_segments(c, B, (cols + 8 * nt - 1) / (8 * nt), max_pages, sms)) return 0;
  return *starts_at + (size_t)sms * sizeof(int4);
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
