// fsa_cache_chunk.cu -- attention of a chunk of new tokens over the paged 4-bit cache.
//
//   o = softmax(scale q K^T) V  over the keys a row sees, K and V the values the cache
//   stands for (codes times block scales), q as given, sums in fp32.
//
// A kv head's query rows (its G heads' rows of each token, in order) go 256 at a time, two tiles
// of 128, over the key tiles of 128 that some of them see:
//   - bound by the products, 4 D flops a seen pair: tcgen05 kind::f16 MMAs.  The block-scaled
//     kinds cannot take V's scales, which run across its product's summation, nor q unrounded.  So
//     four warps turn a tile's codes into 16-bit operands in shared memory, once for 256 rows.
//   - A cache row's bytes are in the order of other fragments (fsa_cache.h); here a word becomes
//     a 16-byte piece of its row, so the operands' columns are permuted: those of K alike in q, which is
//     permuted as it is loaded, those of V in the output's columns, which are put in order as they are
//     stored.  K is K-major; V needs no transposition, as the second operand of a product over the keys it
//     is MN-major.
//   - All operands are f16.  A code is one conversion, its scale one product: exact for E4M3 scales, and for E8M0
//     scales of 2^-23 .. 2^13.  Those have fp32's range: a key with others is divided by a power of two that makes its
//     largest scale 2^13, and its scores are multiplied by that (its blocks below 2^-36 of its largest lose bits); 32 keys
//     with others in V have V, and P with it, as bf16.  q has a power of two a row (exact down to 2^-18 of its row's
//     maximum, off by at most 2^-29 of it below).
//   - S, then P over it, and O stay in tensor memory: 128 columns each for both row tiles.  While
//     the softmax of one row tile runs, the other's products do.  P is rounded to f16 (2^-11 of each
//     weight, 2^-32 absolute; where V is bf16 to that, 2^-8); sums and maxima are fp32.  The running maximum
//     is raised only when a score beats it by more than 2^8 in the softmax.
//   - The work, (sequence, row block, kv head, key tile), is one list split evenly over one CTA per
//     SM (a segment's start weighing as EXTRA tiles); parts of a segment that several CTAs share are
//     joined by a second kernel.  Lengths are read on the device.
//   - A row that sees a token whose values are not finite (the scale's NaN) is NaN as a whole; the others
//     are as without it (its V is zero in the operand, and a bit tells the rows).
//
// Measured (one GB300, cuBLAS at 1943 TFLOP/s in bf16): 2048 tokens over 128K keys, 32/8 heads of 128: NVFP4 1570
// TFLOP/s (2.73 to 2.82 ms), E2M1 1380 (3.16); heads of 64: 921 (2.37) and 711 (3.07).  Eight sequences of 8192 keys,
// 64 tokens each, NVFP4: 73 us, where fsa_attention_cache takes 322.  Values of which one block of 32 is zeros take no longer.
// What bounds it: of the about 3100 cycles of a tile of 128 dims (NVFP4) its products take 2050 at the nominal rate; a row
// tile's chain, its scores, their maximum (800 cycles), exponentials (1050), products, is as long, and the two row tiles'
// chains cover each other but for their ends.  The operand warps work 2100 of these cycles.  E2M1 is slower by what tells
// the rare scales and by their ways, which cost the softmax registers and fetches (exponentials 1400, K 1650).  With 64
// dims the products are half as long and the rest is not.  Instructions are fetched too slowly for all of the code to be
// straight (0.4 to 0.9 of the 7 to 11 cycles between a warp's instructions wait for them): what runs once a piece is in
// loops.  A piece costs about 12000 cycles beside its tiles: q (2500 to 8000, by where it lies), the first scores, the last
// products, the rows' way out (4000).
#include <algorithm>
#include <atomic>
#include "fsa_cache.h"
#include "fsa_mx.cuh"

namespace fsa {
namespace {

constexpr int ROWS = 256;             // of a block: two tiles of 128
constexpr int KEYS = 128;             // of a tile
// What a segment's start costs a CTA, in tiles.  us with 1, 2, 3, 4, 5, 6, 8 of them: eight turns over 600 to 8192 keys 142, 135,
// 129, 127, 123, 124, 123; 300 and 500 tokens over 40000 and 9000 keys 215, 211, 211, 209, 205, 207, 209; 40 short ones over 520 to 900
// 105, 98, 94, 96, 95, 95, 93; 64 tokens each over 24 of 1000 to 4000 (E2M1) 106, 103, 102, 98, 96, 98, 98; eight windows of 2048 130,
// 126, 128, 125, 124, 124, 124.  (5 would do a little better than 3, but 3 is in the stated limit of the list's length.)
constexpr int EXTRA = 3;
constexpr int THREADS = 512;          // warps 0..7 softmax (a row a thread), 8..11 operands, 12 copies, 13 MMA
constexpr int RAW = 3;                // stages of 64 keys of codes
constexpr float LAZY = 8.0f;          // log2 of how far a score may beat the running maximum
constexpr float UP = 7.0f;            // weights carry 2^7: at most 2^15, in f16
constexpr float NONE = -INFINITY;

template <int D, int CF>
struct Cfg {
  using Gr = CacheGroup<D, CF>;
  static constexpr int NKA = D / 64;                     // 128-byte atoms of a row
  static constexpr int ATOM = KEYS * 128;                // bytes of 128 rows of one
  static constexpr int TILE = NKA * ATOM;                // bytes of an operand tile (Q, K or V)
  static constexpr int STAGE = 4 * Gr::BYTES;            // 64 keys
  static constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = 4 * TILE, OFF_RAW = 6 * TILE;
  static constexpr int OFF_BAR = (OFF_RAW + RAW * STAGE + 63) / 64 * 64;
  static constexpr int OFF_FLAGS = OFF_BAR + 256;        // [4 tiles] of absent keys, keys with a NaN in V, V as bf16, keys with a shift: a word a warp
  static constexpr int OFF_MISC = OFF_FLAGS + 4 * 64;    // absent groups of the raw stages, tmem base, abort flag, warp sums
  static constexpr int OFF_WALK = OFF_MISC + 128;        // where each warp is in the list
  static constexpr int OFF_PRE = OFF_WALK + 16 * 80;     // [THREADS] prefix sums of the list
  static constexpr int OFF_SHIFT = OFF_PRE + THREADS * 4;                    // E8M0: [4 tiles][KEYS] powers of two out of K
  static constexpr int SMEM = OFF_SHIFT + (CF == CF_MX ? 4 * KEYS * 2 : 0) + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // tensor memory: + 128 (S), + D (O), + P_STEP (P) for the second row tile.  With D 64 P has columns of its own, and the next
  // tile's scores are computed while this one's softmax runs (NVFP4 882 TFLOP/s instead of 818, E2M1 714 instead of 706);
  // with D 128 it lies over the scores, for want of columns.
  static constexpr bool APART = D == 64;
  static constexpr uint32_t T_S = 0, T_O = 256, T_P = APART ? 384 : 0, P_STEP = APART ? 64 : 128;
  static constexpr int PART = ROWS * (D + 2);            // floats of a partial result: rows, maxima, sums
};

// ---------------------------------------------------------------------- the work list
struct Span {
  int qlen, len, kmax;      // rows' tokens, keys, keys that some row of the block sees
  int rows;                 // of the block
  int low;                  // the first key of the first row's window
  int lead, w0, tiles;      // tiles of the first keys, first tile of some window, tiles in all
};
// virtual sequence vb = b * p.CT + block of rows
__device__ __forceinline__ Span span_of(const CacheAttnArgs& p, int vb) {
  Span s;
  const int b = vb / p.CT, r0 = (vb - b * p.CT) * ROWS;
  s.qlen = p.q_lens ? min(max(p.q_lens[b], 0), p.Sq) : p.Sq;
  s.len = (int)min((int64_t)max(p.lens[b], 0), (int64_t)p.max_pages << p.c.page_shift);
  s.rows = min(ROWS, s.qlen * p.G - r0);
  s.kmax = s.low = s.lead = s.w0 = s.tiles = 0;
  if (s.rows <= 0) return s;
  s.kmax = p.causal ? max(0, s.len - s.qlen + (r0 + s.rows - 1) / p.G + 1) : s.len;
  const int end = (s.kmax + KEYS - 1) / KEYS;
  if (p.window) {
    s.low = max(0, s.len - s.qlen + r0 / p.G + 1 - p.window);
    s.w0 = min(s.low / KEYS, end);
    s.lead = min((p.sinks + KEYS - 1) / KEYS, s.w0);
  }
  s.tiles = s.lead + end - s.w0;
  return s;
}
// what it weighs (a block that sees nothing is written too)
__device__ __forceinline__ int units_of(const CacheAttnArgs& p, const Span& s) {
  return s.rows <= 0 ? 0 : p.whole ? 1 : max(s.tiles, 1) + EXTRA;
}
// `total` units over n CTAs: the first `more` of them take base + 1, the others base.
struct Shares {
  int base, more;
  __device__ __forceinline__ Shares(int total, int n) {
    base = n > 0 ? total / n : 0;
    more = total - base * n;
  }
  __device__ __forceinline__ int first(int w) const { return base * w + min(w, more); }
  __device__ __forceinline__ int of(int unit) const {
    const int cut = (base + 1) * more;
    return unit < cut ? unit / (base + 1) : more + (unit - cut) / base;
  }
};
// A CTA's walk through its share: piece after piece, the same for all of its warps.
struct Walk {
  int lo, hi, vb, hkv, unit;
  Span sp;
  int t0, t1, rest;         // the piece: tiles t0 .. t1 - 1 of its segment, and the units behind it
  __device__ __forceinline__ void start(const CacheAttnArgs& p, const int* pre, int chunk, int lo_, int hi_) {
    lo = lo_;
    hi = hi_;
    vb = hkv = unit = t0 = t1 = rest = 0;
    sp = Span{};
    if (lo >= hi) return;
    int j = 0;                                           // the last chunk that begins at or before lo
    for (int x = THREADS / 2; x; x >>= 1)
      if (j + x < THREADS && pre[j + x] <= lo) j += x;
    int acc = pre[j], n;
    for (vb = j * chunk;; ++vb) {
      sp = span_of(p, vb);
      n = units_of(p, sp);
      if (lo < acc + n * p.c.Hkv) break;
      acc += n * p.c.Hkv;
    }
    hkv = (lo - acc) / n;
    unit = lo - acc - hkv * n;
  }
  // false: the share is done
  __device__ __forceinline__ bool next(const CacheAttnArgs& p) {
    while (lo < hi) {
      int n = units_of(p, sp);
      if (unit == n) {                                   // on to the next segment
        unit = 0;
        if (++hkv == p.c.Hkv) {
          hkv = 0;
          do { sp = span_of(p, ++vb); } while (sp.rows <= 0);
          n = units_of(p, sp);
        }
      }
      const int u1 = min(n, unit + hi - lo);
      if (p.whole) { t0 = 0; t1 = sp.tiles; }
      else { t0 = max(0, unit - EXTRA); t1 = min(sp.tiles, max(0, u1 - EXTRA)); }
      const bool empty = sp.tiles == 0 && u1 == n;       // a block that sees nothing: whoever has its end writes it
      lo += u1 - unit;
      unit = u1;
      rest = n - u1;
      if (t1 > t0 || empty) return true;
    }
    return false;
  }
};
static_assert(sizeof(Walk) <= 80, "");
// A warp's next piece.  The walk itself waits in shared memory, out of the registers.
struct Piece {
  int vb, hkv, t0, t1, low, lead, w0, rows, kmax, qlen, len, last;     // last: the CTA that has the segment's end
  bool begins, ends;
  __device__ __forceinline__ int at(int t) const { return t < lead ? t : t - lead + w0; }
};
__device__ __forceinline__ bool next_piece(const CacheAttnArgs& p, Walk* slot, const Shares& sh, Piece& c) {
  __syncwarp();
  Walk w = *slot;
  if (!w.next(p)) return false;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) *slot = w;
  c = {w.vb, w.hkv, w.t0, w.t1, w.sp.low, w.sp.lead, w.sp.w0, w.sp.rows, w.sp.kmax, w.sp.qlen, w.sp.len, p.whole ? 0 : sh.of(w.lo + w.rest - 1), w.t0 == 0, w.t1 == w.sp.tiles};
  return true;
}

// ---------------------------------------------------------------- operands from codes
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t byte_of(const uint32_t (&w)[2], int i) { return (w[i / 4] >> (8 * (i % 4))) & 0xFFu; }
// E8M0 scales as factors of f16, twice in a word: exact from 2^-23 to 2^13, whose products with a code are too
constexpr uint32_t LEAST_F16 = 127 - 23, MOST_F16 = 127 + 13;
__device__ __forceinline__ uint32_t e8m0_f16(uint32_t byte) {
  return (byte > 112u ? (byte - 112u) << 10 : 1u << (byte - 103u)) * 0x10001u;
}
// K's, `shift` powers of two less; the least are zeros then, and NaN stays
__device__ __forceinline__ uint32_t e8m0_f16_shifted(uint32_t byte, int shift) {
  const int b = (int)byte - shift;
  return byte == 0xFFu ? 0x7E007E00u : b < 103 ? 0u : e8m0_f16((uint32_t)b);
}
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t byte) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(byte * 0x101u));
  return r;
}

// 16-byte piece of an operand's row: in atoms of 64 columns, swizzled
__device__ __forceinline__ void put_piece(uint8_t* row_at, int row, int piece, const uint32_t (&o)[4]) {
  *reinterpret_cast<uint4*>(row_at + (piece >> 3) * (KEYS * 128) + (((piece & 7) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
}

// A row's 16-byte pieces.  Neighbouring lanes take them in turn, so that neither these loads nor the stores of a
// quarter of the warp share banks (D 64: the loads do, two and two).
template <int D>
__device__ __forceinline__ int piece_of(int row, int c) { return D == 128 ? (c + (row >> 1)) & 3 : c; }
template <int D>
struct Row {
  uint4 u[D / 32];
  __device__ __forceinline__ void load(int row, const uint8_t* src) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) u[c] = *reinterpret_cast<const uint4*>(src + 16 * piece_of<D>(row, c));
  }
};
// How a row's words become a row of an operand: f(word, its place among the four of 16 bytes, o).
template <int D, class F>
__device__ __forceinline__ void put_row(uint8_t* dst, int row, const Row<D>& r, F f) {
  uint8_t* const at = dst + row * 128;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const uint32_t w[4] = {r.u[c].x, r.u[c].y, r.u[c].z, r.u[c].w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t o[4];
      f(w[x], x, o);
      put_piece(at, row, 4 * piece_of<D>(row, c) + x, o);
    }
  }
}
// A row of K.  Word 4t + w (D 64: 2t + w) holds elements 32w + 4t + 0..3 and 16 on, whose scales are those of
// block w (E8M0) or 2w and 2w + 1 (E4M3).  gone: its codes are not there.  shift: of E8M0 scales, see above.
template <int D, int CF>
__device__ __forceinline__ void put_key(uint8_t* dst, int row, const Row<D>& src, const uint32_t (&sb)[2], bool gone, int shift) {
  if constexpr (CF == CF_MX) {
    uint32_t f[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) f[i] = gone ? 0u : e8m0_f16_shifted(byte_of(sb, i), shift);
    put_row<D>(dst, row, src, [&](uint32_t w, int x, uint32_t (&o)[4]) {
      cvt_e2m1x8_f16(w, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = hmul2(o[e], f[x % (D / 32)]);
    });
  } else {
    uint32_t f[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) f[i] = gone ? 0u : e4m3_f16(byte_of(sb, i));
    put_row<D>(dst, row, src, [&](uint32_t w, int x, uint32_t (&o)[4]) {
      cvt_e2m1x8_f16(w, o);
      const int b = x % (D / 32);
      o[0] = hmul2(o[0], f[2 * b]);
      o[1] = hmul2(o[1], f[2 * b]);
      o[2] = hmul2(o[2], f[2 * b + 1]);
      o[3] = hmul2(o[3], f[2 * b + 1]);
    });
  }
}
// A word times a scale in fp32, as bf16 (the rare ways: small, and out of the way of the others' registers)
__device__ __forceinline__ uint32_t scaled_bf16(uint32_t f16x2, float f) {
  float lo, hi;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}" : "=f"(lo), "=f"(hi) : "r"(f16x2));
  return cvt_bf16x2(lo * f, hi * f);
}
// A row of V.  Word 2g + y (D 64: g) holds elements 64y + 2g, + 1, and 16, 32 and 48 on.  A scale that is NaN
// counts as zero, and so does the least E8M0 one, a block of zeros' (2^-127: of values below 2^-124).
template <int D, int CF>
__device__ __forceinline__ void put_value(uint8_t* dst, int row, const Row<D>& src, const uint32_t (&sb)[2], bool gone) {
  constexpr int SB = CacheGroup<D, CF>::SB;
  uint32_t f[SB];
#pragma unroll
  for (int i = 0; i < SB; ++i) {
    const uint32_t byte = byte_of(sb, i);
    const bool none = gone || (CF == CF_MX ? byte - 1u >= 254u : (byte & 0x7Fu) == 0x7Fu);
    f[i] = none ? 0u : CF == CF_MX ? e8m0_f16(byte) : e4m3_f16(byte);
  }
  put_row<D>(dst, row, src, [&](uint32_t w, int x, uint32_t (&o)[4]) {
    cvt_e2m1x8_f16(w, o);
    const int y = D == 128 ? x % 2 : 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = hmul2(o[e], CF == CF_MX ? f[2 * y + e / 2] : f[4 * y + e]);
  });
}
// The same as bf16, with any E8M0 scale (byte << 23 is 0 for the least).
template <int D>
__device__ __forceinline__ void put_value_far(uint8_t* dst, int row, const uint8_t* src, uint32_t sb, bool gone) {
#pragma unroll 1
  for (int i = 0; i < D / 8; ++i) {
    const int y = D == 128 ? i % 2 : 0;
    uint32_t o[4];
    cvt_e2m1x8_f16(*reinterpret_cast<const uint32_t*>(src + 4 * i), o);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t byte = sb >> (8 * (2 * y + e / 2)) & 0xFFu;
      o[e] = scaled_bf16(o[e], gone || byte == 0xFFu ? 0.f : __uint_as_float(byte << 23));
    }
    put_piece(dst + row * 128, row, i, o);
  }
}

// A warp's 32 rows of a tile of q, from `row0` on, in the order of K's columns; src: this lane's row (zeros without one).
// Neighbouring lanes take 16-byte pieces of a row.  Returns what the scores of this lane's row are to be multiplied by.
template <int D>
__device__ __forceinline__ float put_queries(uint8_t* dst, int row0, const uint16_t* src, float sign, float scale_log2) {
  constexpr int L = D / 8, RPI = 32 / L, AHEAD = 8;                // lanes of a row, rows and loads at a time
  const int lane = threadIdx.x & 31, ch = lane % L, sub = lane / L;
  const int w = ch / 4, h = ch & 1, side = ch >> 1 & 1;            // elements 32w + 16 side + 8h + 0..7
  float cq = scale_log2;
#pragma unroll 1
  for (int k0 = 0; k0 < 32 / RPI; k0 += AHEAD) {
    uint4 u[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const uint16_t* const from = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(src), RPI * (k0 + k) + sub));
      u[k] = from ? *reinterpret_cast<const uint4*>(from + 8 * ch) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      uint32_t t[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
      // (as fsa_cache_attn.cu has q)
      uint32_t m = __vmaxu2(__vimax3_u16x2(t[0] & 0x7FFF7FFFu, t[1] & 0x7FFF7FFFu, t[2] & 0x7FFF7FFFu), t[3] & 0x7FFF7FFFu);
#pragma unroll
      for (int x = 1; x < L; x *= 2) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
      m = max(m & 0xFFFFu, m >> 16);
      const int e = (int)(m >> 7) - 127;                   // floor(log2) of the row's maximum
      const int up = e == 128 || m == 0 ? 0 : min(max(4 - e, -126), 126);
      const float f = e == 128 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(up + 127) << 23) * sign;
      const float c = fmaxf(scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23), 1.4e-45f);      // (0 times -inf is NaN)
      const float theirs = __shfl_sync(0xFFFFFFFFu, c, lane % RPI * L);
      if (lane / RPI == k0 + k) cq = theirs;
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = cvt_f16x2(__uint_as_float(t[i] << 16) * f, __uint_as_float(t[i] & 0xFFFF0000u) * f);
      // elements 16 on have the same places: the lane that has them takes the upper halves of both, this one the lower
      const uint32_t x0 = __shfl_xor_sync(0xFFFFFFFFu, side ? t[0] : t[2], 2), x1 = __shfl_xor_sync(0xFFFFFFFFu, side ? t[1] : t[3], 2);
      const uint32_t ax[2] = {side ? x0 : t[0], side ? x1 : t[1]}, bx[2] = {side ? t[2] : x0, side ? t[3] : x1};
      const uint32_t o[4] = {ax[0], ax[1], bx[0], bx[1]};
      const int row = row0 + RPI * (k0 + k) + sub;
      put_piece(dst + row * 128, row, (D / 32) * (2 * h + side) + w, o);
    }
  }
  return cq;
}

// ------------------------------------------------------------------------ small things
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void upk2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Instruction descriptors of f16 operands, and the bit of a second operand that is MN-major
__device__ __forceinline__ constexpr uint32_t idesc_f16(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }
constexpr uint32_t MN_MAJOR_B = 1u << 16;
// bits i of a word with base + i < n
__device__ __forceinline__ uint32_t below(int n, int base) {
  const int k = n - base;
  return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
}

// Scores of 32 keys: -inf where the row does not see the key; their maximum.
__device__ __forceinline__ float mask32(uint32_t (&r)[32], uint32_t seen) {
  float m = NONE;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    if (!(seen >> e & 1)) r[e] = 0xFF800000u;
    m = fmaxf(m, __uint_as_float(r[e]));
  }
  return m;
}

struct Out {                // where a row goes
  int64_t at, lse_at;
};
__device__ __forceinline__ Out out_of(const CacheAttnArgs& p, int b, int hkv, int row) {
  const int i = row / p.G, h = hkv * p.G + row - i * p.G;
  return {b * p.os.b + i * p.os.s + h * p.os.h, ((int64_t)b * p.Sq + i) * p.H + h};
}
// 4 consecutive dims
__device__ __forceinline__ void put4(const CacheAttnArgs& p, int64_t at, float4 v) {
  if (p.out_bf16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(cvt_bf16x2(v.x, v.y), cvt_bf16x2(v.z, v.w));
  else *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
}

// ---------------------------------------------------------------------------- the kernel
template <int D, int CF>
__global__ void __launch_bounds__(THREADS, 1) cache_chunk_kernel(const CacheAttnArgs p) {
  using C = Cfg<D, CF>;
  using Gr = CacheGroup<D, CF>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  // A stage takes halves of tiles in turn, read by warps 8, 9 and by 10, 11.  Either pair has barriers of its own for them, and
  // so sees every phase: by one that both use, a pair ahead of a copy for the other would take that one's phase for its own.
  uint64_t* const raw_full = bars;             // [2][RAW] codes have landed
  uint64_t* const raw_empty = bars + 2 * RAW;  // [RAW] and been read (2 warps)
  uint64_t* const k_full = bars + 3 * RAW;     // [2] operand written (4 warps)
  uint64_t* const k_empty = k_full + 2;        // [2] and multiplied
  uint64_t* const v_full = k_full + 4;
  uint64_t* const v_empty = k_full + 6;
  uint64_t* const s_full = k_full + 8;         // [2] row tile's scores are there
  uint64_t* const p_full = k_full + 10;        // [2] and its probabilities (4 warps)
  uint64_t* const o_full = k_full + 12;        // [2] and its output
  uint64_t* const q_full = k_full + 14;        // [2] q is there (4 warps; only where the row tile has rows)
  uint64_t* const s_free = k_full + 16;        // [2] APART: the scores have been read (4 warps)
  uint64_t* const o_done = k_full + 18;        // [2] APART: a tile's products with V are done
  uint64_t* const drain = k_full + 20;
  uint32_t* const flags = reinterpret_cast<uint32_t*>(sm + C::OFF_FLAGS);      // [4 tiles][4][4]
  uint32_t* const absent = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);      // [RAW]
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC + 16);
  int* const abort_flag = reinterpret_cast<int*>(sm + C::OFF_MISC + 20);
  int* const wsum = reinterpret_cast<int*>(sm + C::OFF_MISC + 32);             // [16]
  int* const pre = reinterpret_cast<int*>(sm + C::OFF_PRE);
  const AbortCtl ac{abort_flag, p.status, p.timeout_ns};

  griddep_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < RAW; ++i) { mbar_init(raw_full + i, 1); mbar_init(raw_full + RAW + i, 1); mbar_init(raw_empty + i, 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4); mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 4); mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1); mbar_init(p_full + i, 4);
      mbar_init(o_full + i, 1); mbar_init(q_full + i, 4);
      mbar_init(s_free + i, 4); mbar_init(o_done + i, 1);
    }
    mbar_init(drain, 1);
    sts_vol(abort_flag, 0);
    fence_mbar_init();
  }
  if (warp == 13) tmem_alloc(tmem_slot, 512);
  griddep_wait();                              // before any tensor is read

  // the list's length and its prefix sums, a chunk of virtual sequences a thread
  const int VB = p.B * p.CT, chunk = (VB + THREADS - 1) / THREADS;
  int mine = 0;
  for (int vb = threadIdx.x * chunk; vb < min(VB, ((int)threadIdx.x + 1) * chunk); ++vb) mine += units_of(p, span_of(p, vb)) * p.c.Hkv;
  int inc = mine;
#pragma unroll
  for (int x = 1; x < 32; x *= 2) {
    const int up = __shfl_up_sync(0xFFFFFFFFu, inc, x);
    if (lane >= x) inc += up;
  }
  if (lane == 31) wsum[warp] = inc;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  pre[threadIdx.x] = before + inc - mine;
  __syncthreads();
  const uint32_t tbase = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  // no more CTAs than have a segment's start and a tile each
  const int NW = min((int)gridDim.x, p.whole ? total : max(1, total / (EXTRA + 1)));
  const Shares sh(total, NW);
  const bool works = (int)blockIdx.x < NW && total > 0;
  Walk* const walk = reinterpret_cast<Walk*>(sm + C::OFF_WALK) + warp;
  {
    Walk w;
    w.start(p, pre, chunk, works ? sh.first(blockIdx.x) : 0, works ? sh.first(blockIdx.x + 1) : 0);
    if (lane == 0) *walk = w;
  }

  if (warp < 8) {
    // ============================================================ softmax, a row a thread
    // (8 warps of 176, 4 of 96, 4 of 64: the launch's 16 of 128.  184, 96, 48: NVFP4 2% more, E2M1 2% less; 168, 104, 72: NVFP4 4%
    // less, E2M1 2% more)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    const int rt = warp >> 2, rl = threadIdx.x & 127;
    const uint32_t tl = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t tS = tl + C::T_S + 128 * rt, tP = tl + C::T_P + C::P_STEP * rt, tO = tl + C::T_O + D * rt;
    uint32_t n = 0, pieces = 0, slot = 0;      // tiles and pieces of this row tile, tiles of the CTA
    int4 start = make_int4(-1, 0, 0, 0);
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
      return __all_sync(0xFFFFFFFFu, mbar_wait<false>(bar, parity, ac));
    };
    Piece pc;
    while (ok && next_piece(p, walk, sh, pc)) {
      const int b = pc.vb / p.CT, row = (pc.vb - b * p.CT) * ROWS + 128 * rt + rl;
      const bool active = pc.rows > 128 * rt, valid = 128 * rt + rl < pc.rows;
      const int T = pc.t1 - pc.t0;
      if (pc.begins && !pc.ends) start = make_int4(pc.vb * p.c.Hkv + pc.hkv, pc.last, pc.qlen, pc.len);
      if (!active) { slot += T; continue; }
      float cq = 1.f;
      int lim = INT32_MAX;                                         // (rows that are none need no masks)
      {
        const int i = row / p.G, h = pc.hkv * p.G + row - i * p.G;
        if (T > 0) {
          cq = put_queries<D>(sm + C::OFF_Q + rt * C::TILE, 32 * (warp & 3), valid ? p.q + b * p.qs.b + i * p.qs.s + h * p.qs.h : nullptr, p.q_sign, p.scale_log2);
          fence_proxy_async_smem();
          __syncwarp();
          mbar_arrive_elect(q_full + rt);
        }
        if (valid) lim = p.causal ? max(0, pc.len - pc.qlen + i + 1) : pc.len;
      }
      const int wlo = p.window && valid ? lim - p.window : 0;
      float M = NONE;
      uint64_t l2 = pk2(0.f, 0.f), l3 = l2;
      int j = 0;
      if (pc.rows <= 128 * rt + 32 * (warp & 3))                 // none of the warp's rows is one: it only goes along
        for (; ok && j < T; ++j, ++n, ++slot) {
          ok = wait(s_full + rt, n & 1);
          tc_fence_before();
          __syncwarp();
          if constexpr (C::APART) {
            mbar_arrive_elect(s_free + rt);
            if (ok && j > 0) ok = wait(o_done + rt, (n - 1) & 1);        // (so that the last tile's p_full has had all its arrivals)
          }
          mbar_arrive_elect(p_full + rt);
        }
#pragma unroll 1
      for (; ok && j < T; ++j, ++n, ++slot) {
        const int k0 = pc.at(pc.t0 + j) * KEYS;
        ok = wait(s_full + rt, n & 1);
        if (!ok) break;
        tc_fence_after();
        // The maximum of all, then block after block of 32 (64 scores at a time in registers; the last two are read twice).
        // Halves as a loop where that is no slower: the fetching of instructions counts here (NVFP4 1564 to 1596 TFLOP/s).
        uint32_t ra[32], rb[32];
        const uint32_t* const fl = flags + 16 * (slot & 3);
        uint32_t told;
        bool wide = false, far = false;                  // V, and P with it, is bf16 for some keys; some keys have a shift
        {
          const uint4 a = reinterpret_cast<const uint4*>(fl)[0], c = reinterpret_cast<const uint4*>(fl)[1];
          told = a.x | a.y | a.z | a.w | c.x | c.y | c.z | c.w;
          if constexpr (CF == CF_MX) {
            const uint4 t = reinterpret_cast<const uint4*>(fl)[2];
            wide = (t.x | t.y | t.z | t.w) != 0;
            const uint4 f = reinterpret_cast<const uint4*>(fl)[3];
            far = (f.x | f.y | f.z | f.w) != 0;
          }
        }
        // the keys that the row does not see (all rows of a warp go along)
        const bool masked = __any_sync(0xFFFFFFFFu, told != 0 || k0 + KEYS > lim || (k0 < wlo && k0 + KEYS > p.sinks));
        uint32_t seen[4] = {};
        if (masked) {
          uint32_t bad = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            seen[c] = below(lim, k0 + 32 * c) & ~fl[c];
            if (p.window) seen[c] &= ~below(wlo, k0 + 32 * c) | below(p.sinks, k0 + 32 * c);
            bad |= seen[c] & fl[4 + c];
          }
          if (bad) l2 = pk2(__uint_as_float(0x7FC00000u), 0.f);
        }
        if (CF == CF_MX && far) {                        // (rare: eight scores at a time, each times its key's power of two)
#pragma unroll 1
          for (int c = 0; c < KEYS / 8; ++c) {
            if (fl[12 + c / 4] == 0) continue;           // (the same for all: none of these 32 keys has one)
            uint32_t o[8];
            TmemLd<8>::run(tS + 8 * c, o);
            const int4 by8 = reinterpret_cast<const int4*>(sm + C::OFF_SHIFT)[KEYS / 8 * (slot & 3) + c];
            const int by2[4] = {by8.x, by8.y, by8.z, by8.w};
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {                // (in two steps: it may lie beyond a float's powers of two)
              const int by = e & 1 ? by2[e / 2] >> 16 : (int)(int16_t)by2[e / 2], half = by >> 1;
              o[e] = __float_as_uint(__uint_as_float(o[e]) * __uint_as_float((uint32_t)(127 + half) << 23) * __uint_as_float((uint32_t)(127 + by - half) << 23));
            }
            TmemSt<8>::run(tS + 8 * c, o);
          }
          tc_wait_st();
        }
        float top = NONE;
#pragma unroll 1
        for (int c = 2; c >= 0; c -= 2) {
          float ma, mb;
          tmem_ld32_max(tS + 32 * c, ra, ma);
          tmem_ld32_max(tS + 32 * c + 32, rb, mb);
          tc_wait_ld();
          if (masked) { ma = mask32(ra, c ? seen[2] : seen[0]); mb = mask32(rb, c ? seen[3] : seen[1]); }
          top = fmaxf(top, fmaxf(ma, mb));
        }
        const float x = top * cq;
        float alpha = 1.f;
        if (M == NONE) {
          M = x;
        } else if (x - M > LAZY) {
          alpha = ex2_approx(M - x);
          M = x;
          l2 = ffma2(l2, pk2(alpha, alpha), pk2(0.f, 0.f));
          l3 = ffma2(l3, pk2(alpha, alpha), pk2(0.f, 0.f));
        }
        // (the scores of this tile are there, so the products of the tile before, or APART of the one before that, are
        // done; those of this tile wait for this warp, so the barrier's parity tells)
        if (j > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
          if constexpr (C::APART) {
            ok = wait(o_done + rt, (n - 1) & 1);
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < D; c += 8) {
            uint32_t o[8];
            TmemLd<8>::run(tO + c, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            TmemSt<8>::run(tO + c, o);
          }
        }
        const float nM = M == NONE ? 0.f : UP - M;       // no key yet: every score is -inf, every weight 0
        const uint64_t c2 = pk2(cq, cq), nM2 = pk2(nM, nM);
        auto weigh = [&](uint32_t (&r)[32], int c, auto pack) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, bb;
            upk2(ffma2(pk2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), c2, nM2), a, bb);
            a = ex2_approx(a);
            bb = ex2_approx(bb);
            if (e & 1) l3 = fadd2(l3, pk2(a, bb));
            else l2 = fadd2(l2, pk2(a, bb));
            r[2 * e] = __float_as_uint(a);
            r[2 * e + 1] = __float_as_uint(bb);
          }
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pw[e] = pack(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
          TmemSt<16>::run(tP + 16 * c, pw);              // (over scores that have been read, or apart)
        };
        if constexpr (C::APART) {
          // P of the tile before has been multiplied before its columns are written again
          if (j > 0) {
            ok = wait(o_done + rt, (n - 1) & 1);
            if (!ok) break;
            tc_fence_after();
          }
        }
        if (CF == CF_MX && wide) {                       // (rare: block after block, read again)
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            tmem_ld_cols<32>(tS + 32 * c, ra);
            tc_wait_ld();
            if (masked) mask32(ra, c == 0 ? seen[0] : c == 1 ? seen[1] : c == 2 ? seen[2] : seen[3]);
            const bool w = fl[8 + c] != 0;
            weigh(ra, c, [&](float a, float bb) { return w ? cvt_bf16x2(a, bb) : cvt_f16x2(a, bb); });
          }
        } else {
          auto f16 = [](float a, float bb) { return cvt_f16x2(a, bb); };
          // (as a loop NVFP4 1402 TFLOP/s instead of 1564, E2M1 1309 instead of 1354, but with 64 dims 714 instead of 678)
#pragma unroll (CF == CF_MX && D == 64 ? 1 : 2)
          for (int c = 0; c < 4; c += 2) {
            if (c > 0) {
              tc_wait_ld();
              if constexpr (C::APART) {
                tc_fence_before();
                __syncwarp();
                mbar_arrive_elect(s_free + rt);
              }
              if (masked) { mask32(ra, seen[2]); mask32(rb, seen[3]); }
            }
            weigh(ra, c, f16);
            if (c == 0) tmem_ld_cols<32>(tS + 64, ra);
            weigh(rb, c + 1, f16);
            if (c == 0) tmem_ld_cols<32>(tS + 96, rb);
          }
        }
        if constexpr (C::APART && CF == CF_MX) {
          if (wide) {
            tc_fence_before();
            __syncwarp();
            mbar_arrive_elect(s_free + rt);
          }
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_elect(p_full + rt);
      }
      if (!ok) break;
      if (T > 0) {
        ok = wait(o_full + rt, pieces & 1);
        if (!ok) break;
        ++pieces;
        tc_fence_after();
      }
      float la, lb, lc, ld;
      upk2(l2, la, lb);
      upk2(l3, lc, ld);
      const float l = (la + lb) + (lc + ld);
      const bool whole = pc.begins && pc.ends, none = l == 0.f;
      const float inv = !whole ? 1.f : none ? 0.f : 1.f / l;
      const Out out = out_of(p, b, pc.hkv, row);
      float* const part = p.partials + (int64_t)(2 * blockIdx.x + (pc.begins ? 1 : 0)) * C::PART;
      // Rows go out by way of the warp's rows of Q, whose products are done, so that neighbouring lanes store
      // neighbouring dims.  Loops stay loops: this runs once a piece, and what it costs is the fetching of its instructions.
      constexpr int AT_ONCE = D / 4;                       // rows of 64 floats that fit there
      uint8_t* const mine = sm + C::OFF_Q + rt * C::TILE + 32 * (warp & 3) * 128;
      auto staged = [&](int r, int c) {                  // four floats c of row r
        const int x = c ^ (r & 7);
        return reinterpret_cast<float4*>(mine + (x & 7) * 16 + (D == 128 ? (x >> 3) * C::ATOM + r * 128 : (2 * r + (x >> 3)) * 128));
      };
      const int rows = min(32, pc.rows - 128 * rt - 32 * (warp & 3));            // of the warp
      const bool zeros = T == 0 || (whole && none);
#pragma unroll 1
      for (int y = 0; y < D / 64; ++y) {
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += AT_ONCE) {
#pragma unroll 1
          for (int g = 0; g < 8; g += 2) {               // dims 64y + 16s + 2g, + 1 at 2s, 2s + 1 of each eight
            uint32_t o[2][8];
            TmemLd<8>::run(tO + 8 * (g * (D / 64) + y), o[0]);
            TmemLd<8>::run(tO + 8 * ((g + 1) * (D / 64) + y), o[1]);
            tc_wait_ld();
            if (D == 128 || (lane & AT_ONCE) == r0) {
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!zeros)
                  v = make_float4(__uint_as_float(o[0][2 * s]) * inv, __uint_as_float(o[0][2 * s + 1]) * inv,
                                  __uint_as_float(o[1][2 * s]) * inv, __uint_as_float(o[1][2 * s + 1]) * inv);
                *staged(lane % AT_ONCE, 4 * s + g / 2) = v;
              }
            }
          }
          __syncwarp();
          const int c = lane & 15, d = 64 * y + 4 * c;
#pragma unroll 1
          for (int k0 = 0; k0 < AT_ONCE / 2; k0 += 4) {
            int64_t to[4];
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = 2 * (k0 + k) + (lane >> 4);
              to[k] = __shfl_sync(0xFFFFFFFFu, out.at, r0 + at);
              v[k] = *staged(at, c);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = r0 + 2 * (k0 + k) + (lane >> 4);
              if (r >= rows) continue;
              if (whole) put4(p, to[k] + d, v[k]);
              else *reinterpret_cast<float4*>(part + (128 * rt + 32 * (warp & 3) + r) * D + d) = v[k];
            }
          }
          __syncwarp();
        }
      }
      if (valid) {
        if (!whole) {
          part[ROWS * D + 128 * rt + rl] = M;
          part[ROWS * (D + 1) + 128 * rt + rl] = l;
        } else if (p.lse) {
          p.lse[out.lse_at] = none ? NONE : (M - UP + log2f(l)) * 0.69314718055994530942f;
        }
      }
      tc_fence_before();
    }
    if (threadIdx.x == 0 && !p.whole) p.starts[blockIdx.x] = ok ? start : make_int4(-1, 0, 0, 0);
  } else if (warp < 12) {
    // ============================================================ operands from codes, a key a thread
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    const int dw = warp - 8, row = 32 * dw + lane;
    uint32_t n = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, ac)); };
    Piece pc;
    while (ok && next_piece(p, walk, sh, pc)) {
      for (int t = pc.t0; t < pc.t1; ++t, ++n) {
        const uint32_t pair = dw >> 1, rs = (2 * n + pair) % RAW, kb = n & 1;
        ok = wait(raw_full + RAW * pair + rs, (n / RAW) & 1) && (n < 2 || wait(k_empty + kb, (n / 2 - 1) & 1));
        if (!ok) break;
        const int grp = 2 * (dw & 1) + (lane >> 4);      // of the stage's four
        const int key = pc.at(t) * KEYS + row;
        bool gone = (absent[rs] >> grp & 1) || key >= pc.kmax;
        if (p.window) gone = gone || (key < pc.low && key >= p.sinks);       // (no row of the block sees it)
        const uint8_t* const base = sm + C::OFF_RAW + rs * C::STAGE + grp * Gr::BYTES;
        uint32_t ks[2] = {0u, 0u}, vs[2] = {0u, 0u};
        const uint8_t *kp = base + Gr::KS + (lane & 15) * Gr::SB, *vp = base + Gr::VS + (lane & 15) * Gr::SB;
        if constexpr (Gr::SB == 8) {
          const uint2 a = *reinterpret_cast<const uint2*>(kp), c = *reinterpret_cast<const uint2*>(vp);
          ks[0] = a.x; ks[1] = a.y; vs[0] = c.x; vs[1] = c.y;
        } else if constexpr (Gr::SB == 4) {
          ks[0] = *reinterpret_cast<const uint32_t*>(kp);
          vs[0] = *reinterpret_cast<const uint32_t*>(vp);
        } else {
          ks[0] = *reinterpret_cast<const uint16_t*>(kp);
          vs[0] = *reinterpret_cast<const uint16_t*>(vp);
        }
        bool nan = false, far = false, kfar = false;     // (the least scale is that of a block of zeros, and not far)
        uint32_t kmax = 0;
#pragma unroll
        for (int i = 0; i < Gr::SB; ++i) {
          const uint32_t byte = byte_of(vs, i);
          nan |= CF == CF_MX ? byte == 0xFFu : (byte & 0x7Fu) == 0x7Fu;
          far |= CF == CF_MX && byte - 1u < 254u && (byte < LEAST_F16 || byte > MOST_F16);
          if constexpr (CF == CF_MX) {
            const uint32_t k = byte_of(ks, i);
            if (k != 0xFFu && k != 0u && !gone) {
              kfar |= k < LEAST_F16 || k > MOST_F16;
              kmax = max(kmax, k);
            }
          }
        }
        const uint32_t gones = __ballot_sync(0xFFFFFFFFu, gone), nans = __ballot_sync(0xFFFFFFFFu, nan && !gone);
        const uint32_t fars = CF == CF_MX ? __ballot_sync(0xFFFFFFFFu, far && !gone) : 0u;
        // (a key with a scale that is not exact in f16: divided by what makes its largest 2^13)
        const int shift = CF == CF_MX && kfar ? (int)kmax - (int)MOST_F16 : 0;
        const uint32_t kfars = CF == CF_MX ? __ballot_sync(0xFFFFFFFFu, shift != 0) : 0u;
        uint32_t* const fl = flags + 16 * (n & 3);
        if (lane == 0) {
          fl[dw] = gones;
          fl[4 + dw] = nans;
          if (CF == CF_MX) {
            fl[8 + dw] = fars;
            fl[12 + dw] = kfars;
          }
        }
        if (CF == CF_MX && kfars) reinterpret_cast<int16_t*>(sm + C::OFF_SHIFT)[KEYS * (n & 3) + row] = (int16_t)shift;
        Row<D> r;
        r.load(row, base + Gr::K + (lane & 15) * (D / 2));
        put_key<D, CF>(sm + C::OFF_K + kb * C::TILE, row, r, ks, gone, shift);
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_elect(k_full + kb);
        const uint8_t* const src = base + Gr::V + (lane & 15) * (D / 2);
        uint8_t* const dst = sm + C::OFF_V + kb * C::TILE;
        if (CF == CF_MX && fars) {
          ok = n < 2 || wait(v_empty + kb, (n / 2 - 1) & 1);
          if (!ok) break;
          put_value_far<D>(dst, row, src, vs[0], gone);
          __syncwarp();
          mbar_arrive_elect(raw_empty + rs);
        } else {                                         // (the stage is free before V's place is)
          r.load(row, src);
          __syncwarp();
          mbar_arrive_elect(raw_empty + rs);
          ok = n < 2 || wait(v_empty + kb, (n / 2 - 1) & 1);
          if (!ok) break;
          put_value<D, CF>(dst, row, r, vs, gone);
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_elect(v_full + kb);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 12) {
      // ========================================================== copies: 16 groups of 16 keys at a time
      uint32_t n = 0;                          // stages
      bool ok = true;
      Piece w;
      while (ok && next_piece(p, walk, sh, w)) {
        const int b = w.vb / p.CT;
        const uint8_t* const head = p.c.pages + ((int64_t)w.hkv << (p.c.page_shift - 4)) * Gr::BYTES;
        const int32_t* const table = p.table + (int64_t)b * p.max_pages;
        // the page of lane's group of tiles t .. t + 3 (-1: none, or no row sees any of its keys)
        auto look_up = [&](int t) {
          const int v = t + (lane >> 3), pos = w.at(v) * KEYS + 16 * (lane & 7);
          int page = -1;
          if (v < w.t1 && pos < w.kmax && (pos < p.sinks || pos + 16 > w.low)) {
            page = table[pos >> p.c.page_shift];
            if ((uint32_t)page >= (uint32_t)p.c.num_pages) {
              page = -1;
              if (p.status) atomicExch(p.status, -1);    // FSA_ERR_INVALID_ARG
            }
          }
          return page;
        };
        int ahead = look_up(w.t0);
        for (int t = w.t0; ok && t < w.t1; t += 4) {
          const int page = ahead;
          if (t + 4 < w.t1) ahead = look_up(t + 4);
          const uint32_t here = __ballot_sync(0xFFFFFFFFu, page >= 0);
          for (int x = 0; ok && x < 2 * min(4, w.t1 - t); ++x, ++n) {
            const uint32_t rs = n % RAW;
            uint64_t* const full = raw_full + RAW * (n & 1) + rs;
            ok = n < RAW || __all_sync(0xFFFFFFFFu, mbar_wait(raw_empty + rs, (n / RAW - 1) & 1, ac));
            if (!ok) break;
            const uint32_t four = here >> (4 * x) & 15u;
            if (lane == 0) {
              absent[rs] = four ^ 15u;
              mbar_expect_tx(full, __popc(four) * Gr::BYTES);
            }
            __syncwarp();
            if ((lane >> 2) == x && page >= 0) {
              const int pos = w.at(t + (lane >> 3)) * KEYS + 16 * (lane & 7);
              const int inside = (pos & ((1 << p.c.page_shift) - 1)) / 16;
              bulk_load(sm + C::OFF_RAW + rs * C::STAGE + (lane & 3) * Gr::BYTES, head + page * p.c.page_bytes + inside * Gr::BYTES,
                        Gr::BYTES, full);
            }
            __syncwarp();
          }
        }
      }
      // the copies in flight end before the CTA does
      for (uint32_t x = n > RAW ? n - RAW : 0; x < n; ++x) mbar_drain(raw_full + RAW * (x & 1) + x % RAW, (x / (2 * RAW)) & 1, ac);
    } else if (warp == 13) {
      // ========================================================== products
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, mbar_wait<false>(bar, parity, ac)); };
      // the operands' descriptors; what is added to one is its offset over 16
      const uint64_t dQ = smem_desc(smem_u32(sm + C::OFF_Q), 16, 1024, 2), dK = smem_desc(smem_u32(sm + C::OFF_K), 16, 1024, 2);
      const uint64_t dV = smem_desc(smem_u32(sm + C::OFF_V), C::ATOM, 1024, 2);      // MN-major: 64 dims an atom, 8 keys 1024 bytes
      uint32_t n = 0, nq[2] = {0, 0}, np[2] = {0, 0};
      bool ok = true;
      // (one lane issues them all: with an election for each, and its address worked out there, the issue took longer
      // than the products)
      auto scores = [&](int rt, uint32_t kb) {
        if (elect_one()) {
          const uint64_t q = dQ + rt * (C::TILE / 16), k = dK + kb * (C::TILE / 16);
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_f16_ss(tbase + C::T_S + 128 * rt, q + ((i / 4) * C::ATOM + (i % 4) * 32) / 16, k + ((i / 4) * C::ATOM + (i % 4) * 32) / 16,
                       idesc_f16(128), i > 0);
          tc_commit(s_full + rt);
        }
        __syncwarp();
      };
      auto products = [&](int rt, uint32_t vb, bool more, uint4 wide) {
        if (elect_one()) {
          const uint64_t v = dV + vb * (C::TILE / 16);
          const uint32_t of[4] = {wide.x, wide.y, wide.z, wide.w};
#pragma unroll
          for (int i = 0; i < KEYS / 16; ++i)
            mma_f16_ts(tbase + C::T_O + D * rt, tbase + C::T_P + C::P_STEP * rt + 8 * i, v + i * (2048 / 16),
                       MN_MAJOR_B | (CF == CF_MX && of[i / 2] ? idesc_f16_bf16(D) : idesc_f16(D)), more || i > 0);
          if (C::APART) tc_commit(o_done + rt);
        }
        __syncwarp();
      };
      Piece w;
      while (ok && next_piece(p, walk, sh, w)) {
        const int T = w.t1 - w.t0, tiles = w.rows > 128 ? 2 : 1;
        if (T == 0) continue;
        ok = wait(k_full + (n & 1), (n / 2) & 1);
        for (int rt = 0; ok && rt < tiles; ++rt) {
          ok = wait(q_full + rt, nq[rt] & 1);
          if (!ok) break;
          ++nq[rt];
          tc_fence_after();
          scores(rt, n & 1);
        }
        if (!ok) break;
        tc_commit_p(elect_u32(), k_empty + (n & 1));
        for (int j = 0; ok && j < T; ++j, ++n) {
          ok = wait(v_full + (n & 1), (n / 2) & 1);
          uint4 wide = make_uint4(0u, 0u, 0u, 0u);         // of each operand warp's keys: V and P are bf16
          if constexpr (CF == CF_MX) wide = reinterpret_cast<const uint4*>(flags + 16 * (n & 3))[2];
          if (C::APART && j + 1 < T) {         // the next scores first
            ok = ok && wait(k_full + ((n + 1) & 1), ((n + 1) / 2) & 1);
            for (int rt = 0; ok && rt < tiles; ++rt) {
              ok = wait(s_free + rt, np[rt] & 1);
              if (!ok) break;
              tc_fence_after();
              scores(rt, (n + 1) & 1);
            }
            if (ok) tc_commit_p(elect_u32(), k_empty + ((n + 1) & 1));
          }
          for (int rt = 0; ok && rt < tiles; ++rt) {
            ok = wait(p_full + rt, np[rt] & 1);
            if (!ok) break;
            ++np[rt];
            tc_fence_after();
            products(rt, n & 1, j > 0, wide);
            if (j + 1 == T) {
              tc_commit_p(elect_u32(), o_full + rt);
            } else if (!C::APART) {
              if (rt == 0) ok = wait(k_full + ((n + 1) & 1), ((n + 1) / 2) & 1);
              if (!ok) break;
              tc_fence_after();
              scores(rt, (n + 1) & 1);
            }
          }
          if (!ok) break;
          tc_commit_p(elect_u32(), v_empty + (n & 1));
          if (!C::APART && j + 1 < T) tc_commit_p(elect_u32(), k_empty + ((n + 1) & 1));
        }
      }
      tc_commit_p(elect_u32(), drain);         // all products end before tensor memory is freed
      mbar_drain(drain, 0, ac);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tbase, 512);
}

// Joins the parts of the segments that several CTAs share.  Block (c, y) takes the one that
// begins in CTA c and goes on, 8 rows of it, a warp a row and a lane D/32 dims: CTA c's second part and the
// first part of each later CTA up to the last.  The first parts' rows set out together with all maxima and sums.
constexpr int JOIN_ROWS = 8, JOIN_THREADS = 256, JOIN_AHEAD = 4;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) cache_chunk_join_kernel(const CacheAttnArgs p) {
  constexpr int PART = ROWS * (D + 2), PER = D / 32;
  griddep_launch();
  griddep_wait();                              // the first kernel's results are complete
  const int4 st = p.starts[blockIdx.x];        // segment, last CTA, its rows' tokens, its keys
  if (st.x < 0) return;
  const int lane = threadIdx.x & 31, vb = st.x / p.c.Hkv, hkv = st.x - vb * p.c.Hkv, b = vb / p.CT;
  const int n = st.y - (int)blockIdx.x + 1, r = blockIdx.y * JOIN_ROWS + threadIdx.x / 32;
  if (r >= min(ROWS, st.z * p.G - (vb - b * p.CT) * ROWS)) return;
  const float* const parts = p.partials + (int64_t)2 * blockIdx.x * PART;
  auto part = [&](int k) { return parts + (k == 0 ? (int64_t)PART : (int64_t)2 * k * PART); };
  auto row = [&](int k, float (&v)[PER]) {
    const float* const src = part(k) + r * D + PER * lane;
    if constexpr (PER == 4) {
      const float4 u = *reinterpret_cast<const float4*>(src);
      v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
      const float2 u = *reinterpret_cast<const float2*>(src);
      v[0] = u.x; v[1] = u.y;
    }
  };
  float v[JOIN_AHEAD][PER];
#pragma unroll
  for (int k = 0; k < JOIN_AHEAD; ++k)
    if (k < n) row(k, v[k]);
  float mk = NONE, lk = 0.f, m = NONE;         // of part `lane`
  if (lane < n) {
    mk = part(lane)[ROWS * D + r];
    lk = part(lane)[ROWS * (D + 1) + r];
    m = mk;
  }
  for (int k = lane + 32; k < n; k += 32) m = fmaxf(m, part(k)[ROWS * D + r]);
#pragma unroll
  for (int x = 16; x; x /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
  float l = 0.f, o[PER] = {};
  for (int k0 = 0; k0 < n; k0 += 32) {
    if (k0 > 0) {
      const bool in = k0 + lane < n;
      mk = in ? part(k0 + lane)[ROWS * D + r] : NONE;
      lk = in ? part(k0 + lane)[ROWS * (D + 1) + r] : 0.f;
    }
    const float f = lk == 0.f ? 0.f : exp2f(mk - m);     // (a part that saw nothing counts nothing)
    l = fmaf(f, lk, l);
    auto add = [&](int k, const float (&u)[PER]) {
      const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
      if (fk != 0.f) {
#pragma unroll
        for (int e = 0; e < PER; ++e) o[e] = fmaf(fk, u[e], o[e]);
      }
    };
    int k = 0;
    if (k0 == 0) {
#pragma unroll
      for (int x = 0; x < JOIN_AHEAD; ++x)
        if (x < n) add(x, v[x]);
      k = JOIN_AHEAD;
    }
#pragma unroll 8
    for (; k < min(32, n - k0); ++k) {
      float u[PER];
      row(k0 + k, u);
      add(k, u);
    }
  }
#pragma unroll
  for (int x = 16; x; x /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.0f / l;
  const Out out = out_of(p, b, hkv, (vb - b * p.CT) * ROWS + r);
  if constexpr (PER == 4) {
    put4(p, out.at + 4 * lane, none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv));
  } else {
    const float x = none ? 0.f : o[0] * inv, y = none ? 0.f : o[1] * inv;
    if (p.out_bf16) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + out.at + 2 * lane) = cvt_bf16x2(x, y);
    else *reinterpret_cast<float2*>(static_cast<float*>(p.out) + out.at + 2 * lane) = make_float2(x, y);
  }
  if (lane == 0 && p.lse) p.lse[out.lse_at] = none ? NONE : (m - UP + log2f(l)) * 0.69314718055994530942f;
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

template <int D, int CF>
cudaError_t launch(const CacheAttnArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<D, CF>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(cache_chunk_kernel<D, CF>, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  const int64_t segments = (int64_t)a.B * a.CT * a.c.Hkv;
  const unsigned grid = a.whole ? (unsigned)std::min<int64_t>(segments, sms) : (unsigned)sms;
  e = launch_early(cache_chunk_kernel<D, CF>, dim3(grid), THREADS, C::SMEM, st, a);
  if (e != cudaSuccess || a.whole) return e;
  return launch_early(cache_chunk_join_kernel<D>, dim3(grid, ROWS / JOIN_ROWS), JOIN_THREADS, 0, st, a);
}

}  // namespace

int cache_chunk_blocks(int rows) { return (rows + ROWS - 1) / ROWS; }

// Segments of at most 4 tiles are not shared: a CTA each, no second kernel (64 tokens over 512 keys, NVFP4, in tables
// of 512 and of 576 tokens, which are shared: 4 sequences 18 and 25 us, 32 34 and 52, 64 67 and 82; 256 of 256 keys
// 180 and 207).
bool cache_chunk_whole(const Cache& c, int max_pages) { return ((int64_t)max_pages << c.page_shift) <= 4 * KEYS; }

// parts of the CTAs, two each; where segments begin that go on
size_t cache_chunk_workspace(const Cache& c, int max_pages, int sms, size_t* starts_at) {
  *starts_at = (size_t)2 * sms * ROWS * (c.D + 2) * sizeof(float);
  return cache_chunk_whole(c, max_pages) ? 0 : *starts_at + (size_t)sms * sizeof(int4);
}

cudaError_t launch_cache_chunk(const CacheAttnArgs& a, int sms, cudaStream_t st) {
  if (a.c.D == 128) return a.c.cf == CF_MX ? launch<128, CF_MX>(a, sms, st) : launch<128, CF_NV>(a, sms, st);
  return a.c.cf == CF_MX ? launch<64, CF_MX>(a, sms, st) : launch<64, CF_NV>(a, sms, st);
}

}  // namespace fsa
