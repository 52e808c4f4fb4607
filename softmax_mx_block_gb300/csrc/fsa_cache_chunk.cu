// fsa_cache_chunk.cu -- attention of a chunk of new tokens over the paged 4-bit cache.
//
//   o = softmax(scale q K^T) V  over the keys a row sees, K and V the values the cache
//   stands for (codes times block scales), q as given, sums in fp32.
//
// A kv head's query rows (its G heads' rows of each token, in order) go 256 at a time, two tiles
// of 128, over the key tiles of 128 that some of them see:
//   - bound by the products, 4 D flops a seen pair: tcgen05 kind::f16 MMAs on bf16.  The block-scaled
//     kinds cannot take V's scales, which run across its product's summation, nor q unrounded.  A
//     code times its scale is exact in bf16, so four warps turn a tile's codes into bf16 operands in
//     shared memory, once for 256 rows (as long as both products of one tile of 128 rows take).
//   - A cache row's bytes are in the order of other fragments (fsa_cache.h); here a word becomes
//     a 16-byte piece of its row, nibbles i and i + 4 side by side, so the operands' columns are
//     permuted: those of K alike in q, which is permuted as it is loaded, those of V in the output's
//     columns, which are put in order as they are stored.  K is K-major; V needs no transposition, as
//     the second operand of a product over the keys it is MN-major.
//   - E2M1's exponent and fraction put into bf16's lowest bits are the value times 2^-126, a zero
//     or a subnormal included; one product with the scale times 2^(126 - 16) gives the operand, 2^-16
//     of the value (the largest scales need a second one).  The softmax factor and the end make up for it.
//   - S, then P over it, and O stay in tensor memory: 128 columns each for both row tiles.  While
//     the softmax of one row tile runs, the other's products do.  P is rounded to bf16 (2^-8 of each
//     weight; the output's own rounding is as large); sums and maxima are fp32.  The running maximum
//     is raised only when a score beats it by more than 2^8 in the softmax.
//   - The work, (sequence, row block, kv head, key tile), is one list split evenly over one CTA per
//     SM (a segment's start weighing as EXTRA tiles); parts of a segment that several CTAs share are
//     joined by a second kernel.  Lengths are read on the device.
//   - A row that sees a token whose values are not finite (the scale's NaN) is NaN as a whole; the others
//     are as without it (its V is zero in the operand, and a bit tells the rows).
#include <algorithm>
#include <atomic>
#include "fsa_cache.h"
#include "fsa_mx.cuh"

namespace fsa {
namespace {

constexpr int ROWS = 256;             // of a block: two tiles of 128
constexpr int KEYS = 128;             // of a tile
constexpr int EXTRA = 3;              // what a segment's start costs a CTA, in tiles
constexpr int THREADS = 512;          // warps 0..7 softmax (a row a thread), 8..11 operands, 12 copies, 13 MMA
constexpr int RAW = 3;                // stages of 64 keys of codes
constexpr float LAZY = 8.0f;          // log2 of how far a score may beat the running maximum
constexpr float SHIFT_UP = 65536.0f;  // 2^16, the operands being 2^-16 of K and V
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
  static constexpr int OFF_FLAGS = OFF_BAR + 256;        // [4 tiles][4 warps] of {absent keys, keys with a NaN in V}
  static constexpr int OFF_MISC = OFF_FLAGS + 128;       // absent groups of the raw stages, tmem base, abort flag, warp sums
  static constexpr int OFF_PRE = OFF_MISC + 128;         // [THREADS] prefix sums of the list
  static constexpr int SMEM = OFF_PRE + THREADS * 4 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t T_S = 0, T_O = 256;          // tensor memory: + 128 (S), + D (O) for the second row tile
  static constexpr int PART = ROWS * (D + 2);            // floats of a partial result: rows, maxima, sums
};

// ---------------------------------------------------------------------- the work list
struct Span {
  int qlen, len, kmax;      // rows' tokens, keys, keys that some row of the block sees
  int rows;                 // of the block
  int lead, w0, tiles;      // tiles of the first keys, first tile of some window, tiles in all
  __device__ __forceinline__ int at(int t) const { return t < lead ? t : t - lead + w0; }
};
// virtual sequence vb = b * p.CT + block of rows
__device__ __forceinline__ Span span_of(const CacheAttnArgs& p, int vb) {
  Span s;
  const int b = vb / p.CT, r0 = (vb - b * p.CT) * ROWS;
  s.qlen = p.q_lens ? min(max(p.q_lens[b], 0), p.Sq) : p.Sq;
  s.len = (int)min((int64_t)max(p.lens[b], 0), (int64_t)p.max_pages << p.c.page_shift);
  s.rows = min(ROWS, s.qlen * p.G - r0);
  s.kmax = s.lead = s.w0 = s.tiles = 0;
  if (s.rows <= 0) return s;
  s.kmax = p.causal ? max(0, s.len - s.qlen + (r0 + s.rows - 1) / p.G + 1) : s.len;
  const int end = (s.kmax + KEYS - 1) / KEYS;
  if (p.window) {
    s.w0 = min(max(0, s.len - s.qlen + r0 / p.G + 1 - p.window) / KEYS, end);
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
  __device__ __forceinline__ Walk(const CacheAttnArgs& p, const int* pre, int chunk, int lo_, int hi_) : lo(lo_), hi(hi_) {
    vb = hkv = unit = 0;
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
  __device__ __forceinline__ bool begins() const { return t0 == 0; }
  __device__ __forceinline__ bool ends() const { return t1 == sp.tiles; }
};

// ---------------------------------------------------------------- operands from codes
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The eight codes of a word as bf16 of value * 2^-126: nibbles i and i + 4 in word i.
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&o)[4]) {
  constexpr uint32_t SIGN = 0x80008000u, MAG = 0x01C001C0u;
  o[0] = ((w << 12) & SIGN) | ((w << 6) & MAG);
  o[1] = ((w << 8) & SIGN) | ((w << 2) & MAG);
  o[2] = ((w << 4) & SIGN) | ((w >> 2) & MAG);
  o[3] = (w & SIGN) | ((w >> 6) & MAG);
}
// A block scale as a bf16 factor 2^(126 - 16) * scale, in both halves of a word, and what is
// missing from it (more: its factor, 1 but for E8M0 scales over 2^17)
__device__ __forceinline__ uint32_t e8m0_factor(uint32_t byte) {
  const uint32_t f = byte == 0xFFu ? 0x7FC0u : min(byte + 110u, 254u) << 7;
  return f * 0x10001u;
}
__device__ __forceinline__ uint32_t e8m0_more(uint32_t byte) { return (byte > 144u && byte != 0xFFu ? (byte - 144u + 127u) << 7 : 0x3F80u) * 0x10001u; }
// (up to 2^118: exact, as the scale's four bits are)
__device__ __forceinline__ uint32_t e4m3_factor(uint32_t byte) {
  const float f = e4m3_to_f32(byte) * 0x1p110f;
  return (__float_as_uint(f) >> 16) * 0x10001u;
}
__device__ __forceinline__ uint32_t low_high(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7610); }   // a's low half, b's high

// One row (key) of K or of V: its codes at `src`, scale bytes `sb`, into row `row` of the operand.
template <int D, int CF, bool VALUES>
__device__ __forceinline__ void put_operand(uint8_t* dst, int row, const uint8_t* src, const uint32_t (&sb)[2], bool gone) {
  constexpr int PIECES = D / 32;                         // of 16 bytes (four words) of codes
  constexpr int SB = CacheGroup<D, CF>::SB;
  uint32_t f[SB], more[SB];
  bool big = false;
#pragma unroll
  for (int i = 0; i < SB; ++i) {
    const uint32_t byte = (sb[i / 4] >> (8 * (i % 4))) & 0xFFu;
    if constexpr (CF == CF_MX) {
      f[i] = e8m0_factor(byte);
      more[i] = e8m0_more(byte);
      big |= byte > 144u && byte != 0xFFu;
      if (VALUES && byte == 0xFFu) f[i] = 0u;
    } else {
      f[i] = e4m3_factor(byte);
      if (VALUES && (byte & 0x7Fu) == 0x7Fu) f[i] = 0u;
    }
    if (gone) f[i] = 0u;
  }
  // two factors a word (pairs 0, 1 and pairs 2, 3 of its four), by the word's place among the four
  uint32_t fa[4], fb[4], ma[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    if constexpr (!VALUES) {                             // word 4t + w (D 64: 2t + w): elements 32w + 4t + 0..3, + 16 .. 19
      const int w = x % (D / 32);
      fa[x] = fb[x] = CF == CF_MX ? f[w] : low_high(f[2 * w % SB], f[(2 * w + 1) % SB]);
      ma[x] = CF == CF_MX ? more[w] : 0u;
    } else {                                             // word 2g + y (D 64: g): elements 64y + 2g + 0, 1, + 16, 17, + 32, 33, + 48, 49
      const int y = D == 128 ? x % 2 : 0;
      if constexpr (CF == CF_MX) {
        fa[x] = fb[x] = low_high(f[2 * y], f[2 * y + 1]);
        ma[x] = low_high(more[2 * y], more[2 * y + 1]);
      } else {
        fa[x] = low_high(f[(4 * y) % SB], f[(4 * y + 2) % SB]);
        fb[x] = low_high(f[(4 * y + 1) % SB], f[(4 * y + 3) % SB]);
        ma[x] = 0u;
      }
    }
  }
  uint8_t* const out = dst + row * 128;
#pragma unroll
  for (int c = 0; c < PIECES; ++c) {
    // neighbouring lanes take the pieces in turn, so that neither the loads nor the stores of a
    // quarter of the warp share banks (D 64: the loads do, two and two)
    const int cc = D == 128 ? (c + (row >> 1)) & 3 : c;
    const uint4 u = *reinterpret_cast<const uint4*>(src + 16 * cc);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t o[4];
      spread(w[x], o);
      o[0] = bmul2(o[0], fa[x]);
      o[1] = bmul2(o[1], fa[x]);
      o[2] = bmul2(o[2], fb[x]);
      o[3] = bmul2(o[3], fb[x]);
      if (CF == CF_MX && big) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = bmul2(o[e], ma[x]);
      }
      const int piece = 4 * cc + x;                      // of the row's D/8
      *reinterpret_cast<uint4*>(out + (piece >> 3) * (KEYS * 128) + (((piece & 7) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Row `row` of a tile of q, in the order of K's columns.
template <int D>
__device__ __forceinline__ void put_query(uint8_t* dst, int row, const uint16_t* src, uint32_t flip, uint32_t keep) {
  uint8_t* const out = dst + row * 128;
#pragma unroll
  for (int w = 0; w < D / 32; ++w)
#pragma unroll
    for (int h = 0; h < 2; ++h) {                        // elements 32w + 8h + 0..7 and 16 on: words of t = 2h, 2h + 1
      uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
      if (src) {
        a = *reinterpret_cast<const uint4*>(src + 32 * w + 8 * h);
        b = *reinterpret_cast<const uint4*>(src + 32 * w + 8 * h + 16);
      }
      const uint32_t ax[4] = {a.x, a.y, a.z, a.w}, bx[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = (__byte_perm(ax[2 * k + e / 2], bx[2 * k + e / 2], e & 1 ? 0x7632 : 0x5410) ^ flip) & keep;
        const int piece = (D / 32) * (2 * h + k) + w;
        *reinterpret_cast<uint4*>(out + (piece >> 3) * (KEYS * 128) + (((piece & 7) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
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
// bits i of a word with base + i < n
__device__ __forceinline__ uint32_t below(int n, int base) {
  const int k = n - base;
  return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
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
  uint64_t* const raw_full = bars;             // [RAW] codes have landed
  uint64_t* const raw_empty = bars + RAW;      // [RAW] and been read (2 warps)
  uint64_t* const k_full = bars + 2 * RAW;     // [2] operand written (4 warps)
  uint64_t* const k_empty = k_full + 2;        // [2] and multiplied
  uint64_t* const v_full = k_full + 4;
  uint64_t* const v_empty = k_full + 6;
  uint64_t* const s_full = k_full + 8;         // [2] row tile's scores are there
  uint64_t* const p_full = k_full + 10;        // [2] and its probabilities (4 warps)
  uint64_t* const o_full = k_full + 12;        // [2] and its output
  uint64_t* const q_full = k_full + 14;        // [2] q is there (4 warps; only where the row tile has rows)
  uint64_t* const drain = k_full + 16;
  uint2* const flags = reinterpret_cast<uint2*>(sm + C::OFF_FLAGS);
  uint32_t* const absent = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC);      // [RAW]
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC + 16);
  int* const abort_flag = reinterpret_cast<int*>(sm + C::OFF_MISC + 20);
  int* const wsum = reinterpret_cast<int*>(sm + C::OFF_MISC + 32);             // [16]
  int* const pre = reinterpret_cast<int*>(sm + C::OFF_PRE);
  const AbortCtl ac{abort_flag, p.status, p.timeout_ns};

  griddep_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < RAW; ++i) { mbar_init(raw_full + i, 1); mbar_init(raw_empty + i, 2); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4); mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 4); mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1); mbar_init(p_full + i, 4);
      mbar_init(o_full + i, 1); mbar_init(q_full + i, 4);
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
  Walk w(p, pre, chunk, works ? sh.first(blockIdx.x) : 0, works ? sh.first(blockIdx.x + 1) : 0);

  if (warp < 8) {
    // ============================================================ softmax, a row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int rt = warp >> 2, rl = threadIdx.x & 127;
    const uint32_t tl = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t tS = tl + C::T_S + 128 * rt, tO = tl + C::T_O + D * rt;
    uint32_t n = 0, pieces = 0, slot = 0;      // tiles and pieces of this row tile, tiles of the CTA
    int4 start = make_int4(-1, 0, 0, 0);
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
      return __all_sync(0xFFFFFFFFu, mbar_wait<false>(bar, parity, ac));
    };
    while (ok && w.next(p)) {
      const Span& sp = w.sp;
      const int b = w.vb / p.CT, row = (w.vb - b * p.CT) * ROWS + 128 * rt + rl;
      const bool active = sp.rows > 128 * rt, valid = 128 * rt + rl < sp.rows;
      const int i = row / p.G, h = w.hkv * p.G + row - i * p.G;
      const int T = w.t1 - w.t0;
      if (active && T > 0) {
        put_query<D>(sm + C::OFF_Q + rt * C::TILE, rl, valid ? p.q + b * p.qs.b + i * p.qs.s + h * p.qs.h : nullptr,
                     p.q_sign < 0.f ? 0x80008000u : 0u, p.q_sign == 0.f ? 0u : 0xFFFFFFFFu);
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_elect(q_full + rt);
      }
      if (w.begins() && !w.ends()) start = make_int4(w.vb * p.c.Hkv + w.hkv, sh.of(w.lo + w.rest - 1), sp.qlen, sp.len);
      const int lim = !valid ? 0 : p.causal ? max(0, sp.len - sp.qlen + i + 1) : sp.len;
      const int wlo = p.window ? lim - p.window : 0;
      float M = NONE;
      uint64_t l2 = pk2(0.f, 0.f), l3 = l2;
      if (!active) { slot += T; continue; }
      for (int j = 0; j < T; ++j, ++n, ++slot) {
        const int k0 = sp.at(w.t0 + j) * KEYS;
        ok = wait(s_full + rt, n & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t raw[128];
        float bm[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_max(tS + 32 * c, raw + 32 * c, bm[c]);
        const uint4 fl0 = *reinterpret_cast<const uint4*>(flags + 4 * (slot & 3)), fl1 = *reinterpret_cast<const uint4*>(flags + 4 * (slot & 3) + 2);
        const uint32_t gone[4] = {fl0.x, fl0.z, fl1.x, fl1.z}, nans[4] = {fl0.y, fl0.w, fl1.y, fl1.w};
        const bool told = (fl0.x | fl0.y | fl0.z | fl0.w | fl1.x | fl1.y | fl1.z | fl1.w) != 0;
        tc_wait_ld();
        // the keys that the row does not see (all rows of a warp go along)
        if (__any_sync(0xFFFFFFFFu, told || k0 + KEYS > lim || (k0 < wlo && k0 + KEYS > p.sinks))) {
          uint32_t bad = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int base = k0 + 32 * c;
            uint32_t seen = below(lim, base) & ~gone[c];
            if (p.window) seen &= ~below(wlo, base) | below(p.sinks, base);
            bad |= seen & nans[c];
            float m = NONE;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(seen >> e & 1)) raw[32 * c + e] = 0xFF800000u;
              m = fmaxf(m, __uint_as_float(raw[32 * c + e]));
            }
            bm[c] = m;
          }
          if (bad) l2 = pk2(__uint_as_float(0x7FC00000u), 0.f);
        }
        const float x = fmaxf(fmaxf(bm[0], bm[1]), fmaxf(bm[2], bm[3])) * p.scale_log2;
        float alpha = 1.f;
        if (M == NONE) {
          M = x;
        } else if (x - M > LAZY) {
          alpha = ex2_approx(M - x);
          M = x;
          l2 = ffma2(l2, pk2(alpha, alpha), pk2(0.f, 0.f));
          l3 = ffma2(l3, pk2(alpha, alpha), pk2(0.f, 0.f));
        }
        // (the scores of this tile are there, so the products of the tile before are done)
        if (j > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            TmemLd<16>::run(tO + c, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            TmemSt<16>::run(tO + c, o);
          }
        }
        const float nM = M == NONE ? 0.f : -M;           // no key yet: every score is -inf, every weight 0
        const uint64_t c2 = pk2(p.scale_log2, p.scale_log2), nM2 = pk2(nM, nM);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a, bb;
            upk2(ffma2(pk2(__uint_as_float(raw[32 * c + 2 * e]), __uint_as_float(raw[32 * c + 2 * e + 1])), c2, nM2), a, bb);
            a = ex2_approx(a);
            bb = ex2_approx(bb);
            if (e & 1) l3 = fadd2(l3, pk2(a, bb));
            else l2 = fadd2(l2, pk2(a, bb));
            pw[e] = cvt_bf16x2(a, bb);
          }
          TmemSt<16>::run(tS + 16 * c, pw);
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
      const bool whole = w.begins() && w.ends(), none = l == 0.f;
      const float inv = whole ? (none ? 0.f : SHIFT_UP / l) : SHIFT_UP;
      const Out out = out_of(p, b, w.hkv, row);
      float* const part = p.partials + (int64_t)(2 * blockIdx.x + (w.begins() ? 1 : 0)) * C::PART;
#pragma unroll
      for (int y = 0; y < D / 64; ++y) {
        uint32_t o[8][8];
        if (T > 0) {
#pragma unroll
          for (int g = 0; g < 8; ++g) TmemLd<8>::run(tO + 8 * (g * (D / 64) + y), o[g]);
          tc_wait_ld();
        }
        if (!valid) continue;
        // dim 64y + 2g + {0, 32, 1, 33, 16, 48, 17, 49} of each eight
        constexpr int FROM[4][2] = {{0, 2}, {4, 6}, {1, 3}, {5, 7}};
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int g = 0; g < 8; g += 2) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (T > 0 && !(whole && none))
              v = make_float4(__uint_as_float(o[g][FROM[s][0]]) * inv, __uint_as_float(o[g][FROM[s][1]]) * inv,
                              __uint_as_float(o[g + 1][FROM[s][0]]) * inv, __uint_as_float(o[g + 1][FROM[s][1]]) * inv);
            const int d = 64 * y + 16 * s + 2 * g;
            if (whole) put4(p, out.at + d, v);
            else *reinterpret_cast<float4*>(part + (128 * rt + rl) * D + d) = v;
          }
      }
      if (valid) {
        if (!whole) {
          part[ROWS * D + 128 * rt + rl] = M;
          part[ROWS * (D + 1) + 128 * rt + rl] = l;
        } else if (p.lse) {
          p.lse[out.lse_at] = none ? NONE : (M + log2f(l)) * 0.69314718055994530942f;
        }
      }
      tc_fence_before();
    }
    if (threadIdx.x == 0 && !p.whole) p.starts[blockIdx.x] = ok ? start : make_int4(-1, 0, 0, 0);
  } else if (warp < 12) {
    // ============================================================ operands from codes, a key a thread
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const int dw = warp - 8, row = 32 * dw + lane;
    uint32_t n = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, ac)); };
    while (ok && w.next(p)) {
      for (int t = w.t0; t < w.t1; ++t, ++n) {
        const int k0 = w.sp.at(t) * KEYS;
        const uint32_t half = 2 * n + (dw >> 1), rs = half % RAW, kb = n & 1;
        ok = wait(raw_full + rs, (half / RAW) & 1) && (n < 2 || wait(k_empty + kb, (n / 2 - 1) & 1));
        if (!ok) break;
        const int grp = 2 * (dw & 1) + (lane >> 4);      // of the stage's four
        const bool gone = (absent[rs] >> grp & 1) || k0 + row >= w.sp.kmax;
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
        bool nan = false;
#pragma unroll
        for (int i = 0; i < Gr::SB; ++i) {
          const uint32_t byte = (vs[i / 4] >> (8 * (i % 4))) & 0xFFu;
          nan |= CF == CF_MX ? byte == 0xFFu : (byte & 0x7Fu) == 0x7Fu;
        }
        const uint32_t gones = __ballot_sync(0xFFFFFFFFu, gone), nans = __ballot_sync(0xFFFFFFFFu, nan && !gone);
        if (lane == 0) flags[4 * (n & 3) + dw] = make_uint2(gones, nans);
        put_operand<D, CF, false>(sm + C::OFF_K + kb * C::TILE, row, base + Gr::K + (lane & 15) * (D / 2), ks, gone);
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_elect(k_full + kb);
        ok = n < 2 || wait(v_empty + kb, (n / 2 - 1) & 1);
        if (!ok) break;
        put_operand<D, CF, true>(sm + C::OFF_V + kb * C::TILE, row, base + Gr::V + (lane & 15) * (D / 2), vs, gone);
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_elect(v_full + kb);
        mbar_arrive_elect(raw_empty + rs);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 12) {
      // ========================================================== copies: 16 groups of 16 keys at a time
      uint32_t n = 0;                          // stages
      bool ok = true;
      while (ok && w.next(p)) {
        const int b = w.vb / p.CT;
        const uint8_t* const head = p.c.pages + ((int64_t)w.hkv << (p.c.page_shift - 4)) * Gr::BYTES;
        const int32_t* const table = p.table + (int64_t)b * p.max_pages;
        // the page of lane's group of tiles t .. t + 3 (-1: none)
        auto look_up = [&](int t) {
          const int v = t + (lane >> 3), pos = w.sp.at(v) * KEYS + 16 * (lane & 7);
          int page = -1;
          if (v < w.t1 && pos < w.sp.kmax) {
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
            ok = n < RAW || __all_sync(0xFFFFFFFFu, mbar_wait(raw_empty + rs, (n / RAW - 1) & 1, ac));
            if (!ok) break;
            const uint32_t four = here >> (4 * x) & 15u;
            if (lane == 0) {
              absent[rs] = four ^ 15u;
              mbar_expect_tx(raw_full + rs, __popc(four) * Gr::BYTES);
            }
            __syncwarp();
            if ((lane >> 2) == x && page >= 0) {
              const int pos = w.sp.at(t + (lane >> 3)) * KEYS + 16 * (lane & 7);
              const int inside = (pos & ((1 << p.c.page_shift) - 1)) / 16;
              bulk_load(sm + C::OFF_RAW + rs * C::STAGE + (lane & 3) * Gr::BYTES, head + page * p.c.page_bytes + inside * Gr::BYTES,
                        Gr::BYTES, raw_full + rs);
            }
            __syncwarp();
          }
        }
      }
      // the copies in flight end before the CTA does
      for (uint32_t x = n > RAW ? n - RAW : 0; x < n; ++x) mbar_drain(raw_full + x % RAW, (x / RAW) & 1, ac);
    } else if (warp == 13) {
      // ========================================================== products
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, mbar_wait<false>(bar, parity, ac)); };
      const uint32_t sQ = smem_u32(sm + C::OFF_Q), sK = smem_u32(sm + C::OFF_K), sV = smem_u32(sm + C::OFF_V);
      uint32_t n = 0, nq[2] = {0, 0}, np[2] = {0, 0};
      bool ok = true;
      auto scores = [&](int rt, uint32_t kb) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = (i / 4) * C::ATOM + (i % 4) * 32;
          mma_f16_ss_p(elect_u32(), tbase + C::T_S + 128 * rt, smem_desc(sQ + rt * C::TILE + off, 16, 1024, 2),
                       smem_desc(sK + kb * C::TILE + off, 16, 1024, 2), idesc_f16_bf16(128), i > 0);
        }
        tc_commit_p(elect_u32(), s_full + rt);
      };
      auto products = [&](int rt, uint32_t vb, bool more) {
#pragma unroll
        for (int i = 0; i < KEYS / 16; ++i)              // V is MN-major: 64 dims an atom, 8 keys 1024 bytes
          mma_f16_ts_p(elect_u32(), tbase + C::T_O + D * rt, tbase + C::T_S + 128 * rt + 8 * i,
                       smem_desc(sV + vb * C::TILE + 2048 * i, C::ATOM, 1024, 2), idesc_f16_bf16(D) | 1u << 16, more || i > 0);
      };
      while (ok && w.next(p)) {
        const int T = w.t1 - w.t0, tiles = w.sp.rows > 128 ? 2 : 1;
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
          for (int rt = 0; ok && rt < tiles; ++rt) {
            ok = wait(p_full + rt, np[rt] & 1);
            if (!ok) break;
            ++np[rt];
            tc_fence_after();
            products(rt, n & 1, j > 0);
            if (j + 1 < T) {
              if (rt == 0) ok = wait(k_full + ((n + 1) & 1), ((n + 1) / 2) & 1);
              if (!ok) break;
              tc_fence_after();
              scores(rt, (n + 1) & 1);
            } else {
              tc_commit_p(elect_u32(), o_full + rt);
            }
          }
          if (!ok) break;
          tc_commit_p(elect_u32(), v_empty + (n & 1));
          if (j + 1 < T) tc_commit_p(elect_u32(), k_empty + ((n + 1) & 1));
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
// begins in CTA c and goes on, 32 rows of it: CTA c's second part and the first part of each
// later CTA up to the last.  A warp a row, a lane D/32 dims.
constexpr int JOIN_ROWS = 32, JOIN_THREADS = 256;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) cache_chunk_join_kernel(const CacheAttnArgs p) {
  constexpr int PART = ROWS * (D + 2), PER = D / 32;
  griddep_launch();
  griddep_wait();                              // the first kernel's results are complete
  const int4 st = p.starts[blockIdx.x];        // segment, last CTA, its rows' tokens, its keys
  if (st.x < 0) return;
  const int lane = threadIdx.x & 31, vb = st.x / p.c.Hkv, hkv = st.x - vb * p.c.Hkv, b = vb / p.CT;
  const int n = st.y - (int)blockIdx.x + 1;
  const float* const parts = p.partials + (int64_t)2 * blockIdx.x * PART;
  auto part = [&](int k) { return parts + (k == 0 ? (int64_t)PART : (int64_t)2 * k * PART); };
  const int rows = min(ROWS, st.z * p.G - (vb - b * p.CT) * ROWS);
  for (int r = blockIdx.y * JOIN_ROWS + threadIdx.x / 32; r < min(rows, ((int)blockIdx.y + 1) * JOIN_ROWS); r += JOIN_THREADS / 32) {
    float m = NONE;
    for (int k = lane; k < n; k += 32) m = fmaxf(m, part(k)[ROWS * D + r]);
#pragma unroll
    for (int x = 16; x; x /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    float l = 0.f, o[PER] = {};
    for (int k0 = 0; k0 < n; k0 += 32) {
      float f = 0.f;
      if (k0 + lane < n) {
        const float* const pk = part(k0 + lane);
        const float mk = pk[ROWS * D + r], lk = pk[ROWS * (D + 1) + r];
        f = lk == 0.f ? 0.f : exp2f(mk - m);
        l = fmaf(f, lk, l);
      }
#pragma unroll 8
      for (int k = 0; k < min(32, n - k0); ++k) {
        const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
        const float* const src = part(k0 + k) + r * D + PER * lane;
        float v[PER];
        if constexpr (PER == 4) {
          const float4 u = *reinterpret_cast<const float4*>(src);
          v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
        } else {
          const float2 u = *reinterpret_cast<const float2*>(src);
          v[0] = u.x; v[1] = u.y;
        }
        if (fk != 0.f) {                       // (a part that saw nothing counts nothing)
#pragma unroll
          for (int e = 0; e < PER; ++e) o[e] = fmaf(fk, v[e], o[e]);
        }
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
    if (lane == 0 && p.lse) p.lse[out.lse_at] = none ? NONE : (m + log2f(l)) * 0.69314718055994530942f;
  }
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

// Segments of at most 4 tiles are not shared: a CTA each, no second kernel.
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
