// fsa_append_rope.cu -- the projection's q, k and v of new tokens on their way to the attention:
// q normalised, rotated and written as bf16, k normalised, rotated and put into the 4-bit cache
// beside v, in one pass.
//
// q is that of fsa_qk_norm_rope, bit for bit, v that of fsa_cache_append.  k is rounded once:
// its codes and scales are those of the exact values
//   y = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = pos * inv_freq
// (through bf16 they would be rounded twice).  They are computed in fp32, whose error is
// known: with Y the row's largest |y|, |a| + |b| <= 2 Y for every pair; the angle is off by at most 2^-23.3 (a part of
// a turn by 2^-26, for positions up to 2^24), cos and sin by an ulp, 2^-24, their products with the weights and
// the two products of a pair by 2^-24 each: 2^-21.1 Y together.  The norm's factor is off by 2^-21.7 of y (seven additions
// on the way to a sum of exact squares, half of that, and 2^-23.4), a quotient by an E4M3 scale by 2^-22.4, the two
// below by 2^-24: in all 1.05 2^-20 Y.  So each block is rounded twice, from y - 1.25 2^-20 Y and from y + 1.25 2^-20 Y;
// where scale and codes agree, as in all but about one warp in 150, they are the exact ones, and what is left open
// is computed again to 2^-43.  Elements that neither a norm nor an angle touches are
// exact as they are, and rounded as fsa_cache_append does.
//
// To move: 4 H + 4 Hkv + 2 Hkv (0.53 or 0.56) bytes a token and dim.  A block has the queries of a few
// tokens or the keys and values of a few: the sines of a token are computed once a block, for the rows of q (D/16
// lanes each, both elements of a pair in a lane) or of k (D/8 lanes, 8 consecutive elements a lane, as the
// quantisation wants them; a pair's other element comes from another lane).
//
// Measured (one GB300, calls in a graph, 32+8 heads of 128, NVFP4, against fsa_qk_norm_rope and fsa_cache_append in
// turn): 64 tokens 5.7 to 7.2 us (5.8; by whether a warp has something open), 512 8.3 (9.7), 1024 11.5 (11.9), 2048 17.7
// (15.4), 16384 93.8 (76.2), where memory takes 52; 16384 tokens of 8+8 heads 73.6 (47.2).  From about a
// thousand tokens on it is bound by instructions, 61.5 M a warp for 16384 tokens, 2.3 of 4 a cycle: half of them turn the
// keys, whose two roundings and whose register need beside the rare ways cost what the saved pass over k gives; the
// codes are those of the exact keys, which the two calls' are not.  Rows that all go through fp64 (NaN, or far over
// ordinary size) take 3.9 ms.
#include <algorithm>
#include "fsa_cache_codes.cuh"
#include "fsa_rope.cuh"

namespace fsa {
namespace {

constexpr float SURE = 0x1.4p-20f;      // of a row's largest |y|: more than the fp32 arithmetic is off by
// Blocks of an SM: where there are more than run at once (16384 tokens, 32+8 heads: 12 96.2 us, 11 97.4, 10 99.0; 80
// registers and some spills), and where all do (no spills: 64 tokens 5.7 us instead of 6.1).
constexpr int APPEND_MANY = 12, APPEND_FEW = 8;

struct Place {
  int pos;             // what it turns by, if no positions are given
  bool live;           // a row of its sequence
  uint8_t* group;      // head 0 of its group of the cache, or null; `row` of its 16
  int row;
};

// Token tok (of B * S): where it goes.  look: its page is wanted.
__device__ __forceinline__ Place place_of(const AppendRopeArgs& a, uint32_t tok, int group_bytes, bool look) {
  const int b = (int)(tok / (uint32_t)a.r.S), s = (int)(tok - (uint32_t)b * (uint32_t)a.r.S);
  const int fresh = a.which ? min(max(a.which[b], 0), a.r.S) : a.r.S;
  const int64_t at = (int64_t)a.lens[b] - fresh + s;
  Place p{(int)max(at, (int64_t)INT32_MIN), s < fresh, nullptr, (int)(at & 15)};
  if (!look || !p.live || at < 0) return p;
  const int64_t pi = at >> a.c.page_shift;
  if (pi >= a.max_pages) return p;
  const int page = a.table[(int64_t)b * a.max_pages + pi];
  if (page < 0 || page >= a.c.num_pages) {
    if (a.status) atomicExch(a.status, -1);       // FSA_ERR_INVALID_ARG
    return p;
  }
  p.group = a.c.pages + page * a.c.page_bytes + ((int)(at & ((1 << a.c.page_shift) - 1)) / 16) * (int64_t)group_bytes;
  return p;
}

// What a lane of a key's row has: 8 consecutive elements, in two fours; each four turns as a whole
// (half is a multiple of 4): with which pairs, and on which side of them.
struct Lane8 {
  f2 own[4], other[4];       // an element is multiplied by own, its pair's other one by other
  uint32_t turned;           // bit u: four u turns
  bool exact;                // no element of the lane is touched
};

template <bool INTER>
__device__ __forceinline__ void pair_of(int e, int half, int& pair, int& other, bool& second) {
  if (INTER) { pair = e >> 1; other = e ^ 1; second = e & 1; }
  else { second = e >= half; pair = second ? e - half : e; other = second ? e - half : e + half; }
}

template <int D, bool INTER>
__device__ __forceinline__ void set_lane(Lane8& f, const RopeArgs& a, const float2* sines, int l) {
  f.turned = 0;
  bool still = true;
  float own[8], by[8];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e0 = 8 * l + 4 * u;
    const bool turns = e0 < 2 * a.half;
    f.turned |= turns ? 1u << u : 0u;
#pragma unroll
    for (int e = 4 * u; e < 4 * u + 4; ++e) {
      const float w = a.wk ? bf16_to_f32(a.wk[8 * l + e]) : 1.f;
      own[e] = w;
      by[e] = 0.f;
      if (turns) {
        int pair, other;
        bool second;
        pair_of<INTER>(8 * l + e, a.half, pair, other, second);
        const float2 t = sines[pair];
        const float wo = a.wk ? bf16_to_f32(a.wk[other]) : 1.f;
        own[e] = w * t.x;
        by[e] = second ? wo * t.y : -wo * t.y;
        still &= t.x == 1.f && t.y == 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.own[i] = make(own[2 * i], own[2 * i + 1]);
    f.other[i] = make(by[2 * i], by[2 * i + 1]);
  }
  f.exact = !a.norm && still;
}

// The other elements of the pairs of a lane's eight, from the lanes of the row that have them.
template <int D, bool INTER>
__device__ __forceinline__ uint4 others_of(uint4 x, int half, int row, int l) {
  if constexpr (INTER) {
    return make_uint4(__funnelshift_l(x.x, x.x, 16), __funnelshift_l(x.y, x.y, 16), __funnelshift_l(x.z, x.z, 16),
                      __funnelshift_l(x.w, x.w, 16));
  } else {
    const int hq = half / 4;
    const bool flip = hq & 1;
    uint4 r;
    // four u of this lane takes four 2l + u +- hq, whose place in its lane is u or, flipped, the other
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int su = 2 * l + u, from = su < hq ? su + hq : su < 2 * hq ? su - hq : su;
      const bool high = flip ? u == 0 : u == 1;
      const uint32_t a = __shfl_sync(0xFFFFFFFFu, high ? x.z : x.x, row + from / 2);
      const uint32_t b = __shfl_sync(0xFFFFFFFFu, high ? x.w : x.y, row + from / 2);
      if (u == 0) { r.x = a; r.y = b; } else { r.z = a; r.w = b; }
    }
    return r;
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }

// What the fp32 values of a lane's eight say of their codes.
struct Codes {
  uint32_t codes, sb;
  uint32_t open;       // nibbles that the values' error leaves open
  bool scale_open;     // whether it leaves the block's scale open
};

constexpr float SIXTH = 0.16666667163372039795f;      // (half an ulp over 1/6)
constexpr float RAISE = 1.0f + 0x1p-20f, ABOVE = 1.0f + 0x1p-22f, BELOW = 1.0f - 0x1p-22f;

// The scale byte of a block whose maximum lies in tlo .. thi, and whether that leaves it open.
template <int CF>
__device__ __forceinline__ void scale_of(float tlo, float thi, Codes& r) {
  if constexpr (CF == CF_MX) {
    const uint32_t m = __float_as_uint(thi) >> 23;               // exponent, less 2 (zero and subnormal: 0)
    r.sb = (uint32_t)max((int)m - 2, 0);
    r.scale_open = m >= 0xFF || r.sb != (uint32_t)max((int)(__float_as_uint(tlo) >> 23) - 2, 0);
  } else {
    // (known: raised by 2^-20 and cut, ties stay ties, fsa_cache_codes.cuh)
    const bool known = thi == tlo;
    r.sb = cvt_e4m3x2(known ? cut12(thi * (SIXTH * RAISE)) : thi * (SIXTH * ABOVE), 0.f) & 0xFFu;
    r.scale_open = !(thi < 3e38f) || (!known && r.sb != (cvt_e4m3x2(tlo * (SIXTH * BELOW), 0.f) & 0xFFu));
  }
}
// What quotients by it are: a factor (0 for a zero scale, whose codes are zeros without signs)
template <int CF>
__device__ __forceinline__ float quotient_of(uint32_t sb) {
  if constexpr (CF == CF_MX) return __uint_as_float((254u - min(sb, 253u)) << 23);
  const float s = e4m3_to_f32(sb);
  float mul;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(mul) : "f"(s));
  return s > 0.f ? mul : 0.f;
}

// The codes of 8 values rs (y +- d) of a lane under the block's scale.
template <int CF>
__device__ __forceinline__ void codes_of(const f2 (&y)[4], float d, float rs, Codes& r) {
  // (finite for a row of zeros too, whose scale is the least)
  const float mul = fminf(quotient_of<CF>(r.sb) * rs, 3.4e38f), dm = d * mul;
  const f2 m2 = make(mul, mul), lo2 = make(-dm, -dm), hi2 = make(dm, dm);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    split(fma(y[i], m2, lo2), lo[2 * i], lo[2 * i + 1]);
    split(fma(y[i], m2, hi2), hi[2 * i], hi[2 * i + 1]);
  }
  r.codes = cvt_e2m1x8(hi);
  r.open = r.codes ^ cvt_e2m1x8(lo);
  if (CF == CF_NV && mul == 0.f) r.codes = r.open = 0u;
}

// The same where the values are as they are (and rs is 1): ties stay ties.
template <int CF>
__device__ __forceinline__ void codes_of_exact(const f2 (&y)[4], Codes& r) {
  const float mul = quotient_of<CF>(r.sb) * (CF == CF_NV ? RAISE : 1.f);
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(y[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = CF == CF_NV ? cut12(x[e] * mul) : x[e] * mul;
  r.codes = cvt_e2m1x8(x);
  r.open = 0u;
  if (CF == CF_NV && mul == 0.f) r.codes = 0u;
}

// Taylor's coefficients of sin(x) / x and cos(x) over x^2, from the last one that counts on [-pi/4, pi/4]
__constant__ double SERIES[8][2] = {{-1.0 / 1307674368000.0, -1.0 / 87178291200.0}, {1.0 / 6227020800.0, 1.0 / 479001600.0},
                                    {-1.0 / 39916800.0, -1.0 / 3628800.0}, {1.0 / 362880.0, 1.0 / 40320.0}, {-1.0 / 5040.0, -1.0 / 720.0},
                                    {1.0 / 120.0, 1.0 / 24.0}, {-1.0 / 6.0, -0.5}, {1.0, 1.0}};
__constant__ float BORDERS[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};       // of E2M1; a tie goes up at every second

// cos and sin of t (|t| below 2^51): quarter turns taken off with pi / 2 as two doubles, then the series.
__device__ __forceinline__ void cos_sin64(double t, double& c, double& s) {
  constexpr double HALF_PI = 1.5707963267948965580, REST = 6.1232339957367658861e-17;       // their sum: pi / 2
  const double k = rint(t * 0.63661977236758138243);
  const double x = ::fma(-k, REST, ::fma(-k, HALF_PI, t)), z = x * x;
  double p = 0.0, q = 0.0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    p = ::fma(p, z, SERIES[i][0]);
    q = ::fma(q, z, SERIES[i][1]);
  }
  p *= x;
  const int quarter = (int)((long long)k & 3);
  c = quarter & 1 ? p : q;
  s = quarter & 1 ? q : p;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter & 2) s = -s;
}

// A value as the sum of two floats, the second below half an ulp of the first.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two sum2(float h, float l) {        // |h| >= |l|
  const float s = h + l;
  return {s, l - (s - h)};
}
__device__ __forceinline__ bool over(Two a, Two b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }
// n 2^-63
__device__ __forceinline__ Two fraction63(uint64_t n) {
  const float h = (float)n;                                      // (2^63 at most)
  return {h * 0x1p-63f, (float)(int64_t)(n - (uint64_t)h) * 0x1p-63f};
}

// cos and sin of p * freq to 2^-42, in integers: freq / 2 pi with 96 fraction bits times p leaves the turn's 64;
// quarter turns taken off, the rest times 2 pi is x <= pi / 4 with 63, and Taylor's series with x^2 as a
// fraction of 64, term after term from below.
__device__ __forceinline__ void cos_sin63(int p, double freq, Two& c, Two& s) {
  const uint64_t bits = (uint64_t)__double_as_longlong(freq);
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const int down = 1075 - 30 - (int)(bits >> 52 & 0x7FF);        // freq = m 2^(-30 - down)
  const unsigned __int128 q = (unsigned __int128)m * 0xA2F9836E4E44152Aull;               // 2^66 / 2 pi
  // (of a frequency of 2^23 and more whole turns are cut off on the left)
  const unsigned __int128 turn96 = down >= 128 || down <= -128 ? 0 : down >= 0 ? q >> down : q << -down;
  const uint64_t turn = (uint64_t)((turn96 * (p < 0 ? 0u - (uint32_t)p : (uint32_t)p)) >> 32);
  const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(turn - ((uint64_t)quarter << 62));
  const uint64_t x = __umul64hi((uint64_t)llabs(rest) * 4, 0xC90FDAA22168C235ull);          // pi / 4
  const uint64_t z = __umul64hi(x, x) << 2;
  constexpr uint64_t ONE = 1ull << 63;
  uint64_t a = ONE / 39916800 - __umul64hi(ONE / 6227020800ull, z), b = ONE / 479001600 - __umul64hi(ONE / 87178291200ull, z);
  a = ONE / 362880 - __umul64hi(a, z);  b = ONE / 3628800 - __umul64hi(b, z);
  a = ONE / 5040 - __umul64hi(a, z);    b = ONE / 40320 - __umul64hi(b, z);
  a = ONE / 120 - __umul64hi(a, z);     b = ONE / 720 - __umul64hi(b, z);
  a = ONE / 6 - __umul64hi(a, z);       b = ONE / 24 - __umul64hi(b, z);
  a = ONE - __umul64hi(a, z);           b = ONE / 2 - __umul64hi(b, z);
  b = ONE - __umul64hi(b, z);
  a = __umul64hi(a, x) << 1;
  Two sn = fraction63(a), co = fraction63(b);
  if (rest < 0) sn = {-sn.h, -sn.l};
  c = quarter & 1 ? sn : co;
  s = quarter & 1 ? co : sn;
  if ((quarter & 3) == 1 || (quarter & 3) == 2) c = {-c.h, -c.l};
  if (((quarter & 2) != 0) != ((p < 0) != (freq < 0.0))) s = {-s.h, -s.l};
}

// 1 / sqrt(x), whatever its size
__device__ __noinline__ double rsqrt64(double x) { return 1.0 / sqrt(x); }

// The scale byte of a block with maximum `top`, as the definition has it.
template <int CF>
__device__ __noinline__ uint32_t scale64(double top, bool finite) {
  if constexpr (CF == CF_MX) {
    const int e = min(max((int)((uint32_t)__double2hiint(top) >> 20 & 0x7FF) - 1023 - 2, -127), 127);
    return finite ? (uint32_t)(e + 127) : 0xFFu;
  } else {
    const double t = fmin(top / 6.0, 448.0);
    const int ex = max((int)((uint32_t)__double2hiint(t) >> 20 & 0x7FF) - 1023, -6);
    const double n = rint(t * __hiloint2double((1023 + 3 - ex) << 20, 0));              // 8..16 steps, or fewer when subnormal
    return !finite ? 0x7Fu : (uint32_t)(n < 8.0 ? n : (ex + 7) * 8 + n - 8.0);
  }
}

// 16 bits on to the next element
__device__ __forceinline__ void next_element(uint4& w) {
  w.x = __funnelshift_r(w.x, w.y, 16);
  w.y = __funnelshift_r(w.y, w.z, 16);
  w.z = __funnelshift_r(w.z, w.w, 16);
  w.w = __funnelshift_r(w.w, w.x, 16);
}

// The codes that are open (and all of a block whose scale is) in fp64 from the definition, for values of any
// size; all lanes of a warp, D/8 a row.  An fp64 operation that waits for the one before takes 75 to 110 cycles
// here, so this is for the rows that close_codes does not take.
template <int D, bool INTER, int CF>
__device__ __noinline__ Codes close_codes64(const RopeArgs& a, uint4 own, uint4 others, const int32_t* pos, int place, int l, Codes r) {
  constexpr int L = D / 8, PER = CF == CF_MX ? 4 : 2;
  double rr = 1.0;
  if (a.norm) {
    double ss = 0.0;
    uint4 w = own;
#pragma unroll 1
    for (int e = 0; e < 8; ++e, next_element(w)) {
      const double x = lo_bf16(w.x);
      ss = ::fma(x, x, ss);
    }
#pragma unroll 1
    for (int m = 1; m < L; m *= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, m);
    const double mean = ::fma(ss, 1.0 / D, (double)a.eps);
    if (mean > 0x1p-90 && mean < 0x1p100) {
      const double y = (double)rsqrtf((float)mean), e = ::fma(-mean * y, y, 1.0);      // |e| < 2^-20: the next term is e^3
      rr = ::fma(y * e, ::fma(0.375, e, 0.5), y);
    } else {
      rr = rsqrt64(mean);
    }
  }
  const uint32_t open = r.scale_open ? 0xFFFFFFFFu : r.open;
  double top = 0.0;
  bool finite = true;
  // a first time for the block's maximum, where its scale is open, then for the codes
#pragma unroll 1
  for (int pass = __any_sync(0xFFFFFFFFu, r.scale_open) ? 0 : 1; pass < 2; ++pass) {
    uint4 w = own, v = others;
    const float scale = CF == CF_MX ? __uint_as_float(min(r.sb, 254u) > 0u ? min(r.sb, 254u) << 23 : 1u << 22) : e4m3_to_f32(r.sb);
#pragma unroll 1
    for (int e = 0; e < 8; ++e, next_element(w), next_element(v)) {
      const bool mine = open >> (4 * e) & 15u;
      if (!__any_sync(0xFFFFFFFFu, mine)) continue;
      const int at = 8 * l + e;
      double y = lo_bf16(w.x);
      if (a.wk) y *= (double)bf16_to_f32(a.wk[at]);
      if (mine && at < 2 * a.half) {
        int pair, other;
        bool second;
        pair_of<INTER>(at, a.half, pair, other, second);
        double z = lo_bf16(v.x);                         // (interleaved: a word's two, exchanged)
        if (a.wk) z *= (double)bf16_to_f32(a.wk[other]);
        const int axis = pair >= a.first2 ? 2 : pair >= a.first1 ? 1 : 0;
        double sn, c;
        const int p = pos ? pos[axis] : place;
        const double t = (double)p * a.inv_freq[pair];
        if (fabs(t) >= 0x1p51 && fabs(t) < INFINITY) {    // (in fp64 its part of a turn would be lost)
          Two c2, s2;
          cos_sin63(p, a.inv_freq[pair], c2, s2);
          c = (double)c2.h + c2.l;
          sn = (double)s2.h + s2.l;
        } else {
          cos_sin64(t, c, sn);
        }
        y = ::fma(z, second ? sn : -sn, y * c);
      }
      y *= rr;
      if (pass == 0) {
        finite &= isfinite(y);
        top = fmax(top, fabs(y));
        continue;
      }
      uint32_t code = 0;
#pragma unroll 1
      for (int i = 0; i < 7; ++i) {
        const double border = (double)(BORDERS[i] * scale), m = fabs(y);                // (exact)
        code += m > border || ((i & 1) && m == border);
      }
      code |= signbit(y) ? 8u : 0u;
      if (!finite || (CF == CF_NV && scale == 0.f)) code = 0u;
      if (mine) r.codes = (r.codes & ~(15u << (4 * e))) | code << (4 * e);
    }
    if (pass == 0) {
#pragma unroll 1
      for (int m = 1; m < PER; m *= 2) {
        top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
        finite &= (bool)__shfl_xor_sync(0xFFFFFFFFu, (int)finite, m);
      }
      if (r.scale_open) r.sb = scale64<CF>(top, finite);
    }
  }
  return r;
}

// The open ones of a lane's eight again, for rows of ordinary size, in pairs of floats (about 2^-43 of a row's largest
// |y|; no fp64): their codes, or, `scales`, the byte of the block's scale, open then being those that may be its maximum.
template <int D, bool INTER, int CF>
__device__ __noinline__ Codes close_codes(const RopeArgs& a, uint4 own, uint4 others, const int32_t* pos, int place, int l, Codes r, bool scales) {
  constexpr int L = D / 8, PER = CF == CF_MX ? 4 : 2;
  Two rr{1.f, 0.f};
  if (a.norm) {
    float hi = 0.f, lo = 0.f;                            // squares of bf16 are exact in fp32; a sum and what it drops
    auto add = [&](float x) {
      const float s = hi + x, t = s - hi;
      lo += (hi - (s - t)) + (x - t);
      hi = s;
    };
    uint4 w = own;
#pragma unroll 1
    for (int e = 0; e < 8; ++e, next_element(w)) add(__fmul_rn(lo_bf16(w.x), lo_bf16(w.x)));
#pragma unroll 1
    for (int m = 1; m < L; m *= 2) {
      const float h = __shfl_xor_sync(0xFFFFFFFFu, hi, m), k = __shfl_xor_sync(0xFFFFFFFFu, lo, m);
      add(h);
      lo += k;
    }
    hi *= 1.0f / D;
    lo *= 1.0f / D;
    add(a.eps);
    const Two mean = sum2(hi, lo);
    // 1 / sqrt: y and the next term of Newton's series, e = 1 - mean y^2 exactly but for 2^-47
    const float y = rsqrtf(mean.h), y2 = y * y, y2l = fmaf(y, y, -y2), g = mean.h * y2;
    const float e = ((1.f - g) - fmaf(mean.h, y2, -g)) - fmaf(mean.h, y2l, mean.l * y2);
    rr = sum2(y, y * e * fmaf(0.375f, e, 0.5f));
  }
  Two top{0.f, 0.f};
  {
    uint4 w = own, v = others;
    const float scale = CF == CF_MX ? __uint_as_float(max(r.sb, 1u) << 23) : e4m3_to_f32(r.sb);       // (rows of ordinary size: sb > 0)
#pragma unroll 1
    for (int e = 0; e < 8; ++e, next_element(w), next_element(v)) {
      const bool mine = r.open >> (4 * e) & 15u;
      if (!__any_sync(0xFFFFFFFFu, mine)) continue;
      const int at = 8 * l + e;
      float x = lo_bf16(w.x);                            // times its weight: 16 bits
      if (a.wk) x *= bf16_to_f32(a.wk[at]);
      Two y{x, 0.f};
      if (mine && at < 2 * a.half) {
        int pair, other;
        bool second;
        pair_of<INTER>(at, a.half, pair, other, second);
        float z = lo_bf16(v.x);                          // (interleaved: a word's two, exchanged)
        if (a.wk) z *= bf16_to_f32(a.wk[other]);
        if (!second) z = -z;
        const int axis = pair >= a.first2 ? 2 : pair >= a.first1 ? 1 : 0;
        Two c, sn;
        cos_sin63(pos ? pos[axis] : place, a.inv_freq[pair], c, sn);
        const float f = x * c.h, g = z * sn.h, q = f + g, t = q - f;
        const float rest = ((f - (q - t)) + (g - t)) + (fmaf(x, c.h, -f) + fmaf(x, c.l, fmaf(z, sn.h, -g) + z * sn.l));
        y = sum2(q, rest);
      }
      const float f = y.h * rr.h;
      y = sum2(f, fmaf(y.h, rr.h, -f) + fmaf(y.h, rr.l, y.l * rr.h));
      const bool negative = signbit(y.h);
      if (negative) y = {-y.h, -y.l};
      if (scales) {
        if (mine && over(y, top)) top = y;
        continue;
      }
      uint32_t code = 0;
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        const Two border{(i < 4 ? 0.25f + 0.5f * i : i == 4 ? 2.5f : i == 5 ? 3.5f : 5.f) * scale, 0.f};        // (exact)
        code += over(y, border) || ((i & 1) && y.h == border.h && y.l == 0.f);
      }
      code |= negative ? 8u : 0u;
      if (CF == CF_NV && scale == 0.f) code = 0u;
      if (mine) r.codes = (r.codes & ~(15u << (4 * e))) | code << (4 * e);
    }
    if (scales) {
#pragma unroll 1
      for (int m = 1; m < PER; m *= 2) {
        const Two o{__shfl_xor_sync(0xFFFFFFFFu, top.h, m), __shfl_xor_sync(0xFFFFFFFFu, top.l, m)};
        if (over(o, top)) top = o;
      }
      if (r.scale_open) {
        if constexpr (CF == CF_MX) {
          const uint32_t bits = __float_as_uint(top.h);
          r.sb = (uint32_t)max((int)(bits >> 23) - ((bits & 0x7FFFFFu) == 0 && top.l < 0.f) - 2, 0);
        } else {                                         // the two E4M3 values that come into question, and their middle
          const float t = top.h * SIXTH;
          const uint32_t b0 = cvt_e4m3x2(t * BELOW, 0.f) & 0xFFu, b1 = cvt_e4m3x2(t * ABOVE, 0.f) & 0xFFu;
          const Two middle{(e4m3_to_f32(b0) + e4m3_to_f32(b1)) * 3.f, 0.f};               // (exact)
          r.sb = b0 == b1 || over(middle, top) ? b0 : over(top, middle) ? b1 : b0 & 1 ? b1 : b0;
        }
      }
    }
  }
  return r;
}

// One row of k, a lane's eight elements: its codes and scale into the cache (all lanes of a warp).  in: the row is
// there and has a place.
template <int D, bool INTER, int CF>
__device__ __forceinline__ void put_key(const AppendRopeArgs& p, const Lane8& f, uint4 ku, bool in, const int32_t* pos, int place,
                                        uint8_t* codes, uint8_t* scales) {
  using Gr = CacheGroup<D, CF>;
  constexpr int LK = D / 8, PER = CF == CF_MX ? 4 : 2;            // lanes of a row, of a block
  const RopeArgs& a = p.r;
  const int l = threadIdx.x % LK, row0 = threadIdx.x % 32 - l;
  const bool all = 2 * a.half == D;
  const uint4 others = a.half > 0 ? others_of<D, INTER>(ku, a.half, row0, l) : ku;
  const uint32_t w[4] = {ku.x, ku.y, ku.z, ku.w}, v[4] = {others.x, others.y, others.z, others.w};
  f2 y[4], sq[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 o = unpack(w[i]), z = mul(o, f.own[i]);
    sq[i] = mul(o, o);                                          // (exact)
    y[i] = fma(unpack(v[i]), f.other[i], z);
    if (!all && !(f.turned >> (i / 2) & 1)) y[i] = z;         // (an element that does not turn takes nothing of another)
  }
  float t[8], ss, s1;
#pragma unroll
  for (int i = 0; i < 4; ++i) split(y[i], t[2 * i], t[2 * i + 1]);
  // (maxima that keep NaN, of an element, a weight or an angle: the row is not sure then)
  const float own_top = max_nan(max_nan(max_nan(fabsf(t[0]), fabsf(t[1])), max_nan(fabsf(t[2]), fabsf(t[3]))),
                                max_nan(max_nan(fabsf(t[4]), fabsf(t[5])), max_nan(fabsf(t[6]), fabsf(t[7]))));
  float top = own_top;
#pragma unroll
  for (int m = 1; m < PER; m *= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));          // the block's
  float most = top;
#pragma unroll
  for (int m = PER; m < LK; m *= 2) most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, m));      // the row's
  float rs = 1.f;
  bool sure = true;
  if (a.norm) {
    split(add(add(sq[0], sq[1]), add(sq[2], sq[3])), ss, s1);
    ss += s1;
#pragma unroll
    for (int m = 1; m < LK; m *= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, m);
    const float mean = ss * (1.0f / D) + a.eps;
    rs = rsqrtf(mean);
    rs = fmaf(rs * 0.5f, fmaf(-mean * rs, rs, 1.f), rs);        // (a step of Newton's: off by 2^-23.4)
    sure = mean > 0x1p-90f && mean < 0x1p120f;                // (squares below fp32's range are nothing beside that)
  }
  sure = sure && most * rs < 0x1p120f && (most * rs > 0x1p-90f || most == 0.f);
  float d = most * SURE;
  if (!a.norm && f.exact) d = 0.f;
  // a maximum of the block lies in tlo .. thi (some lanes' values may be exact, others not)
  float tlo = fmaxf(top - d, 0.f), thi = top + d;
  if (!a.norm) {
    tlo = fmaxf(own_top - d, 0.f);
    thi = sure ? own_top + d : INFINITY;
#pragma unroll
    for (int m = 1; m < PER; m *= 2) {
      tlo = fmaxf(tlo, __shfl_xor_sync(0xFFFFFFFFu, tlo, m));
      thi = fmaxf(thi, __shfl_xor_sync(0xFFFFFFFFu, thi, m));
    }
  }
  Codes kc;
  scale_of<CF>(tlo * rs, thi * rs, kc);
  kc.scale_open = in && (kc.scale_open || !sure);
  kc.open = 0u;
  bool done = false;                                          // (for the warp)
  if (__any_sync(0xFFFFFFFFu, kc.scale_open)) {
    // (an open block far below its row's largest |y|: its elements may lie below fp32's normal range)
    const bool ordinary = !kc.scale_open || (sure && top > most * 0x1p-15f);
    done = !__all_sync(0xFFFFFFFFu, ordinary);
    if (!done) {
#pragma unroll
      for (int e = 0; e < 8; ++e) kc.open |= kc.scale_open && fabsf(t[e]) + d >= tlo ? 15u << (4 * e) : 0u;
      kc = close_codes<D, INTER, CF>(a, ku, others, pos, place, l, kc, true);
    }
  }
  if (d == 0.f && !a.norm) codes_of_exact<CF>(y, kc);
  else codes_of<CF>(y, d, rs, kc);
  if (!in) kc.open = 0u;
  if (done) {
    kc = close_codes64<D, INTER, CF>(a, ku, others, pos, place, l, kc);
  } else if (__any_sync(0xFFFFFFFFu, kc.open != 0u)) {
    kc = close_codes<D, INTER, CF>(a, ku, others, pos, place, l, kc, false);
  }
  const uint32_t kw = k_to_cache<LK>(kc.codes, row0, l);
  if (in) {
    *reinterpret_cast<uint32_t*>(codes + Gr::K) = kw;
    if (l % PER == 0) scales[0] = (uint8_t)kc.sb;
  }
}
template <int D, int CF>
__device__ __forceinline__ void put_value(uint4 vu, bool in, uint8_t* codes, uint8_t* scales) {
  using Gr = CacheGroup<D, CF>;
  constexpr int LK = D / 8, PER = CF == CF_MX ? 4 : 2;
  const int l = threadIdx.x % LK, row0 = threadIdx.x % 32 - l;
  uint32_t vsb;
  const uint32_t vw = v_to_cache<LK>(quantise8<CF>(vu, vsb), row0, l);
  if (in) {
    *reinterpret_cast<uint32_t*>(codes + Gr::V) = vw;
    if (l % PER == 0) scales[Gr::VS - Gr::KS] = (uint8_t)vsb;
  }
}

// A block has the queries of a few tokens, or the keys and values of a few more: of `groups` of kv_tokens tokens
// each, kv_tokens / tokens blocks of queries and one of keys and values.
template <int D, int P, bool INTER, int CF, int BLOCKS>
__global__ void __launch_bounds__(ROPE_THREADS, BLOCKS) append_rope_kernel(const __grid_constant__ AppendRopeArgs p, int tokens, int kv_tokens) {
  constexpr int L = D / (2 * P), GROUPS = ROPE_THREADS / L;       // lanes of a row of q
  constexpr int LK = D / 8, KGROUPS = ROPE_THREADS / LK;          // of k and v
  constexpr int PER = CF == CF_MX ? 4 : 2;                        // lanes of a block of k and v
  using Gr = CacheGroup<D, CF>;
  const RopeArgs& a = p.r;
  __shared__ __align__(16) float2 sines[ROPE_TOKENS * D / 2];     // cos, sin of [token][pair]
  griddep_launch();
  griddep_wait();
  const uint32_t total = (uint32_t)a.B * (uint32_t)a.S;
  const uint32_t per = (uint32_t)(kv_tokens / tokens) + 1, part = blockIdx.x / per, sub = blockIdx.x - part * per;
  const bool queries = sub < per - 1;
  const uint32_t first = part * (uint32_t)kv_tokens + (queries ? sub * (uint32_t)tokens : 0u);
  if (first >= total) return;
  const int ntok = (int)min((uint32_t)(queries ? tokens : kv_tokens), total - first);

  auto turn = [&] {                                               // the block's sines
    if (a.half > 0) {
      const int by = ROPE_THREADS / a.half;       // tokens at a time
      const int i = threadIdx.x % a.half;
      if ((int)threadIdx.x < by * a.half) {
        float fh, fl;
        turns_of(a.inv_freq[i], fh, fl);
        const int axis = i >= a.first2 ? 2 : i >= a.first1 ? 1 : 0;
        for (int t = threadIdx.x / a.half; t < ntok; t += by) {
          const int pos = a.pos ? a.pos[((int64_t)first + t) * a.axes + axis] : place_of(p, first + t, 0, false).pos;
          sines[t * a.half + i] = cos_sin(pos, fh, fl);
        }
      }
    }
    __syncthreads();
  };

  if (queries) {
    // this thread: lane of a row of token j, rows h, h + step, .. of its heads
    const int lane = threadIdx.x % L, group = threadIdx.x / L;
    const int step = GROUPS / tokens, j = group / step;
    const uint32_t lanes = (uint32_t)((1ull << L) - 1) << (threadIdx.x % 32 / L * L);
    const bool turns = P * lane < a.half, all = a.half == D / 2;
    const int at0 = INTER || !turns ? 2 * P * lane : P * lane;
    const int at1 = INTER || !turns ? 2 * P * lane + P : a.half + P * lane;
    const uint32_t tok = first + min(j, ntok - 1);
    const int b = (int)(tok / (uint32_t)a.S), s = (int)(tok - (uint32_t)b * (uint32_t)a.S);
    const int n = j < ntok && place_of(p, tok, 0, false).live ? a.H : 0;
    int h = group - j * step;
    const uint16_t* src = a.q + b * a.qs.b + s * a.qs.s + h * a.qs.h;
    uint16_t* dst = a.qo + b * a.qos.b + s * a.qos.s + h * a.qos.h;
    const int64_t sstep = step * a.qs.h, dstep = step * a.qos.h;
    Raw<P> x[ROPE_ROWS];
    auto load = [&] {
#pragma unroll
      for (int r = 0; r < ROPE_ROWS; ++r)
        if (h + r * step < n) x[r].load(src + r * sstep, at0, at1);
    };
    load();                                                       // on their way while the sines are computed
    turn();
    Factors<P, INTER> f;
    // (threads past the pairs hold 2P consecutive elements, unturned)
    f.set(sines + j * a.half + P * lane, turns, a.wq, at0, at1);
#pragma unroll 1
    while (h < n) {
#pragma unroll
      for (int r = 0; r < ROPE_ROWS; ++r)
        if (h + r * step < n) {
          turn_row<D, P, INTER>(x[r], f, lanes, turns, all, a.norm, a.eps);
          x[r].store(dst + r * dstep, at0, at1);
        }
      h += ROPE_ROWS * step;
      src += ROPE_ROWS * sstep;
      dst += ROPE_ROWS * dstep;
      load();
    }
    return;
  }

  // lane l of a row of token j, rows h, h + step, .. of k's and v's heads, two of each on their way
  const int l = threadIdx.x % LK, group = threadIdx.x / LK;
  const int step = KGROUPS / kv_tokens, j = group / step;
  const uint32_t tok = first + min(j, ntok - 1);
  const int b = (int)(tok / (uint32_t)a.S), s = (int)(tok - (uint32_t)b * (uint32_t)a.S);
  int h = group - j * step;
  const uint16_t* ksrc = a.k + b * a.ks.b + s * a.ks.s + h * a.ks.h + 8 * l;
  const uint16_t* vsrc = p.v + b * p.vs.b + s * p.vs.s + h * p.vs.h + 8 * l;
  const int64_t kstep = step * a.ks.h, vstep = step * p.vs.h;
  const bool live = j < ntok && place_of(p, tok, 0, false).live;
  uint4 ku, vu, kn, vn;                           // this row's, and the next one's on their way
  auto load = [&](int on, uint4& k, uint4& v) {   // row `on` from here
    const bool in = live && h + on * step < a.Hkv;
    k = in ? *reinterpret_cast<const uint4*>(ksrc + on * kstep) : make_uint4(0u, 0u, 0u, 0u);
    v = in ? *reinterpret_cast<const uint4*>(vsrc + on * vstep) : make_uint4(0u, 0u, 0u, 0u);
  };
  load(0, ku, vu);                                // before the place is looked up
  load(1, kn, vn);
  const Place at = place_of(p, tok, Gr::BYTES, live);
  const bool kept = at.group != nullptr;
  const int64_t head = ((int64_t)1 << (p.c.page_shift - 4)) * Gr::BYTES;
  uint8_t* const codes = at.group + at.row * (D / 2) + 4 * l;     // of head 0
  uint8_t* const scales = at.group + Gr::KS + at.row * Gr::SB + l / PER;
  const int32_t* const pos = a.pos ? a.pos + (int64_t)tok * a.axes : nullptr;
  turn();
  Lane8 f;
  set_lane<D, INTER>(f, a, sines + j * a.half, l);
  // every lane of a warp goes along (their rows end together); the loop has one row's code, not two: what is to
  // be fetched counts
#pragma unroll 1
  for (int n = a.Hkv; n > 0; n -= step) {
    const bool in = kept && h < a.Hkv;
    const int64_t to = h * head;
    put_key<D, INTER, CF>(p, f, ku, in, pos, at.pos, codes + to, scales + to);
    put_value<D, CF>(vu, in, codes + to, scales + to);
    ku = kn;
    vu = vn;
    load(2, kn, vn);
    h += step;
    ksrc += kstep;
    vsrc += vstep;
  }
}

template <int D, int P, bool INTER, int CF>
cudaError_t launch(const AppendRopeArgs& a, unsigned grid, int tokens, int kv_tokens, int sms, cudaStream_t st) {
  return launch_early(grid > (unsigned)(APPEND_FEW * sms) ? append_rope_kernel<D, P, INTER, CF, APPEND_MANY> : append_rope_kernel<D, P, INTER, CF, APPEND_FEW>,
                      dim3(grid), ROPE_THREADS, 0, st, a, tokens, kv_tokens);
}
template <int D, int P>
cudaError_t launch(const AppendRopeArgs& a, unsigned grid, int tokens, int kv_tokens, int sms, cudaStream_t st) {
  if (a.c.cf == CF_MX)
    return a.r.interleaved ? launch<D, P, true, CF_MX>(a, grid, tokens, kv_tokens, sms, st) : launch<D, P, false, CF_MX>(a, grid, tokens, kv_tokens, sms, st);
  return a.r.interleaved ? launch<D, P, true, CF_NV>(a, grid, tokens, kv_tokens, sms, st) : launch<D, P, false, CF_NV>(a, grid, tokens, kv_tokens, sms, st);
}

}  // namespace

cudaError_t launch_append_rope(const AppendRopeArgs& a, int sms, cudaStream_t st) {
  const int64_t total = (int64_t)a.r.B * a.r.S;
  const bool wide = a.r.half % 8 == 0;          // (as for fsa_qk_norm_rope)
  int tokens = std::max(1, ROPE_THREADS / (a.r.D / (wide ? 16 : 8)) / 4), kv_tokens = ROPE_TOKENS;
  while (tokens > 1 && 2 * total <= APPEND_FEW * (int64_t)tokens * sms) tokens /= 2;
  while (kv_tokens > tokens && 2 * total <= APPEND_FEW * (int64_t)kv_tokens * sms) kv_tokens /= 2;
  const unsigned grid = (unsigned)((total + kv_tokens - 1) / kv_tokens * (kv_tokens / tokens + 1));
  if (a.r.D == 128) return wide ? launch<128, 8>(a, grid, tokens, kv_tokens, sms, st) : launch<128, 4>(a, grid, tokens, kv_tokens, sms, st);
  return wide ? launch<64, 8>(a, grid, tokens, kv_tokens, sms, st) : launch<64, 4>(a, grid, tokens, kv_tokens, sms, st);
}

}  // namespace fsa
