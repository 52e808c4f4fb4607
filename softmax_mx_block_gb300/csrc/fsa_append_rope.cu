// fsa_append_rope.cu -- the projection's q, k and v of new tokens on their way to the attention:
// q normalised, rotated and written as bf16, k normalised, rotated and put into the 4-bit cache
// beside v, in one pass.
//
// q is that of fsa_qk_norm_rope, bit for bit, v that of fsa_cache_append.  k is rounded once:
// its codes and scales are those of the exact values
//   y = x / sqrt(mean(x^2) + eps) * w,  (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = pos * inv_freq
// (through bf16 they would be rounded twice).  They are computed in fp32, whose error is
// known: with Y the row's largest |y|, |a| + |b| <= 2 Y for every pair, the angle is off by at most
// 2^-22.3 (an ulp of a part of a turn, for positions up to 2^24), cos and sin by 2^-23 and the two products by
// 2^-24 each, together 2^-20.2 Y; the norm's factor by 2^-21.4 of y, a quotient by an E4M3 scale by 2^-22.4: in
// all 2^-19.4 Y.  So each block is rounded twice, from y - 2^-19 Y and from y + 2^-19 Y; where scale and
// codes agree, as in all but about one warp in 100, they are the exact ones, and what is left open is
// computed in fp64.  Elements that neither a norm nor an angle touches are exact as they are, and
// rounded as fsa_cache_append does.
//
// Bound by memory: 4 H + 4 Hkv + 2 Hkv (0.53 or 0.56) bytes a token and dim.  A block takes a
// few tokens with all their heads, as fsa_qk_norm_rope does: the sines of a token are computed
// once, for the rows of q (D/16 lanes each, both elements of a pair in a lane) and of k (D/8 lanes,
// 8 consecutive elements a lane, as the quantisation wants them; a pair's other element comes from
// another lane).
#include <algorithm>
#include "fsa_cache_codes.cuh"
#include "fsa_rope.cuh"

namespace fsa {
namespace {

constexpr float SURE = 0x1p-19f;      // of a row's largest |y|: more than the fp32 arithmetic is off by
constexpr int KV_ROWS = 2;            // rows of a thread in flight, of k and of v each

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
  float own[8], other[8];    // an element is multiplied by own, its pair's other one by other
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
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int e0 = 8 * l + 4 * u;
    const bool turns = e0 < 2 * a.half;
    f.turned |= turns ? 1u << u : 0u;
#pragma unroll
    for (int e = 4 * u; e < 4 * u + 4; ++e) {
      const float w = a.wk ? bf16_to_f32(a.wk[8 * l + e]) : 1.f;
      f.own[e] = w;
      f.other[e] = 0.f;
      if (turns) {
        int pair, other;
        bool second;
        pair_of<INTER>(8 * l + e, a.half, pair, other, second);
        const float2 t = sines[pair];
        const float wo = a.wk ? bf16_to_f32(a.wk[other]) : 1.f;
        f.own[e] = w * t.x;
        f.other[e] = second ? wo * t.y : -wo * t.y;
        still &= t.x == 1.f && t.y == 0.f;
      }
    }
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

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// What the fp32 values of a lane's eight say of their codes.
struct Codes {
  uint32_t codes, sb;
  uint32_t open;       // nibbles that the values' error leaves open
  bool scale_open;     // whether it leaves the block's scale open
};

// 8 values y +- d of a lane (d >= 0; 0: exactly y) as codes and scale byte.
template <int CF>
__device__ __forceinline__ Codes codes_of(const float (&y)[8], float d) {
  Codes r;
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
  float tlo = fmaxf(top - d, 0.f), thi = top + d;
#pragma unroll
  for (int m = 1; m < (CF == CF_MX ? 4 : 2); m *= 2) {
    tlo = fmaxf(tlo, __shfl_xor_sync(0xFFFFFFFFu, tlo, m));
    thi = fmaxf(thi, __shfl_xor_sync(0xFFFFFFFFu, thi, m));
  }
  const bool exact = d == 0.f;
  float mul;
  if constexpr (CF == CF_MX) {
    const uint32_t m = __float_as_uint(thi) >> 23;               // exponent, less 2 (zero and subnormal: 0)
    r.sb = (uint32_t)max((int)m - 2, 0);
    r.scale_open = m >= 0xFF || r.sb != (uint32_t)max((int)(__float_as_uint(tlo) >> 23) - 2, 0);
    mul = __uint_as_float((254u - r.sb) << 23);
  } else {
    // (1/6 as a float is half an ulp above it; raised by 2^-20 and cut, ties stay ties: fsa_cache_codes.cuh)
    constexpr float SIXTH = 0.16666667163372039795f, RAISE = 1.0f + 0x1p-20f, LESS = 1.0f - 0x1p-20f;
    const bool known = thi == tlo;
    r.sb = cvt_e4m3x2(known ? cut12(thi * (SIXTH * RAISE)) : thi * (SIXTH * RAISE), 0.f) & 0xFFu;
    r.scale_open = !(thi < 3e38f) || (!known && r.sb != (cvt_e4m3x2(tlo * (SIXTH * LESS), 0.f) & 0xFFu));
    const float s = e4m3_to_f32(r.sb);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(mul) : "f"(s));
    mul = s > 0.f ? (exact ? mul * RAISE : mul) : 0.f;           // (codes of a zero scale are zeros, without signs)
  }
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = (y[e] + d) * mul;
    if (CF == CF_NV && exact) x[e] = cut12(x[e]);
  }
  r.codes = cvt_e2m1x8(x);
  if (CF == CF_NV && mul == 0.f) r.codes = 0u;
  r.open = 0u;
  if (!exact && !(CF == CF_NV && mul == 0.f)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (y[e] - d) * mul;
    r.open = r.codes ^ cvt_e2m1x8(x);
  }
  return r;
}

// The codes that are open (and all of a block whose scale is) in fp64 from the definition; all
// lanes of a warp, D/8 a row.  One GB300's fp64 pipe takes 16 cycles a warp instruction and a sine with its
// cosine about 50, so what is not needed is left out, and the sum of squares is kept as two floats.
template <int D, bool INTER, int CF>
__device__ __noinline__ void close_codes(const RopeArgs& a, uint4 own, uint4 others, const int32_t* pos, int place, int l, Codes& r) {
  constexpr int L = D / 8, PER = CF == CF_MX ? 4 : 2;
  const uint32_t w[4] = {own.x, own.y, own.z, own.w}, v[4] = {others.x, others.y, others.z, others.w};
  double rr = 1.0;
  if (a.norm) {
    float hi = 0.f, lo = 0.f;                        // squares of bf16 are exact in fp32; a sum and what it drops
    auto add = [&](float x) {
      const float s = hi + x, t = s - hi;
      lo += (hi - (s - t)) + (x - t);
      hi = s;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      add(__fmul_rn(lo_bf16(w[i]), lo_bf16(w[i])));
      add(__fmul_rn(hi_bf16(w[i]), hi_bf16(w[i])));
    }
#pragma unroll
    for (int m = 1; m < L; m *= 2) {
      const float h = __shfl_xor_sync(0xFFFFFFFFu, hi, m), k = __shfl_xor_sync(0xFFFFFFFFu, lo, m);
      add(h);
      lo += k;
    }
    double mean = ((double)hi + (double)lo) * (1.0 / D) + (double)a.eps;
    const bool within = hi < 0x1p100f && mean > 0x1p-90;
    if (within) {
      const double y = (double)rsqrtf((float)mean), e = ::fma(-mean * y, y, 1.0);      // |e| < 2^-20: the next term is e^3
      rr = ::fma(y * e, ::fma(0.375, e, 0.5), y);
    }
    if (!__all_sync(0xFFFFFFFFu, within)) {          // beyond fp32's range (the warp's rows go along: they shuffle)
      double ss = 0.0;
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const double x = e & 1 ? hi_bf16(w[e >> 1]) : lo_bf16(w[e >> 1]);
        ss += x * x;
      }
#pragma unroll
      for (int m = 1; m < L; m *= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, m);
      if (!within) rr = 1.0 / sqrt(ss / D + (double)a.eps);
    }
  }
  if (r.scale_open) r.open = 0xFFFFFFFFu;
  bool finite = true;
  double top = 0.0, y[8];
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    const bool mine = r.open >> (4 * e) & 15u;
    y[e] = 0.0;
    if (!__any_sync(0xFFFFFFFFu, mine)) continue;
    const int at = 8 * l + e;
    double x = e & 1 ? hi_bf16(w[e >> 1]) : lo_bf16(w[e >> 1]);
    if (a.norm) x *= rr * (a.wk ? (double)bf16_to_f32(a.wk[at]) : 1.0);
    if (mine && at < 2 * a.half) {
      int pair, other;
      bool second;
      pair_of<INTER>(at, a.half, pair, other, second);
      double z = e & 1 ? hi_bf16(v[e >> 1]) : lo_bf16(v[e >> 1]);       // (interleaved: a word's two, exchanged)
      if (a.norm) z *= rr * (a.wk ? (double)bf16_to_f32(a.wk[other]) : 1.0);
      const int axis = pair >= a.first2 ? 2 : pair >= a.first1 ? 1 : 0;
      const double t = (double)(pos ? pos[axis] : place) * a.inv_freq[pair];
      double sn, c;
      sincos(t, &sn, &c);
      x = second ? x * c + z * sn : x * c - z * sn;
    }
    y[e] = x;
    finite &= isfinite(x);
    top = fmax(top, fabs(x));
  }
#pragma unroll
  for (int m = 1; m < PER; m *= 2) {
    top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    finite &= (bool)__shfl_xor_sync(0xFFFFFFFFu, (int)finite, m);
  }
  double scale;
  if constexpr (CF == CF_MX) {
    if (r.scale_open) {
      const int e = min(max((int)((uint32_t)__double2hiint(top) >> 20 & 0x7FF) - 1023 - 2, -127), 127);
      r.sb = finite ? (uint32_t)(e + 127) : 0xFFu;
    }
    scale = __hiloint2double((int)(1023 - 127 + min(r.sb, 254u)) << 20, 0);
  } else {
    if (r.scale_open) {
      const double t = fmin(top / 6.0, 448.0);
      const int ex = max((int)((uint32_t)__double2hiint(t) >> 20 & 0x7FF) - 1023, -6);
      const double n = rint(t * __hiloint2double((1023 + 3 - ex) << 20, 0));          // 8..16 steps, or fewer when subnormal
      r.sb = !finite ? 0x7Fu : (uint32_t)(n < 8.0 ? n : (ex + 7) * 8 + n - 8.0);
    }
    scale = (double)e4m3_to_f32(r.sb);
  }
  // the borders times the scale are exact
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    const bool mine = r.open >> (4 * e) & 15u;
    if (!__any_sync(0xFFFFFFFFu, mine)) continue;
    const double m = fabs(y[e]);
    uint32_t code = (m > 0.25 * scale) + (m >= 0.75 * scale) + (m > 1.25 * scale) + (m >= 1.75 * scale) + (m > 2.5 * scale) +
                    (m >= 3.5 * scale) + (m > 5.0 * scale);
    code |= signbit(y[e]) ? 8u : 0u;
    if (CF == CF_NV && scale == 0.0) code = 0u;
    if (mine) r.codes = (r.codes & ~(15u << (4 * e))) | (finite ? code : 0u) << (4 * e);
  }
}

template <int D, int P, bool INTER, int CF, int BLOCKS>
__global__ void __launch_bounds__(ROPE_THREADS, BLOCKS) append_rope_kernel(const AppendRopeArgs p, int tokens) {
  constexpr int L = D / (2 * P), GROUPS = ROPE_THREADS / L;       // lanes of a row of q
  constexpr int LK = D / 8, KGROUPS = ROPE_THREADS / LK;          // of k and v
  constexpr int PER = CF == CF_MX ? 4 : 2;                        // lanes of a block
  using Gr = CacheGroup<D, CF>;
  const RopeArgs& a = p.r;
  __shared__ __align__(16) float2 sines[ROPE_TOKENS * D / 2];     // cos, sin of [token][pair]
  griddep_launch();
  griddep_wait();
  const uint32_t total = (uint32_t)a.B * (uint32_t)a.S;
  const uint32_t first = blockIdx.x * (uint32_t)tokens;
  const int ntok = (int)min((uint32_t)tokens, total - first);
  // with two blocks for the same tokens, the first has their queries and the second their keys and values
  const bool queries = gridDim.y == 1 || blockIdx.y == 0, keys = gridDim.y == 1 || blockIdx.y == 1;

  // this thread: lane of a row of token j, rows h0, h0 + step, .. of q's heads
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int step = GROUPS / tokens, j = group / step, h0 = group - j * step;
  const uint32_t lanes = (uint32_t)((1ull << L) - 1) << (threadIdx.x % 32 / L * L);
  const bool turns = P * lane < a.half, all = a.half == D / 2;
  const int at0 = INTER || !turns ? 2 * P * lane : P * lane;
  const int at1 = INTER || !turns ? 2 * P * lane + P : a.half + P * lane;
  const uint32_t tok = first + min(j, ntok - 1);
  const int b = (int)(tok / (uint32_t)a.S), s = (int)(tok - (uint32_t)b * (uint32_t)a.S);
  const int nq = queries && j < ntok && place_of(p, tok, 0, false).live ? a.H : 0;

  const uint16_t* src = a.q + b * a.qs.b + s * a.qs.s + h0 * a.qs.h;
  uint16_t* dst = a.qo + b * a.qos.b + s * a.qos.s + h0 * a.qos.h;
  Raw<P> x[ROPE_ROWS];
  int h = h0;
  auto load = [&] {
#pragma unroll
    for (int r = 0; r < ROPE_ROWS; ++r)
      if (h + r * step < nq) x[r].load(src + r * step * a.qs.h, at0, at1);
  };
  load();                                                         // on their way while the sines are computed

  // and lane l of a row of token kj, rows kh, kh + kstep, .. of k's and v's heads
  const int l = threadIdx.x % LK, kgroup = threadIdx.x / LK, row0 = threadIdx.x % 32 - l;
  const int kstep = KGROUPS / tokens, kj = kgroup / kstep;
  const uint32_t ktok = first + min(kj, ntok - 1);
  Place at = place_of(p, ktok, Gr::BYTES, keys && kj < ntok);
  if (kj >= ntok) at.live = false;
  const int kb = (int)(ktok / (uint32_t)a.S), ks = (int)(ktok - (uint32_t)kb * (uint32_t)a.S);
  int kh = kgroup - kj * kstep;
  const uint16_t* ksrc = a.k + kb * a.ks.b + ks * a.ks.s + kh * a.ks.h + 8 * l;
  const uint16_t* vsrc = p.v + kb * p.vs.b + ks * p.vs.s + kh * p.vs.h + 8 * l;
  const int64_t head = ((int64_t)1 << (p.c.page_shift - 4)) * Gr::BYTES;
  const bool kept = at.group != nullptr;
  uint8_t* codes = at.group + kh * head + at.row * (D / 2) + 4 * l;
  uint8_t* scales = at.group + kh * head + Gr::KS + at.row * Gr::SB + l / PER;
  uint4 ku[KV_ROWS], vu[KV_ROWS];
  auto load_kv = [&] {
#pragma unroll
    for (int r = 0; r < KV_ROWS; ++r) {
      const bool in = kept && kh + r * kstep < a.Hkv;
      ku[r] = in ? *reinterpret_cast<const uint4*>(ksrc + r * kstep * a.ks.h) : make_uint4(0u, 0u, 0u, 0u);
      vu[r] = in ? *reinterpret_cast<const uint4*>(vsrc + r * kstep * p.vs.h) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  if (!queries) load_kv();                                        // (the queries' rows would keep them waiting)

  if (a.half > 0) {
    const int per = ROPE_THREADS / a.half;        // tokens at a time
    const int i = threadIdx.x % a.half;
    if ((int)threadIdx.x < per * a.half) {
      float fh, fl;
      turns_of(a.inv_freq[i], fh, fl);
      const int axis = i >= a.first2 ? 2 : i >= a.first1 ? 1 : 0;
      for (int t = threadIdx.x / a.half; t < ntok; t += per) {
        const int pos = a.pos ? a.pos[((int64_t)first + t) * a.axes + axis] : place_of(p, first + t, 0, false).pos;
        sines[t * a.half + i] = cos_sin(pos, fh, fl);
      }
    }
  }
  __syncthreads();
  if (queries) {
    Factors<P, INTER> f;
    // (threads past the pairs hold 2P consecutive elements, unturned)
    f.set(sines + j * a.half + P * lane, turns, a.wq, at0, at1);
#pragma unroll 1
    while (h < nq) {
#pragma unroll
      for (int r = 0; r < ROPE_ROWS; ++r)
        if (h + r * step < nq) {
          turn_row<D, P, INTER>(x[r], f, lanes, turns, all, a.norm, a.eps);
          x[r].store(dst + r * step * a.qos.h, at0, at1);
        }
      h += ROPE_ROWS * step;
      src += ROPE_ROWS * step * a.qs.h;
      dst += ROPE_ROWS * step * a.qos.h;
      load();
    }
  }
  if (!keys) return;

  // every lane of a warp goes along (their rows end together)
  Lane8 f;
  set_lane<D, INTER>(f, a, sines + kj * a.half, l);
#pragma unroll 1
  for (int n = a.Hkv; n > 0; n -= KV_ROWS * kstep) {
    if (queries || n < a.Hkv) load_kv();
#pragma unroll
    for (int r = 0; r < KV_ROWS; ++r) {
      if (n <= r * kstep) break;                                  // (the same for all)
      const uint4 others = a.half > 0 ? others_of<D, INTER>(ku[r], a.half, row0, l) : ku[r];
      const uint32_t w[4] = {ku[r].x, ku[r].y, ku[r].z, ku[r].w}, v[4] = {others.x, others.y, others.z, others.w};
      float y[8], ss = 0.f, top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float own = e & 1 ? hi_bf16(w[e / 2]) : lo_bf16(w[e / 2]), other = e & 1 ? hi_bf16(v[e / 2]) : lo_bf16(v[e / 2]);
        ss = fmaf(own, own, ss);
        y[e] = own * f.own[e];
        // (an element that does not turn takes nothing of another)
        if (f.turned >> (e / 4) & 1) y[e] = fmaf(other, f.other[e], y[e]);
        top = fmaxf(top, fabsf(y[e]));
      }
      float rs = 1.f;
      bool sure = true;
      if (a.norm) {
#pragma unroll
        for (int m = 1; m < LK; m *= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, m);
        const float mean = ss * (1.0f / D) + a.eps;
        rs = rsqrtf(mean);
        sure = mean > 0x1p-90f && mean < 0x1p120f;                // (squares below fp32's range are nothing beside that)
      }
#pragma unroll
      for (int m = 1; m < LK; m *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= rs;
      top *= rs;
      sure = sure && top < 0x1p120f && (top > 0x1p-90f || top == 0.f);
      uint32_t vsb;
      const bool in = kept && kh + r * kstep < a.Hkv;
      // (maxima drop NaN: an element that is not finite leaves its block open)
      constexpr uint32_t MAG = 0x7FFF7FFFu;
      const uint32_t most = __vmaxu2(__vimax3_u16x2(w[0] & MAG, w[1] & MAG, w[2] & MAG),
                                     __vimax3_u16x2(w[3] & MAG, __vmaxu2(v[0] & MAG, v[1] & MAG), __vmaxu2(v[2] & MAG, v[3] & MAG)));
      const bool finite = max(most & 0xFFFFu, most >> 16) < 0x7F80u;
      Codes kc = codes_of<CF>(y, !finite ? INFINITY : f.exact ? 0.f : top * SURE);
      kc.scale_open = in && (kc.scale_open || !sure);
      kc.open = in ? kc.open : 0u;
      if (__any_sync(0xFFFFFFFFu, kc.scale_open || kc.open != 0u)) {
        Codes c = kc;                                             // (in memory only here)
        close_codes<D, INTER, CF>(a, ku[r], others, a.pos ? a.pos + (int64_t)ktok * a.axes : nullptr, at.pos, l, c);
        kc = c;
      }
      const uint32_t kw = k_to_cache<LK>(kc.codes, row0, l);
      const uint32_t vw = v_to_cache<LK>(quantise8<CF>(vu[r], vsb), row0, l);
      if (in) {
        *reinterpret_cast<uint32_t*>(codes + r * kstep * head + Gr::K) = kw;
        *reinterpret_cast<uint32_t*>(codes + r * kstep * head + Gr::V) = vw;
        if (l % PER == 0) {
          scales[r * kstep * head] = (uint8_t)kc.sb;
          scales[r * kstep * head + Gr::VS - Gr::KS] = (uint8_t)vsb;
        }
      }
    }
    kh += KV_ROWS * kstep;
    ksrc += KV_ROWS * kstep * a.ks.h;
    vsrc += KV_ROWS * kstep * p.vs.h;
    codes += KV_ROWS * kstep * head;
    scales += KV_ROWS * kstep * head;
  }
}

template <int D, int P, bool INTER>
cudaError_t launch(const AppendRopeArgs& a, dim3 grid, int tokens, cudaStream_t st) {
  return a.c.cf == CF_MX ? launch_early(append_rope_kernel<D, P, INTER, CF_MX, 8>, grid, ROPE_THREADS, 0, st, a, tokens)
                         : launch_early(append_rope_kernel<D, P, INTER, CF_NV, 8>, grid, ROPE_THREADS, 0, st, a, tokens);
}
template <int D, int P>
cudaError_t launch(const AppendRopeArgs& a, dim3 grid, int tokens, cudaStream_t st) {
  return a.r.interleaved ? launch<D, P, true>(a, grid, tokens, st) : launch<D, P, false>(a, grid, tokens, st);
}

}  // namespace

cudaError_t launch_append_rope(const AppendRopeArgs& a, int sms, cudaStream_t st) {
  const int64_t total = (int64_t)a.r.B * a.r.S;
  const bool wide = a.r.half % 8 == 0;          // (as for fsa_qk_norm_rope)
  int tokens = std::max(1, ROPE_THREADS / (a.r.D / (wide ? 16 : 8)) / 4);
  while (tokens > 1 && 2 * total <= 8 * (int64_t)tokens * sms) tokens /= 2;
  const int64_t blocks = (total + tokens - 1) / tokens;
  const dim3 grid((unsigned)blocks, 2 * blocks <= 8 * (int64_t)sms ? 2 : 1);
  if (a.r.D == 128) return wide ? launch<128, 8>(a, grid, tokens, st) : launch<128, 4>(a, grid, tokens, st);
  return wide ? launch<64, 8>(a, grid, tokens, st) : launch<64, 4>(a, grid, tokens, st);
}

}  // namespace fsa
