// fsa_rope.cuh -- RMS norm and rotation of a row, shared by the kernel that prepares queries
// and keys (fsa_rope.cu) and the one that also puts the keys into the cache (fsa_append_rope.cu):
// paired fp32 arithmetic, a row's elements in a lane, the angles' frequencies in turns.
#pragma once
#include "fsa_cache.h"
#include "fsa_ptx.cuh"

namespace fsa {

constexpr int ROPE_THREADS = 64;   // 8 or 16 rows at once; small blocks end one by one (256 threads: video 495 us, 64: 479)
constexpr int ROPE_TOKENS = 4;     // of a block, at most
constexpr int ROPE_ROWS = 2;       // rows of a thread in flight

// two floats in one register pair
struct f2 {
  uint64_t v;
};
__device__ __forceinline__ f2 make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(f2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ f2 mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ f2 unpack(uint32_t w) { return make(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t pack(f2 a) {
  float lo, hi;
  split(a, lo, hi);
  return cvt_bf16x2(lo, hi);
}
// P pairs of elements in the order that the arithmetic takes them: a firsts, b seconds.
// A lane of a row holds 2P elements: `a` at at0 .. and `b` at at1 .., P consecutive each, or,
// interleaved, 2P consecutive ones from at0 on (at1 = at0 + P).
template <int P>
struct Raw {
  uint32_t w[P];           // P/2 words from at0, P/2 from at1
  __device__ __forceinline__ void load(const uint16_t* x, int at0, int at1) {
    if constexpr (P == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(x + at0), v = *reinterpret_cast<const uint4*>(x + at1);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
      w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(x + at0), v = *reinterpret_cast<const uint2*>(x + at1);
      w[0] = u.x; w[1] = u.y; w[2] = v.x; w[3] = v.y;
    }
  }
  __device__ __forceinline__ void store(uint16_t* x, int at0, int at1) const {
    if constexpr (P == 8) {
      *reinterpret_cast<uint4*>(x + at0) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(x + at1) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      *reinterpret_cast<uint2*>(x + at0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(x + at1) = make_uint2(w[2], w[3]);
    }
  }
};

// The first and the second elements of pairs 2e and 2e + 1.
template <int P, bool INTER>
__device__ __forceinline__ void firsts_seconds(const Raw<P>& x, int e, f2& a, f2& b) {
  if (INTER) {             // words 2e and 2e + 1
    const uint32_t u = x.w[2 * e], v = x.w[2 * e + 1];
    a = make(__uint_as_float(u << 16), __uint_as_float(v << 16));
    b = make(__uint_as_float(u & 0xFFFF0000u), __uint_as_float(v & 0xFFFF0000u));
  } else {
    a = unpack(x.w[e]);
    b = unpack(x.w[P / 2 + e]);
  }
}

// What the first and the second element of each of the thread's pairs are multiplied by,
// two pairs a register: first result a * c[0] + b * c[1], second a * c[2] + b * c[3].
template <int P, bool INTER>
struct Factors {
  f2 c[4][P / 2];
  __device__ __forceinline__ void set(const float2* t, bool turns, const uint16_t* w, int at0, int at1) {
    Raw<P> raw;                                     // the weights, as a row
    if (w) raw.load(w, at0, at1);
    else
#pragma unroll
      for (int e = 0; e < P; ++e) raw.w[e] = 0x3F803F80u;       // ones
#pragma unroll
    for (int e = 0; e < P / 2; ++e) {
      f2 wa, wb;
      firsts_seconds<P, INTER>(raw, e, wa, wb);
      const float4 cs = turns ? reinterpret_cast<const float4*>(t)[e] : make_float4(1.f, 0.f, 1.f, 0.f);   // cos, sin of two
      const f2 co = make(cs.x, cs.z), si = make(cs.y, cs.w);
      c[0][e] = mul(wa, co);
      c[1][e] = mul(wb, make(-cs.y, -cs.w));
      c[2][e] = mul(wa, si);
      c[3][e] = mul(wb, co);
    }
  }
};

// One row, normalised and turned.  lanes: those of the row; turns: this thread's elements do
// (all: every thread's).
template <int D, int P, bool INTER>
__device__ __forceinline__ void turn_row(Raw<P>& x, const Factors<P, INTER>& f, uint32_t lanes, bool turns, bool all, bool norm,
                                         float eps) {
  constexpr int L = D / (2 * P);
  f2 a[P / 2], b[P / 2];
#pragma unroll
  for (int e = 0; e < P / 2; ++e) firsts_seconds<P, INTER>(x, e, a[e], b[e]);
  float rs = 1.0f;
  if (norm) {
    f2 sa = mul(a[0], a[0]), sb = mul(b[0], b[0]);
#pragma unroll
    for (int e = 1; e < P / 2; ++e) {
      sa = fma(a[e], a[e], sa);
      sb = fma(b[e], b[e], sb);
    }
    float s0, s1, s2, s3;
    split(sa, s0, s1);
    split(sb, s2, s3);
    float ss = (s0 + s1) + (s2 + s3);
#pragma unroll
    for (int m = L / 2; m; m >>= 1) ss += __shfl_xor_sync(lanes, ss, m, L);
    rs = rsqrtf(ss * (1.0f / D) + eps);
  }
  const f2 rr = make(rs, rs);
#pragma unroll
  for (int e = 0; e < P / 2; ++e) {
    f2 p = fma(a[e], f.c[0][e], mul(b[e], f.c[1][e]));
    f2 q = fma(b[e], f.c[3][e], mul(a[e], f.c[2][e]));
    if (!all) {            // an element that does not turn takes nothing of another
      p.v = turns ? p.v : mul(a[e], f.c[0][e]).v;
      q.v = turns ? q.v : mul(b[e], f.c[3][e]).v;
    }
    p = mul(rr, p);
    q = mul(rr, q);
    if (INTER) {
      float p0, p1, q0, q1;
      split(p, p0, p1);
      split(q, q0, q1);
      x.w[2 * e] = cvt_bf16x2(p0, q0);
      x.w[2 * e + 1] = cvt_bf16x2(p1, q1);
    } else {
      x.w[e] = pack(p);
      x.w[P / 2 + e] = pack(q);
    }
  }
}

// inv_freq / 2 pi as a sum of two floats, without fp64 arithmetic (few lanes have it): the
// double's leading 24 and following 29 bits, times 1 / 2 pi as two floats.
__device__ __forceinline__ void turns_of(double freq, float& fh, float& fl) {
  const uint32_t hi = (uint32_t)__double2hiint(freq), lo = (uint32_t)__double2loint(freq);
  const int e = (int)(hi >> 20 & 0x7FF) - 1023;
  fh = fl = 0.f;
  if (e < -100) return;                             // no angle at any position
  const float lead = __uint_as_float((hi & 0x80000000u) | (uint32_t)(min(e, 128) + 127) << 23 | (hi & 0xFFFFFu) << 3 | lo >> 29);
  const float rest = copysignf((float)(lo & 0x1FFFFFFFu) * __uint_as_float((uint32_t)max(e + 127 - 52, 0) << 23), lead);
  constexpr float ch = 0.15915494309189535f, cl = (float)(0.15915494309189533576888376337251436 - (double)ch);
  fh = __fmul_rn(lead, ch);
  fl = fmaf(lead, ch, -fh) + fmaf(lead, cl, rest * ch);
}

// cos and sin of position p times a frequency of fh + fl turns.
__device__ __forceinline__ float2 cos_sin(int p, float fh, float fl) {
  const float ph = (float)p, pl = (float)((int64_t)p - (int64_t)ph);       // p = ph + pl exactly
  const float g = __fmul_rn(ph, fh);          // rounded: l below holds what this drops
  const float l = fmaf(ph, fh, -g) + fmaf(ph, fl, pl * fh);
  const float part = (g - rintf(g)) + l;      // of a turn
  float sn, c;
  sincospif(2.0f * part, &sn, &c);
  return make_float2(c, sn);
}

}  // namespace fsa
