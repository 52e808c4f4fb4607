// fsa_rope.cu -- queries and keys on their way from the projection to the attention:
// RMS norm of each head and rotation by position, in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * w                       (fp32)
//   t = pos[axis(i)] * inv_freq[i],  (a, b) -> (a cos t - b sin t, a sin t + b cos t)
// for the pairs (a, b) = (y[i], y[i + half]) or (y[2i], y[2i + 1]); one rounding to bf16.
//
// The angle is held in turns: inv_freq / 2 pi in fp64 once per thread, as the sum of two
// floats, so pos * inv_freq keeps about 2^-48 of its size and its whole turns come off
// exactly.  An fp32 product alone would be off by 0.06 rad at position 2^20.
//
// The work is bound by memory (4 bytes an element).  A block takes a few tokens with
// all their heads: the sines of a token are computed once, by all threads, through shared
// memory, and then stay in the registers of the threads that have that token, multiplied
// by the norm's weights.  D/16 lanes hold a row, 16 elements each, chosen so that both
// elements of a pair are in one thread, and the arithmetic goes two floats at a time.
//
// Measured (one GB300): 75600 patches of 40 + 40 heads of 128 471 us (6.6 TB/s, 0.97 of the copy
// bandwidth), 16K tokens of 32 + 8 heads 59.5 us (0.83: about 7 us to start and to run out, and
// heads before positions cost 5%, their rows of two tokens being 512 bytes), 64 tokens of a
// decode step 3.6 us.
#include <algorithm>
#include "fsa_cache.h"
#include "fsa_ptx.cuh"

namespace fsa {
namespace {

constexpr int ROPE_THREADS = 64;   // 8 or 16 rows at once; small blocks end one by one (256 threads: video 495 us, 64: 479)
constexpr int ROPE_TOKENS = 4;     // of a block, at most
constexpr int ROPE_ROWS = 2;       // rows of a thread in flight
// Blocks of an SM: 12 of at most 80 registers where there are more blocks than run at once (8:
// video 543 us), 8 of 128 registers, without spills, where all do (12: the half-rotated
// batch of 4593 tokens 7.3 us, 8: 5.5).
constexpr int ROPE_MANY = 12, ROPE_FEW = 8;

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

template <int D, int P, bool INTER, int BLOCKS>
__global__ void __launch_bounds__(ROPE_THREADS, BLOCKS) qk_norm_rope_kernel(const RopeArgs a, int tokens) {
  constexpr int L = D / (2 * P), GROUPS = ROPE_THREADS / L;
  __shared__ __align__(16) float2 sines[ROPE_TOKENS * D / 2];     // cos, sin of [token][pair]
  griddep_launch();
  griddep_wait();
  const uint32_t total = (uint32_t)a.B * (uint32_t)a.S;
  const uint32_t first = blockIdx.x * (uint32_t)tokens;
  const int ntok = (int)min((uint32_t)tokens, total - first);
  // this thread: lane of a row of token j, rows h0, h0 + step, .. of q's heads and then k's
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int step = GROUPS / tokens, j = group / step, h0 = group - j * step;
  const uint32_t lanes = (uint32_t)((1ull << L) - 1) << (threadIdx.x % 32 / L * L);
  const bool turns = P * lane < a.half, all = a.half == D / 2;
  const int at0 = INTER || !turns ? 2 * P * lane : P * lane;
  const int at1 = INTER || !turns ? 2 * P * lane + P : a.half + P * lane;
  const uint32_t tok = first + min(j, ntok - 1);
  const int b = (int)(tok / (uint32_t)a.S), s = (int)(tok - (uint32_t)b * (uint32_t)a.S);
  const int nq = j < ntok ? a.H : 0, nk = j < ntok ? a.Hkv : 0;

  const uint16_t* src = a.q + b * a.qs.b + s * a.qs.s + h0 * a.qs.h;
  uint16_t* dst = a.qo + b * a.qos.b + s * a.qos.s + h0 * a.qos.h;
  int64_t sstep = step * a.qs.h, dstep = step * a.qos.h;
  Raw<P> x[ROPE_ROWS];
  int h = h0, n = nq;
  auto load = [&] {
#pragma unroll
    for (int r = 0; r < ROPE_ROWS; ++r)
      if (h + r * step < n) x[r].load(src + r * sstep, at0, at1);
  };
  load();                                                         // on their way while the sines are computed
  if (a.half > 0) {
    const int per = ROPE_THREADS / a.half;        // tokens at a time
    const int i = threadIdx.x % a.half;
    if ((int)threadIdx.x < per * a.half) {
      float fh, fl;
      turns_of(a.inv_freq[i], fh, fl);
      const int axis = i >= a.first2 ? 2 : i >= a.first1 ? 1 : 0;
      for (int t = threadIdx.x / a.half; t < ntok; t += per) {
        const int p = a.pos[((int64_t)first + t) * a.axes + axis];
        const float ph = (float)p, pl = (float)((int64_t)p - (int64_t)ph);       // p = ph + pl exactly
        const float g = __fmul_rn(ph, fh);          // rounded: l below holds what this drops
        const float l = fmaf(ph, fh, -g) + fmaf(ph, fl, pl * fh);
        const float part = (g - rintf(g)) + l;      // of a turn
        float sn, c;
        sincospif(2.0f * part, &sn, &c);
        sines[t * a.half + i] = make_float2(c, sn);
      }
    }
  }
  __syncthreads();
  Factors<P, INTER> f;
  const float2* const t = sines + j * a.half + P * lane;
  // (threads past the pairs hold 2P consecutive elements, unturned)
  f.set(t, turns, a.wq, at0, at1);
#pragma unroll 1
  for (bool keys = false;; keys = true) {
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
    if (keys) return;
    src = a.k + b * a.ks.b + s * a.ks.s + h0 * a.ks.h;
    dst = a.ko + b * a.kos.b + s * a.kos.s + h0 * a.kos.h;
    sstep = step * a.ks.h;
    dstep = step * a.kos.h;
    h = h0;
    n = nk;
    load();
    f.set(t, turns, a.wk, at0, at1);
  }
}

template <int D, int P, bool INTER>
cudaError_t launch_rows(const RopeArgs& a, unsigned grid, int tokens, int sms, cudaStream_t st) {
  return launch_early(grid > (unsigned)(ROPE_FEW * sms) ? qk_norm_rope_kernel<D, P, INTER, ROPE_MANY>
                                                        : qk_norm_rope_kernel<D, P, INTER, ROPE_FEW>,
                      dim3(grid), ROPE_THREADS, 0, st, a, tokens);
}
template <int D, int P>
cudaError_t launch_rows(const RopeArgs& a, unsigned grid, int tokens, int sms, cudaStream_t st) {
  return a.interleaved ? launch_rows<D, P, true>(a, grid, tokens, sms, st) : launch_rows<D, P, false>(a, grid, tokens, sms, st);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, int sms, cudaStream_t st) {
  const int64_t total = (int64_t)a.B * a.S;
  // 16 elements a lane halve the shuffles and the addresses of a row; 8 where the rotated
  // part is an odd multiple of 8
  const bool wide = a.half % 8 == 0;
  // Tokens of a block: four of its groups of lanes each (with the pairs' frequencies and the
  // weights, which a block starts with, used for a quarter of a token's heads; with half
  // as many tokens the video took 10% longer); fewer while all blocks still run at once, 8 an
  // SM (us without / with: 1000 tokens of 32 + 8 heads of 128 7.5 / 5.6, of 8 + 8 5.1 / 4.4; 1800 of
  // 14 + 2 heads of 64 5.2 / 4.2).  Up to 12 an SM, 1800 tokens of 32 + 8 heads would take 9.3
  // instead of 10.1, but of 8 + 8 5.8 instead of 5.3; beyond that two waves, 2000 of 8 + 8 7.4
  // instead of 5.3.
  int tokens = std::max(1, ROPE_THREADS / (a.D / (wide ? 16 : 8)) / 4);
  while (tokens > 1 && 2 * total <= ROPE_FEW * (int64_t)tokens * sms) tokens /= 2;
  const unsigned grid = (unsigned)((total + tokens - 1) / tokens);
  if (a.D == 128) return wide ? launch_rows<128, 8>(a, grid, tokens, sms, st) : launch_rows<128, 4>(a, grid, tokens, sms, st);
  return wide ? launch_rows<64, 8>(a, grid, tokens, sms, st) : launch_rows<64, 4>(a, grid, tokens, sms, st);
}

}  // namespace fsa
