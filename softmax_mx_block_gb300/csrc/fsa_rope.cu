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
// by the norm's weights.  D/8 lanes hold a row, 8 elements each, chosen so that both
// elements of a pair are in one thread, and the arithmetic goes two floats at a time.
#include "fsa_cache.h"
#include "fsa_ptx.cuh"

namespace fsa {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_TOKENS = 4;
constexpr int ROPE_ROWS = 4;       // rows of a thread in flight

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
__device__ __forceinline__ float weight_at(const uint16_t* w, int d) { return w ? __uint_as_float((uint32_t)w[d] << 16) : 1.0f; }

// A thread's share of one tensor (q or k) for its token: rows h = first, first + step, ..
template <int D>
struct Rows {
  const uint16_t* src;     // this lane's elements of the first row
  uint16_t* dst;
  int64_t sstep, dstep;    // to the next row
  int n;                   // rows left
  uint2 u0[ROPE_ROWS], u1[ROPE_ROWS];
  __device__ __forceinline__ Rows(const uint16_t* x, const Strides& xs, uint16_t* o, const Strides& os, int heads, int b, int s,
                                  int first, int step) {
    src = x + b * xs.b + s * xs.s + first * xs.h;
    dst = o + b * os.b + s * os.s + first * os.h;
    sstep = step * xs.h;
    dstep = step * os.h;
    n = heads > first ? (heads - first + step - 1) / step : 0;
  }
  __device__ __forceinline__ void load(int at0, int at1) {
#pragma unroll
    for (int r = 0; r < ROPE_ROWS; ++r)
      if (r < n) {
        u0[r] = *reinterpret_cast<const uint2*>(src + r * sstep + at0);
        u1[r] = *reinterpret_cast<const uint2*>(src + r * sstep + at1);
      }
  }
};

// The loaded rows, normalised, turned and stored.  c0..c3: what the first and the second
// element of each pair are multiplied by, for the first and the second result.  turns: this
// thread's elements do (all: every thread's).
template <int D, bool INTER>
__device__ __forceinline__ void finish_rows(Rows<D>& x, int at0, int at1, const f2 (&c)[4][2], uint32_t lanes, bool turns, bool all,
                                            bool norm, float eps) {
  constexpr int L = D / 8;
#pragma unroll
  for (int r = 0; r < ROPE_ROWS; ++r) {
    if (r >= x.n) break;
    // elements in the order that pairs take them: a = firsts, b = seconds of the 4 pairs
    f2 a[2], b[2];
    if (INTER) {
      float v[8];
      split(unpack(x.u0[r].x), v[0], v[1]);
      split(unpack(x.u0[r].y), v[2], v[3]);
      split(unpack(x.u1[r].x), v[4], v[5]);
      split(unpack(x.u1[r].y), v[6], v[7]);
      a[0] = make(v[0], v[2]); a[1] = make(v[4], v[6]);
      b[0] = make(v[1], v[3]); b[1] = make(v[5], v[7]);
    } else {
      a[0] = unpack(x.u0[r].x); a[1] = unpack(x.u0[r].y);
      b[0] = unpack(x.u1[r].x); b[1] = unpack(x.u1[r].y);
    }
    float rs = 1.0f;
    if (norm) {
      float lo, hi;
      split(fma(a[0], a[0], fma(a[1], a[1], fma(b[0], b[0], mul(b[1], b[1])))), lo, hi);
      float ss = lo + hi;
#pragma unroll
      for (int m = L / 2; m; m >>= 1) ss += __shfl_xor_sync(lanes, ss, m, L);
      rs = rsqrtf(ss * (1.0f / D) + eps);
    }
    const f2 rr = make(rs, rs);
    f2 p[2], q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f2 ap = mul(b[e], c[1][e]), aq = mul(a[e], c[2][e]);
      p[e] = fma(a[e], c[0][e], ap);
      q[e] = fma(b[e], c[3][e], aq);
      if (!all) {                                   // an element that does not turn takes nothing of another
        p[e].v = turns ? p[e].v : mul(a[e], c[0][e]).v;
        q[e].v = turns ? q[e].v : mul(b[e], c[3][e]).v;
      }
      p[e] = mul(rr, p[e]);
      q[e] = mul(rr, q[e]);
    }
    uint2 o0, o1;
    if (INTER) {
      float pv[4], qv[4];
      split(p[0], pv[0], pv[1]); split(p[1], pv[2], pv[3]);
      split(q[0], qv[0], qv[1]); split(q[1], qv[2], qv[3]);
      o0 = make_uint2(cvt_bf16x2(pv[0], qv[0]), cvt_bf16x2(pv[1], qv[1]));
      o1 = make_uint2(cvt_bf16x2(pv[2], qv[2]), cvt_bf16x2(pv[3], qv[3]));
    } else {
      o0 = make_uint2(pack(p[0]), pack(p[1]));
      o1 = make_uint2(pack(q[0]), pack(q[1]));
    }
    *reinterpret_cast<uint2*>(x.dst + r * x.dstep + at0) = o0;
    *reinterpret_cast<uint2*>(x.dst + r * x.dstep + at1) = o1;
  }
  x.src += ROPE_ROWS * x.sstep;
  x.dst += ROPE_ROWS * x.dstep;
  x.n -= ROPE_ROWS;
}

// The factors of the thread's 4 pairs: first result a * c0 + b * c1, second a * c2 + b * c3.
template <bool INTER>
__device__ __forceinline__ void factors(const float4& t0, const float4& t1, const uint16_t* w, int at0, int at1, f2 (&c)[4][2]) {
  const float cs[4] = {t0.x, t0.z, t1.x, t1.z}, sn[4] = {t0.y, t0.w, t1.y, t1.w};
  float f[4][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float wa = weight_at(w, INTER ? at0 + 2 * e : at0 + e), wb = weight_at(w, INTER ? at0 + 2 * e + 1 : at1 + e);
    f[0][e] = wa * cs[e];
    f[1][e] = -wb * sn[e];
    f[2][e] = wa * sn[e];
    f[3][e] = wb * cs[e];
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    c[x][0] = make(f[x][0], f[x][1]);
    c[x][1] = make(f[x][2], f[x][3]);
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS) qk_norm_rope_kernel(const RopeArgs a, int tokens) {
  constexpr int L = D / 8, GROUPS = ROPE_THREADS / L;
  __shared__ __align__(16) float2 cs[ROPE_TOKENS * D / 2];        // cos, sin of [token][pair]
  const uint32_t total = (uint32_t)a.B * (uint32_t)a.S;
  const uint32_t first = blockIdx.x * (uint32_t)tokens;
  const int ntok = (int)min((uint32_t)tokens, total - first);
  // this thread: lane of a row of token j, heads h0, h0 + step, ..
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int step = GROUPS / tokens, j = group / step, h0 = group - j * step;
  const uint32_t lanes = (uint32_t)((1ull << L) - 1) << (threadIdx.x % 32 / L * L);
  const int at0 = INTER || 4 * lane >= a.half ? 8 * lane : 4 * lane;
  const int at1 = INTER || 4 * lane >= a.half ? 8 * lane + 4 : a.half + 4 * lane;
  const uint32_t tok = first + min(j, ntok - 1);
  const int b = (int)(tok / (uint32_t)a.S), s = (int)(tok - (uint32_t)b * (uint32_t)a.S);
  Rows<D> q(a.q, a.qs, a.qo, a.qos, j < ntok ? a.H : 0, b, s, h0, step);
  q.load(at0, at1);                                               // on their way while the sines are computed
  if (a.half > 0) {
    const int per = ROPE_THREADS / a.half;        // tokens at a time
    const int i = threadIdx.x % a.half;
    if ((int)threadIdx.x < per * a.half) {
      const double f = a.inv_freq[i] * 0.15915494309189533576888376337251436;   // 1 / (2 pi)
      const float fh = (float)f, fl = (float)(f - (double)fh);
      const int axis = i >= a.first2 ? 2 : i >= a.first1 ? 1 : 0;
      for (int x = threadIdx.x / a.half; x < ntok; x += per) {
        const int p = a.pos[((int64_t)first + x) * a.axes + axis];
        const float ph = (float)p, pl = (float)((int64_t)p - (int64_t)ph);       // p = ph + pl exactly
        const float h = __fmul_rn(ph, fh);          // rounded: l below holds what this drops
        const float l = fmaf(ph, fh, -h) + fmaf(ph, fl, pl * fh);
        const float turns = (h - rintf(h)) + l;
        float sn, c;
        sincospif(2.0f * turns, &sn, &c);
        cs[x * a.half + i] = make_float2(c, sn);
      }
    }
  }
  __syncthreads();
  if (j >= ntok) return;
  float4 t0 = make_float4(1.f, 0.f, 1.f, 0.f), t1 = t0;           // past the pairs: no turn
  if (4 * lane < a.half) {
    const float4* t = reinterpret_cast<const float4*>(cs + j * a.half + 4 * lane);
    t0 = t[0];
    t1 = t[1];
  }
  // (threads past the pairs hold 8 consecutive elements: as pairs (x, x + 4) of them, or as
  // neighbours when interleaved, unturned)
  const bool turns = 4 * lane < a.half, all = a.half == D / 2;
  f2 c[4][2];
  factors<INTER>(t0, t1, a.wq, at0, at1, c);
  while (true) {
    finish_rows<D, INTER>(q, at0, at1, c, lanes, turns, all, a.norm, a.eps);
    if (q.n <= 0) break;
    q.load(at0, at1);
  }
  Rows<D> k(a.k, a.ks, a.ko, a.kos, a.Hkv, b, s, h0, step);
  if (k.n <= 0) return;
  k.load(at0, at1);
  factors<INTER>(t0, t1, a.wk, at0, at1, c);
  while (true) {
    finish_rows<D, INTER>(k, at0, at1, c, lanes, turns, all, a.norm, a.eps);
    if (k.n <= 0) break;
    k.load(at0, at1);
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  const int64_t total = (int64_t)a.B * a.S;
  const int tokens = total >= 4096 ? ROPE_TOKENS : 1;
  const unsigned grid = (unsigned)((total + tokens - 1) / tokens);
  if (a.D == 128) {
    if (a.interleaved) qk_norm_rope_kernel<128, true><<<grid, ROPE_THREADS, 0, st>>>(a, tokens);
    else qk_norm_rope_kernel<128, false><<<grid, ROPE_THREADS, 0, st>>>(a, tokens);
  } else {
    if (a.interleaved) qk_norm_rope_kernel<64, true><<<grid, ROPE_THREADS, 0, st>>>(a, tokens);
    else qk_norm_rope_kernel<64, false><<<grid, ROPE_THREADS, 0, st>>>(a, tokens);
  }
  return cudaGetLastError();
}

}  // namespace fsa
