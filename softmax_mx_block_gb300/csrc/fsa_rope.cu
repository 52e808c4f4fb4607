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
// all their heads: the sines of a token are computed once, by all threads, and read by
// every head from shared memory.  D/8 lanes hold a row, 8 elements each, chosen so
// that both elements of a pair are in one thread.
#include "fsa_cache.h"
#include "fsa_ptx.cuh"

namespace fsa {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_TOKENS = 4;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The heads of one tensor (q or k) for the block's tokens.
template <int D, bool INTER>
__device__ __forceinline__ void rope_rows(const uint16_t* __restrict__ x, const Strides& xs, uint16_t* __restrict__ o,
                                          const Strides& os, const uint16_t* __restrict__ weight, int heads,
                                          int ntok, const int2* __restrict__ tok, const float2* __restrict__ cs,
                                          int half, bool norm, float eps) {
  constexpr int L = D / 8;                        // lanes of a row
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  // the two 4-element chunks of this thread
  int at0 = 8 * lane, at1 = 8 * lane + 4;
  if (!INTER && 4 * lane < half) { at0 = 4 * lane; at1 = half + 4 * lane; }
  // (threads past the pairs hold 8 consecutive elements from 2*half on: 8*lane)
  const bool turns = 4 * lane < half;
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = e < 4 ? at0 + e : at1 + e - 4;
    w[e] = weight ? __uint_as_float((uint32_t)weight[d] << 16) : 1.0f;
  }
  const uint32_t lanes = (uint32_t)((1ull << L) - 1) << (threadIdx.x % 32 / L * L);
  const int rows = ntok * heads;
  for (int r = group; r < rows; r += ROPE_THREADS / L) {
    const int j = r / heads, h = r - j * heads;
    const int2 bs = tok[j];
    const uint16_t* src = x + bs.x * xs.b + bs.y * xs.s + h * xs.h;
    uint2 u0, u1;
    u0 = *reinterpret_cast<const uint2*>(src + at0);
    u1 = *reinterpret_cast<const uint2*>(src + at1);
    float v[8] = {bf_lo(u0.x), bf_hi(u0.x), bf_lo(u0.y), bf_hi(u0.y),
                  bf_lo(u1.x), bf_hi(u1.x), bf_lo(u1.y), bf_hi(u1.y)};
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
      for (int m = L / 2; m; m >>= 1) ss += __shfl_xor_sync(lanes, ss, m, L);
      const float rs = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * rs * w[e];
    }
    if (turns) {
      const float2* c = cs + j * half + 4 * lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = c[e];                    // cos, sin
        const int a = INTER ? 2 * e : e, b = INTER ? 2 * e + 1 : e + 4;
        const float va = v[a], vb = v[b];
        v[a] = va * t.x - vb * t.y;
        v[b] = va * t.y + vb * t.x;
      }
    }
    uint16_t* dst = o + bs.x * os.b + bs.y * os.s + h * os.h;
    *reinterpret_cast<uint2*>(dst + at0) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
    *reinterpret_cast<uint2*>(dst + at1) = make_uint2(cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7]));
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS) qk_norm_rope_kernel(const RopeArgs a, int tokens) {
  __shared__ float2 cs[ROPE_TOKENS * D / 2];
  __shared__ int2 tok[ROPE_TOKENS];
  const int64_t total = (int64_t)a.B * a.S;
  const int64_t first = (int64_t)blockIdx.x * tokens;
  const int ntok = (int)min((int64_t)tokens, total - first);
  if (threadIdx.x < ntok) {
    const int64_t t = first + threadIdx.x;
    tok[threadIdx.x] = make_int2((int)(t / a.S), (int)(t % a.S));
  }
  if (a.half > 0) {
    const int per = ROPE_THREADS / a.half;        // tokens at a time
    const int i = threadIdx.x % a.half;
    if ((int)threadIdx.x < per * a.half) {
      const double f = a.inv_freq[i] * 0.15915494309189533576888376337251436;   // 1 / (2 pi)
      const float fh = (float)f, fl = (float)(f - (double)fh);
      const int axis = i >= a.first2 ? 2 : i >= a.first1 ? 1 : 0;
      for (int j = threadIdx.x / a.half; j < ntok; j += per) {
        const int p = a.pos[(first + j) * a.axes + axis];
        const float ph = (float)p, pl = (float)((int64_t)p - (int64_t)ph);       // p = ph + pl exactly
        const float h = __fmul_rn(ph, fh);          // rounded: l below holds what this drops
        const float l = fmaf(ph, fh, -h) + fmaf(ph, fl, pl * fh);
        const float turns = (h - rintf(h)) + l;
        float s, c;
        sincospif(2.0f * turns, &s, &c);
        cs[j * a.half + i] = make_float2(c, s);
      }
    }
  }
  __syncthreads();
  rope_rows<D, INTER>(a.q, a.qs, a.qo, a.qos, a.wq, a.H, ntok, tok, cs, a.half, a.norm, a.eps);
  rope_rows<D, INTER>(a.k, a.ks, a.ko, a.kos, a.wk, a.Hkv, ntok, tok, cs, a.half, a.norm, a.eps);
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
