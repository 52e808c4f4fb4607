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
#include "fsa_rope.cuh"

namespace fsa {
namespace {

// Blocks of an SM: 12 of at most 80 registers where there are more blocks than run at once (8:
// video 543 us), 8 of 128 registers, without spills, where all do (12: the half-rotated
// batch of 4593 tokens 7.3 us, 8: 5.5).
constexpr int ROPE_MANY = 12, ROPE_FEW = 8;

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
        sines[t * a.half + i] = cos_sin(p, fh, fl);
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
