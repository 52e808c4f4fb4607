// fsa_cache.h -- the paged 4-bit K/V cache (fsa.h): its layout, and the launch
// descriptors of the kernels that write, read and attend over it and of the kernel
// that prepares queries and keys.
//
// A page holds page_size tokens of every kv head: [Hkv][page_size/16] groups.  A
// group is 16 tokens of one head, contiguous so that one bulk copy fetches it whole:
//   16 rows of K codes (D/2 bytes), 16 rows of V codes, 16 rows of K scales (SB
//   bytes), 16 rows of V scales;  SB = D/32 (E2M1, E8M0 scales) or D/16 (NVFP4, E4M3).
// The bytes of a code row are in the order in which the attention kernel's threads
// take them for their matrix fragments (fsa_cache_attn.cu):
//   K: byte t*(D/8) + 2s + h holds elements 16s + 4t + 2h (low nibble) and + 1
//   V: byte g*(D/16) + i     holds elements 16i + 2g (low nibble) and + 1
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace fsa {

constexpr int CF_MX = 0, CF_NV = 1;   // E2M1 with E8M0 scales per 32, NVFP4 with E4M3 scales per 16

template <int D, int CF>
struct CacheGroup {
  static constexpr int SB = CF == CF_MX ? D / 32 : D / 16;   // scale bytes of a row
  static constexpr int K = 0, V = 8 * D, KS = 16 * D, VS = 16 * D + 16 * SB;
  static constexpr int BYTES = 16 * D + 32 * SB;
};

struct Cache {
  uint8_t* pages;
  int64_t page_bytes;
  int num_pages;
  int page_shift;       // log2 of the tokens of a page
  int Hkv, D, cf;
};

struct Strides { int64_t b, s, h; };   // in elements; the head dimension is contiguous

struct CacheIo {          // append and read
  Cache c;
  uint16_t* k;            // append: source, read: destination (may be null)
  uint16_t* v;
  Strides ks, vs;
  const int32_t* table;   // [B][max_pages]
  const int32_t* lens;    // [B]
  const int32_t* which;   // append: new tokens of each sequence (null: S), read: first position (null: 0)
  int B, S, max_pages;
  int32_t* status;
};

struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* qo;
  uint16_t* ko;
  Strides qs, ks, qos, kos;
  const uint16_t* wq;     // null: ones
  const uint16_t* wk;
  const int32_t* pos;     // [B][S][axes]
  const double* inv_freq; // [half]
  int B, S, H, Hkv, D, half, axes, first1, first2;   // pairs from first1 on turn by axis 1, from first2 on by axis 2
  int norm, interleaved;
  float eps;
};

struct AppendRopeArgs {   // r.k is read only (r.ko is null); r.pos null: by their places in the sequences
  RopeArgs r;
  Cache c;
  const uint16_t* v;
  Strides vs;
  const int32_t* table;   // [B][max_pages]
  const int32_t* lens;    // [B]
  const int32_t* which;   // new tokens of each sequence (null: S)
  int max_pages;
  int32_t* status;
};

struct CacheAttnArgs {
  Cache c;
  const uint16_t* q;
  Strides qs, os;
  void* out;              // bf16 or fp32
  float* lse;             // [B][Sq][H] or null
  const int32_t* table;
  const int32_t* lens;
  const int32_t* q_lens;  // null: Sq each
  float* partials;        // workspace: two partial results a CTA
  int4* starts;           // workspace: per CTA, the segment that begins in it and goes on, and the CTA where it ends
  int B, H, Sq, G, CT, max_pages, causal, out_bf16;
  int window, sinks;      // of the keys before a row the last `window` and the first `sinks` (window 0: all)
  int whole;              // chunks: a segment is one CTA's (CT: blocks of 256 rows)
  uint32_t g_mul;         // col / G is the high word of col * g_mul (0: it is not)
  float scale_log2;       // |scale| log2 e, or 1 when the scale is 0
  float q_sign;           // the scale's sign (0 for a zero scale)
  int32_t* status;
  uint64_t timeout_ns;
};

// Launch a kernel that begins with griddep_launch and griddep_wait (fsa_ptx.cuh): its blocks
// may be set up while the stream's previous kernel still runs, and wait for its end
// themselves.  Where the previous kernel is one of these too, that hides about 1 us.
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_cache_append(const CacheIo& a, cudaStream_t st);
cudaError_t launch_cache_read(const CacheIo& a, cudaStream_t st);
cudaError_t launch_qk_norm_rope(const RopeArgs& a, int sms, cudaStream_t st);
cudaError_t launch_append_rope(const AppendRopeArgs& a, int sms, cudaStream_t st);

// columns (query rows of one kv head) of a pass, by eights, and the workspace of a call
int cache_attn_ntiles(int cols);
size_t cache_attn_workspace(const Cache& c, int B, int H, int Sq, int max_pages, int window, int sinks, int sms, size_t* starts_at);
cudaError_t launch_cache_attn(const CacheAttnArgs& a, int nt, int sms, cudaStream_t st);
cudaError_t launch_cache_attn_window(const CacheAttnArgs& a, int nt, int sms, cudaStream_t st);      // a.window > 0

// chunks: blocks of a sequence's rows (of a kv head), whether its segments are one CTA's each
int cache_chunk_blocks(int rows);
bool cache_chunk_whole(const Cache& c, int max_pages);
size_t cache_chunk_workspace(const Cache& c, int max_pages, int sms, size_t* starts_at);
cudaError_t launch_cache_chunk(const CacheAttnArgs& a, int sms, cudaStream_t st);

}  // namespace fsa
