// fsa_cache_api.cu -- the C ABI of the serving operators (fsa.h): argument checks and
// dispatch for the query/key preparation, the paged cache and the attention over it.
#include <cmath>
#include <climits>
#include <cstdint>
#include <cuda_runtime.h>
#include "fsa.h"
#include "fsa_cache.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

bool page_ok(int page_size) { return page_size >= 16 && page_size <= 1024 && (page_size & (page_size - 1)) == 0; }

size_t page_bytes_of(int page_size, int Hkv, int D, int fmt) {
  return (size_t)Hkv * page_size * (D + 2 * (fmt == FSA_FMT_E2M1 ? D / 32 : D / 16));
}

// FSA_OK and the kernels' form of a cache, or the error
int take_cache(const fsa_cache* c, fsa::Cache* out) {
  if (!c || !c->pages || !aligned(c->pages, 16) || !page_ok(c->page_size) || c->Hkv <= 0 || c->Hkv > 65535 ||
      (c->D != 64 && c->D != 128) || c->num_pages <= 0 || c->num_pages > INT_MAX)
    return FSA_ERR_INVALID_ARG;
  if (c->fmt != FSA_FMT_E2M1 && c->fmt != FSA_FMT_NVFP4) return FSA_ERR_UNSUPPORTED_FMT;
  out->pages = static_cast<uint8_t*>(c->pages);
  out->page_bytes = (int64_t)page_bytes_of(c->page_size, c->Hkv, c->D, c->fmt);
  out->num_pages = (int)c->num_pages;
  out->page_shift = log2_of(c->page_size);
  out->Hkv = c->Hkv;
  out->D = c->D;
  out->cf = c->fmt == FSA_FMT_E2M1 ? fsa::CF_MX : fsa::CF_NV;
  return FSA_OK;
}

// strides of a [B][S][h][D] tensor whose rows move as 16-byte aligned pieces; those of an
// output must keep its rows apart
bool take_strides(const fsa_strides* st, int B, int S, int H, bool output, fsa::Strides* out) {
  if (!st) return false;
  const int64_t v[3] = {st->b, st->s, st->h};
  const int n[3] = {B, S, H};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (v[i] % 8 != 0 || v[i] < 0 || (output && v[i] == 0))) return false;
  out->b = B > 1 ? v[0] : 0;
  out->s = S > 1 ? v[1] : 0;
  out->h = H > 1 ? v[2] : 0;
  return true;
}

bool pages_ok(int max_pages, int page_size) { return max_pages > 0 && (int64_t)max_pages * page_size <= (1 << 30); }

bool table_ok(const int32_t* table, int max_pages, int page_size) {
  return table && aligned(table, 4) && pages_ok(max_pages, page_size);
}

int cache_io(const fsa_cache* cache, const void* k, const void* v, const fsa_strides* ks, const fsa_strides* vs, int B,
             int S, const int32_t* table, int max_pages, const int32_t* lens, const int32_t* which, int32_t* status,
             bool output, fsa::CacheIo* a) {
  const int st = take_cache(cache, &a->c);
  if (st != FSA_OK) return st;
  if (B <= 0 || S <= 0 || !lens || !aligned(lens, 4) || !aligned(which, 4) || !aligned(status, 4) ||
      !table_ok(table, max_pages, cache->page_size) || !aligned(k, 16) || !aligned(v, 16))
    return FSA_ERR_INVALID_ARG;
  if ((int64_t)B * (S / 8 + 2) > INT_MAX / cache->Hkv) return FSA_ERR_INVALID_ARG;        // the kernels' units, counted in 32 bits
  if (k && !take_strides(ks, B, S, cache->Hkv, output, &a->ks)) return FSA_ERR_INVALID_ARG;
  if (v && !take_strides(vs, B, S, cache->Hkv, output, &a->vs)) return FSA_ERR_INVALID_ARG;
  a->k = static_cast<uint16_t*>(const_cast<void*>(k));
  a->v = static_cast<uint16_t*>(const_cast<void*>(v));
  a->table = table;
  a->lens = lens;
  a->which = which;
  a->B = B;
  a->S = S;
  a->max_pages = max_pages;
  a->status = status;
  return FSA_OK;
}

// (a failed call's error is reported here, and not to whoever asks the runtime next)
int launch_status(cudaError_t e) {
  if (e == cudaSuccess) return FSA_OK;
  cudaGetLastError();
  return FSA_ERR_LAUNCH;
}

bool sm_count(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && *sms > 0)
    return true;
  cudaGetLastError();
  return false;
}

// The kernels count rows and, over all sequences, heads and passes of columns, tiles of 32
// keys (and what a segment's start weighs, at most 8) in 32 bits.
bool attn_shape_ok(int B, int H, int Hkv, int Sq, int D, int max_pages, int page_size) {
  if (!(B > 0 && H > 0 && Hkv > 0 && H % Hkv == 0 && Sq > 0 && (D == 64 || D == 128) && pages_ok(max_pages, page_size) &&
        (int64_t)B * H <= (1 << 27) / Sq))
    return false;
  const int64_t passes = ((int64_t)Sq * (H / Hkv) + 7) / 8, tiles = ((int64_t)max_pages * page_size + 31) / 32 + 8;
  return (int64_t)B * Hkv <= INT_MAX / passes / tiles;
}

}  // namespace

extern "C" {

int fsa_cache_page_bytes(int page_size, int Hkv, int D, int fmt, size_t* bytes) {
  if (!bytes || !page_ok(page_size) || Hkv <= 0 || Hkv > 65535 || (D != 64 && D != 128)) return FSA_ERR_INVALID_ARG;
  if (fmt != FSA_FMT_E2M1 && fmt != FSA_FMT_NVFP4) return FSA_ERR_UNSUPPORTED_FMT;
  *bytes = page_bytes_of(page_size, Hkv, D, fmt);
  return FSA_OK;
}

int fsa_cache_append(const fsa_cache* cache, const void* k, const void* v, const fsa_strides* k_strides,
                     const fsa_strides* v_strides, int B, int S, const int32_t* block_table, int max_pages,
                     const int32_t* lens, const int32_t* new_lens, int32_t* status, void* stream) {
  fsa::CacheIo a{};
  if (!k || !v) return FSA_ERR_INVALID_ARG;
  const int st = cache_io(cache, k, v, k_strides, v_strides, B, S, block_table, max_pages, lens, new_lens, status,
                          false, &a);
  if (st != FSA_OK) return st;
  return launch_status(fsa::launch_cache_append(a, static_cast<cudaStream_t>(stream)));
}

int fsa_cache_read(const fsa_cache* cache, void* k, void* v, const fsa_strides* k_strides,
                   const fsa_strides* v_strides, int B, int S, const int32_t* block_table, int max_pages,
                   const int32_t* lens, const int32_t* start, int32_t* status, void* stream) {
  fsa::CacheIo a{};
  if (!k && !v) return FSA_ERR_INVALID_ARG;
  const int st = cache_io(cache, k, v, k_strides, v_strides, B, S, block_table, max_pages, lens, start, status, true,
                          &a);
  if (st != FSA_OK) return st;
  return launch_status(fsa::launch_cache_read(a, static_cast<cudaStream_t>(stream)));
}

int fsa_qk_norm_rope(const fsa_norm_rope* r, void* stream) {
  if (!r || !r->q || !r->k || !r->q_out || !r->k_out || r->B <= 0 || r->S <= 0 || r->H <= 0 || r->Hkv <= 0 ||
      (r->D != 64 && r->D != 128) || (int64_t)r->B * r->S > INT_MAX || r->rotary < 0 || r->rotary > r->D ||
      r->rotary % 8 != 0 || (r->norm != 0 && r->norm != 1) || (r->interleaved != 0 && r->interleaved != 1) ||
      (r->norm && !(r->eps >= 0.0f && std::isfinite(r->eps))) || (!r->norm && (r->q_weight || r->k_weight)))
    return FSA_ERR_INVALID_ARG;
  fsa::RopeArgs a{};
  if (r->rotary > 0) {
    if (r->n_axes < 1 || r->n_axes > 3 || !r->pos || !r->inv_freq) return FSA_ERR_INVALID_ARG;
    int64_t pairs = 0;
    for (int i = 0; i < r->n_axes; ++i) {
      if (r->sections[i] < 0) return FSA_ERR_INVALID_ARG;
      pairs += r->sections[i];
    }
    if (pairs != r->rotary / 2) return FSA_ERR_INVALID_ARG;
  }
  for (const void* p : {r->q, r->k, r->q_weight, r->k_weight, (const void*)r->q_out, (const void*)r->k_out})
    if (!aligned(p, 16)) return FSA_ERR_INVALID_ARG;
  if (!aligned(r->pos, 4) || !aligned(r->inv_freq, 8)) return FSA_ERR_INVALID_ARG;
  if (!take_strides(&r->q_strides, r->B, r->S, r->H, false, &a.qs) ||
      !take_strides(&r->k_strides, r->B, r->S, r->Hkv, false, &a.ks) ||
      !take_strides(&r->q_out_strides, r->B, r->S, r->H, true, &a.qos) ||
      !take_strides(&r->k_out_strides, r->B, r->S, r->Hkv, true, &a.kos))
    return FSA_ERR_INVALID_ARG;
  a.q = static_cast<const uint16_t*>(r->q);
  a.k = static_cast<const uint16_t*>(r->k);
  a.qo = static_cast<uint16_t*>(r->q_out);
  a.ko = static_cast<uint16_t*>(r->k_out);
  a.wq = static_cast<const uint16_t*>(r->q_weight);
  a.wk = static_cast<const uint16_t*>(r->k_weight);
  a.pos = r->pos;
  a.inv_freq = r->inv_freq;
  a.B = r->B; a.S = r->S; a.H = r->H; a.Hkv = r->Hkv; a.D = r->D;
  a.half = r->rotary / 2;
  a.axes = r->rotary > 0 ? r->n_axes : 1;
  a.first1 = a.axes > 1 ? r->sections[0] : a.half;
  a.first2 = a.axes > 2 ? r->sections[0] + r->sections[1] : a.half;
  a.norm = r->norm;
  a.interleaved = r->interleaved;
  a.eps = r->eps;
  int sms = 0;
  if (!sm_count(&sms)) return FSA_ERR_NO_DEVICE;
  return launch_status(fsa::launch_qk_norm_rope(a, sms, static_cast<cudaStream_t>(stream)));
}

int fsa_attention_cache_workspace(const fsa_cache* cache, int B, int H, int Sq, int max_pages, size_t* bytes) {
  fsa::Cache c;
  if (!bytes) return FSA_ERR_INVALID_ARG;
  const int st = take_cache(cache, &c);
  if (st != FSA_OK) return st;
  if (!attn_shape_ok(B, H, c.Hkv, Sq, c.D, max_pages, cache->page_size)) return FSA_ERR_INVALID_ARG;
  int sms = 0;
  if (!sm_count(&sms)) return FSA_ERR_NO_DEVICE;
  size_t starts_at;
  *bytes = fsa::cache_attn_workspace(c, B, H, Sq, max_pages, sms, &starts_at);
  return FSA_OK;
}

int fsa_attention_cache(const fsa_cache_attn* c, void* stream) {
  if (!c) return FSA_ERR_INVALID_ARG;
  fsa::CacheAttnArgs a{};
  const int st = take_cache(c->cache, &a.c);
  if (st != FSA_OK) return st;
  const int Hkv = a.c.Hkv, D = a.c.D;
  if (!c->q || !c->out || !c->lens || !attn_shape_ok(c->B, c->H, Hkv, c->Sq, D, c->max_pages, c->cache->page_size) ||
      !table_ok(c->block_table, c->max_pages, c->cache->page_size) || !(std::fabs(c->scale) <= 1e30f) ||
      (c->causal != 0 && c->causal != 1) || (c->out_dtype != FSA_OUT_F32 && c->out_dtype != FSA_OUT_BF16) ||
      !aligned(c->q, 16) || !aligned(c->out, 16) || !aligned(c->workspace, 16) || !aligned(c->lens, 4) ||
      !aligned(c->q_lens, 4) || !aligned(c->lse, 4) || !aligned(c->status, 4))
    return FSA_ERR_INVALID_ARG;
  if (!take_strides(&c->q_strides, c->B, c->Sq, c->H, false, &a.qs) ||
      !take_strides(&c->out_strides, c->B, c->Sq, c->H, true, &a.os))
    return FSA_ERR_INVALID_ARG;
  int sms = 0;
  if (!sm_count(&sms)) return FSA_ERR_NO_DEVICE;
  const int G = c->H / Hkv, nt = fsa::cache_attn_ntiles(c->Sq * G);
  size_t starts_at;
  const size_t need = fsa::cache_attn_workspace(a.c, c->B, c->H, c->Sq, c->max_pages, sms, &starts_at);
  if (need > 0 && (!c->workspace || c->workspace_bytes < need)) return FSA_ERR_INVALID_ARG;
  a.q = static_cast<const uint16_t*>(c->q);
  a.out = c->out;
  a.lse = c->lse;
  a.table = c->block_table;
  a.lens = c->lens;
  a.q_lens = c->q_lens;
  a.partials = static_cast<float*>(c->workspace);
  a.starts = reinterpret_cast<int4*>(static_cast<char*>(c->workspace) + starts_at);
  a.B = c->B; a.H = c->H; a.Sq = c->Sq; a.G = G;
  a.CT = (c->Sq * G + 8 * nt - 1) / (8 * nt);
  // floor(2^32 / G) + 1 exceeds 2^32 / G by at most 1, so the product is exact for columns
  // below 2^32 / G
  a.g_mul = G > 1 && (uint64_t)c->Sq * G * G < (1ull << 32) ? (uint32_t)((1ull << 32) / G + 1) : 0;
  a.max_pages = c->max_pages;
  a.causal = c->causal;
  a.out_bf16 = c->out_dtype == FSA_OUT_BF16;
  a.q_sign = c->scale > 0.0f ? 1.0f : c->scale < 0.0f ? -1.0f : 0.0f;
  a.scale_log2 = c->scale == 0.0f ? 1.0f : (float)(std::fabs((double)c->scale) * 1.4426950408889634073599246810018921);
  a.status = c->status;
  a.timeout_ns = (uint64_t)(c->timeout_ms ? c->timeout_ms : 4000u) * 1000000ull;
  return launch_status(fsa::launch_cache_attn(a, nt, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
