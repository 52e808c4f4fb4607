/*
 * fsa.h -- C ABI of libfsa: MX block-scaled attention forward with a
 * reformulated softmax, for NVIDIA GB300 (sm_103a).
 *
 * Sources (by page title and section):
 *   "Fused-Softmax for efficient quantized attention" (The Singularity Report),
 *       abstract: QK^T and PV as MXFP8/MXFP6/MXFP4 GEMMs; softmax reformulated
 *       and approximated so its dominant work folds into the GEMMs; BF16
 *       attention as the comparison point.
 *   "Moving softmax to matrix operations speeds up AI inference by over 2x"
 *       (zot.news), summary, "Read it as" and the "How it works" figure: max
 *       subtraction and exponentiation folded into the score GEMM; the row
 *       maximum frozen speculatively with a fallback; a fast exponential;
 *       "Exp + MX Quant" fused; probabilities summed on the matrix unit.
 *   "EFQ-Softmax: Exp-Free Quantization for Softmax" (paper-with-me),
 *       abstract: per 32-element block an exponent-only scale from the local
 *       maximum and nonnegative E2M1 probability codes from one affine rule;
 *       the same operand feeds the P~V numerator and the P~1 denominator;
 *       final normalisation in high precision.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers, allocated and owned by the
 *     caller; the library keeps no reference after the call returns.  The
 *     library allocates no device memory on any entry point below.
 *   - `stream` is a cudaStream_t passed as void*; NULL means the legacy
 *     default stream.  Work is enqueued asynchronously; no entry point
 *     synchronises.
 *   - Return value: FSA_OK (0) or a negative FSA_ERR_* code.  Argument errors
 *     are detected on the host before any launch; nothing is enqueued then.
 *   - Shapes: B batch, H query heads, Hkv key/value heads (H % Hkv == 0; query
 *     head h reads kv head h / (H/Hkv)), Sq queries, Sk keys, head dim D in
 *     {64, 128}; the attention calls also need B*H <= 65535, Sq <= 65535*128
 *     and Sk <= 2^20 (else INVALID_ARG).  The key limit is one of accuracy: the
 *     fp32 accumulator in tensor memory, to which every key tile adds its
 *     products, drifts by a per-row factor that grows with the number of key
 *     tiles, as adds that drop low-order bits would (measured at 2^20 keys:
 *     below 5e-4 of the output, within the 2e-3 parity bound; at 2^22 keys up
 *     to 7e-3 with 8-bit P~).
 *     Causal masking is bottom-right aligned: key j is visible to
 *     query i iff j <= i + Sk - Sq.  A query with no visible key gets a zero
 *     output row.
 */
#ifndef FSA_H
#define FSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- status */
#define FSA_OK                   0
#define FSA_ERR_INVALID_ARG     -1  /* null pointer, bad shape, misaligned pointer */
#define FSA_ERR_UNSUPPORTED_FMT -2  /* e.g. E2M1_EFQ as a QK^T operand format */
#define FSA_ERR_LAUNCH          -3  /* CUDA runtime/driver error at launch */
#define FSA_ERR_TIMEOUT         -4  /* a bounded on-chip wait gave up (reported via fsa_stats) */
#define FSA_ERR_NO_DEVICE       -5  /* no sm_100-family device with tcgen05 */

/* ------------------------------------------------------- element formats */
/* OCP MX element types; E2M1_EFQ is the E2M1 operand produced by the EFQ
 * direct-code rule and is valid only as the PV format. */
typedef enum {
  FSA_FMT_E4M3 = 0,      /* MXFP8 */
  FSA_FMT_E2M3 = 1,      /* MXFP6 */
  FSA_FMT_E2M1 = 2,      /* MXFP4, P by exp then round-to-nearest-even */
  FSA_FMT_E2M1_EFQ = 3,  /* MXFP4, P by the EFQ affine rule (fmt_pv only) */
  FSA_FMT_E3M2 = 4,      /* MXFP6, the OCP MX E3M2 element type (bias 3, max 28) */
  FSA_FMT_NVFP4 = 5      /* NVFP4: E2M1 codes with one E4M3 scale per 16 elements
                          * (FSA_MX_ROWS only, i.e. Q and K, fmt_qk only); an
                          * operand format adjacent to the MX ones the
                          * Fused-Softmax brief names (abstract), from NVIDIA's
                          * public FP4 definition without its per-tensor scale */
} fsa_fmt;

/* ------------------------------------------------------------ MX tensors */
/* An MX tensor holds element codes plus one E8M0 scale byte (2^(byte-127))
 * per 32 consecutive elements along the contraction dimension.
 *
 * FSA_MX_ROWS (Q and K; blocks along D).  Source x[B][H][S][D] bf16.
 *   codes : [B*H][S][row_bytes], row_bytes = D (E4M3, E2M3, E3M2) or D/2
 *           (E2M1).  E4M3: one byte per element.  E2M3 and E3M2: each group of
 *           16 elements is 12 bytes of 6-bit codes packed least-significant-bit
 *           first, followed by 4 zero bytes.  E2M1: two elements per byte, the
 *           even element in the low nibble.
 *   scales: [B*H][ceil(S/128)][512] bytes: for row r of a 128-row tile and
 *           block b (b < D/32), byte (r%32)*16 + (r/32)*4 + b.  Slots with no
 *           data (rows >= S, blocks >= D/32) hold 0x7F.
 * FSA_MX_COLS_T (V; blocks along S, stored transposed, K-major for PV).
 *   codes : [B*H][D][Sp] elements, Sp = S rounded up to 128, packed as above
 *           along the key axis; codes of keys >= S are 0.
 *   scales: [B*H][Sp/128][512] bytes: for d (row of V^T) and key block b of
 *           a 128-key tile, byte (d%32)*16 + (d/32)*4 + b.  Rows d >= D hold
 *           0x7F; blocks of keys wholly >= S hold 0x7F.
 * The block scale is E = clamp(floor(log2 amax) - emax, -127, 127) (emax 8
 * for E4M3, 4 for E3M2, 2 for E2M3/E2M1), codes = round-to-nearest-even, saturating, of
 * x * 2^-E; a block with a non-finite element gets scale 0xFF.
 * FSA_FMT_NVFP4 (FSA_MX_ROWS only): codes as E2M1 above; one E4M3 scale byte
 *   per 16 elements along D: the E4M3 value nearest amax/6 (ties to even,
 *   saturating at 448), codes the E2M1 values nearest x/scale (saturating at 6;
 *   a zero scale gives zero codes; a non-finite block gets scale 0x7F, the
 *   E4M3 NaN, and zero codes).  scales: [B*H][ceil(S/128)][D/64][512] bytes:
 *   for row r of a 128-row tile and 16-element block b (b < D/16), byte
 *   (b/4)*512 + (r%32)*16 + (r/32)*4 + b%4; rows >= S hold 0x38 (1.0).   */
typedef enum { FSA_MX_ROWS = 0, FSA_MX_COLS_T = 1 } fsa_mx_layout;

typedef struct {
  void*    codes;    /* device, 16-byte aligned */
  uint8_t* scales;   /* device, 16-byte aligned */
  int32_t  fmt;      /* fsa_fmt of the codes (E4M3, E2M3, E2M1, E3M2 or NVFP4) */
  int32_t  layout;   /* fsa_mx_layout */
  int32_t  B, H, S, D;
} fsa_mx_tensor;

/* Bytes of the codes and scales buffers for an MX tensor. */
int fsa_mx_sizes(int B, int H, int S, int D, int layout, int fmt, size_t* codes_bytes, size_t* scales_bytes);

/* Quantise x_bf16 [B][H][S][D] (device, 16-byte aligned) into out->codes /
 * out->scales with the given layout and element format.  The shape, layout
 * and format fields of *out are written by the call.  One kernel launch on
 * `stream`, which writes every byte of both buffers; nothing is allocated and
 * nothing synchronises, so the call may be captured in a CUDA graph.  Cited:
 * MXFP8/6/4 GEMM operands ("Fused-Softmax for efficient quantized
 * attention", abstract). */
int fsa_mx_quantize(const void* x_bf16, int B, int H, int S, int D, int layout, int fmt,
                    fsa_mx_tensor* out, void* stream);

/* The operands of one attention call in one kernel launch: q [B][H][Sq][D]
 * and k [B][Hkv][Sk][D] into FSA_MX_ROWS tensors of format fmt_qk, v
 * [B][Hkv][Sk][D] into an FSA_MX_COLS_T tensor of format fmt_v (E2M1 for an
 * EFQ P~ V product).  Codes and scales are identical to three
 * fsa_mx_quantize calls; argument checks, field writes and launch behaviour
 * are the same as there.  Errors: FSA_ERR_INVALID_ARG (null or misaligned
 * pointer, bad shape), FSA_ERR_UNSUPPORTED_FMT (E2M1_EFQ as a storage
 * format), FSA_ERR_LAUNCH. */
int fsa_mx_quantize_qkv(const void* q_bf16, const void* k_bf16, const void* v_bf16, int B, int H, int Hkv,
                        int Sq, int Sk, int D, int fmt_qk, int fmt_v, fsa_mx_tensor* q_out,
                        fsa_mx_tensor* k_out, fsa_mx_tensor* v_out, void* stream);

/* ------------------------------------------------------ options and stats */
typedef enum {
  FSA_EXP_POLY = 0,   /* cubic interpolant of 2^f on the FMA pipe for every element */
  FSA_EXP_MUFU = 1,   /* hardware ex2.approx for every element */
  FSA_EXP_SPLIT = 2   /* key positions 4k+3 (of each 32-key block) the cubic, the others ex2.approx */
} fsa_exp_mode;

typedef enum {
  FSA_OUT_F32 = 0,    /* O as fp32 */
  FSA_OUT_BF16 = 1    /* O as bf16: the fp32 result rounded to nearest even */
} fsa_out_dtype;

/* Debug dumps of every key tile the kernel processes (a test instrument: the
 * P~ codes are the method's product, and the EFQ-Softmax page, abstract, defines
 * them as nonnegative E2M1 codes under exponent-only block scales).  All
 * pointers are device memory of the caller.  Query row r (r = (b*H + h)*Sq + i)
 * is dumped to slot row_slot[r] (row_slot NULL: slot r; a negative slot: not
 * dumped); N is the number of slots, NKT = ceil(Sk/128) key tiles.  Entries of
 * tiles a query tile does not process are left untouched (callers initialise
 * them).  The debug instance computes the same outputs as the production kernel,
 * bit for bit.
 *   s        : float    [N][NKT*128]  raw fp32 scores of the MMA (masked keys -inf)
 *   m        : float    [N][NKT]      frozen maximum M used for the tile's P~
 *   p        : uint32_t [N][NKT][32]  P~ code words as written to tensor memory:
 *                                     one byte per code (E4M3; E2M3 in the low 6
 *                                     bits) in words 0..31, or two E2M1 codes per
 *                                     byte (even key in the low nibble) in words 0..15
 *   p_scales : uint32_t [N][NKT]      byte b = E8M0 scale of the tile's 32-key block b
 *   row_slot : int32_t  [B*H*Sq]      optional slot of each query row */
typedef struct {
  float*    s;
  float*    m;
  uint32_t* p;
  uint32_t* p_scales;
  const int32_t* row_slot;
} fsa_debug_dump;

/* The EFQ direct-code rule (EFQ-Softmax page, abstract: an exponent-only block
 * scale from the local maximum, shifted scores in a normalised residual domain,
 * codes by a single affine rule; the page prints no constants).  Per 32-key block
 * with maximum shifted score tmax (log2 units):
 *     E    = clamp(floor(tmax + efq_phi) - 2, -127, 127)
 *     code = clamp(rne(efq_a * (t - E) + efq_b), 0, 7)
 * computed as one fused multiply-add per raw score s (t - E = s*c - (M + E)).
 * The defaults come from a scan of the rule family against fp64 exact attention
 * on the long-context workload (the error-floor criterion of the Fused-Softmax
 * brief, abstract). */
#define FSA_EFQ_A_DEFAULT   1.6875f
#define FSA_EFQ_B_DEFAULT   3.4375f
#define FSA_EFQ_PHI_DEFAULT 0.625f

typedef struct {
  float    delta;        /* fallback margin in log2 units, >= 0 (default 8): a later tile falls
                            back only when its maximum exceeds the frozen one by more than
                            delta; per-block scales make a stale maximum cost no precision.
                            0 is the literal test "any score exceeds the frozen maximum" */
  int32_t  exp_mode;     /* fsa_exp_mode (default FSA_EXP_MUFU: on sm_103a the hardware exp2
                            issues at twice the rate of earlier parts, and the cubic's
                            extra FMA-pipe instructions cost more than they save) */
  float    efq_a;        /* EFQ slope a (default FSA_EFQ_A_DEFAULT), finite, 0 < a <= 16 */
  float    efq_b;        /* EFQ offset b (default FSA_EFQ_B_DEFAULT), finite, |b| <= 64 */
  float    efq_phi;      /* EFQ block-scale reference point (default FSA_EFQ_PHI_DEFAULT), 0 <= phi < 1 */
  uint32_t timeout_ms;   /* limit of each on-chip wait (0: 4000 ms) */
  int32_t* row_fallbacks;/* optional device int32 [B][H][Sq]: fallback count per row */
  int32_t  inject_stall; /* test hook: 1 makes the MMA warp wait on a barrier nobody
                            arrives on, so the bounded wait expires (status TIMEOUT) */
  int32_t  schedule;     /* fsa_schedule (default FSA_SCHED_AUTO); the result does not
                            depend on it: both schedules compute bit-identical outputs */
  int32_t  out_dtype;    /* fsa_out_dtype of `out` (default FSA_OUT_F32) */
  int32_t  reserved;
  const fsa_debug_dump* debug;  /* optional (NULL: none): run the debug instance, which
                            also writes the per-tile dumps; per-query-tile schedule,
                            exp modes POLY and MUFU (else FSA_ERR_UNSUPPORTED_FMT) */
} fsa_opts;

typedef enum {
  FSA_SCHED_AUTO = 0,        /* persistent when query tiles average at most 32 key tiles
                                (short causal prefill), else one CTA per query tile; the
                                BF16 entry point always takes one CTA per query tile */
  FSA_SCHED_PER_TILE = 1,    /* one CTA per 128-row query tile */
  FSA_SCHED_PERSISTENT = 2   /* one CTA per SM, each walking a list of query tiles: a CTA's
                                setup, first loads, pipeline fill and drain are paid once
                                per SM instead of once per query tile */
} fsa_schedule;

typedef struct {                      /* device memory, zeroed by the caller */
  unsigned long long fallback_events; /* (row, tile) pairs whose score beat the frozen max */
  unsigned long long row_tiles;       /* (row, tile) pairs with at least one visible key */
  int32_t status;                     /* FSA_OK or FSA_ERR_TIMEOUT; after TIMEOUT the output
                                         is undefined */
  int32_t reserved;
} fsa_stats;

void fsa_default_opts(fsa_opts* opts);

/* ------------------------------------------------------------- attention */
/* O[B][H][Sq][D] fp32 = softmax(scale * Q K^T) V computed by the fused MX
 * algorithm: QK^T as a block-scaled MMA into tensor memory; the row maximum
 * frozen from the first key tile of 128, with a fallback that rescales the
 * accumulator when a later tile's maximum exceeds it by more than delta; per
 * 32-key block an exponent-only scale from the block maximum and codes by
 * exp-then-round (fmt_pv E4M3/E2M3/E2M1) or the EFQ rule (E2M1_EFQ);
 * P~ [V^|1] as a block-scaled MMA whose extra ones column accumulates the
 * denominator; O = O_acc / l in fp32.
 * q, k: FSA_MX_ROWS tensors in fmt_qk; v: FSA_MX_COLS_T tensor in the
 * element format of fmt_pv (E2M1 for E2M1_EFQ).  out: device fp32, 16-byte
 * aligned.  scale: softmax scale (e.g. 1/sqrt(D)). */
int fsa_attention_fwd(const fsa_mx_tensor* q, const fsa_mx_tensor* k, const fsa_mx_tensor* v, float* out,
                      int B, int H, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                      int fmt_qk, int fmt_pv, void* stream);

/* As fsa_attention_fwd with options and statistics: the frozen-maximum margin
 * (the fallback of "Moving softmax to matrix operations...", "Read it as"), the
 * exp2 path of the exp-then-round formats (its "fast method"), the EFQ rule's
 * constants (EFQ-Softmax page, abstract), the output dtype (`out` is fp32 or
 * bf16 [B][H][Sq][D] per opts->out_dtype, 16-byte aligned), the schedule, the
 * wait limit and the debug dumps.  opts NULL: defaults.  stats: device
 * fsa_stats (NULL: none; without stats a wait that times out is not reported).
 * Errors as fsa_attention_fwd, plus FSA_ERR_INVALID_ARG for options out of
 * range (negative or non-finite delta, exp_mode, EFQ constants, schedule,
 * out_dtype) and FSA_ERR_UNSUPPORTED_FMT for a debug run of a format pair or
 * exp mode without a debug instance. */
int fsa_attention_fwd_ex(const fsa_mx_tensor* q, const fsa_mx_tensor* k, const fsa_mx_tensor* v, void* out,
                         int B, int H, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                         int fmt_qk, int fmt_pv, const fsa_opts* opts, fsa_stats* stats, void* stream);

/* As fsa_attention_fwd_ex, with Q given as bf16 [B][H][Sq][D] (device, 16-byte
 * aligned) and quantised to fmt_qk inside the attention kernel's prologue, so Q
 * makes no round trip through HBM as MX codes (the Fused-Softmax brief, abstract:
 * MX operands of the attention GEMMs; the codes and scales are those of
 * fsa_mx_quantize, so the output is bit-identical to quantising Q first).  Runs
 * one CTA per query tile with the hardware exp2 (or EFQ P codes): a request for
 * the persistent schedule, another exp mode or a debug dump returns
 * FSA_ERR_UNSUPPORTED_FMT.  Other errors as fsa_attention_fwd_ex. */
int fsa_attention_fwd_qbf16(const void* q_bf16, const fsa_mx_tensor* k, const fsa_mx_tensor* v, void* out,
                            int B, int H, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                            int fmt_qk, int fmt_pv, const fsa_opts* opts, fsa_stats* stats, void* stream);

/* Rearrange V [B][Hkv][S][D] bf16 into V^T [B][Hkv][D][Sp] bf16 (Sp = S
 * rounded up to 128, zero padded) for the BF16 kernel. */
int fsa_bf16_transpose_v(const void* v, void* vt, int B, int Hkv, int S, int D, void* stream);

/* In-house baseline: the same kernel skeleton with BF16 operands and exact
 * online softmax (standard attention of the "How it works" figure, tiled with
 * the running maximum and historical rescaling that the EFQ page keeps
 * unchanged; rescale only when the maximum grows by more than 8 in log2
 * units).  q [B][H][Sq][D], vt from fsa_bf16_transpose_v, k [B][Hkv][Sk][D],
 * all bf16 device, 16-byte aligned; out fp32. */
int fsa_attention_fwd_bf16(const void* q, const void* k, const void* vt, float* out,
                           int B, int H, int Hkv, int Sq, int Sk, int D, int causal, float scale,
                           fsa_stats* stats, void* stream);

/* ------------------------------------------------- hybrid-format layer schedule */
/* One attention layer of a model that picks its MX formats per layer (the
 * Fused-Softmax brief, abstract: a hybrid MXFP6/MXFP4 schedule on a video
 * model).  Fields as the arguments of fsa_attention_fwd_ex; `out` is fp32 or
 * bf16 per the call's opts->out_dtype; `delta` is this layer's frozen-maximum
 * margin (>= 0); `stats` optional device fsa_stats of this layer. */
typedef struct {
  const fsa_mx_tensor* q;
  const fsa_mx_tensor* k;
  const fsa_mx_tensor* v;
  void*   out;
  int32_t B, H, Hkv, Sq, Sk, D, causal;
  float   scale;
  int32_t fmt_qk, fmt_pv;
  float   delta;
  fsa_stats* stats;
} fsa_layer;

/* Run n_layers layers back to back on `stream`, each with its own formats and
 * margin and the remaining options of `opts` (NULL: defaults; a debug dump is
 * refused, the per-row fallback buffer is not used).  Every layer's arguments
 * are checked before the first launch: on an argument error nothing is
 * enqueued.  Errors as fsa_attention_fwd_ex. */
int fsa_attention_fwd_layers(const fsa_layer* layers, int n_layers, const fsa_opts* opts, void* stream);

/* Host-side margin update driven by the fallback counts of a previous run (the
 * speculative maximum of "Moving softmax to matrix operations...", "Read it
 * as", falls back when the guess is wrong; a larger margin trades fallbacks for
 * accumulator headroom).  stats: HOST copies of each layer's fsa_stats; delta:
 * host array of the layers' margins, updated in place: a layer whose fallback
 * rate (events / row-tiles) is above target_rate gets delta + step, at most
 * max_delta; layers without evidence (status not FSA_OK, no row-tiles) keep
 * theirs.  FSA_ERR_INVALID_ARG for null arrays, step <= 0, a negative target or
 * maximum, or a delta outside [0, max_delta]. */
int fsa_tune_delta(const fsa_stats* stats, int n_layers, float target_rate, float step, float max_delta,
                   float* delta);

/* ------------------------------------------------------- from host memory */
/* Inputs and output of one attention call in HOST memory (page-locked memory lets
 * the copies run asynchronously and overlap; pageable memory works, without the
 * overlap).  q [B][H][Sq][D], k and v [B][Hkv][Sk][D] bf16; out [B][H][Sq][D] fp32
 * or bf16 per opts->out_dtype. */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void*       out;
} fsa_host_io;

/* The caller's device buffers for the same call: q, k, v bf16 of the host shapes,
 * out of the output's shape and dtype, and the three MX tensors (codes and scales
 * of fsa_mx_sizes bytes for q and k in FSA_MX_ROWS / fmt_qk and v in
 * FSA_MX_COLS_T / the storage format of fmt_pv).  All 16-byte aligned. */
typedef struct {
  void*          q;
  void*          k;
  void*          v;
  fsa_mx_tensor* q_mx;
  fsa_mx_tensor* k_mx;
  fsa_mx_tensor* v_mx;
  void*          out;
} fsa_device_io;

/* The attention of fsa_attention_fwd_ex (the Fused-Softmax brief, abstract; the
 * pages say nothing of where the operands live) on operands in host memory.  The
 * call is split into n_chunks groups of whole kv heads (a kv head with its H/Hkv
 * query heads; n_chunks <= 0: min(B*Hkv, 8), fewer when a group would hold under two
 * query tiles per SM), and for each group: Q, K and V are
 * copied host to device on a stream of the library's own, quantised
 * (fsa_mx_quantize_qkv) and attended on `stream` once they have landed, and O
 * copied back on a second stream of its own while the next group computes.  The
 * output is bit-identical to quantising and attending the whole call at once (every
 * head is computed by the same kernels on the same data).  Nothing is allocated on
 * the device; the two streams and the events are created by the call and released
 * when their work completes.  On return the work is enqueued: `stream` completes
 * after the last copy back, so synchronising it makes host->out valid.  The MX
 * tensors' shape, layout and format fields are written as fsa_mx_quantize_qkv
 * would.  opts as fsa_attention_fwd_ex (row_fallbacks: device [B][H][Sq]; a debug
 * dump is refused); stats accumulates over the groups.  Not for CUDA graph capture.
 * Errors: FSA_ERR_INVALID_ARG (null or misaligned pointer, bad shape or option),
 * FSA_ERR_UNSUPPORTED_FMT, FSA_ERR_LAUNCH (a stream, event, copy or launch failed;
 * what was enqueued before the failure still completes before `stream` does). */
int fsa_attention_fwd_host(const fsa_host_io* host, const fsa_device_io* dev, int B, int H, int Hkv, int Sq,
                           int Sk, int D, int causal, float scale, int fmt_qk, int fmt_pv, const fsa_opts* opts,
                           fsa_stats* stats, int n_chunks, void* stream);

/* ---------------------------------------------------------- serving: q and k */
/* Strides of a bf16 tensor indexed [B][S][heads][D], in elements; D is contiguous.
 * Those of dimensions longer than 1 are non-negative multiples of 8, and not 0 for an
 * output.  (Heads before positions, as fsa_mx_quantize takes them, is a choice of
 * strides.) */
typedef struct {
  int64_t b, s, h;
} fsa_strides;

/* Queries and keys from the projection to the attention, in one pass: RMS norm of each
 * head, y = x / sqrt(mean(x^2) + eps) * weight, and rotation of pairs of its elements by
 * the position.  Pair i < rotary/2 is (y[i], y[i + rotary/2]), or (y[2i], y[2i+1]) when
 * interleaved; it turns by pos[b][s][axis] * inv_freq[i].  sections[a] consecutive pairs
 * turn by axis a (one axis for text; time, height and width for images and video);
 * elements from `rotary` on pass unrotated.  fp32 arithmetic, angles good to 2^-24 of a
 * turn up to position 2^24 (2^-16 at 2^31) for |inv_freq| up to 1 and in proportion beyond,
 * one rounding to bf16.  The norm is of each head by itself, with one weight of D for all of
 * them; a model that normalises all heads of its projection together has this call without
 * norm for the rotation.
 *   q [B][S][H][D], k [B][S][Hkv][D]: bf16, device, 16-byte aligned, strided
 *   q_out, k_out: as q and k, strides of their own; may be q and k themselves (same
 *     pointer and strides), and must not overlap them or each other otherwise
 *   q_weight, k_weight: bf16 [D], 16-byte aligned, or NULL for ones (NULL without norm)
 *   pos: int32 [B][S][n_axes]; inv_freq: double [rotary/2] (radians a position);
 *     both device, unused when rotary is 0
 * One launch, nothing allocated: may be captured.  Errors: FSA_ERR_INVALID_ARG (null or
 * misaligned pointer, bad shape or strides, rotary not a multiple of 8 in 0..D, n_axes
 * not 1..3, sections that do not sum to rotary/2, eps negative or not finite),
 * FSA_ERR_NO_DEVICE, FSA_ERR_LAUNCH. */
typedef struct {
  const void*    q;
  const void*    k;
  void*          q_out;
  void*          k_out;
  fsa_strides    q_strides, k_strides, q_out_strides, k_out_strides;
  const void*    q_weight;
  const void*    k_weight;
  const int32_t* pos;
  const double*  inv_freq;
  int32_t        B, S, H, Hkv, D, rotary, n_axes;
  int32_t        sections[3];
  int32_t        norm;          /* 1: RMS norm, 0: none */
  int32_t        interleaved;
  float          eps;
} fsa_norm_rope;

int fsa_qk_norm_rope(const fsa_norm_rope* args, void* stream);

/* ------------------------------------------------------- serving: the K/V cache */
/* A pool of pages that holds keys and values in 4 bits (the MXFP4 and NVFP4 operand
 * formats above).  Blocks run along D for V as well as for K, so that a token is written
 * once and never again.  fmt FSA_FMT_E2M1: 32 elements a block, E8M0 scale; FSA_FMT_NVFP4:
 * 16 elements, E4M3 scale; scale and code rules as for the MX tensors above.
 * A page is [Hkv][page_size/16] groups of 16 tokens.  A group is
 *   16 rows of K codes, 16 rows of V codes      D/2 bytes each
 *   16 rows of K scales, 16 rows of V scales    D/32 (E2M1) or D/16 (NVFP4) bytes each
 * with the scale of block j in byte j, two codes to a byte (the even element in the low
 * nibble), and the bytes of a code row in the order of the attention's fragments:
 *   K: byte t*(D/8) + 2s + h holds elements 16s + 4t + 2h and the next (t < 4, h < 2)
 *   V: byte g*(D/16) + i holds elements 16i + 2g and the next (g < 8)
 * Which pages belong to a sequence, in order, is said by a row of a block table
 * (int32 [B][max_pages]); the caller hands out the pages. */
typedef struct {
  void*   pages;       /* device, 16-byte aligned, num_pages * fsa_cache_page_bytes */
  int64_t num_pages;   /* <= 2^31 - 1 */
  int32_t page_size;   /* tokens: a power of two, 16..1024 */
  int32_t Hkv, D;      /* Hkv 1..65535, D 64 or 128 */
  int32_t fmt;         /* FSA_FMT_E2M1 or FSA_FMT_NVFP4 */
} fsa_cache;

/* Bytes of a page (a multiple of 64). */
int fsa_cache_page_bytes(int page_size, int Hkv, int D, int fmt, size_t* bytes);

/* Quantise new keys and values into the cache.  k, v: bf16 [B][S][Hkv][D], strided,
 * 16-byte aligned.  lens[b] (int32, device): tokens of sequence b with the new ones;
 * new_lens[b]: how many are new, at most S (NULL: S each).  Row i < new_lens[b] becomes
 * token lens[b] - new_lens[b] + i; rows behind (padding) are not read.  Tokens at negative
 * positions or past the block table are dropped.  A page number outside 0..num_pages-1 is
 * not followed: its tokens are dropped, and *status (device int32, optional) becomes
 * FSA_ERR_INVALID_ARG.  Two tokens of one call must not share a place (two sequences whose
 * tables name one page for their new tokens); what such a place then holds is unspecified.
 * max_pages * page_size <= 2^30, B * (S/8 + 2) * Hkv < 2^31.  One launch, nothing allocated: may be captured.  Errors:
 * FSA_ERR_INVALID_ARG, FSA_ERR_UNSUPPORTED_FMT (fmt), FSA_ERR_LAUNCH. */
int fsa_cache_append(const fsa_cache* cache, const void* k, const void* v, const fsa_strides* k_strides,
                     const fsa_strides* v_strides, int B, int S, const int32_t* block_table, int max_pages,
                     const int32_t* lens, const int32_t* new_lens, int32_t* status, void* stream);

/* The projection's q, k and v of new tokens in one pass: q normalised and rotated into q_out
 * as fsa_qk_norm_rope does (the same bits), k normalised and rotated and v as they are into
 * the cache as fsa_cache_append puts them.  k is rounded once, to 4 bits: its codes and scales
 * are those of the exact values, for positions up to 2^24 and |inv_freq| up to 1 (angles
 * pos * inv_freq rounded to 64 bits); beyond, of values within the error of fsa_qk_norm_rope.
 * That is what it is for: from about a thousand new tokens on the two calls are the faster ones (16384 tokens
 * of 32+8 heads of 128: 94 us, and 76 for the two), for some hundreds this one.  A call whose rows of k
 * are all beyond 2^60, or not finite, takes 40 times as long.
 *   args: as fsa_qk_norm_rope, without k_out (NULL).  pos may be NULL with one axis: a token
 *     then turns by its place in its sequence, lens[b] - new_lens[b] + i.  q_out may be q, and
 *     must not overlap k or v.
 *   v: bf16 [B][S][Hkv][D] and its strides, block_table, lens, new_lens, status, dropped
 *     tokens and bad pages: as fsa_cache_append.  Row i < new_lens[b] of q is written whether
 *     its token is dropped or not; rows behind are neither read nor written.
 * One launch, nothing allocated: may be captured.  Errors: FSA_ERR_INVALID_ARG (as the two
 * calls; Hkv or D other than the cache's), FSA_ERR_UNSUPPORTED_FMT, FSA_ERR_NO_DEVICE,
 * FSA_ERR_LAUNCH. */
int fsa_cache_append_rope(const fsa_norm_rope* args, const fsa_cache* cache, const void* v, const fsa_strides* v_strides,
                          const int32_t* block_table, int max_pages, const int32_t* lens, const int32_t* new_lens,
                          int32_t* status, void* stream);

/* The values that the cache stands for (exact in bf16): row i of sequence b is token
 * start[b] + i (start NULL: 0) where that lies in 0..lens[b]-1; other rows of k and v are
 * left as they were.  k or v may be NULL.  Tokens past the block table, or of a page number
 * outside the pool, read as zeros (the latter sets *status as above).  Shapes, limits and
 * errors as fsa_cache_append. */
int fsa_cache_read(const fsa_cache* cache, void* k, void* v, const fsa_strides* k_strides,
                   const fsa_strides* v_strides, int B, int S, const int32_t* block_table, int max_pages,
                   const int32_t* lens, const int32_t* start, int32_t* status, void* stream);

/* Attention of few query rows over the cache (decode steps, guessed tokens; the cache is read
 * again for each 16 rows a kv head, so from about 60 on, with 64 dims from about 80, fsa_attention_chunk is
 * faster over many keys, eight sequences of 2048 or one of 32768; over fewer keys later: eight sequences of 500
 * from 90, one from some hundreds): O = softmax(scale Q K^T) V on the values the cache stands for; q is not
 * quantised, sums and softmax statistics are fp32, probabilities times V's scales are
 * rounded to f16 before the product with the codes of V (2^-11 relative, 2^-10 with
 * NVFP4; for products far below the largest block scale in V that the row sees, an absolute
 * 2^-33 of it, or of 2^-80 where all E8M0 scales are smaller; with NVFP4 block scales over 8 in V times the
 * scale).  V may have any magnitude that bf16 has.  Query head h reads kv head h / (H/Hkv).  Row i < q_lens[b] of sequence b
 * stands at position lens[b] - q_lens[b] + i and sees the keys up to its own position
 * (causal) or all lens[b]; lens counts the rows' own tokens, which are in the cache
 * already.  A row that sees nothing gives zeros (lse -inf).  Rows behind q_lens[b] are not
 * written.  The lengths are read on the device: a captured call follows them.
 *   q, out: [B][Sq][H][D] strided, 16-byte aligned; out bf16 or fp32 by out_dtype
 *   scale: of any sign, |scale| <= 1e30.  Keys of magnitudes up to 2^115, scale times q finite
 *     in fp32, and |scale| times the sum of |q k| below 2^126: a row beyond that may be NaN or
 *     zeros; the rows beside it are as without it
 *   lse: optional fp32 [B][Sq][H], natural log of the sum of exp(scale q k)
 *   lens: int32 [B], cut to max_pages * page_size; q_lens: int32 [B], cut to 0..Sq, or NULL (Sq)
 *   workspace: fsa_attention_cache_workspace bytes, 16-byte aligned; needs no initial
 *     value, and is the call's own while it runs (calls that may run at once, captured ones
 *     included, need one each)
 *   status: optional device int32: FSA_ERR_INVALID_ARG where a page number lay outside the
 *     pool (its keys are not seen), FSA_ERR_TIMEOUT where a wait for a copy ran out
 *     (timeout_ms; 0: 4000), the output then being undefined
 * B * Sq * H <= 2^27; B * Hkv * (Sq * H/Hkv / 8 + 1) * (max_pages * page_size / 32 + 9) < 2^31
 * (the kernels count tiles over all sequences in 32 bits).  Errors: FSA_ERR_INVALID_ARG, FSA_ERR_UNSUPPORTED_FMT,
 * FSA_ERR_NO_DEVICE, FSA_ERR_LAUNCH.  The work is laid out for the current device, which
 * must be the one of the pointers and the stream. */
typedef struct {
  const void*      q;
  void*            out;
  float*           lse;
  const fsa_cache* cache;
  const int32_t*   block_table;
  const int32_t*   lens;
  const int32_t*   q_lens;
  void*            workspace;
  size_t           workspace_bytes;
  int32_t*         status;
  fsa_strides      q_strides, out_strides;
  int32_t          B, H, Sq, max_pages, causal, out_dtype;
  float            scale;
  uint32_t         timeout_ms;
} fsa_cache_attn;

/* Bytes of the workspace of such a call on the current device: 0 where it needs none (short
 * block tables), and its workspace may then be NULL. */
int fsa_attention_cache_workspace(const fsa_cache* cache, int B, int H, int Sq, int max_pages, size_t* bytes);
int fsa_attention_cache(const fsa_cache_attn* args, void* stream);

/* As fsa_attention_cache, causal, with a window: of the keys up to its own position a row at
 * position p sees the last `window` (j > p - window; its own token is one) and the first
 * `sinks` of the sequence (j < sinks).  Only the pages of keys that some row sees are read.
 * window >= 1, sinks >= 0, args->causal 1, else FSA_ERR_INVALID_ARG.  The workspace is
 * fsa_attention_cache_window_workspace bytes. */
int fsa_attention_cache_window_workspace(const fsa_cache* cache, int B, int H, int Sq, int max_pages, int window, int sinks,
                                         size_t* bytes);
int fsa_attention_cache_window(const fsa_cache_attn* args, int window, int sinks, void* stream);

/* What fsa_attention_cache computes, for chunks of new tokens (a prompt's, or the next turn's
 * of a conversation): rows go 256 a kv head at a time over the cache, whose codes are turned
 * into 16-bit operands once for each 256.  Scores are sums of exact products in fp32, sums and
 * maxima fp32; q goes as f16, exact down to 2^-18 of its row's largest magnitude and off by at
 * most 2^-29 of that below.  Probabilities are rounded to f16 for the product with V
 * (2^-11 of each, or an absolute 2^-32 of the largest value for small ones); with E2M1, where V's block scales in
 * a tile's 32 keys (seen by the row or by others of its 256) leave 2^-23 .. 2^13, to bf16 (2^-8) for these keys; a block of
 * zeros has no such scale.  E2M1 keys up to 2^115, values up to 2^100; blocks of a key below 2^-36 of its largest lose bits,
 * as do keys below 2^-100 and values below 2^-126; a block of values that are all below 2^-124 counts as zeros.
 * |scale| times a row's largest sum of |q k| below 2^26: beyond, where a score's rounding in fp32 is more
 * than the softmax's distances, the row may be NaN or zeros.
 * A row that sees a token with a non-finite key or value is NaN as a whole, and so is a row of
 * q that is not finite; the rows beside it are as without it.
 * window and sinks as above; window 0: none (sinks 0 too), causal or not.
 * args as there, with a workspace of fsa_attention_chunk_workspace bytes: none for block tables of up to 512
 * tokens, else 2 * SMs * 256 * (D + 2) floats and a little more, whatever the rows (40 MB with 128 dims).
 * B * Sq * H <= 2^27; B * Hkv * ceil(Sq * H/Hkv / 256) * (ceil(max_pages * page_size / 128) + 4) < 2^31. */
int fsa_attention_chunk_workspace(const fsa_cache* cache, int B, int H, int Sq, int max_pages, size_t* bytes);
int fsa_attention_chunk(const fsa_cache_attn* args, int window, int sinks, void* stream);

/* ------------------------------------------------------ tensor-core peak probe */
/* Measurement instrument (the roofline denominator of the attention kernels; the
 * Fused-Softmax brief, abstract, quotes its kernels' throughput on the block-
 * scaled matrix cores).  Launches n_ctas CTAs (one per SM) that each issue
 * `iters` iterations of dense M=128, N=n (128 or 256), K=128 products from
 * shared-memory operand tiles into tensor memory, as 8 kind::f16 bf16 MMAs
 * (kind 0), 4 kind::mxf8f6f4 E4M3 block-scaled MMAs (kind 1), 2 kind::mxf4
 * E2M1 block-scaled MMAs (kind 2) or 2 kind::mxf4nvf4 MMAs on the same MXFP4
 * operands (E2M1, E8M0 scales, scale_vec::2X; kind 3).  *flops (host, optional) receives the
 * launch's 2*M*N*K*iters*n_ctas; time the launch with events on `stream`.
 * status: optional device int32, set to FSA_ERR_TIMEOUT if the final wait
 * (2 s) expires.  Errors: FSA_ERR_INVALID_ARG, FSA_ERR_LAUNCH. */
int fsa_mma_peak(int kind, int n, int n_ctas, long long iters, int32_t* status, double* flops, void* stream);

const char* fsa_status_string(int status);
int fsa_version(void);

#ifdef __cplusplus
}
#endif
#endif /* FSA_H */
