/*
 * fa4fp4.h -- C ABI of the GB300 (sm_103a) block-scaled FP4 attention library
 * with Direct-P.
 *
 * The method is the one described in "Hardware-Aware FP4 FlashAttention-4"
 * (arXiv:2609.04105; gist.science technical summary and the arXiv abstract):
 * Q and K quantized to E2M1 with power-of-two (E8M0) scales per 32 elements,
 * S = Q K^T on FP4 tensor cores, each score's offset from the running row max
 * mapped straight to an E2M1 probability code, P V on FP4 tensor cores with an
 * online-softmax rescale of O, and a causal backward that rebuilds P from the
 * saved quantized Q and K and uses FP8 E4M3 operands.
 *
 * Conventions shared by every call:
 *   - Pointers are DEVICE pointers, allocated and owned by the caller, except
 *     the host buffers of fa4fp4_fwd_host.  The library never allocates or
 *     frees memory and never synchronizes, except in fa4fp4_sync_status.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Every compute call is asynchronous on it; the return value
 *     reports host-side argument validation and launch errors only.  Device
 *     watchdog errors (a pipeline wait that ran out of time) are reported by
 *     fa4fp4_sync_status.
 *   - Tensors are dense and row-major in the layouts stated below; every
 *     pointer must be 16-byte aligned (FA4FP4_ERR_ALIGNMENT otherwise).
 *   - Supported shapes: d in {64, 128}; N >= 1; B, H >= 0; Hq % Hkv == 0;
 *     causal attention uses the same N for queries and keys, aligned top-left
 *     (key n is visible to query i iff n <= i).
 *   - An empty problem (B == 0, or H == 0 / Hq == 0) is a no-op: the call
 *     checks its shape and options, then returns FA4FP4_OK without inspecting
 *     its pointers (they may be NULL) and without launching anything.  (Sums
 *     over an empty problem that are outputs, fa4fp4_norm_rope_bwd's weight
 *     gradients and fa4bf16_cross_bwd's dk and dv, are written: zeros.)
 *   - softmax_scale <= 0 selects 1/sqrt(d).
 *   - No C++ exception crosses this boundary; there is no CPU fallback.
 *
 * Quantized tensor layouts ("qtensor": a codes buffer plus a scales buffer):
 *   blocks along d (FA4FP4_BLOCKS_ALONG_D), logical x[B][H][N][d]:
 *       codes  [B][H][N][d/2] bytes (MXFP4: two E2M1 codes per byte, element
 *              2i in the low nibble) or [B][H][N][d] bytes (MXFP8: E4M3)
 *       scales [B][H][N][d/32] E8M0 bytes
 *   blocks along N (FA4FP4_BLOCKS_ALONG_N), stored transposed, Np = N rounded
 *   up to a multiple of 128, positions >= N hold +0:
 *       codes  [B][H][d][Np/2] (MXFP4) or [B][H][d][Np] (MXFP8)
 *       scales [B][H][d][Np/32]
 */
#ifndef FA4FP4_H
#define FA4FP4_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA4FP4_API __attribute__((visibility("default")))
#else
#define FA4FP4_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA4FP4_OK = 0,
  FA4FP4_ERR_INVALID_ARG = 1,    /* null pointer, negative size, bad enum */
  FA4FP4_ERR_UNSUPPORTED = 2,    /* d not in {64,128}, Hq % Hkv != 0, ... */
  FA4FP4_ERR_ALIGNMENT = 3,      /* a pointer is not 16-byte aligned */
  FA4FP4_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed */
  FA4FP4_ERR_DEVICE_TIMEOUT = 5, /* a kernel's bounded wait expired */
  FA4FP4_ERR_WORKSPACE = 6,      /* workspace missing or too small */
  FA4FP4_ERR_DEVICE_INDEX = 7,   /* a cache call met a page index, length or count out of range */
  FA4FP4_ERR_DEVICE_NONFINITE = 8 /* a NaN or infinity was given to the cache */
} fa4fp4_status;

typedef enum { FA4FP4_FMT_MXFP4 = 0, FA4FP4_FMT_MXFP8_E4M3 = 1 } fa4fp4_format;
typedef enum { FA4FP4_BLOCKS_ALONG_D = 0, FA4FP4_BLOCKS_ALONG_N = 1 } fa4fp4_axis;
typedef enum { FA4FP4_OUT_F32 = 0, FA4FP4_OUT_BF16 = 1 } fa4fp4_out_dtype;

/* Bytes of the codes buffer of a quantized tensor; *scale_bytes (if not NULL)
 * receives the bytes of its scales buffer.  Returns 0 for invalid arguments. */
FA4FP4_API size_t fa4fp4_qtensor_bytes(int B, int H, int N, int d, int fmt, int axis, size_t* scale_bytes);

/* Block quantization (technical summary, Methodology 1 "Format Selection";
 * Methodology 2 "Gradient Formats").  x_bf16 is [B][H][N][d] bf16.  Each block
 * of 32 elements along `axis` gets the E8M0 exponent X = floor(log2(amax)) -
 * emax (emax 2 for E2M1, 8 for E4M3; OCP MX rule; clamped to [-127,127]); each
 * element is x * 2^-X rounded to nearest-even on the element grid, saturating,
 * with its sign kept.  Writes codes/scales in the layouts above. */
FA4FP4_API fa4fp4_status fa4fp4_quantize(const void* x_bf16, int B, int H, int N, int d, int fmt, int axis,
                              void* codes, void* scales, void* stream);

/* The three forward inputs in one launch: q [B][Hq][N][d] and k [B][Hkv][N][d]
 * to MXFP4 with blocks along d, v [B][Hkv][N][d] to MXFP4 with blocks along N
 * (the transposed V^T layout), byte for byte what fa4fp4_quantize writes for
 * each of them (same rule, layouts and sizes: fa4fp4_qtensor_bytes);
 * technical summary, Methodology 1 ("Format Selection": MXFP4 Q, K and V).
 * The transposes of V share the grid with the row blocks of Q and K.  All
 * buffers are device memory owned by the caller, 16-byte aligned; errors as
 * fa4fp4_fwd's dimension checks (d in {64,128}, Hq a multiple of Hkv). */
FA4FP4_API fa4fp4_status fa4fp4_quantize_qkv(const void* q_bf16, const void* k_bf16, const void* v_bf16,
                                             int B, int Hq, int Hkv, int N, int d, void* q_codes,
                                             void* q_scales, void* k_codes, void* k_scales,
                                             void* vt_codes, void* vt_scales, void* stream);

/* Direct-P forward (technical summary, Methodology 1 "Direct Mapping" and
 * "Consistent Normalization"; abstract).
 *   q: MXFP4 along d, [B][Hq][N][d];  k: MXFP4 along d, [B][Hkv][N][d];
 *   vt: MXFP4 along N (transposed V), [B][Hkv][d][Np].
 *   Query head h reads kv head h / (Hq/Hkv).
 * Per 128-query tile, key tiles of 128 are visited in ascending order; for
 * key tile j the running max m_j = max(m_{j-1}, row max of S_j); each score s
 * gets the E2M1 code #{k : fmaf(s, c, -fl32(m_j*c)) >= T_k}, c =
 * fl32(softmax_scale*log2 e), T_k the smallest FP32 x with RNE_E2M1(6*2^x) >=
 * the k-th E2M1 magnitude; P blocks carry the unit E8M0 scale; O and the
 * normalizer l are rescaled by 2^(c(m_{j-1}-m_j)) before P_j V_j is added and
 * l accumulates the same code values.  Output o = O/l ([B][Hq][N][d], f32 or
 * bf16 per out_dtype) and, if lse != NULL, lse[B][Hq][N] = softmax_scale*m +
 * ln(l/6) (f32). */
FA4FP4_API fa4fp4_status fa4fp4_fwd(const void* q_codes, const void* q_scales, const void* k_codes,
                         const void* k_scales, const void* vt_codes, const void* vt_scales,
                         int B, int Hq, int Hkv, int N, int d, float softmax_scale, int causal,
                         void* o, int out_dtype, float* lse, void* stream);

/* The inference step end to end on HOST buffers: bf16 q [B][Hq][N][d] and k,
 * v [B][Hkv][N][d] in host memory, o (f32 or bf16 per out_dtype,
 * [B][Hq][N][d]) and lse (nullable, f32 [B][Hq][N]) written to host memory;
 * on the device, fa4fp4_quantize_qkv and fa4fp4_fwd (technical summary,
 * Methodology 1: MXFP4 Q, K, V and the Direct-P forward), with the same
 * results as those two calls on the same data.  The pages have no
 * counterpart; this is the library's end-to-end entry point.  The work is cut
 * into chunks of consecutive (batch element, kv head) units with their query
 * heads, the last chunk a single unit; each chunk's inputs are copied in on
 * an internal stream, quantized and attended alternately on `stream` and a
 * second internal stream, and copied out on a third, two chunks' staging
 * buffers in flight, so that the copies overlap the compute.
 * Host buffers should be page-locked (cudaHostAlloc / cudaHostRegister) for
 * the copies to overlap; q, k, v, o must be 16-byte aligned and lse 4-byte
 * aligned.  `workspace` is DEVICE memory of at least
 * fa4fp4_fwd_host_workspace_bytes(B, Hq, Hkv, N, d) bytes, 16-byte aligned
 * (FA4FP4_ERR_WORKSPACE if missing or too small), used as staging; calls in
 * flight at the same time need their own workspaces.  The call is
 * asynchronous on `stream`: later work on `stream` sees o and lse in host
 * memory, and the call starts after earlier work on `stream`.  The first call
 * on a device creates three streams and seven events on it, kept until the
 * process exits.  Other errors as fa4fp4_fwd's; all checks are made before
 * anything is enqueued, and a CUDA failure while enqueuing returns
 * FA4FP4_ERR_CUDA with the chunks before it already enqueued. */
FA4FP4_API size_t fa4fp4_fwd_host_workspace_bytes(int B, int Hq, int Hkv, int N, int d);
FA4FP4_API fa4fp4_status fa4fp4_fwd_host(const void* q_host, const void* k_host, const void* v_host, int B,
                                         int Hq, int Hkv, int N, int d, float softmax_scale, int causal,
                                         void* o_host, int out_dtype, float* lse_host, void* workspace,
                                         size_t workspace_bytes, void* stream);

/* The FP8 P/V training route of the forward (technical summary, Methodology 2
 * "Stability Constraint" and Training Performance: the retained training route
 * keeps FP8 probabilities and values).  Same arguments, layouts and errors as
 * fa4fp4_fwd except V: v8_codes/v8_scales is V quantized to MXFP8 with blocks
 * along N (fa4fp4_quantize with FA4FP4_FMT_MXFP8_E4M3, FA4FP4_BLOCKS_ALONG_N:
 * E4M3 codes [B][Hkv][d][Np], scales [B][Hkv][d][Np/32]).  Per 128-key tile
 * in ascending order: S = Q K^T on FP4 tensor cores, running max m, p =
 * 2^x with x = fl32(fl32(s - m) c) in FP32 (hardware exponential; the row max
 * gets p = 1 exactly), P rounded to E4M3
 * with one E8M0 scale per 32 keys (the least X with amax <= 448 * 2^X, so no
 * element saturates), O += P V and l += P 1 on
 * FP8 tensor cores (kind::mxf8f6f4), eager rescale when m grows.  Outputs
 * O / l and LSE = softmax_scale * m + ln(l). */
FA4FP4_API fa4fp4_status fa4fp4_fwd_fp8pv(const void* q_codes, const void* q_scales, const void* k_codes,
                                          const void* k_scales, const void* v8_codes, const void* v8_scales,
                                          int B, int Hq, int Hkv, int N, int d, float softmax_scale, int causal,
                                          void* o, int out_dtype, float* lse, void* stream);

/* NVFP4 block quantization along d (technical summary, Methodology 1
 * "Format Selection": NVFP4 for Q and K, for its fine-grained scaling; the
 * public NVFP4 layout).  x_bf16 is [B][H][N][d] bf16.  Writes codes
 * [B][H][N][d/2] (E2M1, element 2i in the low nibble), scales [B][H][N][d/16]
 * (unsigned E4M3, one per 16 elements) and *ts, the tensor's FP32 scale, in
 * device memory.  Every step is an FP32 operation rounded to nearest: ts =
 * amax/2688 (1 for an all-zero tensor), block scale E4M3(amax_b / (6 ts)),
 * element E2M1(x / (block scale * ts)), saturating, sign kept; a block whose
 * scale rounds to zero gets signed zeros.  Three launches on `stream` (tensor
 * amax, tensor scale, blocks); *ts is also their scratch word. */
FA4FP4_API fa4fp4_status fa4fp4_quantize_nvfp4(const void* x_bf16, int B, int H, int N, int d, void* codes,
                                               void* scales, float* ts, void* stream);

/* The forward with NVFP4 Q and K (from fa4fp4_quantize_nvfp4): q_ts and k_ts
 * point to their device tensor scales.  S = Q K^T runs as tcgen05 kind::mxf4nvf4
 * (UE4M3 scales per 16); the two tensor scales fold into the softmax scale,
 * fl32(fl32(softmax_scale * q_ts) * k_ts), which also enters the LSE.  fp8pv
 * selects the P/V path: 0 = Direct-P with V^T as MXFP4 (fa4fp4_fwd), 1 = the
 * FP8 P/V route with V^T as MXFP8 (fa4fp4_fwd_fp8pv).  Other arguments and
 * errors as fa4fp4_fwd. */
FA4FP4_API fa4fp4_status fa4fp4_fwd_nvfp4(const void* q_codes, const void* q_scales, const float* q_ts,
                                          const void* k_codes, const void* k_scales, const float* k_ts,
                                          const void* vt_codes, const void* vt_scales, int B, int Hq, int Hkv,
                                          int N, int d, float softmax_scale, int causal, int fp8pv, void* o,
                                          int out_dtype, float* lse, void* stream);

/* Direct-P forward (or the FP8 P/V route, fp8pv = 1) with Q in bf16: Q is
 * quantized to MXFP4 (E8M0 per 32 along d, the fa4fp4_quantize rule) inside
 * the forward's prologue, so an inference step reads Q once and needs no
 * separate pass over it (technical summary, Methodology 2 "Gradient Formats":
 * quantization happens where the operands are produced, not as a pass of its
 * own).  q: bf16 [B][Hq][N][d]; k, vt as in fa4fp4_fwd (vt MXFP8 along N when
 * fp8pv = 1).  Results are identical, bit for bit, to fa4fp4_quantize of Q
 * followed by fa4fp4_fwd (fa4fp4_fwd_fp8pv).  Errors as fa4fp4_fwd. */
FA4FP4_API fa4fp4_status fa4fp4_fwd_qbf16(const void* q, const void* k_codes, const void* k_scales,
                               const void* vt_codes, const void* vt_scales, int B, int Hq, int Hkv,
                               int N, int d, float softmax_scale, int causal, int fp8pv, void* o,
                               int out_dtype, float* lse, void* stream);

/* K (MXFP4 along d) and V (MXFP4 along N, transposed) in one launch: the
 * operands fa4fp4_fwd_qbf16 takes quantized.  Byte-identical to two
 * fa4fp4_quantize calls.  k, v: bf16 [B][Hkv][N][d]; outputs in the layouts
 * of fa4fp4_qtensor_bytes. */
FA4FP4_API fa4fp4_status fa4fp4_quantize_kv(const void* k, const void* v, int B, int Hkv, int N, int d,
                                 void* k_codes, void* k_scales, void* vt_codes, void* vt_scales,
                                 void* stream);

/* Bytes of caller-provided workspace fa4fp4_bwd needs. */
FA4FP4_API size_t fa4fp4_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d);

/* Quantized causal backward (technical summary, Methodology 2 "Quantized
 * Causal Backward": P recomputed from the forward's FP4 Q/K and its LSE;
 * FP8 copies of Q, K and V blocked along each product's contraction axis;
 * abstract: FP8 gradient operands).
 *   q4, k4: the forward's MXFP4 Q/K (along d);
 *   q8c, k8c: MXFP8 Q/K blocked along N ([B][H][d][Np] transposed views);
 *   v8r: MXFP8 V blocked along d ([B][Hkv][N][d]);
 *   o: forward output [B][Hq][N][d] (f32 or bf16 per o_dtype);
 *   dout: upstream gradient, bf16 [B][Hq][N][d];  lse: f32 [B][Hq][N].
 * Computes P = 2^x with x = fl32(s' c), s' = S + fl32(-fl32(lse*log2 e) / c)
 * accumulated by the tensor core (S the FP4 product, c = scale*log2 e; within
 * a few units in the last place of fmaf(S, c, -fl32(lse*log2 e))),
 * D = rowsum(dO*O), the MXFP8
 * views of dO (blocks along d and blocks of 32 queries), dP = dO V^T, dS =
 * P*(dP-D), and, with P and dS quantized to MXFP8 (P and dS in blocks of 32
 * queries for dV/dK, dS in blocks of 32 keys for dQ; P's blocks take the
 * least X with amax <= 448 * 2^X, dS's the OCP MX exponent):
 *   dV = P^T dO, dK = scale * dS^T Q, dQ = scale * dS K
 * summed over the query heads of each kv head.  dq [B][Hq][N][d], dk/dv
 * [B][Hkv][N][d], all f32, fully overwritten.  `workspace` must hold
 * fa4fp4_bwd_workspace_bytes(...) bytes (FA4FP4_ERR_WORKSPACE otherwise); it
 * receives the MXFP8 views of dO and, per query row, -fl32(lse*log2 e) / c and
 * -D as bf16 parts (16 bytes), and must not be shared with another
 * call in flight.  d = 64 or 128. */
FA4FP4_API fa4fp4_status fa4fp4_bwd(const void* q4_codes, const void* q4_scales, const void* k4_codes,
                         const void* k4_scales, const void* q8c_codes, const void* q8c_scales,
                         const void* k8c_codes, const void* k8c_scales, const void* v8r_codes,
                         const void* v8r_scales, const void* o, int o_dtype, const void* dout,
                         const float* lse, int B, int Hq, int Hkv, int N, int d,
                         float softmax_scale, int causal, float* dq, float* dk, float* dv,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Size of the fixed device scratch array used by fa4fp4_bwd_noalloc. */
#define FA4FP4_BWD_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/* fa4fp4_bwd for callers that cannot allocate device memory (plugins whose
 * host framework owns every device allocation, runtimes that forbid
 * allocation after start-up, code whose device memory is budgeted up front).
 * The paper has no counterpart: this is a deployment variant of fa4fp4_bwd.
 * Same arguments and results as fa4fp4_bwd without the workspace, and the
 * same status for a bad argument; the scratch is a fixed
 * FA4FP4_BWD_NOALLOC_SCRATCH_BYTES device array inside this library (held by
 * every GPU that loads it until exit).  Returns FA4FP4_ERR_WORKSPACE when
 * fa4fp4_bwd_workspace_bytes(...) exceeds that size.  Allocates nothing.
 * The first call on a device looks up the array's device address on that
 * device; make that first call before any stream capture.  All calls share
 * the array: calls that overlap on the GPU (other streams or host threads)
 * race on it. */
FA4FP4_API fa4fp4_status fa4fp4_bwd_noalloc(
    const void* q4_codes, const void* q4_scales, const void* k4_codes, const void* k4_scales,
    const void* q8c_codes, const void* q8c_scales, const void* k8c_codes, const void* k8c_scales,
    const void* v8r_codes, const void* v8r_scales, const void* o, int o_dtype, const void* dout,
    const float* lse, int B, int Hq, int Hkv, int N, int d, float softmax_scale, int causal,
    float* dq, float* dk, float* dv, void* stream);

/* BF16 FlashAttention forward, the speedup reference for fa4fp4_fwd
 * (technical summary, Results: the BF16 kernel its speedups are measured
 * against).  q [B][Hq][N][d], k/v
 * [B][Hkv][N][d] bf16; exact online softmax with P rounded to bf16 for the
 * P V product.  o as in fa4fp4_fwd; lse (nullable) = natural-log LSE. */
FA4FP4_API fa4fp4_status fa4bf16_fwd(const void* q, const void* k, const void* v, int B, int Hq, int Hkv,
                          int N, int d, float softmax_scale, int causal, void* o, int out_dtype,
                          float* lse, void* stream);

/* Direct-P code map on its own, with the device routines fa4fp4_fwd uses
 * (technical summary, Methodology 1 "Direct Mapping", which allows hardware
 * exponentials for part of the classification).
 * For every score: codes[i] = #{k : fmaf(s[i], c, -fl32(m*c)) >= T_k}.
 * native_exp = 0 computes it with the threshold count; native_exp = 1 with
 * the forward's route: e = ex2(x), codes of 6e(1-2^-18) and 6e(1+2^-18), the
 * threshold count only where those two differ.  Both give identical codes.
 * s: n FP32 scores, codes: n bytes (device arrays). */
FA4FP4_API fa4fp4_status fa4fp4_directp_codes(const float* s, int64_t n, float m, float c,
                                              int native_exp, uint8_t* codes, void* stream);

/* Watchdog self-test: launches one CTA whose pipeline wait can never be
 * satisfied, bounded by limit_ns (0 < limit_ns <= 2e9).  The wait expires,
 * the kernel returns, and the next fa4fp4_sync_status reports
 * FA4FP4_ERR_DEVICE_TIMEOUT; the context stays usable.  Exercises the same
 * bounded-wait routine every kernel of the library uses (2 s limit). */
FA4FP4_API fa4fp4_status fa4fp4_watchdog_selftest(int64_t limit_ns, void* stream);

/* The 8-bit key/value cache: a paged pool of K and V as E4M3 codes with one
 * E8M0 scale per page and head, the calls that fill it, attend over it, read
 * it sparsely and cut it back.
 *
 * A pool has num_pages pages of `page` tokens (16, 32, 64 or 128) for Hkv heads
 * of d (64 or 128):
 *     k_codes, v_codes    [num_pages][Hkv][page][d] E4M3 bytes
 *     k_scales, v_scales  [num_pages][Hkv] E8M0 bytes
 *     k_bounds            [num_pages][Hkv][2][d] E4M3 bytes: the least and the
 *                         greatest K code of the page's tokens, elementwise,
 *                         under the page's K scale
 * and holds any number of sequences: sequence b's token i lies in slot i % page
 * of pool page page_table[b][i / page] (int32, [B][max_pages], device memory),
 * and lens[b] (int32, device memory) is its number of tokens, at most
 * max_pages * page.  Calls that only read may share pages among sequences;
 * fa4fp4_cache_append and the destination of fa4fp4_cache_evict need pages of
 * their own.  Code bytes in [0, lens) are finite (fa4fp4_cache_append writes no
 * others); what lies behind a sequence's end may be anything.
 *
 * The lengths and page indexes are device data, so the host cannot check them.
 * Every kernel does: a page index outside the pool, a length or count outside
 * its range, or a token without room in the table is not followed (its keys
 * count as absent, its tokens are not stored), nothing out of bounds is read or
 * written, and the next fa4fp4_sync_status returns FA4FP4_ERR_DEVICE_INDEX.
 *
 * page_table, lens, q_lens, n_new, pages, weights and lse inputs need 4-byte
 * alignment, all else 16-byte.  num_pages, max_pages >= 1; B <= 65535, Hkv <=
 * 32767, max_pages * page <= 2^30, B * Hq * T < 2^31.  T == 0 is an empty
 * problem too.  The calls read the structure during the call only. */
typedef struct {
  void* k_codes;
  void* v_codes;
  void* k_scales;
  void* v_scales;
  void* k_bounds;
  int num_pages, Hkv, page, d;
} fa4fp4_cache;

/* Stores the new tokens k, v (bf16 [B][Hkv][T][d]) of every sequence behind its
 * lens[b] tokens: n_new[b] <= T of them (NULL: T).  lens is not changed.  Per
 * page, head and tensor: X = the least integer >= -127 with |x| <= 448 * 2^X
 * for all new tokens x of the page, at least the page's exponent when the page
 * already holds tokens (in slots before lens[b]); codes E4M3(x * 2^-X) rounded
 * to nearest even; when X grows the older codes become E4M3(code * 2^(X_old -
 * X)).  (The OCP exponent of fa4fp4_quantize would saturate magnitudes above
 * 448 * 2^X.)  k_bounds follows.  Slots behind the new end are not touched.  A
 * NaN is stored as 0, an infinity as the largest code of its sign; neither
 * counts for X, and the next fa4fp4_sync_status returns
 * FA4FP4_ERR_DEVICE_NONFINITE. */
FA4FP4_API fa4fp4_status fa4fp4_cache_append(const fa4fp4_cache* cache, const void* k, const void* v,
                                             const int* page_table, const int* lens, const int* n_new, int B,
                                             int max_pages, int T, void* stream);

/* Attention of T new query tokens per sequence over the cache.  q: bf16
 * [B][Hq][T][d], query head h reads kv head h / (Hq / Hkv); lens counts the new
 * tokens in (append first); sequence b has q_lens[b] <= T query tokens (NULL:
 * T), its last ones: token t sees keys 0 .. lens[b] - q_lens[b] + t when
 * causal, else all.  pages != NULL (int32 [B][Hkv][T][n_sel], as
 * fa4fp4_cache_select writes it): token t of kv head hk sees, of those keys,
 * only the ones in the pages listed for it (indexes into the sequence's row of
 * page_table, -1 for none; a page listed twice counts twice); n_sel = 0
 * without it.
 *   s = softmax_scale * q.k, o = softmax(s) v, lse = ln sum e^s (nullable)
 * o: [B][Hq][T][d], f32 or bf16 per out_dtype; lse: f32 [B][Hq][T].  A token
 * that sees no key gets o = 0 and lse = -inf; rows t >= q_lens[b] are not
 * written.  The products are exact in the codes, the sums FP32.  P is rounded
 * to f16 (half a step: 2^-11) under a power of two that takes V's page scales
 * in, so that a P far below the largest V of its 128 keys (seen or not) is off by
 * 2^-36 of that V at most, or by 2^-90 of a far larger sum that it is added to;
 * f32 output takes P as a sum of two f16 (2^-22).  Scores up to
 * 2^22 in magnitude; beyond, the rounding of their maximum takes P out of its
 * range.  The result does not depend on anything but the arguments.  (More than
 * 64 rows Hq / Hkv * T are fastest with bf16 output and without pages: f32 output
 * reads the keys again for every 16 rows.)  `workspace`: at least
 * fa4fp4_cache_fwd_workspace_bytes(...) bytes of device memory
 * (FA4FP4_ERR_WORKSPACE otherwise), for this call alone while it runs; it needs no
 * initialisation, but after FA4FP4_ERR_DEVICE_TIMEOUT zeros before its next use. */
FA4FP4_API size_t fa4fp4_cache_fwd_workspace_bytes(int B, int Hq, int Hkv, int T, int d, int page, int max_pages,
                                                   int n_sel);
FA4FP4_API fa4fp4_status fa4fp4_cache_fwd(const fa4fp4_cache* cache, const void* q, const int* page_table,
                                          const int* lens, const int* q_lens, const int* pages, int B, int Hq, int T,
                                          int max_pages, int n_sel, float softmax_scale, int causal, void* o,
                                          int out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream);

/* The pages whose keys could score highest, for every query token and kv head.
 * Among the pages that hold keys which token t sees (causal), the one with its
 * last visible key is taken, and of the others those with the highest
 *   sum over the kv head's query heads, sum over dims of max(q lo, q hi)
 * (lo, hi: the page's bounds as values), ties to the lowest page, n_sel in all;
 * all of them where there are no more.  pages (int32 [B][Hkv][T][n_sel])
 * receives them in ascending order, then -1; rows t >= q_lens[b] are all -1.
 * The set is that of the real-valued bounds: FP32 sums decide only where their
 * error bounds allow it, the rest is evaluated in 64 bits.  max_pages <= 2^18.
 * `workspace` as for fa4fp4_cache_fwd; up to 16384 pages it needs none (its size
 * is 0 and it may be NULL). */
FA4FP4_API size_t fa4fp4_cache_select_workspace_bytes(int B, int Hkv, int T, int max_pages);
FA4FP4_API fa4fp4_status fa4fp4_cache_select(const fa4fp4_cache* cache, const void* q, const int* page_table,
                                             const int* lens, const int* q_lens, int B, int Hq, int T, int max_pages,
                                             int n_sel, int* pages, void* workspace, size_t workspace_bytes,
                                             void* stream);

/* The attention weight that every cached token received from these queries:
 *   weight_out[b][hk][j] = weight_in[b][hk][j] + sum over the query heads of hk
 *                          and the tokens t that see j of e^(s - lse)
 * for j < lens[b], with fa4fp4_cache_fwd's arguments and the lse that it wrote
 * (rows with an infinite lse add nothing).  The scores are sums of exact products
 * in the tensor cores' FP32, which cuts where it adds, and the exponential is the
 * native one: for scores of ordinary size what is received is off by 2^-23 of its
 * norm, a single weight by up to 2^-20.  weights: f32 [B][Hkv][max_pages * page];
 * weight_out may be weight_in; entries j >= lens[b] are not written.  `workspace`
 * as for fa4fp4_cache_fwd; below 80 query rows per kv head (Hq / Hkv * T) it
 * needs none (its size is 0 and it may be NULL). */
FA4FP4_API size_t fa4fp4_cache_weigh_workspace_bytes(int B, int Hq, int Hkv, int T, int d);
FA4FP4_API fa4fp4_status fa4fp4_cache_weigh(const fa4fp4_cache* cache, const void* q, const float* lse,
                                            const int* page_table, const int* lens, const int* q_lens, int B, int Hq,
                                            int T, int max_pages, float softmax_scale, int causal,
                                            const float* weight_in, float* weight_out, void* workspace,
                                            size_t workspace_bytes, void* stream);

/* Cuts every sequence back to `budget` tokens per kv head: the `recent` newest
 * and of the others those with the largest weight (f32 [B][Hkv][max_pages *
 * page]; NaN below everything), ties to the lowest position; all where there
 * are no more than `budget`.  The kept tokens go, in order, into the pages
 * dst_table[b][0 ..] (int32 [B][dst_pages] with dst_pages * page >= budget;
 * pages of the same pool that no sequence of the call reads and no other row
 * writes), fitted to the destination's scales by the append's rule.  Sequence b
 * is then dst_table's row with new_lens[b] = min(lens[b], budget) tokens (new_lens
 * may be lens).
 * kept: int32 [B][Hkv][budget], the kept positions in ascending order, then -1.
 * weight_out (nullable): f32 [B][Hkv][dst_pages * page], the kept tokens'
 * weights, then 0; not the weight array itself.  0 <= recent <= budget,
 * budget >= 1. */
FA4FP4_API fa4fp4_status fa4fp4_cache_evict(const fa4fp4_cache* cache, const int* page_table, const int* lens,
                                            const float* weight, const int* dst_table, int B, int max_pages,
                                            int dst_pages, int budget, int recent, int* new_lens, int* kept,
                                            float* weight_out, void* stream);

/* Operators around the attention calls: norm and rotation of queries and keys,
 * and attention of queries to keys of another length.  Their tensors may be
 * strided views (slices of a fused projection, transposes of [B][N][H][d]):
 * logical [B][H][N][d], element (b, h, n, i) at ptr + b stride_b + h stride_h + n
 * stride_n + i, strides in elements.  The last dimension is dense; ptr is 16-byte
 * aligned, and so is every row: strides (of dimensions larger than 1) are
 * multiples of 16 bytes, at least 0 and at most 2^40 bytes.  An input may have
 * strides of 0 (a broadcast).  The rows of an output overlap neither each other nor,
 * where not said otherwise, anything else of the call.  d is 64 or 128; B N is at
 * most 2^30, heads are at most 2^20, rows in all at most 2^36, and for the attention B
 * Hq Nq and B Hkv Nk are below 2^31, B Hq at most 2^24 (FA4FP4_ERR_UNSUPPORTED). */
typedef struct {
  void* ptr;
  int64_t stride_b, stride_h, stride_n;
} fa4fp4_heads;

/* The rotation by position.  Channel pair i < d / 2 is (i, i + d / 2), or (2i,
 * 2i + 1) when interleaved, and turns by positions[axis(i)] * freqs[i] radians;
 * the first sections[0] pairs belong to axis 0, the next sections[1] to axis 1 and
 * so on (1 to 4 axes, sections sum to d / 2).  positions: int32 in DEVICE memory,
 * [B][axes][N], or [axes][N] for all sequences when shared, 4-byte aligned, of any
 * sign.  sections and freqs (64-bit, d / 2 of them, finite) are HOST arrays, read
 * during the call only.  Angles are reduced to a turn in 64-bit integers, so they
 * are as exact at far positions as at near ones: for |freqs[i]| up to 2^40 an angle
 * in [-pi, pi] is off by 2^-21 at most (its roundings to FP32), and its sine and
 * cosine by another 2^-21 (the native functions). */
typedef struct {
  const int* positions;
  int shared;
  int axes;
  const int* sections;
  const double* freqs;
  int interleaved;
} fa4fp4_rotation;

/* The norm of every row of d channels: n = x w / sqrt(mean(x^2) + eps), w the
 * weight of its tensor ([d], f32 or bf16 by weight_dtype (fa4fp4_out_dtype), device
 * memory, 16-byte aligned; NULL: ones).  eps >= 0.  Rows of any size: squares that
 * would pass FP32's range at either end are formed in other units. */
typedef struct {
  const void* q_weight;
  const void* k_weight;
  int weight_dtype;
  float eps;
} fa4fp4_norm;

/* Norm and rotation of queries and keys in one pass: q bf16 [B][Hq][N][d], k bf16
 * [B][Hkv][N][d] (NULL: queries alone; Hkv is then 0), norm NULL for the rotation
 * alone, rotation NULL for the norm alone (not both NULL).  All arithmetic is FP32
 * (the angles as above), rounded once to bf16.  q_out may be q and k_out may be k.
 * Hq and Hkv need not divide each other. */
FA4FP4_API fa4fp4_status fa4fp4_norm_rope(const fa4fp4_heads* q, const fa4fp4_heads* k, int B, int Hq, int Hkv,
                                          int N, int d, const fa4fp4_norm* norm,
                                          const fa4fp4_rotation* rotation, const fa4fp4_heads* q_out,
                                          const fa4fp4_heads* k_out, void* stream);

/* Its gradients: from q, k as they went in and the outputs' gradients dq_out,
 * dk_out (f32, as fa4fp4_bwd writes them, or bf16, by dout_dtype), with g the
 * gradient turned back, r = 1 / sqrt(mean(x^2) + eps), u = g w:
 *   dx = r (u - x r mean(u x r)),  dw = sum over b, h, n of g x r
 * dq, dk: bf16; dq_weight, dk_weight: f32 [d] (NULL where not wanted; without a
 * norm they must be NULL).  All sums are FP32, in an order that depends on the
 * shapes and the GPU's number of multiprocessors alone.  `workspace`: at least
 * fa4fp4_norm_rope_bwd_workspace_bytes(...) bytes of device memory (its size is 0,
 * and it may be NULL, for an empty problem), for this call alone while it runs; it
 * needs no initialisation.  Without a dq_weight or dk_weight it is not used and may
 * be NULL.  dq may be q, and dk may be k. */
FA4FP4_API size_t fa4fp4_norm_rope_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d);
FA4FP4_API fa4fp4_status fa4fp4_norm_rope_bwd(const fa4fp4_heads* dq_out, const fa4fp4_heads* dk_out, int dout_dtype,
                                              const fa4fp4_heads* q, const fa4fp4_heads* k, int B, int Hq, int Hkv,
                                              int N, int d, const fa4fp4_norm* norm,
                                              const fa4fp4_rotation* rotation, const fa4fp4_heads* dq,
                                              const fa4fp4_heads* dk, float* dq_weight, float* dk_weight,
                                              void* workspace, size_t workspace_bytes, void* stream);

/* BF16 attention of queries to keys of another length (cross attention to an
 * encoder's states), beside fa4bf16_fwd: q bf16 [B][Hq][Nq][d], k and v bf16
 * [B][Hkv][Nk][d], query head h reads kv head h / (Hq / Hkv), no causal mask.
 * kv_lens (int32 [B], device memory, 4-byte aligned; NULL: Nk) is each sequence's
 * number of keys; keys behind it may be anything, NaN too.  A length outside 0 ..
 * Nk is taken as the nearer end and the next fa4fp4_sync_status returns
 * FA4FP4_ERR_DEVICE_INDEX.
 *   s = softmax_scale * q.k, o = softmax(s) v, lse = ln sum e^s (nullable)
 * o: bf16; lse: f32 [B][Hq][Nq], dense.  Without a key o = 0 and lse = -inf.  The
 * rows of q, k and v do not overlap (stride_n >= d; FA4FP4_ERR_UNSUPPORTED); heads
 * and sequences may be broadcast.
 * Products are exact, sums FP32; P is rounded to bf16 (half a step: 2^-8) for the
 * product with V, its sum is taken before that.  No sum of P V passes FP32's range
 * on its way to o, whatever the values and the number of keys; weights below 2^-117
 * Nk of a row's largest may count as 0.  Scores below FP32's range have no weight; a
 * row without any other is one without a key.  Scores that are NaN, or above FP32's
 * range, give NaN for the row's o and lse.  A row's largest score is good up to 2^30
 * in magnitude: FP32's steps are 64 there.  Nq and Nk may be 0 (k and v are then
 * not read; no query is an empty problem). */
FA4FP4_API fa4fp4_status fa4bf16_cross_fwd(const fa4fp4_heads* q, const fa4fp4_heads* k, const fa4fp4_heads* v,
                                           const int* kv_lens, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                                           float softmax_scale, const fa4fp4_heads* o, float* lse, void* stream);

/* Its gradients, from the o and lse that it wrote and the gradient dout of o
 * (bf16): with P = e^(s - lse), dP = dO V^T, D = rowsum(dO o), dS = P (dP - D),
 *   dV = P^T dO, dK = softmax_scale dS^T Q, dQ = softmax_scale dS K
 * dV and dK summed over the query heads of their kv head.  dq, dk, dv: bf16, fully
 * written (zeros for keys behind kv_lens and for queries without a key).  P and dS
 * are rounded to bf16 for the products, the sums are FP32 and are added in an order
 * that depends on the shapes and the GPU's number of multiprocessors alone.  lse is
 * FP32, and P is off by about 2^-22 |lse| of itself for it: rows of |lse| above 2^20
 * have no use for gradients, and may make them infinite or NaN above 2^28.  The rows
 * of o and dout do not overlap either; their heads and sequences may be broadcast.
 * `workspace`: at least fa4bf16_cross_bwd_workspace_bytes(...) bytes of device
 * memory (FA4FP4_ERR_WORKSPACE otherwise), for this call alone while it runs; it
 * needs no initialisation.  Nq == 0 or Hq == 0 gives zeros for dk and dv, Nk == 0
 * zeros for dq. */
FA4FP4_API size_t fa4bf16_cross_bwd_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d);
FA4FP4_API fa4fp4_status fa4bf16_cross_bwd(const fa4fp4_heads* q, const fa4fp4_heads* k, const fa4fp4_heads* v,
                                           const fa4fp4_heads* o, const fa4fp4_heads* dout, const float* lse,
                                           const int* kv_lens, int B, int Hq, int Hkv, int Nq, int Nk, int d,
                                           float softmax_scale, const fa4fp4_heads* dq, const fa4fp4_heads* dk,
                                           const fa4fp4_heads* dv, void* workspace, size_t workspace_bytes,
                                           void* stream);

/* Synchronizes `stream`, then returns FA4FP4_ERR_CUDA for a pending CUDA error
 * or, for what kernels reported, FA4FP4_ERR_DEVICE_TIMEOUT if any bounded wait
 * expired, FA4FP4_ERR_DEVICE_INDEX or FA4FP4_ERR_DEVICE_NONFINITE for what the
 * cache calls met, else FA4FP4_OK.  One kind a call, in this order: what a call
 * returns is cleared by it, the other kinds are returned by the next ones. */
FA4FP4_API fa4fp4_status fa4fp4_sync_status(void* stream);

/* Static description of a status code. */
FA4FP4_API const char* fa4fp4_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FA4FP4_H */
