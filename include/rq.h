/*
 * rq.h -- C ABI of librq.so, the quantized linear layer for GB300 (sm_103a).
 *
 * The operations follow the three source pages of realizar 0.8.4 (docs.rs):
 *   [gemm.rs]  src/cuda/executor/layers/cublas_prefill/gemm.rs
 *   [mod.rs]   src/cuda/executor/layers/cublas_prefill/mod.rs
 *   [q6k.rs]   src/cuda/executor/q6k_gemv_indexed.rs
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers are DEVICE pointers (cudaMalloc / torch CUDA tensors) unless
 *    the name ends in _host.  The caller owns every pointer it passes in.
 *  - `stream` is a cudaStream_t (0 = legacy default stream).  Every call is
 *    asynchronous and stream-ordered: nothing synchronises the host, except
 *    rq_get_device_status and allocations on a cache miss (documented below).
 *  - Arguments are validated on the host before anything is launched; on a
 *    validation error nothing is launched or written and the status says why.
 *    A failed launch returns RQ_ERR_CUDA.  No entry point traps or aborts.
 *  - Matrices are row-major and densely packed (row stride = row length).
 *  - Shapes: M = tokens (rows of x and y), N = output features (weight rows),
 *    K = input features.  Quantized weights need K % 256 == 0.
 *  - Not thread-safe per rq_ctx: one thread and one stream at a time per ctx.
 *  - One CUDA device per process (one process per GPU): a kernel's
 *    shared-memory and cluster-size opt-ins are made once, on the device
 *    current at its first launch, and reused.
 */
#ifndef RQ_H
#define RQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RQ_ABI_VERSION 1

typedef enum {
    RQ_OK = 0,
    RQ_ERR_NULL = 1,       /* a required pointer is NULL                      */
    RQ_ERR_SHAPE = 2,      /* a size is out of range or misaligned            */
    RQ_ERR_QTYPE = 3,      /* unsupported weight quantization type            */
    RQ_ERR_NOT_CACHED = 4, /* reserved: a weight has no FP8 cache entry       */
    RQ_ERR_ALLOC = 5,      /* device or host allocation failed                */
    RQ_ERR_CUDA = 6,       /* a CUDA call or kernel launch failed             */
    RQ_ERR_TIMEOUT = 7,    /* a kernel gave up on a pipeline wait (see below) */
    RQ_ERR_ARCH = 8,       /* device lacks sm_103 features (tcgen05, TMA)     */
    RQ_ERR_INDEX = 9       /* a kernel met an index outside its array (a cache
                              slot, a page, a position); rq_get_device_status */
} rq_status;

/* GGUF tensor type ids. */
typedef enum { RQ_Q4K = 12, RQ_Q6K = 14 } rq_qtype;

/* ABI-identical to cudaStream_t. */
typedef struct CUstream_st *rq_stream_t;

/* Opaque context: owns the FP8 weight cache, the activation FP8 scratch and
 * the device scalars of the prefill path. */
typedef struct rq_ctx rq_ctx;

int rq_abi_version(void);
const char *rq_status_string(rq_status s);

/* ------------------------------------------------------------ context -- */

/* Create a context on the current CUDA device.  Default GEMM threshold 4,
 * or the value of the environment variable RQ_GEMM_THRESHOLD (read once,
 * here), mirroring [mod.rs] cublas_gemm_threshold.
 * Errors: RQ_ERR_NULL (out == NULL), RQ_ERR_ALLOC. */
rq_status rq_ctx_create(rq_ctx **out);

/* Free every buffer the context owns (FP8 weights, scratch, scalars).  The
 * caller must make sure no work using them is still in flight.  NULL is a
 * no-op. */
void rq_ctx_destroy(rq_ctx *ctx);

/* M at or above the threshold goes to the FP8 GEMM, below it to the GEMV
 * ([mod.rs], cublas_gemm_threshold: "Minimum M ... to use GEMM instead of
 * batched GEMV", default 4).  Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (< 1). */
rq_status rq_ctx_set_gemm_threshold(rq_ctx *ctx, int m_threshold);
int rq_ctx_get_gemm_threshold(const rq_ctx *ctx);

/* Host-side counters: activation-cache hits and misses of rq_linear, number
 * of cached FP8 weights and the device bytes they hold.  Any out pointer may
 * be NULL.  Errors: RQ_ERR_NULL (ctx). */
rq_status rq_ctx_get_stats(const rq_ctx *ctx, int64_t *act_hits_host,
                           int64_t *act_misses_host, int64_t *weights_host,
                           int64_t *weight_bytes_host);

/* ---------------------------------------------------- absmax + E4M3 ---- */

/* Per-tensor absmax ([mod.rs], ABSMAX_REDUCE_PTX and gpu_absmax_device):
 * *absmax_bits = IEEE bits of max_i |x[i]| over the n floats of x, starting
 * from +0; NaNs are skipped, +-Inf count as +Inf.  The word is zeroed on
 * `stream` first (no host copy from a stack temporary), then reduced with an
 * unsigned atomic max, which orders non-negative floats correctly.
 *   x: n floats (any alignment).  absmax_bits: one device word (4-aligned).
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (n < 0).  n == 0 yields 0. */
rq_status rq_absmax(const float *x, int64_t n, uint32_t *absmax_bits,
                    rq_stream_t stream);

/* Scaled FP32 -> E4M3 ([mod.rs], F32_TO_E4M3_DEVICE_SCALED_PTX): reads the
 * absmax word A from the device, uses A' = (A == 0 ? 1 : A), s = 448 / A'
 * (correctly rounded fp32 division), writes out[i] = E4M3(fl32(x[i] * s)) and
 * *dequant_out = A' / 448.  Encoder rules: exponent rebias 127 -> 7, mantissa
 * round-to-nearest-even 23 -> 3 bits, values below 2^-6 flush to 0x00,
 * overflow saturates to sign|0x7E (+-448), 0x7F/0xFF are never produced,
 * NaN/Inf inputs give sign(x)|0x7E and +-0 gives 0x00 (decided before the
 * multiply).  Bit-exact with the CPU reference.
 *   x: n floats.  out: n bytes.  dequant_out: one device float.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (n < 0). */
rq_status rq_quant_e4m3(const float *x, int64_t n, const uint32_t *absmax_bits,
                        uint8_t *out, float *dequant_out, rq_stream_t stream);

/* ------------------------------------------------------------- GEMV ---- */

/* Decode GEMV on GGUF Q4_K weights, dequantized inside the dot product
 * ([q6k.rs], q4k_gemv_into; [mod.rs] cublas_gemm_threshold doc: batched GEMV
 * for small M reads Q4_K directly at 0.5625 B/weight):
 *   y[m, n] = sum_k x[m, k] * w(n, k),  0 <= m < M, 0 <= n < N.
 *   w: N rows of K/256 Q4_K super-blocks, 144 B each (fp16 d, fp16 dmin,
 *      12 packed 6-bit scale/min bytes, 128 bytes of 4-bit quants), rows
 *      contiguous; 16-byte aligned.
 *   x: f32 [M x K], 16-byte aligned.  y: f32 [M x N] (written, not added to).
 * Accuracy: for finite x, every output whose sum_k |x[m,k] * w(n,k)| is at
 * least 2^-100 is within 1e-4 * sum_k |x[m,k] * w(n,k)| of the exact result
 * (outputs beyond fp32's range are +-Inf; non-finite x give Inf / NaN as in
 * IEEE arithmetic).  The fast paths prove this per output with an error
 * certificate computed alongside the sum; an output whose certificate fails
 * (extreme ranges of x within 32 values, weights whose two terms cancel on
 * the largest x) is recomputed exactly in fp64 inside the same launch, which
 * is slow but never wrong (see rq_gemv_exact_outputs).  Several tokens run
 * one launch per token (the weight is read once per token).
 * Ordering: the kernel may start streaming w before the kernel launched just
 * before it on the stream has finished (programmatic dependent launch); it
 * reads x and writes y only after that kernel has completed.  So w must not
 * be written by the immediately preceding kernel on the stream (a copy or
 * any earlier kernel is fine).  The same holds for rq_q6k_gemv and for the
 * GEMV route of rq_linear.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (M not in 1..8, N < 1, K < 256,
 * K % 256 != 0, misaligned w or x). */
rq_status rq_q4k_gemv(const void *w, const float *x, float *y, int M, int N,
                      int K, rq_stream_t stream);

/* The same on GGUF Q6_K weights ([q6k.rs], q6k_gemv_indexed_async, which
 * returns InvalidLaunchConfig for a null weight pointer; here the output is
 * caller-owned, nothing is allocated):
 *   w: N rows of K/256 Q6_K super-blocks, 210 B each (ql[128], qh[64],
 *      16 int8 scales, fp16 d), rows contiguous; 4-byte aligned.
 *   weight = d * scale * (q - 32), q the 6-bit quant.
 * Accuracy as rq_q4k_gemv (certificate per output, exact fp64 path when it
 * fails); 2..8 tokens are one launch.
 * Errors: as rq_q4k_gemv (w need only be 4-byte aligned). */
rq_status rq_q6k_gemv(const void *w, const float *x, float *y, int M, int N,
                      int K, rq_stream_t stream);

/* ------------------------------------------------------- FP8 prefill --- */

/* FP8 weight cache ([gemm.rs], get_or_cache_fp8_weight): on the first call
 * for (w, qtype, N, K) the packed weight is dequantized to fp32 in the fixed
 * order w = (d*sc)*q - dmin*m (Q4_K) or (d*scale)*(q-32) (Q6_K), its absmax
 * A_w is taken, and every weight is encoded as in rq_quant_e4m3 with
 * 448 / A_w'.  Unlike the pages, the dequant scale A_w'/448 stays in device
 * memory (no host read-back, no host sync); no fp32 scratch is used (the
 * weight is decoded twice instead).  Later calls return the cached pointers.
 *   *w_fp8: device E4M3 bytes [N x K] owned by ctx, valid until
 *           rq_ctx_destroy.  *w_dequant: one device float owned by ctx.
 * A miss allocates with cudaMalloc (which may synchronise the device).
 * Errors: RQ_ERR_NULL, RQ_ERR_QTYPE, RQ_ERR_SHAPE, RQ_ERR_ALLOC. */
rq_status rq_fp8_weight_cache(rq_ctx *ctx, rq_qtype qtype, const void *w,
                              int N, int K, const uint8_t **w_fp8,
                              const float **w_dequant, rq_stream_t stream);

/* FP8 E4M3 GEMM with a fused fp32 epilogue ([gemm.rs],
 * cublas_prefill_fp8_gemm: raw FP8 products, then the activation scale
 * act_absmax/448 and the weight scale w_absmax/448, both read from device
 * memory, with no host sync):
 *   y[m, n] = (sum_k e4m3(x_fp8[m, k]) * e4m3(w_fp8[n, k]))
 *             * (*x_dequant) * (*w_dequant)            for m < M, n < N.
 * Tensor cores (tcgen05 kind::f8f6f4), fp32 accumulation; agrees with the
 * exact reference within 2e-3*|ref| + 1e-3*rms(row of ref).
 *   x_fp8: E4M3 [M_pad x K], M_pad = (M + 15) / 16 * 16; rows M..M_pad-1
 *          are read but do not affect y.  16-byte aligned.
 *   w_fp8: E4M3 [N x K], 16-byte aligned.   y: f32 [M x N]; rows >= M and
 *          columns >= N are never written.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (M, N < 1, K < 128, K % 128 != 0,
 * misaligned operands), RQ_ERR_CUDA. */
rq_status rq_fp8_gemm(const uint8_t *x_fp8, const float *x_dequant,
                      const uint8_t *w_fp8, const float *w_dequant, float *y,
                      int M, int N, int K, rq_stream_t stream);

/* FP8 activation cache ([gemm.rs], cublas_prefill_fp8_gemm: the
 * activation's per-tensor absmax and E4M3 conversion, and the PMAT-084
 * reuse of that FP8 copy by the next linears that read the same input):
 * returns device pointers to the E4M3 form of x and its dequant scale
 * absmax'/448 (absmax' = absmax, or 1 for an all-zero x), quantizing x into
 * the ctx's scratch on a miss.  The bytes are those of rq_absmax followed by
 * rq_quant_e4m3, with rows M..M_pad-1 zero (M_pad = M rounded up to 16), so
 * the result feeds rq_fp8_gemm directly.  The key is (x, M, K, generation),
 * as for rq_linear, which calls this on its FP8 route.  A call on a stream that
 * is being captured finds only what the same capture quantizes, so that every
 * replay quantizes x anew, and a call that runs at once finds nothing captured:
 * each kind has a scratch of its own, and captured graphs' scratch stays where
 * it is until the ctx is destroyed, however much larger a later call is (a
 * capture may allocate it).  All graphs of a ctx share it: they are replayed,
 * like every call on the ctx, on one stream at a time.
 *   x: f32 [M x K], 16-byte aligned.   *x_fp8: E4M3 [M_pad x K] (owned by
 *   ctx).   *x_dequant: one device float (owned by ctx).
 * The pointers stay valid until a later miss on this ctx needs a larger
 * scratch, those of a captured call until the ctx is destroyed; a later miss of
 * the same or smaller size overwrites the bytes in stream order.  Allocates on a
 * miss that needs a larger scratch.  Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (M, K < 1,
 * x misaligned), RQ_ERR_ALLOC, RQ_ERR_CUDA. */
rq_status rq_fp8_act_cache(rq_ctx *ctx, const float *x, int M, int K,
                           const uint8_t **x_fp8, const float **x_dequant,
                           rq_stream_t stream);

/* Quantized linear layer with M-threshold routing ([mod.rs],
 * cublas_gemm_threshold; [gemm.rs], cublas_prefill_gemm FP8 branch):
 *   M <  threshold: Q4_K / Q6_K GEMV straight from the packed weights
 *                   (M > 8 is processed 8 rows at a time);
 *   M >= threshold: FP8 weight cache (a hit after the first call), then, on
 *                   an activation-cache miss, absmax + E4M3 quantization of
 *                   x into the ctx's [M_pad x K] scratch (pad rows zeroed),
 *                   then the FP8 GEMM.  Up to 2^17 elements, absmax and
 *                   quantization are one launch of one thread-block
 *                   cluster (x read twice, the second time from L2); from
 *                   2^20 elements on, one cooperative kernel while x fits
 *                   on chip in one wave of CTAs (per SM 512 x 24 float4
 *                   in registers plus about 220 KB of shared memory: x
 *                   read once) or, with x held in shared memory, while
 *                   what does not fit is at most 16 MB (128 MB from 2^24
 *                   elements on; only that rest read twice); otherwise
 *                   two kernels, the second reading x backwards (the same
 *                   bytes every way; at ctx creation the environment
 *                   variables RQ_CLUSTER_QUANT_MAX (elements, 0 = never)
 *                   and RQ_ONE_PASS_QUANT=0 turn the first two off).
 * The activation cache ([gemm.rs], PMAT-084 reuse across Q/K/V and gate/up)
 * is keyed by (x, M, K, generation); rq_act_cache_invalidate bumps the
 * generation and must be called when x's contents change in place.  Captured
 * calls quantize x in the graph, whatever was cached before (rq_fp8_act_cache).
 * Errors: those of the routes taken. */
rq_status rq_linear(rq_ctx *ctx, rq_qtype qtype, const void *w, const float *x,
                    float *y, int M, int N, int K, rq_stream_t stream);

/* Linear layers that share one input ([gemm.rs], PMAT-084: Q, K and V read
 * the same activation, and so do gate and up):
 *   y_i = x . W_i^T   for i < count,  W_i: N_i rows of qtypes[i] super-blocks.
 * Routes like rq_linear.  On the FP8 route the activation is quantized once
 * (activation cache) and the group is one GEMM launch over the members'
 * FP8 weights, cached once per group contiguously by rows (member i keeps
 * its own per-tensor scale; its bytes equal rq_fp8_weight_cache's).  On
 * the GEMV route the Q4_K members are one launch (one pass of x) for up to
 * 8 tokens; for a single token the group's Q6_K member joins that launch
 * when it has exactly one (the CTAs split between the two formats); other
 * members are launched one by one.  Results are those of count rq_linear calls within the same
 * tolerances.
 *   count: 1 .. RQ_MAX_GROUP.  qtypes, w, y, N: host arrays of count
 *   entries (w[i], y[i] device pointers as for rq_linear).  All members
 *   share x (f32 [M x K], 16-byte aligned), M and K.
 * The group's FP8 weights are owned by ctx (keyed by the members' pointers,
 * types and shapes) and freed by rq_ctx_destroy.
 * Errors: RQ_ERR_NULL, RQ_ERR_QTYPE, RQ_ERR_SHAPE (count out of range, or
 * as rq_linear), RQ_ERR_ALLOC, RQ_ERR_CUDA. */
#define RQ_MAX_GROUP 4
rq_status rq_linear_group(rq_ctx *ctx, int count, const rq_qtype *qtypes,
                          const void *const *w, const float *x, float *const *y,
                          const int *N, int M, int K, rq_stream_t stream);

/* FP8 linear layer that allocates nothing.  The source pages have no
 * counterpart to this entry point.
 *
 * For callers that cannot call cudaMalloc while serving: code that runs
 * inside a host framework which owns and pre-reserves all device memory (an
 * inference engine's plugin or operator callback, say), or a process under a
 * fixed device-memory budget where a new allocation would fail or stall.
 * Given an E4M3 weight and its dequant scale (for example the pointers
 * rq_fp8_weight_cache returns), it computes the same result as the FP8 route
 * of rq_linear: absmax of x, E4M3 quantization of x, FP8 GEMM with both
 * scales applied to the fp32 accumulator:
 *   y[m, n] = (sum_k e4m3(xq[m, k]) * e4m3(w_fp8[n, k])) * x_deq * (*w_dequant)
 *   x: f32 [M x K], 16-byte aligned.  w_fp8: E4M3 [N x K], 16-byte aligned.
 *   w_dequant: one device float.  y: f32 [M x N].
 * The quantized activation (M_pad x K bytes, M_pad = M rounded up to 16) and
 * two device scalars live in one fixed array inside the library, of
 * RQ_NOALLOC_MAX_ACT_BYTES + 256 bytes, which the GPU holds until the process
 * exits.  No call allocates: no cudaMalloc, cudaFree or allocating library
 * routine.
 *   - The first call looks up the array's device address (with the device
 *     current).  Under CUDA's lazy module loading that lookup may also be
 *     what loads the library's module and reserves the array, so the first
 *     call may take device memory once: make it a warm-up call before
 *     serving or any stream capture, and before fixing a memory budget.
 *   - The library serves one device per process (see the conventions at
 *     the top).  All calls share the array, and it keeps the last call's
 *     contents; each call re-zeroes what must start at zero.  Calls whose
 *     work overlaps on the GPU (on two streams, say) race on the array:
 *     serialise them.
 * Errors: RQ_ERR_NULL; RQ_ERR_SHAPE for M, N < 1, K < 128, K % 128 != 0,
 * misaligned pointers, or M_pad * K > RQ_NOALLOC_MAX_ACT_BYTES (the array
 * is too small for this activation); RQ_ERR_CUDA. */
#define RQ_NOALLOC_MAX_ACT_BYTES (8u * 1024u * 1024u)
rq_status rq_fp8_linear_noalloc(const float *x, const uint8_t *w_fp8,
                                const float *w_dequant, float *y, int M, int N,
                                int K, rq_stream_t stream);

/* Forget the cached FP8 activation (bump the generation). */
rq_status rq_act_cache_invalidate(rq_ctx *ctx);

/* --------------------------------- FP8 product with a fused epilogue --- */

/* What is done to a product's sums before they are stored, in f32:
 *   y = residual + mul * act(sum + bias),  rounded once, to y's type.
 *   bias: f32 [N], 4-byte aligned, or NULL.   act: rq_act.
 *   mul, residual: [M][N] of y's type, consecutive tokens mul_stride /
 *     residual_stride elements apart (at least N), or NULL.  mul is the up
 *     product of a gated layer, say; residual the stream that the block's
 *     output is added to.  Either may be y itself, with y's stride; neither
 *     may overlap y in another way.
 * SiLU z / (1 + e^-z); GELU z/2 (1 + erf(z / sqrt 2)); GELU_TANH z/2 (1 +
 * tanh(sqrt(2/pi) (z + 0.044715 z^3))); RELU max(z, 0) (a NaN stays one).
 * Before the output's rounding they are within 2^-20 of their value, plus, of
 * it, for 16-bit outputs 2^-23 |z| (SiLU) or 2^-23 z^2 (GELU), and for GELU_TANH
 * 2^-21 |b|, b the tanh's argument doubled; and within 2^-120.  The struct is
 * read on the host during the call. */
typedef enum {
    RQ_ACT_NONE = 0,
    RQ_ACT_SILU = 1,
    RQ_ACT_GELU = 2,
    RQ_ACT_GELU_TANH = 3,
    RQ_ACT_RELU = 4
} rq_act;

typedef struct {
    const float *bias;
    int act; /* rq_act */
    const void *mul, *residual;
    int64_t mul_stride, residual_stride;
} rq_epilogue;

/* rq_fp8_gemm with an epilogue and an output of dtype (RQ_F32, RQ_F16,
 * RQ_BF16; see below), tokens y_stride elements apart (at least N):
 *   sum[m, n] = (sum_k e4m3(x_fp8[m, k]) * e4m3(w_fp8[n, k]))
 *               * (*x_dequant) * (*w_dequant).
 * x_fp8, w_fp8 and the scales as for rq_fp8_gemm, for any M from a single
 * token on; y, mul and residual need their element's alignment only.
 * Accuracy of the sums: the tensor cores add in f32 and cut off; measured
 * about 6e-8 of the result for K up to 4096 and 1.5e-6 at K = 18944.
 * epilogue_host NULL: the product alone.  Equal calls give equal bits.
 * Errors: RQ_ERR_NULL, RQ_ERR_QTYPE (dtype or act), RQ_ERR_SHAPE (as
 * rq_fp8_gemm, strides, alignment), RQ_ERR_CUDA. */
rq_status rq_fp8_gemm_epilogue(const uint8_t *x_fp8, const float *x_dequant,
                               const uint8_t *w_fp8, const float *w_dequant,
                               const rq_epilogue *epilogue_host, int dtype, void *y,
                               int64_t y_stride, int M, int N, int K,
                               rq_stream_t stream);

/* The FP8 route of rq_linear with an epilogue, at every M (the threshold does
 * not apply: the weight is read as one byte per value even for one token):
 * FP8 weight cache (rq_linear's, shared with it), FP8 activation of x,
 * rq_fp8_gemm_epilogue.  For M at or above the threshold the activation cache is
 * used, shared with rq_linear and under its rule: rq_act_cache_invalidate must
 * be called when x's contents change in place (rq_residual_norm into the same x,
 * say).  Below it, where rq_linear quantizes nothing, every call quantizes x
 * and leaves nothing in the cache.
 * Call it once with a weight before a capture: the FP8 weight is allocated and
 * made on the first call.
 * Errors: RQ_ERR_QTYPE (qtype, dtype or act), those of rq_linear and of
 * rq_fp8_gemm_epilogue. */
rq_status rq_linear_epilogue(rq_ctx *ctx, rq_qtype qtype, const void *w, const float *x,
                             const rq_epilogue *epilogue_host, int dtype, void *y,
                             int64_t y_stride, int M, int N, int K, rq_stream_t stream);

/* ------------------------------------- norms between a layer's blocks -- */

/* What stands between two blocks, fixed for the layer:
 *   width: values per token, 1 .. 16384.
 *   norms: RQ_NORM_POST and RQ_NORM_PRE, either or both or none.  A norm is
 *     x * rsqrt(mean(x^2) + eps) * weight over the token's values.
 *   post_weight, pre_weight: f32 [width], 4-byte aligned, or NULL for ones.
 *   scale: multiplies the block's output (finite). */
typedef enum { RQ_NORM_POST = 1, RQ_NORM_PRE = 2 } rq_norms;

typedef struct {
    const float *post_weight, *pre_weight;
    int width;
    int norms;
    float eps, scale;
} rq_norm_params;

/* The norm after a block, its gated and scaled sum with the residual stream
 * and the norm before the next block, in one pass over each token:
 *   h' = h + scale * (gate * post(y)),     x = pre(h').
 *   y: [tokens][width] of dtype, the block's output, tokens y_stride elements
 *     apart; NULL for none (h' = h; h_out must be NULL then).
 *   gate: [width] of dtype with gate_stride 0, one for all tokens, or
 *     [tokens][width] with gate_stride elements between tokens; NULL: ones.
 *   h: [tokens][width] of h_dtype, which is dtype or RQ_F32, h_stride.
 *   h_out: like h, dense, or NULL.   x_out: [tokens][width] of dtype, dense,
 *     or NULL (not both).  h_out may be h and x_out may be y where those are
 *     dense; otherwise outputs overlap nothing.
 *   absmax_bits: one device word, or NULL: IEEE bits of the largest |x| over
 *     all tokens, NaNs skipped, as rq_absmax leaves it (so that rq_quant_e4m3
 *     can follow).  Needs dtype RQ_F32 and x_out; written whatever was there.
 * All arithmetic is f32; x is taken from h' before h' is rounded to h_dtype.
 * Strides are at least width; every pointer needs its element's alignment
 * (16-byte aligned rows of a multiple of 16 bytes are read 16 bytes at a
 * time).  tokens == 0 does nothing (but sets *absmax_bits to 0).
 * A linear that reads x_out as cached FP8 codes (rq_linear and
 * rq_linear_epilogue from the threshold on) wants rq_act_cache_invalidate after
 * each call that writes the same x_out.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_QTYPE (dtype, h_dtype, or
 * absmax_bits with 16-bit x), RQ_ERR_CUDA. */
rq_status rq_residual_norm(const rq_norm_params *params_host, int dtype, const void *y,
                           int64_t y_stride, const void *gate, int64_t gate_stride,
                           int h_dtype, const void *h, int64_t h_stride, void *h_out,
                           void *x_out, uint32_t *absmax_bits, int tokens,
                           rq_stream_t stream);

/* -------------------------------------------- the places of a pass ----- */

/* Cache slots, positions and page tables of a pass's new tokens, from the
 * lengths of its sequences, on the GPU:
 *   length: int32 [batch], cached tokens of each sequence (< 0: unused, it has
 *     no new tokens).   count: int32 [batch], its new tokens (below 0 counts as
 *     0), or NULL: new_tokens each.
 *   new_tokens > 0: `rows` = batch * new_tokens rows, row b * new_tokens + i is
 *     new token i of sequence b (the layout of rq_cache_attention); a count
 *     above new_tokens is cut to it and records RQ_ERR_INDEX.
 *   new_tokens == 0: the tokens of the sequences one behind another in `rows`
 *     rows (count is needed); what does not fit has no row and records
 *     RQ_ERR_INDEX.
 *   page_table: int32 [batch][max_pages], in and out.  The first
 *     ceil(length / page_size) entries are read; the entries of pages that the
 *     new tokens begin are written; all others stay as they are.
 *   free_pages: int32 [free_capacity], a stack of unused pages, of which the
 *     first *free_count (a device word) are valid.  New pages are taken from
 *     its end: page i of the pass, counted over the sequences in order, is
 *     free_pages[*free_count - 1 - i].
 *   free_left: one device word, *free_count less the pages that the pass
 *     needs; below zero where the stack did not hold enough.  Must not be
 *     free_count.
 *   slot: int64 [rows], page * page_size + offset; position: int32 [rows], the
 *     token's place in its sequence; sequence: int32 [rows] or NULL.  Rows
 *     without a token (padding, unused sequences) get slot -1, which writes
 *     nothing, position 0 and sequence -1.
 *   row_start: int32 [batch + 1] or NULL, the first row of each sequence and
 *     the rows used.   next_length: int32 [batch] or NULL, length + count (an
 *     unused sequence's length as it is); must not be length.
 * A token whose page is missing (past the table or the stack, or a negative
 * entry) gets slot -1 and records RQ_ERR_INDEX (rq_get_device_status); a
 * missing new page is written as -1 where the table has room.  Drafts that are
 * not kept give their pages back when the count is raised again by as many: the
 * pages lie at the stack's end in the order in which they are taken.
 * page_size: 16, 32, 64, 128 or 256.  batch <= 65536, max_pages >= 1.
 * batch == 0 does nothing but fill `rows` and free_left.  int32 arrays are
 * 4-byte aligned, slot 8-byte.  One launch, no scratch.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_CUDA. */
rq_status rq_batch_plan(const int32_t *length, const int32_t *count, int batch,
                        int new_tokens, int page_size, int32_t *page_table,
                        int max_pages, const int32_t *free_pages, int free_capacity,
                        const int32_t *free_count, int32_t *free_left, int64_t *slot,
                        int32_t *position, int32_t *sequence, int rows,
                        int32_t *row_start, int32_t *next_length, rq_stream_t stream);

/* ------------------------------------------ quantized K/V cache ------- */

/* The steps of a decoder layer between its q/k/v products and its o product,
 * and the step from probabilities to tokens.  The source pages have no
 * counterpart to these entry points: the layer's linears above produce their
 * inputs (f32) and read their outputs.
 *
 * Activations are f32, f16 or bf16; every sum, norm and softmax statistic is
 * f32 (the token draws are exact integers), and a result is rounded once. */
typedef enum { RQ_F32 = 0, RQ_F16 = 1, RQ_BF16 = 2 } rq_dtype;

/* One byte per cached value, one f32 scale per cached row (the head_dim
 * values of one token and kv head): value = code * scale.  With A the row's
 * largest finite magnitude, A' = max(A, 2^-100) and top the format's largest
 * value (448 or 127):  scale = A' / top,  code = rn(x * (top * (1 / A'))),
 * each operation one correctly rounded f32 operation and rn the round to
 * nearest even into the format, limited to +-top.  A value that is not finite
 * takes +-top with its own sign, so the NaN codes of E4M3 are never written.
 * (A caller who fills a cache otherwise leaves none in rows that a query sees;
 * in rows that are not seen they do no harm.) */
typedef enum { RQ_KV_E4M3 = 0, RQ_KV_I8 = 1 } rq_kv_format;

/* A paged cache, described by the caller, who owns its memory:
 *   k, v:  codes [pages][kv_heads][page_size][head_dim], 16-byte aligned.
 *   k_scale, v_scale:  f32 [pages][kv_heads][page_size], 16-byte aligned.
 *   page_size: 16, 32, 64, 128 or 256 tokens.  head_dim: 64, 128 or 256.
 *   pages >= 1, kv_heads >= 1, pages * kv_heads < 2^31.
 * A slot names one token's place: slot = page * page_size + offset.  The
 * struct is read on the host during the call; it need not outlive it. */
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t pages;
    int page_size, kv_heads, head_dim;
    int format; /* rq_kv_format */
} rq_kv_cache;

/* What one layer's norms and rotation of q and k need, fixed for the layer:
 *   q_weight, k_weight: f32 [head_dim] norm weights, 16-byte aligned, or NULL
 *     for no norm of that side.  The norm is x * rsqrt(mean(x^2) + eps) *
 *     weight over each head's head_dim values.
 *   cos_table, sin_table: f32 [positions][rotary_dim / 2], 16-byte aligned
 *     (NULL when rotary_dim is 0).
 *   rotary_dim: the leading coordinates of each head that turn, 0 or a
 *     multiple of 16 up to head_dim; coordinate pairs are (i, i +
 *     rotary_dim / 2), or (2 i, 2 i + 1) when interleaved is nonzero:
 *     (a, b) -> (a cos - b sin, b cos + a sin). */
typedef struct {
    const float *q_weight, *k_weight;
    const float *cos_table, *sin_table;
    int64_t positions;
    int q_heads, kv_heads, head_dim;
    int rotary_dim, interleaved;
    float eps;
} rq_qk_params;

/* Per-head norm and position rotation of q and k in one pass:
 *   q: [tokens][q_heads][head_dim], k: [tokens][kv_heads][head_dim] of dtype,
 *     a token's heads contiguous, consecutive tokens q_stride / k_stride
 *     elements apart (at least the row, and a multiple of 16 bytes).
 *   position: int32 [tokens], rows of the tables (ignored, may be NULL, when
 *     rotary_dim is 0).  A token whose position is outside the tables is not
 *     turned and RQ_ERR_INDEX is recorded for rq_get_device_status.
 *   q_out, k_out: dense, of dtype.  q_out may be q and k_out may be k where
 *     those are dense.
 * q or k may be NULL together with its output: that side is left out.
 * All pointers 16-byte aligned (position: 4).  tokens == 0 does nothing.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_QTYPE (dtype), RQ_ERR_CUDA. */
rq_status rq_qk_norm_rope(const rq_qk_params *params_host, int dtype, const void *q,
                          int64_t q_stride, const void *k, int64_t k_stride,
                          const int32_t *position, void *q_out, void *k_out,
                          int tokens, rq_stream_t stream);

/* The same, with k (after norm and rotation) and v quantized straight from
 * f32 into the cache at slot[t] in the same pass:
 *   v: like k, v_stride.   slot: int64 [tokens], 8-byte aligned; a negative
 *   slot writes nothing for its token, one past the cache writes nothing and
 *   records RQ_ERR_INDEX.  Two tokens of one call must not share a slot.
 * The cache's kv_heads and head_dim must be the params'.  q may be NULL with
 * q_out.  Errors: as rq_qk_norm_rope, and those of rq_kv_write. */
rq_status rq_qkv_to_cache(const rq_qk_params *params_host, int dtype, const void *q,
                          int64_t q_stride, const void *k, int64_t k_stride,
                          const void *v, int64_t v_stride, const int32_t *position,
                          void *q_out, const rq_kv_cache *cache_host,
                          const int64_t *slot, int tokens, rq_stream_t stream);

/* Quantize k and v rows into the cache as they are (no norm, no rotation).
 * Arguments as above.  Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (sizes, strides or
 * alignment), RQ_ERR_QTYPE (dtype or cache format), RQ_ERR_CUDA. */
rq_status rq_kv_write(const rq_kv_cache *cache_host, int dtype, const void *k,
                      int64_t k_stride, const void *v, int64_t v_stride,
                      const int64_t *slot, int tokens, rq_stream_t stream);

/* Read the cache back: k_out, v_out [tokens][kv_heads][head_dim] of dtype,
 * dense, 16-byte aligned: code * scale of slot[t] (one f32 product, then the
 * dtype's rounding), zeros for a negative slot; a slot past the cache reads
 * as zeros and records RQ_ERR_INDEX.  Errors: as rq_kv_write. */
rq_status rq_kv_read(const rq_kv_cache *cache_host, int dtype, const int64_t *slot,
                     void *k_out, void *v_out, int tokens, rq_stream_t stream);

/* Attention of new tokens over the paged quantized cache: single tokens,
 * drafted chains and trees, prompts.  Sequence b has length[b] cached tokens
 * and `new_tokens` new ones, whose keys and values are already in the cache
 * at the places length[b] .. length[b] + new_tokens - 1 of the sequence:
 *   out[b, i, h] = sum_j softmax_j(scale * q[b, i, h] . k[j, h']) v[j, h'],
 *   h' = h / (q_heads / kv_heads),
 * over the places j < length[b], and of the new ones over
 *   tree == NULL:  new tokens 0 .. i (a chain or a prompt);
 *   tree != NULL:  new token j where bit j of tree[b, i] is set (the draft
 *                  itself and those before it on its path, say); bits from
 *                  new_tokens on are ignored.  new_tokens <= 64.
 * A row that sees nothing gives zeros, whatever its q.  length[b] < 0 marks an
 * unused sequence: zeros.  Any other row whose q is not finite gives NaN; so
 * may one whose scores (in powers of two: 1.45 scale q . k) leave f32's range.
 *   q: [batch * new_tokens][q_heads][head_dim] of dtype, consecutive tokens
 *     q_stride elements apart.   out: the same shape, dense.
 *   page_table: int32 [batch][max_pages]; place p of sequence b is offset
 *     p % page_size of page page_table[b, p / page_size].  Entries past the
 *     sequence's last place are not read.  A page outside the cache reads as
 *     page 0, places past max_pages pages are not seen; both record
 *     RQ_ERR_INDEX.
 *   scale: finite, above 0.   q_heads: a multiple of kv_heads.
 * What lies in the cache behind a sequence's places, at later new tokens or
 * under a cleared bit, does not reach a row's output: its bits stay whatever
 * the codes and scales there are.
 * Accuracy: with f32 activations q, the probabilities and both products are
 * carried to about 21 bits (each f32 operand split into two f16 parts, codes
 * exact in f16, f32 sums, whose additions the tensor cores cut off rather than
 * round, and which are therefore taken over into rounded sums every few
 * hundred keys: about 1e-6 of the result whatever the length); with f16 / bf16
 * activations q and the probabilities may be f16 operands (11 bits).  A key's
 * weight is carried relative to the largest value scale that its row has seen:
 * what is below 2^-30 of that is lost.
 * Partial results of split sequences live in scratch owned by ctx: about 61
 * MB, allocated by the first call that needs it (which waits for the stream,
 * and inside a stream capture gives RQ_ERR_ALLOC: call once before) and kept
 * until ctx is destroyed, whatever later calls' sizes.  They are joined in a
 * fixed order, so equal calls give equal bits.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_QTYPE (dtype or format),
 * RQ_ERR_ALLOC, RQ_ERR_CUDA. */
rq_status rq_cache_attention(rq_ctx *ctx, const rq_kv_cache *cache_host, int dtype,
                             const void *q, int64_t q_stride, void *out, int batch,
                             int new_tokens, int q_heads, const int32_t *page_table,
                             int max_pages, const int32_t *length,
                             const uint64_t *tree, float scale, rq_stream_t stream);

/* Host-side counters: calls of rq_cache_attention on ctx that launched the
 * kernel for few query rows per kv head, and the one for many (sizes choose;
 * the results of both keep to what is stated above).  Either pointer may be
 * NULL.  Errors: RQ_ERR_NULL (ctx). */
rq_status rq_ctx_attention_launches(const rq_ctx *ctx, int64_t *few_rows_host,
                                    int64_t *many_rows_host);

/* ------------------------------------- verification of drafted tokens -- */

/* Keep or reject a chain of drafted tokens per sequence, and draw the next
 * token, so that the kept tokens and the drawn one are distributed as the
 * target's own:
 *   token: int32 [batch][drafts].
 *   p: f32 [batch][drafts + 1][vocab], the target's probabilities at the
 *     place of each draft and after the last one.
 *   q: f32 [batch][drafts][vocab], the distributions the drafts were drawn
 *     from, or NULL for drafts that were not drawn (q one-hot).
 *   u: f32 [batch][drafts + 1] random numbers in [0, 1): u[b, i] decides
 *     draft i, u[b, drafts] draws the next token.
 * Draft i with token x is kept if u[i] * q[i][x] < p[i][x] (one f32 product;
 * q one-hot: u[i] < p[i][x]); accepted[b] = drafts kept before the first that
 * is not.  The next token is drawn from the weights max(p - q, 0) at the
 * rejected draft's place (q one-hot: p with the draft's own entry 0), or
 * from p after the last draft; weights that are all zero fall back to p.  A
 * draft token outside 0 .. vocab-1 ends the chain there, and the next token
 * is drawn from p (drafts of unequal number).
 * The draw is exact: weights are whole numbers, floor(min(w, 1) * 2^36) (NaN:
 * 0), and the next token is the first whose running sum exceeds
 * floor(U * total / 2^24), U = floor(u * 2^24) limited to 0 .. 2^24-1, so
 * that it depends on no order of summation; -1 if p has no weight either.
 *   accepted, next: int32 [batch].
 * 0 <= drafts <= 2^30 (token, q may be NULL at 0), 1 <= vocab <= 2^20,
 * 0 <= batch <= 2^27 (0 does nothing).
 * p and q: 4-byte aligned.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_CUDA. */
rq_status rq_verify_chain(const int32_t *token, const float *p, const float *q,
                          const float *u, int32_t *accepted, int32_t *next, int batch,
                          int drafts, int vocab, rq_stream_t stream);

/* The same for trees of drafts that were not drawn at random (a node's
 * likeliest continuations, say): at each node the target's token is drawn
 * and the walk goes on where a draft holds it.
 *   parent: int32 [batch][drafts], parent[b, i] < i, or -1 for the last
 *     token before the drafts; a draft whose parent is outside -1 .. i-1 is
 *     not reached.  p: f32 [batch][drafts + 1][vocab]: row 0 after the last
 *     token, row 1 + i after draft i.   u: f32 [batch][drafts + 1] likewise.
 * Starting at the last token: y is drawn from the node's p with the node's u
 * (exactly as above); the first draft whose parent is the node and whose
 * token is y is accepted and becomes the node; without one, y is the next
 * token.   accepted, next: int32 [batch].   path: int32 [batch][drafts], the
 * accepted drafts in order, then -1.   drafts <= 1024.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_CUDA. */
rq_status rq_verify_tree(const int32_t *token, const int32_t *parent, const float *p,
                         const float *u, int32_t *accepted, int32_t *next,
                         int32_t *path, int batch, int drafts, int vocab,
                         rq_stream_t stream);

/* ---------------------------------------- from logits to tokens -------- */

/* Each row's own filters: device arrays [rows], 4-byte aligned; NULL leaves a
 * filter out for every row.  The struct is read on the host during the call.
 *   temperature T (NULL: 1).  T <= 0 or NaN: the likeliest token alone; below
 *   2^-116 counts as that.
 *   top_k: <= 0 is off.   top_p: >= 1 or NaN is off.   min_p: <= 0 or NaN is
 *   off, above 1 counts as 1. */
typedef struct {
    const float *temperature;
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
} rq_sampling;

/* The distribution that a token is drawn from.  Tokens stand in order of their
 * logits, largest first, equal ones by index, and have whole weights
 *   W = floor(2^42 e^((logit - largest) / T))
 * (2^42 for the largest itself; the others within 2^-32 of their value and one
 * unit of that).  A NaN counts as -Inf; next to +Inf all
 * finite logits weigh 0.  A token stays if
 *   W > 0 and W >= min_p 2^42                                   (min-p),
 *   fewer than top_k of those stand before it                   (top-k), and
 *   the weights before it, of what those two leave, sum to less than top_p
 *   times their total; the first always stays                   (top-p).
 * Sums are whole numbers of 64 bits, so no order of summation matters. */

/* Draw a token per row from u: f32 [rows] random numbers in [0, 1), as
 * rq_verify_chain draws: the first token by index whose running sum of staying
 * weights exceeds floor(U total / 2^24), U = floor(u 2^24) limited to 0 ..
 * 2^24-1.
 *   logits: [rows][vocab] of dtype, rows `stride` elements apart (at least
 *   vocab), aligned to their element.   token: int32 [rows]; -1 for a row of
 *   NaN and -Inf only.
 * 1 <= vocab <= 2^20, 0 <= rows <= 2^27 (0 does nothing).  No scratch.
 * Errors: RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_QTYPE (dtype), RQ_ERR_CUDA. */
rq_status rq_sample(const rq_sampling *sampling_host, int dtype, const void *logits,
                    int64_t stride, const float *u, int32_t *token, int rows, int vocab,
                    rq_stream_t stream);

/* The same distribution written out, as rq_verify_chain and rq_verify_tree
 * take it:  p: f32 [rows][vocab], dense, W / total of the tokens that stay, to
 * 2^-21 of itself whatever W is, and 0 elsewhere (a row of NaN and -Inf only:
 * zeros), so that rq_sample draws no token of p 0; must not overlap the logits.
 * Errors: as rq_sample. */
rq_status rq_token_probs(const rq_sampling *sampling_host, int dtype, const void *logits,
                         int64_t stride, float *p, int rows, int vocab,
                         rq_stream_t stream);

/* ----------------------------------------------------------- tracing --- */

/* Kernel-level tracing of rq_linear, the device-side counterpart of the
 * pages' PREFILL_DETAIL_TRACE phases ([gemm.rs], cublas_prefill_fp8_gemm:
 * absmax+convert / gemm / convert) without their host synchronisations:
 * while tracing is on, every kernel rq_linear launches is bracketed by two
 * CUDA events recorded on the call's stream (as external event nodes when the
 * stream is being captured).  Kinds: */
typedef enum {
    RQ_TRACE_GEMV = 0,    /* Q4_K / Q6_K GEMV                         */
    RQ_TRACE_ABSMAX = 1,  /* (not emitted by rq_linear, which traces the
                             activation's absmax and encoding together
                             as RQ_TRACE_QUANT)                       */
    RQ_TRACE_QUANT = 2,   /* activation absmax + E4M3 quantization    */
    RQ_TRACE_GEMM = 3,    /* FP8 GEMM                                 */
    RQ_TRACE_WCACHE = 4,  /* FP8 weight-cache build (a miss)          */
    RQ_TRACE_KINDS = 5
} rq_trace_kind;

/* Start tracing with room for `capacity` kernels (events are created here,
 * reused across begin/end pairs).  Kernels beyond the capacity are not
 * traced.  Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (capacity < 1),
 * RQ_ERR_ALLOC. */
rq_status rq_ctx_trace_begin(rq_ctx *ctx, int capacity);

/* Restrict tracing to the kinds whose bit (1 << kind) is set in `mask`
 * (all kinds by default): the events of a traced kernel keep it from
 * overlapping its neighbours (programmatic dependent launch), so a caller
 * timing a whole pass traces only the kernels it needs.  Takes effect for
 * kernels launched after the call.  Errors: RQ_ERR_NULL, RQ_ERR_SHAPE (mask
 * 0 or with bits at or above RQ_TRACE_KINDS). */
rq_status rq_ctx_trace_kinds(rq_ctx *ctx, unsigned int mask);

/* Stop tracing, wait for the traced events, and return per kind the number
 * of kernels and their summed device time in milliseconds (arrays of
 * RQ_TRACE_KINDS host entries; either may be NULL).  Errors: RQ_ERR_NULL,
 * RQ_ERR_CUDA. */
rq_status rq_ctx_trace_end(rq_ctx *ctx, int64_t *counts_host, double *ms_host);

/* Synchronise `stream`, then report and clear the library's device error
 * word: RQ_ERR_TIMEOUT if a GEMM, GEMV or attention pipeline wait, or the
 * one-pass quantization's grid barrier, exceeded its time limit (the kernel
 * then stopped early and its output is incomplete), RQ_ERR_INDEX if a cache
 * or attention kernel met a slot, page or position outside its array (it
 * went on without it), RQ_ERR_CUDA if the synchronisation itself failed,
 * RQ_OK otherwise. */
rq_status rq_get_device_status(rq_stream_t stream);

/* Test hook for the timeout path: launches one block that waits on an
 * mbarrier nothing will ever complete, with a wait limit of `limit_ns`
 * nanoseconds, and records a timeout exactly like the GEMM would.  The
 * caller then reads it with rq_get_device_status.  Errors: RQ_ERR_SHAPE
 * (limit_ns outside 1 .. 10^10), RQ_ERR_CUDA. */
rq_status rq_debug_wait_timeout(int64_t limit_ns, rq_stream_t stream);

/* Diagnostics of the GEMVs' accuracy guarantee (rq_q4k_gemv): synchronise
 * `stream`, then return in *count_host the number of GEMV outputs (one per
 * token and row) that were recomputed on the exact fp64 path since the last
 * call, and reset the count.  The count is per process and device; kernels
 * still running on other streams may or may not be included.
 * Errors: RQ_ERR_NULL, RQ_ERR_CUDA. */
rq_status rq_gemv_exact_outputs(rq_stream_t stream, int64_t *count_host);

#ifdef __cplusplus
}
#endif

#endif /* RQ_H */
