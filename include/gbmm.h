/*
 * gbmm.h -- C ABI of the GB300 (sm_103a) dense GEMM / GEMV / expert-ID matmul
 * library (libgbmm.so), with the router, token order and gradients of a
 * mixture-of-experts layer, 4-bit matrix-vector products, the gated
 * feed-forward projection with its gradients and products of 8-bit integers.
 *
 * Conventions shared by every entry point
 *   - Pointers named a, b, c, weights, input, ids, out, expert_counts and
 *     routed_rows are DEVICE pointers (cudaMalloc / torch CUDA memory of the
 *     current device).  The caller owns all device memory; the library never
 *     allocates device memory on a call path and never synchronises the
 *     stream (except gbmm_device_error and the test hooks, which say so).
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default
 *     stream) and runs asynchronously.  Stream order is the only ordering:
 *     reuse of an output or scratch buffer on the same stream is safe, on
 *     another stream the caller must order it.
 *   - Fail-closed: every argument check runs on the host before the first
 *     launch.  A call that returns an error launched nothing and wrote
 *     nothing.  gbmm_last_error() then describes the failure.
 *   - Thread safety: calls may be made from several host threads; the error
 *     string is per thread.
 *   - CUDA graphs: every call can be captured into a graph once the same
 *     call has run on the device outside the capture (the first call on a
 *     device sets kernel attributes, looks up the device error word and loads
 *     modules, which a capture does not allow); replays read whatever
 *     the captured buffers hold.  GroupedPrefill's grouped kernel is launched
 *     with programmatic stream serialisation behind the map kernel and waits
 *     for it before touching global memory, which a capture keeps; the kernels
 *     of gbmm_moe_*, gbmm_gated* and *_i8 are behind whatever precedes them.  Not with
 *     GBMM_DEBUG_SYNC=1 (it synchronises the stream).
 *   - Debugging: with the environment variable GBMM_DEBUG_SYNC=1 (read once
 *     per process) every launch is followed by a stream synchronisation, so a
 *     kernel that fails on the device is reported by the call that launched
 *     it (GBMM_ERR_CUDA, with the kernel's name in gbmm_last_error()) -- the
 *     counterpart of [P1]'s debug wait_until_completed.
 *
 * Sources (page titles and the items on them)
 *   [P1] tract-metal 0.23.6, src/kernels/matmul/mlx_gemm/mod.rs
 *   [P2] mlx-native 0.13.0, src/ops/dense_matmul_id.rs
 *   [P3] rlx-metal 0.2.14, src/mps_blas.rs
 */
#ifndef GBMM_H
#define GBMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GBMM_ABI_VERSION 1u
/* Schema version of the expert-ID capability record, as in [P2]
 * `DENSE_MATMUL_ID_SCHEMA_VERSION`. */
#define GBMM_MATMUL_ID_SCHEMA_VERSION 3u
/* Most experts the grouped route accepts, as in [P2] `GROUPED_MAX_EXPERTS`. */
#define GBMM_GROUPED_MAX_EXPERTS 1024u

#if defined(__GNUC__)
#define GBMM_API __attribute__((visibility("default")))
#else
#define GBMM_API
#endif

typedef struct CUstream_st *gbmm_stream; /* == cudaStream_t */

typedef enum gbmm_status {
    GBMM_OK = 0,
    GBMM_ERR_INVALID_ARGUMENT = 1,  /* a shape, stride, size, flag or alignment rule failed */
    GBMM_ERR_UNSUPPORTED_DTYPE = 2, /* dtype outside the call's set */
    GBMM_ERR_OVERLAP = 3,           /* an output range overlaps an input or scratch range */
    GBMM_ERR_SCRATCH = 4,           /* grouped route: scratch missing or too small */
    GBMM_ERR_KERNEL_UNAVAILABLE = 5,/* a kernel this call needs could not be resolved */
    GBMM_ERR_LAUNCH = 6,            /* the CUDA launch itself failed */
    GBMM_ERR_DEVICE_TIMEOUT = 7,    /* a bounded device-side wait ran out (gbmm_device_error) */
    GBMM_ERR_CUDA = 8               /* another CUDA runtime error */
} gbmm_status;

typedef enum gbmm_dtype {
    GBMM_F32 = 0,
    GBMM_F16 = 1,
    GBMM_BF16 = 2
} gbmm_dtype;

/* ------------------------------------------------------------------------ */
/* Dense GEMM / GEMV                                                          */
/* ------------------------------------------------------------------------ */

/*
 * gbmm_gemm -- C[b] = op(A[b]) * op(B[b]) for b < batch.
 *
 * Defined by [P1] `MlxGemm::dispatch_eval` / `dispatch_metal_mlx_gemm` and
 * [P3] `encode_mps_sgemm_t` (transposeLeft / transposeRight):
 *   C[b,i,j] = sum_{x<k} Aop[b,i,x] * Bop[b,x,j],   i < m, j < n
 *   Aop[b,i,x] = A[b*batch_stride_a + (transpose_a ? x*lda + i : i*lda + x)]
 *   Bop[b,x,j] = B[b*batch_stride_b + (transpose_b ? j*ldb + x : x*ldb + j)]
 *   C[b*batch_stride_c + i*ldc + j] receives the result.
 * So A is stored [k, m] when transpose_a, else [m, k]; B is stored [n, k]
 * when transpose_b, else [k, n]; all row-major with leading dims lda/ldb/ldc.
 *
 * dt: one dtype for A, B and C ([P1] homogeneous datum types); f32, f16 and
 *   bf16.  Products accumulate in f32; f16/bf16 results are rounded to
 *   nearest-even once, from the f32 accumulator.
 * a/b/c + *_offset_bytes: the matrix base; the sum must be aligned to the
 *   element size (offsets are in bytes, as Metal buffer offsets are in [P1]).
 * lda >= (transpose_a ? m : k), ldb >= (transpose_b ? k : n), ldc >= n, in
 *   elements.  Batch strides are in elements and >= 0; A or B may broadcast
 *   one matrix to every batch with stride 0; batches of C must not overlap.
 * C must not overlap A or B (GBMM_ERR_OVERLAP).
 * Edge cases: batch, m or n == 0 is a no-op; k == 0 writes zeros to C.
 *
 * Route (host-side, fixed rules, [P1] `dispatch_eval`):
 *   - skinny/wide (16-bit dt, !transpose_a, transpose_b, batch == 1,
 *     2 <= m <= 15): one HBM-streaming pass over B with a register tile of m
 *     rows of A ([P1] `gemv_wide_config` gate on m);
 *   - m == 1 or n == 1: the GEMV kernels (as gbmm_gemv);
 *   - otherwise the tensor-core GEMM (tcgen05 + TMEM, TMA-fed) when dt is
 *     f16/bf16 and the TMA layout rules hold (K-contiguous A and B, leading
 *     dims and batch strides multiples of 16 bytes, 16-byte aligned bases),
 *     else the FFMA GEMM.
 */
GBMM_API gbmm_status gbmm_gemm(gbmm_dtype dt, int64_t batch, int64_t m, int64_t n, int64_t k,
                      int transpose_a, int transpose_b,
                      const void *a, int64_t a_offset_bytes, int64_t lda, int64_t batch_stride_a,
                      const void *b, int64_t b_offset_bytes, int64_t ldb, int64_t batch_stride_b,
                      void *c, int64_t c_offset_bytes, int64_t ldc, int64_t batch_stride_c,
                      gbmm_stream stream);

/*
 * gbmm_gemv -- the matrix x vector special case of gbmm_gemm ([P1]
 * `dispatch_metal_mlx_gemv`): same arguments and definition, and requires
 * m == 1 or n == 1 (else GBMM_ERR_INVALID_ARGUMENT).  With n != 1 the
 * matrix is B (the vector is row 0 of op(A)); otherwise the matrix is A (the
 * vector is column 0 of op(B)).  A matrix whose rows run along the
 * contraction dim is read as one coalesced, 128-bit-vectorised stream with
 * warp-shuffle reductions; the other orientation reduces across rows.
 */
GBMM_API gbmm_status gbmm_gemv(gbmm_dtype dt, int64_t batch, int64_t m, int64_t n, int64_t k,
                      int transpose_a, int transpose_b,
                      const void *a, int64_t a_offset_bytes, int64_t lda, int64_t batch_stride_a,
                      const void *b, int64_t b_offset_bytes, int64_t ldb, int64_t batch_stride_b,
                      void *c, int64_t c_offset_bytes, int64_t ldc, int64_t batch_stride_c,
                      gbmm_stream stream);

/* ------------------------------------------------------------------------ */
/* Expert-ID matmul                                                           */
/* ------------------------------------------------------------------------ */

/* [P2] `DenseMatmulIdInputLayout` */
enum { GBMM_INPUT_SHARED_PER_TOKEN = 0, GBMM_INPUT_SLOTTED = 1 };
/* [P2] `DenseMatmulIdMultiplicity` */
enum { GBMM_IDS_DISTINCT_PER_TOKEN = 0, GBMM_IDS_MAY_REPEAT = 1 };
/* [P2] `DenseMatmulIdRoute`: chosen by the caller; the library never picks. */
enum { GBMM_ROUTE_DIRECT = 0, GBMM_ROUTE_GROUPED_PREFILL = 1 };

/* [P2] `DenseMatmulIdParams` */
typedef struct gbmm_matmul_id_params {
    uint32_t m;            /* tokens */
    uint32_t n;            /* output features = rows of each expert matrix */
    uint32_t k;            /* input features = columns of each expert matrix */
    uint32_t top_k;        /* expert slots per token */
    uint32_t n_experts;    /* experts in the weight stack */
    uint32_t input_layout; /* GBMM_INPUT_* */
    uint32_t multiplicity; /* GBMM_IDS_* */
    uint32_t route;        /* GBMM_ROUTE_* */
    uint64_t expert_stride_bytes; /* bytes from expert e to expert e+1 */
    /* GBMM_ACT_* (an extension of this library; zero = the pages' f32
     * activation product).  Only the GroupedPrefill route with bf16 or f16
     * weights on the tensor cores reads it; elsewhere every value computes in
     * f32. */
    uint32_t activation_precision;
    uint32_t reserved;     /* must be 0 */
} gbmm_matmul_id_params;

/*
 * Activation precision of the tensor-core grouped GEMM (bf16 or f16 weights,
 * f32 activations).  Tensor cores multiply pairs of one 16-bit type, so the
 * f32 activations must be rounded to the weights' type (for f16 weights each
 * routed row first scaled by a power of two that puts its largest magnitude
 * in [2^14, 2^15), and the result scaled back exactly):
 *   GBMM_ACT_SPLIT (default): x = hi + lo with hi = round(x), lo = round(x - hi),
 *     both multiplied by the weights -- activation error <= 2^-16 |x| (bf16),
 *     2^-22 |x| (f16), the product is f32-accurate and every element meets
 *     2e-3 * sum|w||x|.
 *   GBMM_ACT_BF16: x rounded once, half the tensor work -- activation error
 *     <= 2^-8 |x| for bf16 weights, so an element can differ from the f32
 *     product by up to ~2^-8 * sum|w||x| (about 3.9e-3, above the 2e-3 bound
 *     when all products share a sign; far below it for zero-mean data); for
 *     f16 weights <= 2^-11 |x|, inside the bound.
 */
enum { GBMM_ACT_SPLIT = 0, GBMM_ACT_BF16 = 1 };

/* [P2] `DenseMatmulIdCapability` + `DenseMatmulIdScratchRequirement` */
typedef struct gbmm_matmul_id_capability_t {
    uint32_t schema_version;     /* GBMM_MATMUL_ID_SCHEMA_VERSION */
    uint32_t weight_dtype;       /* gbmm_dtype */
    uint32_t route;              /* GBMM_ROUTE_* */
    uint32_t has_scratch;        /* 1 for the grouped route */
    uint64_t required_weight_bytes; /* (n_experts-1)*expert_stride_bytes + n*k*size */
    uint64_t required_input_bytes;  /* (shared ? m : m*top_k) * k * 4 */
    uint64_t required_ids_bytes;    /* m*top_k*4 */
    uint64_t required_output_bytes; /* m*top_k*n*4 */
    uint64_t expert_counts_bytes;   /* n_experts*4 (grouped), else 0 */
    uint64_t routed_rows_bytes;     /* n_experts*m*4 (grouped), else 0 */
} gbmm_matmul_id_capability_t;

/* [P2] `DenseMatmulIdDispatchReceipt` */
typedef struct gbmm_matmul_id_receipt {
    uint32_t weight_dtype;  /* gbmm_dtype */
    uint32_t route;         /* GBMM_ROUTE_* */
    uint32_t launch_count;  /* kernels enqueued: 1 (Direct) or 2 (GroupedPrefill) */
} gbmm_matmul_id_receipt;

/*
 * Caller-owned scratch of the grouped route ([P2] `DenseMatmulIdScratch`):
 *   expert_counts  u32[max_experts]
 *   routed_rows    u32[max_experts * max_tokens]
 * After a grouped call, expert_counts[e] is the number of routed rows with
 * id e and routed_rows[e*m + i], i < expert_counts[e], lists them in
 * increasing order of the flattened routed row r = t*top_k + s.  Both
 * buffers must outlive the work enqueued on them and must not overlap the
 * weights, input, ids, output or each other.
 */
typedef struct gbmm_matmul_id_scratch {
    uint32_t *expert_counts;
    uint64_t expert_counts_bytes;
    uint32_t *routed_rows;
    uint64_t routed_rows_bytes;
    uint32_t max_experts;
    uint32_t max_tokens;
} gbmm_matmul_id_scratch;

/*
 * gbmm_matmul_id_scratch_bytes -- byte sizes of the scratch buffers for a
 * capacity of (max_experts, max_tokens), as [P2] `DenseMatmulIdScratch::new`
 * computes them (both capacities must be nonzero; overflow is an error).
 * Allocates nothing.
 */
GBMM_API gbmm_status gbmm_matmul_id_scratch_bytes(uint32_t max_experts, uint32_t max_tokens,
                                         uint64_t *expert_counts_bytes,
                                         uint64_t *routed_rows_bytes);

/*
 * gbmm_matmul_id_capability -- fail-closed validation and exact byte
 * extents, with the rules of [P2] `dense_matmul_id_capability`:
 *   m, n, k, top_k, n_experts nonzero; DistinctPerToken with top_k >
 *   n_experts rejected; weight dtype f32/f16/bf16; expert_stride_bytes >=
 *   n*k*size and a multiple of size; all extents overflow-checked in u64;
 *   m*top_k <= UINT32_MAX; GroupedPrefill requires DistinctPerToken and
 *   n_experts <= GBMM_GROUPED_MAX_EXPERTS.
 * Writes *out on success only.  Host-only: needs no GPU.
 */
GBMM_API gbmm_status gbmm_matmul_id_capability(gbmm_dtype weight_dtype, const gbmm_matmul_id_params *p,
                                      gbmm_matmul_id_capability_t *out);

/*
 * gbmm_matmul_id -- expert-ID matrix multiplication ([P2] `dense_matmul_id`).
 *
 * For routed row r = t*top_k + s (t < m, s < top_k) with e = ids[r]:
 *   e >= n_experts: out[r, :] = 0 (the whole row is overwritten, no weight
 *                   address is formed);
 *   otherwise:      out[r, j] = sum_{x<k} W_e[j, x] * xrow(t, s)[x],  j < n,
 * W_e = the row-major [n, k] matrix at byte offset e*expert_stride_bytes of
 * `weights`; xrow(t, s) = input + t*k (SharedPerToken) or input +
 * (t*top_k + s)*k (Slotted); out is f32 [m, top_k, n].  Weights are widened
 * to f32; accumulation is f32.
 *
 * weights/input/ids/out (+ *_bytes): device buffers and their lengths; each
 *   length must cover the capability extent and each pointer must be aligned
 *   to its element type ([P2] `validate_buffer`).
 * out must not overlap weights, input or ids ([P2]
 *   `validate_dense_matmul_id_call`), else GBMM_ERR_OVERLAP.
 * scratch: required for GroupedPrefill (max_experts >= n_experts, max_tokens
 *   >= m, byte lengths >= the requirement; else GBMM_ERR_SCRATCH); may be
 *   NULL for Direct.
 * Routes:
 *   Direct: one launch; each distinct expert selected by the call is
 *     streamed from HBM once and applied to every row that selected it (bf16
 *     or f16 weights with 16-byte aligned rows and at most 1024 routed rows:
 *     on the tensor cores, activations split into hi + lo of the weights'
 *     type -- for f16 each routed row first scaled by a power of two into
 *     f16's range, and scaled back exactly; otherwise on the FFMA pipe).
 *   GroupedPrefill: two launches in stream order -- the routing map
 *     (expert_counts / routed_rows, atomic-free count / scan / scatter; also
 *     zero-fills rows with out-of-range ids), then the grouped GEMM over
 *     each expert's row list (tensor cores for bf16 weights with hi + lo
 *     activations, and for f16 weights with per-row scaled f16 hi + lo; FFMA
 *     for f32 weights and strides TMA cannot read).  The second launch reads
 *     the first's scratch; a later call may reuse the scratch on the same
 *     stream.
 * Both kernels this call needs are resolved before the first launch; if one
 * is unavailable the call fails with nothing enqueued ([P2] `dense_matmul_id`
 * resolves every pipeline before touching the encoder).
 * receipt (may be NULL): written on success.
 */
GBMM_API gbmm_status gbmm_matmul_id(const gbmm_matmul_id_params *p, gbmm_dtype weight_dtype,
                           const void *weights, uint64_t weights_bytes,
                           const float *input, uint64_t input_bytes,
                           const uint32_t *ids, uint64_t ids_bytes,
                           float *out, uint64_t out_bytes,
                           const gbmm_matmul_id_scratch *scratch,
                           gbmm_stream stream, gbmm_matmul_id_receipt *receipt);

/*
 * gbmm_matmul_id_static_scratch -- the GroupedPrefill route of
 * gbmm_matmul_id for callers that cannot allocate device memory.  (The
 * pages have no counterpart: their grouped route always takes caller-owned
 * scratch.)
 *
 * Who needs it: a caller that is handed only the operands and outputs of
 * each call while someone else owns all other device memory (a plugin slot
 * in another runtime), or a serving loop that may not call cudaMalloc once
 * it runs, since an allocation can wait on a device-wide synchronisation.
 * Such a caller cannot supply the expert_counts / routed_rows buffers.
 *
 * What it does: exactly gbmm_matmul_id with route GroupedPrefill (same
 * arguments minus `scratch`, same results, two launches), with the scratch
 * taken from one fixed array compiled into the library.  The array holds
 * GBMM_GROUPED_MAX_EXPERTS counts and GBMM_STATIC_SCRATCH_ROUTED_ROWS_BYTES
 * of routed rows, i.e. n_experts * m <= 1,048,576; it is reserved on every
 * GPU that loads the library until the process exits.  The call allocates
 * nothing and calls no allocating routine.
 *
 * Errors: GBMM_ERR_INVALID_ARGUMENT for a NULL params or a route other than
 * GroupedPrefill; GBMM_ERR_SCRATCH (nothing launched) when n_experts * m * 4
 * exceeds the array; otherwise every rule and status of gbmm_matmul_id.
 *
 * Sharing: every call on every stream of a device uses the same array, and
 * the array keeps the last call's contents.  Nothing in it needs to start at
 * zero (each call rewrites what it reads).  Calls whose work overlaps on the
 * GPU -- concurrent streams, or host threads without stream ordering between
 * them -- race on the array and corrupt each other's results; order them.
 *
 * Set-up: the first call on each device (that device current) looks up the
 * array's device address with cudaGetSymbolAddress and caches it.  With the
 * CUDA runtime's lazy module loading (the default) that lookup is also what
 * loads the array onto the device: a one-time device allocation made by the
 * CUDA runtime, not by this library.  So make one call per device as a
 * warm-up, before serving starts and before any stream capture on it.  The
 * cached address belongs to the device's current context: after
 * cudaDeviceReset (or any reset of the primary context) the array may live
 * at another address, and this entry point must not be called again in that
 * process.
 */
#define GBMM_STATIC_SCRATCH_ROUTED_ROWS_BYTES (4u << 20)
GBMM_API gbmm_status gbmm_matmul_id_static_scratch(const gbmm_matmul_id_params *p,
                                                   gbmm_dtype weight_dtype,
                                                   const void *weights, uint64_t weights_bytes,
                                                   const float *input, uint64_t input_bytes,
                                                   const uint32_t *ids, uint64_t ids_bytes,
                                                   float *out, uint64_t out_bytes,
                                                   gbmm_stream stream,
                                                   gbmm_matmul_id_receipt *receipt);

/* ------------------------------------------------------------------------ */
/* Mixture-of-experts layer: router, expert order, combine                     */
/* ------------------------------------------------------------------------ */
/*
 * What surrounds the expert products, with the gradients that training needs.
 * (The pages have no counterpart: their callers bring ids.)  Shared rules:
 *   - m tokens, top_k expert slots per token; routed row r = t*top_k + s, as in
 *     gbmm_matmul_id.  An id >= n_experts means "no expert"; all of these calls
 *     and gbmm_matmul_id agree on that.  m * top_k < 2^31; n_experts <=
 *     GBMM_GROUPED_MAX_EXPERTS.
 *   - ids, weights and d_weights are tight [m, top_k] (u32 and f32).  Other
 *     matrices have rows ld* elements apart (ld* >= their row length).
 *   - dt (f32, f16, bf16) is the type of the logits, or of every matrix of rows
 *     in the call.  All arithmetic is f32, sums run in a fixed order (results do
 *     not change from call to call), and each output is rounded once.
 *   - Pointers must be aligned to their elements, outputs must not overlap
 *     inputs or each other (GBMM_ERR_OVERLAP), and m == 0 is a no-op (except
 *     that gbmm_moe_sort writes its offsets).  No call allocates or synchronises.
 */

enum { GBMM_SOFTMAX_ALL = 0, GBMM_SOFTMAX_SELECTED = 1 };
/* Most expert slots per token of the router. */
#define GBMM_MOE_MAX_TOP_K 32u

/*
 * gbmm_moe_route -- top-k softmax gate over logits [m, n_experts].
 *
 * score[t,e] = logit[t,e], plus select_bias[e] rounded to f32 when select_bias
 *   (f32 [n_experts]) is not NULL.  An expert is live for a token when its
 *   score is greater than -inf (so a logit or bias of -inf or NaN masks it).
 * ids[t,:] = the live experts of largest score, in descending order, the lowest
 *   index first among equals.  If fewer than top_k are live the remaining slots
 *   get id n_experts and weight 0; every slot of a row without a live expert does.
 * weights[t,s], with e = ids[t,s] and l the logits (without the bias):
 *   GBMM_SOFTMAX_ALL       exp(l_e) / sum of exp(l) over the live experts
 *   GBMM_SOFTMAX_SELECTED  exp(l_e) / sum of exp(l) over the chosen experts
 *   computed with the maximum subtracted.  A live logit of +inf gives NaN weights.
 * n_experts >= 1, 1 <= top_k <= min(n_experts, GBMM_MOE_MAX_TOP_K).
 */
GBMM_API gbmm_status gbmm_moe_route(gbmm_dtype dt, uint32_t m, uint32_t n_experts, uint32_t top_k,
                                    uint32_t softmax, const void *logits, int64_t ld_logits,
                                    const float *select_bias, uint32_t *ids, float *weights,
                                    gbmm_stream stream);

/*
 * gbmm_moe_route_backward -- d_logits [m, n_experts] from d_weights, given the
 * forward call's arguments and its ids and weights (w):
 *   GBMM_SOFTMAX_ALL       d_l[e] = p[e] * (g[e] - c) for live e, p the softmax
 *     over the live experts, g[e] = d_weights[s] where ids[s] == e, else 0
 *   GBMM_SOFTMAX_SELECTED  d_l[ids[s]] = w[s] * (d_weights[s] - c)
 *   with c = sum_s w[s] * d_weights[s] over the slots that have an expert; every
 *   other entry 0.  The selection itself has no gradient.
 * GBMM_SOFTMAX_SELECTED reads neither logits nor select_bias (both may be NULL).
 * ids must be distinct within a token (those of gbmm_moe_route are) or n_experts.
 */
GBMM_API gbmm_status gbmm_moe_route_backward(gbmm_dtype dt, uint32_t m, uint32_t n_experts, uint32_t top_k,
                                             uint32_t softmax, const void *logits, int64_t ld_logits,
                                             const float *select_bias, const uint32_t *ids,
                                             const float *weights, const float *d_weights, void *d_logits,
                                             int64_t ld_d_logits, gbmm_stream stream);

/* gbmm_moe_sort_scratch_bytes -- bytes of scratch that gbmm_moe_sort needs for
 * these sizes (0 is possible); grows with m.  Host-only. */
GBMM_API gbmm_status gbmm_moe_sort_scratch_bytes(uint32_t m, uint32_t top_k, uint32_t n_experts,
                                                 uint64_t *bytes);

/*
 * gbmm_moe_sort -- stable order of the routed rows by expert.
 *   position[r]  the place of routed row r: rows of expert 0 first, in increasing
 *                r, then those of expert 1, ..., last the rows without an expert
 *   order[p]     the routed row at place p (order[position[r]] == r)
 *   offsets[e]   the first place of expert e; offsets[n_experts] (n_experts + 1
 *                entries) = the number of rows that have an expert
 * ids may repeat within a token.  scratch (4-byte aligned; NULL when 0 bytes are
 * needed) of at least gbmm_moe_sort_scratch_bytes(), else GBMM_ERR_SCRATCH; its
 * contents need no preparation, and calls in flight must not share it.
 */
GBMM_API gbmm_status gbmm_moe_sort(uint32_t m, uint32_t top_k, uint32_t n_experts, const uint32_t *ids,
                                   uint32_t *offsets, uint32_t *order, uint32_t *position, void *scratch,
                                   uint64_t scratch_bytes, gbmm_stream stream);

/*
 * Rows to expert order and back.  position and offsets are gbmm_moe_sort's; with
 * both NULL the rows stay in routed order and all count as having an expert
 * (the layout that gbmm_matmul_id writes).  "has an expert": position[r] <
 * offsets[n_experts].  Rows of m tokens (x, y and their gradients, [m, n]) and of
 * m * top_k places (xs, ys and their gradients, [m * top_k, n]).
 *
 * gbmm_moe_dispatch            xs[position[r]] = x[t]; zeros where r has no expert
 * gbmm_moe_dispatch_backward   d_x[t] = sum over s of d_xs[position[r]]
 * gbmm_moe_combine             y[t] = sum over s of weights[r] * ys[position[r]]
 * gbmm_moe_combine_backward    d_ys[position[r]] = weights[r] * d_y[t],
 *                              d_weights[r] = <d_y[t], ys[position[r]]>; both zero
 *                              where r has no expert
 * The sums run over the slots that have an expert (rows of xs or ys without one
 * are not read), in increasing s.  n == 0 is a no-op, except that
 * gbmm_moe_combine_backward then writes zeros to d_weights.
 */
GBMM_API gbmm_status gbmm_moe_dispatch(gbmm_dtype dt, uint32_t m, uint32_t top_k, uint32_t n_experts,
                                       int64_t n, const void *x, int64_t ldx, const uint32_t *position,
                                       const uint32_t *offsets, void *xs, int64_t ldxs, gbmm_stream stream);
GBMM_API gbmm_status gbmm_moe_dispatch_backward(gbmm_dtype dt, uint32_t m, uint32_t top_k,
                                                uint32_t n_experts, int64_t n, const void *d_xs,
                                                int64_t ld_dxs, const uint32_t *position,
                                                const uint32_t *offsets, void *d_x, int64_t ld_dx,
                                                gbmm_stream stream);
GBMM_API gbmm_status gbmm_moe_combine(gbmm_dtype dt, uint32_t m, uint32_t top_k, uint32_t n_experts,
                                      int64_t n, const void *ys, int64_t ldys, const float *weights,
                                      const uint32_t *position, const uint32_t *offsets, void *y,
                                      int64_t ldy, gbmm_stream stream);
GBMM_API gbmm_status gbmm_moe_combine_backward(gbmm_dtype dt, uint32_t m, uint32_t top_k,
                                               uint32_t n_experts, int64_t n, const void *ys, int64_t ldys,
                                               const float *weights, const uint32_t *position,
                                               const uint32_t *offsets, const void *d_y, int64_t ld_dy,
                                               void *d_ys, int64_t ld_dys, float *d_weights,
                                               gbmm_stream stream);

/* ------------------------------------------------------------------------ */
/* Matrix-vector products with 4-bit weights                                  */
/* ------------------------------------------------------------------------ */
/*
 * The decode counterpart of gbmm_gemm (few rows, transpose_b) and of
 * gbmm_matmul_id's Direct route for weights of 4 bits.
 *   W[j,x] = (q[j,x] - z[j,g]) * scale[j,g],  g = x / group,  j < n, x < k
 * q: row j starts at byte j*ldq_bytes; byte i of a row holds column 2i in its low
 *   and column 2i+1 in its high four bits (ldq_bytes >= (k+1)/2; the unused half
 *   of the last byte of an odd k is ignored).  Read fastest: a k that is a multiple
 *   of 64, matrices and rows that start on multiples of 32 bytes, and 16-bit scales;
 *   next, multiples of 16 bytes and any k; every other alignment works.
 * group: 32, 64 or 128 columns; the last one may be ragged.  G = ceil(k/group).
 * scales: [n, G] tight, scale_dt f32, f16 or bf16.  zeros: u8 [n, G] tight, values
 *   0..255, or NULL for 8 everywhere.
 * Codes and zero points enter exactly, and are subtracted before the product: a weight
 * of 0 adds exactly 0.  The values of x enter exactly too, f32 included, except that one far below
 * the largest magnitude of its group of columns (2^28 for f16, 2^31 for bf16, 2^37 for f32)
 * may be off by up to 2^-39 (f32: 2^-61) of that magnitude.  Products accumulate in f32, group by
 * group; a group's sum is multiplied by its scale, and each result is rounded once to its type.
 * The sums' error is below (t ceil(group/16) 2^-22 + (k/32 + 16) 2^-24) * sum |x W|, t = 3 for f32
 * and 1 otherwise.  A row with an infinity, a NaN or a magnitude from 2^112 up is computed in
 * plain f32, each W[j,x] rounded first, and much slower.
 */

/* gbmm_gemv_q4 -- y[i,j] = sum_x x[i,x] * W[j,x] for i < m.  x [m, k] and y
 * [m, n] of type dt, rows ldx / ldy elements apart.  Any m: the weights are read
 * once for each block of up to 8 rows (f32: 4 with groups of 128, else 2), so it is
 * meant for few of them.  m or
 * n == 0 is a no-op, k == 0 writes zeros. */
GBMM_API gbmm_status gbmm_gemv_q4(gbmm_dtype dt, uint32_t m, int64_t n, int64_t k, uint32_t group,
                                  const void *q, int64_t ldq_bytes, const void *scales,
                                  gbmm_dtype scale_dt, const uint8_t *zeros, const void *x, int64_t ldx,
                                  void *y, int64_t ldy, gbmm_stream stream);

/* gbmm_matmul_id_q4 -- out[r,:] = x row of r times matrix ids[r], transposed, for
 * the routed rows r = t*top_k + s; ids >= n_experts give zero rows.  Expert e's q
 * starts at byte e*expert_stride_bytes, its scales and zeros at element e*n*G.
 * input_layout GBMM_INPUT_*: x is [m, k] or [m, top_k, k], out [m, top_k, n], both
 * tight and of type dt.  Each distinct expert among 1024 consecutive routed rows
 * is read once for each block of up to 8 of its rows (fewer where a row more
 * would cost the rest more; the second block finds the weights in L2).  m or n == 0 is a no-op,
 * k == 0 writes zeros. */
GBMM_API gbmm_status gbmm_matmul_id_q4(gbmm_dtype dt, uint32_t m, int64_t n, int64_t k, uint32_t top_k,
                                       uint32_t n_experts, uint32_t input_layout, uint32_t group,
                                       const void *q, int64_t ldq_bytes, int64_t expert_stride_bytes,
                                       const void *scales, gbmm_dtype scale_dt, const uint8_t *zeros,
                                       const void *x, const uint32_t *ids, void *out, gbmm_stream stream);

/* ------------------------------------------------------------------------ */
/* Gated feed-forward projection                                              */
/* ------------------------------------------------------------------------ */
/*
 * The first half of a gated feed-forward block, forward and backward; its second
 * half, the product with the down projection, is gbmm_gemm's (or gbmm_gemm_i8's).
 * dt (f32, f16, bf16) is the type of every matrix of a call.  x [m, k], both weights
 * [n, k], h, gate, up and d_h [m, n], rows ld* elements apart (both weights with the
 * same ldw, both saved projections with the same ld_saved, both weights' gradients
 * with the same ld_dw; two of them may lie side by side in rows of that pitch).
 * m, n and k below 2^31.  Sums are f32 in a fixed order, activations are off by at most
 * 2^-20 of their argument (and 2^-14 of themselves down to f32's smallest normal values),
 * and each output is rounded once.  Pointers must be aligned to
 * their elements, and outputs must not overlap inputs, scratch or each other
 * (GBMM_ERR_OVERLAP).
 */
enum {
    GBMM_GATE_SILU = 0,      /* v / (1 + e^-v) */
    GBMM_GATE_GELU = 1,      /* v (1 + erf(v / sqrt 2)) / 2 */
    GBMM_GATE_GELU_TANH = 2, /* v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2 */
    GBMM_GATE_RELU = 3       /* max(v, 0); slope 0 at 0 */
};

/* gbmm_gated_scratch_bytes -- bytes of scratch with which gbmm_gated runs these sizes at
 * full speed.  aligned: nonzero if x and both weights start on multiples of 16 bytes and ldx
 * and ldw are multiples of 16 bytes (0 is returned then); 0 for any layout.  Host-only. */
GBMM_API gbmm_status gbmm_gated_scratch_bytes(gbmm_dtype dt, int64_t m, int64_t n, int64_t k, int aligned,
                                              uint64_t *bytes);

/*
 * gbmm_gated -- h = act(x w_gate^T) * (x w_up^T), both projections, the activation and
 * the product in one kernel.
 * gate, up: both NULL, or both projections are written too (for gbmm_gated_backward).
 * h is computed from the unrounded projections.
 * scratch: 16-bit operands whose rows do not start on multiples of 16 bytes are laid out
 * again in it; where it is NULL such a call runs on the FFMA pipe, many times slower for large
 * m, and where it is smaller than the layout needs the call fails with GBMM_ERR_SCRATCH.  Its
 * contents need no preparation, and calls in flight must not share it.
 * m or n == 0 is a no-op; k == 0 writes zeros.
 */
GBMM_API gbmm_status gbmm_gated(gbmm_dtype dt, uint32_t activation, int64_t m, int64_t n, int64_t k, const void *x,
                                int64_t ldx, const void *w_gate, const void *w_up, int64_t ldw, void *h, int64_t ldh,
                                void *gate, void *up, int64_t ld_saved, void *scratch, uint64_t scratch_bytes,
                                gbmm_stream stream);

/* gbmm_gated_backward_scratch_bytes -- bytes of scratch that gbmm_gated_backward needs (both
 * projections' gradients, and, where x or the weights are not `aligned` as above, 16-bit rows
 * laid out again).  Host-only. */
GBMM_API gbmm_status gbmm_gated_backward_scratch_bytes(gbmm_dtype dt, int64_t m, int64_t n, int64_t k, int aligned,
                                                       uint64_t *bytes);

/*
 * gbmm_gated_backward -- from d_h, x, the weights and the saved projections:
 *   d_gate = d_h * up * act'(gate)      d_up = d_h * act(gate)     (rounded to dt; not for
 *                                       the weights' gradients of up to four tokens)
 *   d_x [m, k] = d_gate w_gate + d_up w_up
 *   d_w_gate [n, k] = d_gate^T x        d_w_up [n, k] = d_up^T x
 * d_x may be NULL (the weights are not read then), and d_w_gate and d_w_up may both be (x is
 * not read).  Gradients are written, not added.  An m of 0 writes zeros to the weights'
 * gradients, an n of 0 zeros to d_x.
 * scratch: at least gbmm_gated_backward_scratch_bytes(), else GBMM_ERR_SCRATCH; its contents
 * need no preparation, and calls in flight must not share it.
 */
GBMM_API gbmm_status gbmm_gated_backward(gbmm_dtype dt, uint32_t activation, int64_t m, int64_t n, int64_t k,
                                         const void *x, int64_t ldx, const void *w_gate, const void *w_up, int64_t ldw,
                                         const void *gate, const void *up, int64_t ld_saved, const void *d_h,
                                         int64_t ld_dh, void *d_x, int64_t ld_dx, void *d_w_gate, void *d_w_up,
                                         int64_t ld_dw, void *scratch, uint64_t scratch_bytes, gbmm_stream stream);

/* ------------------------------------------------------------------------ */
/* Matrix product in 8-bit integers                                           */
/* ------------------------------------------------------------------------ */

/* Longest contraction of gbmm_gemm_i8: its sums stay inside 32-bit integers. */
#define GBMM_I8_MAX_K 131071

/*
 * gbmm_quantize_i8 -- rows of x [m, k] to codes q [m, k] and a scale for each row:
 *   scale[i] = max |x[i,:]| * (1.0f / 127.0f) in f32;  q[i,x] = the integer nearest to
 *   x[i,x] / scale[i] (the real quotient, ties to even), within -127..127
 * so that x is about q * scale.  A row of zeros (or one whose scale is 0 in f32) gets scale 0
 * and codes 0, a row that holds a NaN or an infinity scale NaN and codes 0.  It serves tokens
 * (rows of activations) and channels (rows of a weight [n, k]) alike.  x of type dt.  m == 0 is
 * a no-op; k == 0 writes scales of 0.
 */
GBMM_API gbmm_status gbmm_quantize_i8(gbmm_dtype dt, int64_t m, int64_t k, const void *x, int64_t ldx, int8_t *q,
                                      int64_t ldq, float *scale, gbmm_stream stream);

/* gbmm_gemm_i8_scratch_bytes -- bytes of scratch that gbmm_gemm_i8 needs (0 is possible).
 * aligned: nonzero if a and b start on multiples of 16 bytes and lda and ldb are multiples of
 * 16; 0 for any layout.  Host-only. */
GBMM_API gbmm_status gbmm_gemm_i8_scratch_bytes(int64_t m, int64_t n, int64_t k, int aligned, uint64_t *bytes);

/*
 * gbmm_gemm_i8 -- c[i,j] = (sum_x a[i,x] b[j,x]) * scale_a[i] * scale_b[j]
 * a [m, k] and b [n, k]: codes from -128 to 127, rows lda / ldb bytes apart, any alignment.
 * The sum is that of integers, exactly; it is rounded to f32, multiplied by scale_a and then by
 * scale_b (f32; NULL for 1), and rounded to dt, the type of c.  k <= GBMM_I8_MAX_K.
 * scratch: at least gbmm_gemm_i8_scratch_bytes(), else GBMM_ERR_SCRATCH; its contents need no
 * preparation, and calls in flight must not share it.  m or n == 0 is a no-op.
 */
GBMM_API gbmm_status gbmm_gemm_i8(gbmm_dtype dt, int64_t m, int64_t n, int64_t k, const int8_t *a, int64_t lda,
                                  const float *scale_a, const int8_t *b, int64_t ldb, const float *scale_b, void *c,
                                  int64_t ldc, void *scratch, uint64_t scratch_bytes, gbmm_stream stream);

/* ------------------------------------------------------------------------ */
/* Errors, diagnostics                                                        */
/* ------------------------------------------------------------------------ */

/* Message of the last failed call on this host thread ("" if none).  The
 * string stays valid until the next call on the thread. */
GBMM_API const char *gbmm_last_error(void);

/* Name of a status code. */
GBMM_API const char *gbmm_status_string(gbmm_status s);

/* GBMM_ABI_VERSION. */
GBMM_API uint32_t gbmm_abi_version(void);

/*
 * gbmm_device_error -- synchronises `stream`, then reads and clears the
 * device error word of the current device.  Kernels set it (instead of
 * trapping) when a bounded wait on an mbarrier runs out; the kernel then
 * drains its own copies in flight, releases its tensor memory and returns.
 * *code receives the word (0 = no error; otherwise bit 0 = a wait ran out,
 * bits 8..15 = which kernel).  Returns GBMM_ERR_DEVICE_TIMEOUT when the word
 * was nonzero, GBMM_OK otherwise.
 */
GBMM_API gbmm_status gbmm_device_error(gbmm_stream stream, uint32_t *code);

/* ------------------------------------------------------------------------ */
/* Test hooks (host-side fault injection and launch accounting)               */
/* ------------------------------------------------------------------------ */

/* Makes the next resolution of kernel `name` fail (one shot), like [P2]'s
 * `KernelRegistry::inject_next_pipeline_lookup_failure`.  NULL clears it.
 * The name "*" makes every resolution fail until cleared: a call that passes
 * validation then returns GBMM_ERR_KERNEL_UNAVAILABLE with nothing launched
 * (tests that hand the library addresses no kernel may touch use it).
 * Kernel names: "gbmm_gemv_rowdot", "gbmm_gemv_coldot", "gbmm_gemv_tc", "gbmm_gemm_simt",
 * "gbmm_gemm_tc", "gbmm_fill_zero", "gbmm_matmul_id_direct",
 * "gbmm_matmul_id_map", "gbmm_matmul_id_grouped", and the names of the gbmm_moe_*,
 * *_q4, gbmm_gated* and *_i8 entry points for theirs; "gbmm_moe_sort_place" is the last of gbmm_moe_sort's three. */
GBMM_API void gbmm_test_inject_kernel_failure(const char *name);

/* Kernels launched by this library since load / the last reset. */
GBMM_API uint64_t gbmm_test_launch_count(void);
GBMM_API void gbmm_test_reset_launch_count(void);

/* Name of the kernel of the most recent launch on this host thread:
 * "gbmm_gemm_tc", "gbmm_gemm_simt", "gbmm_gemm_small", "gbmm_gemv_stream",
 * "gbmm_gemv_rowdot", "gbmm_gemv_coldot", "gbmm_gemv_tc", "gbmm_fill_zero",
 * "gbmm_matmul_id_direct", "gbmm_matmul_id_direct_tc", "gbmm_matmul_id_map",
 * "gbmm_matmul_id_grouped_tc", "gbmm_matmul_id_grouped_simt", "gbmm_bounded_wait_test" for the wait test below, and
 * the names of the gbmm_moe_*, *_q4, gbmm_gated* and *_i8 entry points for theirs. */
GBMM_API const char *gbmm_test_last_kernel(void);

/*
 * gbmm_test_bounded_wait -- launches one tiny kernel that waits on an
 * mbarrier that nothing ever arrives on, with a limit of `limit_ns`
 * nanoseconds (clamped to [1 us, 2 s]).  The wait runs out, the kernel sets
 * the device error word and returns; then this call synchronises and
 * returns what gbmm_device_error returns (GBMM_ERR_DEVICE_TIMEOUT with *code
 * set).  Exercises the timeout path without faulting or hanging the GPU.
 */
GBMM_API gbmm_status gbmm_test_bounded_wait(uint64_t limit_ns, gbmm_stream stream, uint32_t *code);

/*
 * gbmm_test_static_scratch_copy -- enqueues on `stream` a device-to-device
 * copy of the first `bytes` bytes of the fixed scratch array that
 * gbmm_matmul_id_static_scratch uses on the current device, into the
 * caller's device buffer `dst`: the expert counts (u32[GBMM_GROUPED_MAX_EXPERTS])
 * first, then the routed-row lists (u32, expert e's list at entry e * m of
 * that region, m the last call's token count).  Lets a test check the routing
 * map the last call left there.  GBMM_ERR_INVALID_ARGUMENT when `bytes`
 * exceeds the array or `dst` is NULL.
 */
GBMM_API gbmm_status gbmm_test_static_scratch_copy(void *dst, uint64_t bytes, gbmm_stream stream);

/*
 * gbmm_test_few_plan -- how a product of some tens of tokens would be divided on a GPU of `sms`
 * SMs; nothing is launched.  form: 0 gbmm_gated, 1 gbmm_gemm_i8 (both 16-byte-aligned), 2 the d_x
 * of gbmm_gated_backward.  plan: tokens of a tile, CTAs that share a tile, columns of tensor memory
 * that each of them allocates, and CTAs that an SM holds at once; zeros where such a call takes
 * another way.
 */
GBMM_API gbmm_status gbmm_test_few_plan(int form, int64_t m, int64_t n, int64_t k, int32_t sms, int32_t plan[4]);

/* gbmm_test_gated_plan -- the same for gbmm_gated on the FFMA pipe (f32, more than 8 rows): height of
 * a tile (64 columns of both projections wide) and CTAs that divide its contraction; zeros where
 * there would be too many. */
GBMM_API gbmm_status gbmm_test_gated_plan(int64_t m, int64_t n, int64_t k, int32_t sms, int32_t plan[2]);

/*
 * gbmm_test_gradient_plan -- how the products of an f32 gbmm_gated_backward would be divided on a
 * GPU of `sms` SMs; nothing is launched.  need_x, need_w: which gradients are asked for.  plan: edge
 * of a tile of d_x (128 or 64; the weights' tiles are as wide, and 64 rows high, of both weights),
 * CTAs that divide the contraction of one tile of d_x, the same of the weights', and whether the
 * weights' tiles come first.
 */
GBMM_API gbmm_status gbmm_test_gradient_plan(int64_t m, int64_t n, int64_t k, int need_x, int need_w, int32_t sms,
                                             int32_t plan[4]);

#ifdef __cplusplus
}
#endif

#endif /* GBMM_H */
