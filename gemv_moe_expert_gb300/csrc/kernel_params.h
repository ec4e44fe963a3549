// kernel_params.h -- parameter blocks passed by value from the host dispatch
// (api.cu) to the kernels, and the internal launcher declarations.  Plain C++
// structs: no torch types anywhere in the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gbmm {

enum DType : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

inline int dtype_size(int dt) { return dt == kF32 ? 4 : 2; }

// whether rows ld_bytes apart all start on multiples of `unit` bytes
inline bool rows_on(const void *p, int64_t ld_bytes, int unit) {
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && ld_bytes % unit == 0;
}

// device error word bits
constexpr uint32_t kErrWaitTimeout = 1u;

// kernel ids reported in bits 8..15 of the device error word
enum KernelId : uint32_t {
    kKidNone = 0,
    kKidGemmTc = 1,
    kKidGroupedTc = 2,
    kKidBoundedWaitTest = 3,
    kKidGemvStream = 4,
    kKidGemvTc = 5,
    kKidDirectTc = 6,
    kKidGemvColdotStream = 7,
    kKidPairTc = 8,
    kKidFewTc = 9,
};

// What a launcher has done on a device, a bit each; host threads may launch at the same time.
using DeviceBits = std::atomic<unsigned long long>;

// default limit of a bounded device wait (1 s)
constexpr uint64_t kWaitLimitNs = 1000000000ull;

// Matrix-times-vector problem after the host has mapped (batch, m, n, k,
// transposes, strides) onto "rows" outputs, each a dot product of length k.
// All strides in elements.
//   mat(o, x) = mat[bat*mat_bs + o*mat_rs + x*mat_ks]
//   vec_r(x)  = vec[bat*vec_bs + r*vec_rr + x*vec_ks]     (r < nvec)
//   out_r(o)  = out[bat*out_bs + r*out_rr + o*out_os]
struct GemvParams {
    const void *mat;
    const void *vec;
    void *out;
    int64_t rows, k, batch;
    int64_t mat_rs, mat_ks, mat_bs;
    int64_t vec_ks, vec_rr, vec_bs;
    int64_t out_os, out_rr, out_bs;
    int32_t nvec;     // vectors sharing one pass over the matrix (1..16)
    int32_t vec_ok;   // 16-byte vector path legal (host-checked alignment)
    uint32_t *err;            // device error word (streamed kernel's bounded waits)
    uint64_t wait_limit_ns;
};

// General strided GEMM (FFMA pipe).  Same addressing as the public API.
struct GemmParams {
    const void *a;
    const void *b;
    void *c;
    int64_t batch, m, n, k;
    int64_t lda, ldb, ldc;
    int64_t sa, sb, sc;
    int32_t ta, tb;
};

// Tensor-core GEMM: A and B read by TMA through the two tensor maps, each
// K-contiguous (A [batch][m][k], B [batch][n][k]) or, when a_mn / b_mn is
// set, M/N-contiguous (A [batch][k][m], B [batch][k][n]); C written with
// ldc / sc.
struct GemmTcParams {
    void *c;
    int64_t ldc, sc;
    int32_t m, n, k, batch;
    int32_t a_bcast, b_bcast;   // batch stride 0: always batch coordinate 0
    int32_t a_mn, b_mn;         // operand stored M- / N-contiguous
    int32_t c_vec_ok;           // C rows allow 16-byte stores (1) or 32-byte stores (2)
    int32_t tiles_m, tiles_n;
    int32_t num_tiles;
    uint32_t *err;
    uint64_t wait_limit_ns;
};

// Expert-ID matmul (all routes).
struct MatmulIdParams {
    const void *w;
    const float *x;
    const uint32_t *ids;
    float *out;
    uint32_t *counts;        // grouped route scratch
    uint32_t *routed_rows;   // grouped route scratch, row stride m
    int64_t m, n, k, top_k, n_experts;
    int64_t expert_stride_elems;
    int64_t x_token_stride, x_slot_stride;   // elements
    int64_t total_rows;                      // m * top_k
    uint32_t *err;
    uint64_t wait_limit_ns;
};

// Skinny decode GEMV on the tensor cores: y[m, n] (row stride ldc) =
// x[m, k] W[n, k]^T, the operands read through tensor maps.
struct GemvTcParams {
    void *c;
    int64_t ldc;
    int32_t m, n, k;
    int32_t ksplit;  // CTAs per cluster splitting k (1..8), from gemv_tc_split()
    uint32_t *err;
    uint64_t wait_limit_ns;
};

// Top-k softmax router (moe_route.cu).  logits [m, n_experts], rows
// ld_logits elements apart; ids, weights, d_weights [m, top_k] tight.
struct MoeRouteParams {
    const void *logits;
    const float *bias;       // added for the selection only; may be null
    uint32_t *ids;           // written forward, read backward
    float *weights;          // written forward, read backward
    const float *d_weights;  // backward
    void *d_logits;          // backward
    int64_t ld_logits, ld_d_logits;
    uint32_t m, n_experts, top_k;
    int32_t selected;        // softmax over the chosen experts (1) or over every live one (0)
    int32_t logits_vec, bias_vec, d_logits_vec;  // rows divide into aligned runs (set by the launcher)
};

// Stable sort of routed rows by expert (moe_sort.cu).
struct MoeSortParams {
    const uint32_t *ids;  // [rows]
    uint32_t *offsets;    // [n_experts + 1]
    uint32_t *order;      // [rows]
    uint32_t *position;   // [rows]
    uint32_t *scratch;    // moe_sort_scratch_words() words
    uint32_t rows, n_experts;
};

// Rows of n elements in token order (tok, m rows) and in expert order (row,
// m * top_k rows); moe_rows.cu.  position / offsets null: routed row r is row r.
struct MoeRowsParams {
    const void *tok_in;    // dispatch: x; combine backward: d_y
    void *tok_out;         // combine: y; dispatch backward: d_x
    const void *row_in;    // combine, its backward: ys; dispatch backward: d_xs
    void *row_out;         // dispatch: xs; combine backward: d_ys
    const float *weights;  // [m, top_k]; null = 1 (dispatch backward)
    float *d_weights;      // combine backward
    const uint32_t *position;
    const uint32_t *valid;  // offsets + n_experts: rows that have an expert
    int64_t ld_tok_in, ld_tok_out, ld_row_in, ld_row_out;
    int64_t n;
    uint32_t m, top_k;
};

// Matrix-vector products with 4-bit weights (q4.cuh), dense (ids null: every
// row of x through the one matrix) or per expert id (routed row r through
// matrix ids[r]).
struct Q4Params {
    const uint8_t *q;
    const void *scales;
    const uint8_t *zeros;  // null: 8
    const void *x;
    void *out;
    const uint32_t *ids;
    int64_t ldq, expert_stride;  // bytes
    int64_t ldx, x_slot_stride;  // elements; x row of routed row r: (r / top_k) ldx + (r % top_k) x_slot_stride
    int64_t ldo;
    int64_t n, k, groups;        // groups = ceil(k / group)
    int32_t group, scale_dtype;
    uint32_t rows, top_k, n_experts;
    uint32_t first_row;  // per expert id: the launch's first routed row; it takes kQ4LaunchRows at most
};
constexpr uint32_t kQ4Window = 1024;  // routed rows that a CTA searches for its expert's
constexpr uint32_t kQ4LaunchRows = 65535u * kQ4Window;

// Gated projection h = act(x Wg^T) * (x Wu^T) (gated.cu): index 0 is the gate, 1 the up projection.
struct GatedParams {
    const void *x;
    const void *w[2];  // [n, k]
    void *h;
    void *saved[2];    // both projections, or null
    int64_t m, n, k;
    int64_t ldx, ldw, ldh, ld_saved;
    int32_t act;       // GBMM_GATE_*
};

// d_gate and d_up from d_h and the saved projections (gated.cu).
struct GatedGradParams {
    const void *gate, *up, *d_h;
    void *d[2];
    int64_t m, n, ld_saved, ld_dh, ldd;
    int32_t act;
};

// c [m, n] = a[0] b[0] + a[1] b[1], a [m, k] and b [k, n] (gated.cu).
struct SumGemmParams {
    const void *a[2], *b[2];
    void *c;
    int64_t m, n, k, lda, ldb, ldc;
};

// c[i] [n, k] = d[i]^T x, d [m, n] and x [m, k] (gated.cu).
struct OuterGemmParams {
    const void *x, *d[2];
    void *c[2];
    int64_t m, n, k, ldx, ldd, ldc;
};

// Rows laid out again: src [rows, cols] into dst [rows, ldd].  16-bit values, ldd a multiple of 8 (gated.cu); 8-bit
// codes, ldd a multiple of 16, to_size bytes each at dst: 1, or 2 for f16 (i8.cu).
struct RepackParams {
    const void *src;
    void *dst;
    int64_t rows, cols, lds, ldd;
    int32_t to_size;
};

// Rows to 8-bit codes with a scale each, and the product of such codes (i8.cu).
struct QuantizeParams {
    const void *x;
    int8_t *q;
    float *scale;
    int64_t m, k, ldx, ldq;
};
struct GemmI8Params {
    const int8_t *a, *b;
    const float *scale_a, *scale_b;  // null: 1
    void *c;
    int64_t m, n, k, lda, ldb, ldc;
};

// Products of the feed-forward block on CTA pairs (pair_tc.cu): what the tensor maps do not say.
struct PairTcParams {
    void *c;
    void *saved[2];                  // gated: both projections, or null
    const float *scale_a, *scale_b;  // codes; null: 1
    int64_t ldc, ld_saved;
    int32_t m, n, k;                 // k: of one source
    int32_t c_tma, saved_tma;        // the output's maps may be used (its rows start on multiples of 16 bytes)
    int32_t act;
    int32_t tiles_m, tiles_n;  // set by the launcher
    uint32_t *err;
    uint64_t wait_limit_ns;
    // gradients: c [m, n] over both sources of k, and dw[i] [k, n] over m; either may be left out
    void *dw[2];
    int64_t ld_dw;
    int32_t need_c, need_dw, dw_tma;
    int32_t pairs;                              // these and the next are set by the launcher
    int32_t dw_tiles_m, c_units, c_split, dw_units, dw_split, early, behind;
};
struct PairTcMaps {
    CUtensorMap a[2], b[2];
    CUtensorMap out[3];  // c, and both saved projections or both weights' gradients, as 32 x 32 pieces
    CUtensorMap dw_a[2], dw_b;  // gradients: the sources' columns and x, in 64 x 64 boxes
};

// The same products for some tens of tokens (few_tc.cu).
struct FewTcParams {
    void *c;
    void *saved[2];                  // gated: both projections, or null
    const float *scale_a, *scale_b;  // codes; null: 1
    int64_t ldc, ld_saved;
    int32_t m, n, k;
    int32_t act;
    int32_t ksplit, token_blocks;    // these and tmem_cols: few_tc_plan()
    uint32_t tmem_cols;
    uint32_t *err;
    uint64_t wait_limit_ns;
};
struct FewTcMaps {
    CUtensorMap x[2], w[2];  // boxes of 128 bytes x tokens, and x few_tc_rows() (sum: 64) rows; x[1]: only sum
};

// ---- launchers (each returns the launch's cudaError_t) --------------------

cudaError_t launch_fill_zero(int dt, void *c, int64_t batch, int64_t m, int64_t n, int64_t ldc,
                             int64_t sc, cudaStream_t s);
cudaError_t launch_gemv_rowdot(int dt, const GemvParams &p, cudaStream_t s);
cudaError_t launch_gemv_coldot(int dt, const GemvParams &p, cudaStream_t s);
// staged-stream GEMV (stream.cu) and the shapes it takes
bool gemv_stream_eligible(int dt, const GemvParams &p);
cudaError_t launch_gemv_stream(int dt, const GemvParams &p, int num_sms, cudaStream_t s);
// column-dot GEMV fed by TMA (gemv.cu): `map` is a 3-D tensor map over
// (outputs, k, batch) of the matrix with gemv_coldot_stream_box_cols() x
// gemv_coldot_stream_box_rows() boxes, no swizzle
cudaError_t launch_gemv_coldot_stream(int dt, const CUtensorMap &map, const GemvParams &p, cudaStream_t s);
int gemv_coldot_stream_box_cols(int dt);
int gemv_coldot_stream_box_rows();
// skinny decode GEMV on the tensor cores (gemv_tc.cu): W boxes of
// gemv_tc_block_rows() rows, x boxes of gemv_tc_max_tokens() rows, both
// gemv_tc_block_k() wide
cudaError_t launch_gemv_tc(int dt, const CUtensorMap &map_w, const CUtensorMap &map_x, const GemvTcParams &p,
                           cudaStream_t s);
int gemv_tc_block_rows();
int gemv_tc_max_tokens();
int gemv_tc_block_k();
int gemv_tc_split(int64_t n, int64_t k, int num_sms);
cudaError_t launch_gemm_simt(int dt, const GemmParams &p, cudaStream_t s);
cudaError_t launch_gemm_small(int dt, const GemmParams &p, cudaStream_t s);
cudaError_t launch_gemm_tc(int dt, const CUtensorMap &map_a, const CUtensorMap &map_b,
                           const GemmTcParams &p, int num_sms, cudaStream_t s);
// 256 x 256 tiles (gemm_tc_wide_block_m() rows) over CTA pairs (tcgen05 cta_group::2); a
// K-contiguous operand's tensor map has gemm_tc_block_m()-row boxes, an
// M/N-contiguous one 64 x 64 boxes
cudaError_t launch_gemm_tc_pair(int dt, const CUtensorMap &map_a, const CUtensorMap &map_b,
                                const GemmTcParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_matmul_id_direct(int wdt, const MatmulIdParams &p, cudaStream_t s);
cudaError_t launch_matmul_id_map(const MatmulIdParams &p, cudaStream_t s);
cudaError_t launch_matmul_id_grouped_simt(int wdt, const MatmulIdParams &p, cudaStream_t s);
cudaError_t launch_matmul_id_grouped_tc(const CUtensorMap &map_w, const MatmulIdParams &p, int out_vec_ok,
                                        int split, int f16, int num_sms, cudaStream_t s);
cudaError_t launch_bounded_wait_test(uint32_t *err, uint64_t limit_ns, cudaStream_t s);
int grouped_tc_max_experts();
// Direct route on the tensor cores (direct_tc.cu): bf16 or f16 weights
// (wdt) through a 3-D tensor map over (k, n, expert) with direct_tc_block_k()
// x direct_tc_block_rows() boxes; at most direct_tc_max_ids() routed rows and
// direct_tc_max_experts() experts
cudaError_t launch_matmul_id_direct_tc(int wdt, const CUtensorMap &map_w, const MatmulIdParams &p,
                                       int max_distinct, int ksplit, int x_vec_ok, cudaStream_t s);
int direct_tc_split(int64_t n, int64_t k, int64_t max_distinct, int64_t max_rows_per_expert, int num_sms);
int direct_tc_max_ids();
int direct_tc_max_experts();
int direct_tc_block_rows();
int direct_tc_block_k();
int grouped_tc_block_k();

cudaError_t launch_moe_route(int dt, const MoeRouteParams &p, cudaStream_t s);
cudaError_t launch_moe_route_backward(int dt, const MoeRouteParams &p, cudaStream_t s);
uint64_t moe_sort_scratch_words(uint64_t rows, uint32_t n_experts);
int moe_sort_launches(uint64_t rows);
cudaError_t prepare_moe_sort(uint64_t rows);  // before the first of its launches
cudaError_t launch_moe_sort(int step, const MoeSortParams &p, cudaStream_t s);
cudaError_t launch_moe_dispatch(int dt, const MoeRowsParams &p, cudaStream_t s);
cudaError_t launch_moe_combine(int dt, const MoeRowsParams &p, cudaStream_t s);
cudaError_t launch_moe_combine_backward(int dt, const MoeRowsParams &p, cudaStream_t s);
cudaError_t launch_q4_f32(const Q4Params &p, cudaStream_t s);
cudaError_t launch_q4_f16(const Q4Params &p, cudaStream_t s);
cudaError_t launch_q4_bf16(const Q4Params &p, cudaStream_t s);

// gated projection: one warp a column for few rows, FFMA tiles for any number
cudaError_t launch_gated_rowdot(int dt, const GatedParams &p, cudaStream_t s);
cudaError_t launch_gated_simt(int dt, const GatedParams &p, cudaStream_t s);
cudaError_t launch_gated_grad(int dt, const GatedGradParams &p, cudaStream_t s);
// f32
cudaError_t launch_gated_products_simt(const SumGemmParams *x, const OuterGemmParams *w, cudaStream_t s);
void gated_simt_plan(int64_t m, int64_t n, int64_t k, int64_t sms, int32_t plan[2]);
void gated_products_simt_plan(int64_t m, int64_t n, int64_t k, bool need_x, bool need_w, int64_t sms, int32_t plan[4]);
int gated_few_tokens();
cudaError_t launch_gated_outer_few(int dt, const GatedGradParams &p, const OuterGemmParams &w, cudaStream_t s);
cudaError_t launch_repack16(const RepackParams (&p)[3], cudaStream_t s);
cudaError_t launch_lay_out_codes(const RepackParams &a, const RepackParams &b, cudaStream_t s);  // rows 0: nothing to do
// on the tensor cores: gated a[0] = x, b = both weights, all K-contiguous in boxes of pair_tc_rows()
// rows; gradients a and b as in SumGemmParams, b in 64 x 64 boxes; codes a[0] and b[0] (f16) as gated
cudaError_t launch_gated_tc(int dt, const PairTcMaps &maps, const PairTcParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_gated_products_tc(int dt, const PairTcMaps &maps, const PairTcParams &p, int num_sms, cudaStream_t s);
cudaError_t launch_gemm_i8_tc(int dt, const PairTcMaps &maps, const PairTcParams &p, int num_sms, cudaStream_t s);
int pair_tc_rows();
int pair_tc_block_k();
int few_tc_rows(bool codes);
bool few_tc_takes(bool codes, int64_t m, int64_t n, int64_t k);
bool few_tc_half_tokens(int64_t m);
int few_tc_plan(bool codes, int64_t m, int64_t n, int64_t k, int num_sms, FewTcParams *p);
int few_tc_block_k();
int few_tc_ctas_per_sm(bool codes, int tokens);
bool few_tc_takes_sum(int64_t m, int64_t n, int64_t k, bool need_w, int num_sms);
int few_tc_plan_sum(int64_t m, int64_t n, int64_t k, int num_sms, FewTcParams *p);
cudaError_t launch_sum_few(int dt, int tokens, const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s);
cudaError_t launch_gated_few(int dt, int tokens, const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s);
cudaError_t launch_gemm_i8_few(int dt, int tokens, const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s);
cudaError_t launch_quantize_i8(int dt, const QuantizeParams &p, cudaStream_t s);
cudaError_t launch_gemm_i8_dot(int dt, const GemmI8Params &p, cudaStream_t s);

int gemm_tc_block_m();
int gemm_tc_wide_block_m();
int gemm_tc_block_n();
int gemm_tc_block_k();
int device_sm_count();

// device address of the error word on the current device (nullptr on failure)
uint32_t *device_error_word();

}  // namespace gbmm
