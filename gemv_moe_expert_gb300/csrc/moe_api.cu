// moe_api.cu -- the extern "C" entry points of the mixture-of-experts layer
// around the expert products (gbmm_moe_*) and of the 4-bit matrix-vector
// products (gbmm_gemv_q4, gbmm_matmul_id_q4): argument checks, all of them
// before the first launch, then the launchers.
#include "api_checks.h"
#include "api_internal.h"
#include "kernel_params.h"

using namespace gbmm;

namespace {

// m, top_k and n_experts of every gbmm_moe_* call and of gbmm_matmul_id_q4
gbmm_status check_slots(const char *fn, uint32_t m, uint32_t top_k, uint32_t n_experts) {
    if (top_k == 0 || n_experts == 0)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: top_k and n_experts must be nonzero", fn);
    if (n_experts > GBMM_GROUPED_MAX_EXPERTS)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: at most %u experts (got %u)", fn, GBMM_GROUPED_MAX_EXPERTS,
                    n_experts);
    if (static_cast<uint64_t>(m) * top_k > INT32_MAX)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: m * top_k must stay below 2^31 (m=%u top_k=%u)", fn, m, top_k);
    return GBMM_OK;
}

gbmm_status check_route(const char *fn, gbmm_dtype dt, uint32_t m, uint32_t n_experts, uint32_t top_k,
                        uint32_t softmax) {
    if (!known_dtype(dt))
        return fail(GBMM_ERR_UNSUPPORTED_DTYPE, "%s: dtype %d is not f32, f16 or bf16", fn, (int)dt);
    gbmm_status st = check_slots(fn, m, top_k, n_experts);
    if (st != GBMM_OK) return st;
    if (top_k > n_experts || top_k > GBMM_MOE_MAX_TOP_K)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: top_k %u exceeds n_experts %u or %u", fn, top_k, n_experts,
                    GBMM_MOE_MAX_TOP_K);
    if (softmax > GBMM_SOFTMAX_SELECTED)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: unknown softmax %u", fn, softmax);
    return GBMM_OK;
}

// The four calls on rows share their arguments: tok_* are [m, n], row_* are
// [m * top_k, n]; what a call does not have is null with ld = n.
struct RowsCall {
    const char *fn;
    gbmm_dtype dt;
    uint32_t m, top_k, n_experts;
    int64_t n;
    const char *tok_label, *row_label, *row2_label;
    const void *tok;
    int64_t ld_tok;
    bool tok_output;
    const void *row;
    int64_t ld_row;
    bool row_output;
    const void *row2;  // combine backward: d_ys
    int64_t ld_row2;
    bool has_weights, has_d_weights;
    const float *weights;
    const float *d_weights;
    const uint32_t *position, *offsets;
};

gbmm_status check_rows(const RowsCall &c, bool *empty) {
    *empty = false;
    if (!known_dtype(c.dt))
        return fail(GBMM_ERR_UNSUPPORTED_DTYPE, "%s: dtype %d is not f32, f16 or bf16", c.fn, (int)c.dt);
    gbmm_status st = check_slots(c.fn, c.m, c.top_k, c.n_experts);
    if (st != GBMM_OK) return st;
    if (c.n < 0) return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: negative row length", c.fn);
    if (c.ld_tok < c.n || c.ld_row < c.n || (c.row2_label != nullptr && c.ld_row2 < c.n))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: a leading dimension is smaller than the row length %lld", c.fn,
                    (long long)c.n);
    if ((c.position == nullptr) != (c.offsets == nullptr))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: position and offsets come together or not at all", c.fn);
    if (c.m == 0 || (c.n == 0 && !c.has_d_weights)) {
        *empty = true;
        return GBMM_OK;
    }
    const uint64_t rows = static_cast<uint64_t>(c.m) * c.top_k;
    const uint32_t size = static_cast<uint32_t>(dtype_size(c.dt));
    uint64_t tok_bytes, row_bytes, row2_bytes = 0;
    if (!span(c.m, c.n, c.ld_tok, size, &tok_bytes) || !span(rows, c.n, c.ld_row, size, &row_bytes) ||
        (c.row2_label != nullptr && !span(rows, c.n, c.ld_row2, size, &row2_bytes)))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", c.fn);
    const Operand ops[] = {
        {c.tok_label, c.tok, tok_bytes, size, c.tok_output},
        {c.row_label, c.row, row_bytes, size, c.row_output},
        {c.row2_label, c.row2, row2_bytes, size, true},
        {"weights", c.weights, c.has_weights ? rows * 4 : 0, 4, false},
        {"d_weights", c.d_weights, c.has_d_weights ? rows * 4 : 0, 4, true},
        {"position", c.position, c.position ? rows * 4 : 0, 4, false},
        {"offsets", c.offsets, c.offsets ? (static_cast<uint64_t>(c.n_experts) + 1) * 4 : 0, 4, false}};
    return check_operands(c.fn, ops, static_cast<int>(sizeof ops / sizeof ops[0]));
}

MoeRowsParams rows_params(const RowsCall &c) {
    MoeRowsParams p{};
    p.n = c.n;
    p.m = c.m;
    p.top_k = c.top_k;
    p.weights = c.weights;
    p.position = c.position;
    p.valid = c.offsets ? c.offsets + c.n_experts : nullptr;
    return p;
}

// Checks shared by the two 4-bit calls, and the parameter block.
gbmm_status check_q4(const char *fn, gbmm_dtype dt, int64_t n, int64_t k, uint32_t group, int64_t ldq,
                     gbmm_dtype scale_dt, Q4Params *p, uint64_t *matrix_bytes) {
    if (!known_dtype(dt) || !known_dtype(scale_dt))
        return fail(GBMM_ERR_UNSUPPORTED_DTYPE, "%s: dtypes %d and %d must be f32, f16 or bf16", fn, (int)dt,
                    (int)scale_dt);
    if (n < 0 || k < 0 || n > INT32_MAX || k > INT32_MAX)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: n and k must lie in [0, 2^31)", fn);
    if (group != 32 && group != 64 && group != 128)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: group must be 32, 64 or 128 (got %u)", fn, group);
    const int64_t row_bytes = (k + 1) / 2;
    if (ldq < row_bytes)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: ldq_bytes %lld is smaller than a row's %lld", fn, (long long)ldq,
                    (long long)row_bytes);
    if (!span(static_cast<uint64_t>(n), row_bytes, ldq, 1, matrix_bytes))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    p->n = n;
    p->k = k;
    p->group = static_cast<int32_t>(group);
    p->groups = (k + group - 1) / group;
    p->ldq = ldq;
    p->scale_dtype = scale_dt;
    return GBMM_OK;
}

// Per expert id, a launch for each kQ4LaunchRows routed rows.
gbmm_status launch_q4(const char *fn, gbmm_dtype dt, Q4Params p, cudaStream_t s) {
    if (!resolve_kernel(fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    for (;;) {
        const gbmm_status st = finish_launch(dt == GBMM_F32   ? launch_q4_f32(p, s)
                                             : dt == GBMM_F16 ? launch_q4_f16(p, s)
                                                              : launch_q4_bf16(p, s),
                                             fn, s);
        if (st != GBMM_OK || p.ids == nullptr || p.k == 0 || p.rows - p.first_row <= kQ4LaunchRows) return st;
        p.first_row += kQ4LaunchRows;
    }
}

}  // namespace

extern "C" {

gbmm_status gbmm_moe_route(gbmm_dtype dt, uint32_t m, uint32_t n_experts, uint32_t top_k, uint32_t softmax,
                           const void *logits, int64_t ld_logits, const float *select_bias, uint32_t *ids,
                           float *weights, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_moe_route";
    gbmm_status st = check_route(fn, dt, m, n_experts, top_k, softmax);
    if (st != GBMM_OK) return st;
    if (ld_logits < n_experts)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: ld_logits %lld < n_experts %u", fn, (long long)ld_logits,
                    n_experts);
    if (m == 0) return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt));
    const uint64_t slots = static_cast<uint64_t>(m) * top_k * 4;
    uint64_t logit_bytes;
    if (!span(m, n_experts, ld_logits, size, &logit_bytes))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const Operand ops[] = {{"logits", logits, logit_bytes, size, false},
                           {"select_bias", select_bias, select_bias ? n_experts * 4ull : 0, 4, false},
                           {"ids", ids, slots, 4, true},
                           {"weights", weights, slots, 4, true}};
    st = check_operands(fn, ops, 4);
    if (st != GBMM_OK) return st;
    if (!resolve_kernel(fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    MoeRouteParams p{};
    p.logits = logits;
    p.bias = select_bias;
    p.ids = ids;
    p.weights = weights;
    p.ld_logits = ld_logits;
    p.m = m;
    p.n_experts = n_experts;
    p.top_k = top_k;
    p.selected = softmax == GBMM_SOFTMAX_SELECTED;
    return finish_launch(launch_moe_route(dt, p, cuda_stream(stream)), fn, cuda_stream(stream));
}

gbmm_status gbmm_moe_route_backward(gbmm_dtype dt, uint32_t m, uint32_t n_experts, uint32_t top_k, uint32_t softmax,
                                    const void *logits, int64_t ld_logits, const float *select_bias,
                                    const uint32_t *ids, const float *weights, const float *d_weights,
                                    void *d_logits, int64_t ld_d_logits, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_moe_route_backward";
    gbmm_status st = check_route(fn, dt, m, n_experts, top_k, softmax);
    if (st != GBMM_OK) return st;
    const bool all = softmax == GBMM_SOFTMAX_ALL;
    if ((all && ld_logits < n_experts) || ld_d_logits < n_experts)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: a leading dimension is smaller than n_experts %u", fn, n_experts);
    if (m == 0) return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt));
    const uint64_t slots = static_cast<uint64_t>(m) * top_k * 4;
    uint64_t logit_bytes = 0, d_bytes;
    if ((all && !span(m, n_experts, ld_logits, size, &logit_bytes)) ||
        !span(m, n_experts, ld_d_logits, size, &d_bytes))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const Operand ops[] = {{"logits", logits, logit_bytes, size, false},
                           {"select_bias", select_bias, all && select_bias ? n_experts * 4ull : 0, 4, false},
                           {"ids", ids, slots, 4, false},
                           {"weights", weights, slots, 4, false},
                           {"d_weights", d_weights, slots, 4, false},
                           {"d_logits", d_logits, d_bytes, size, true}};
    st = check_operands(fn, ops, 6);
    if (st != GBMM_OK) return st;
    if (!resolve_kernel(fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    MoeRouteParams p{};
    p.logits = logits;
    p.bias = select_bias;
    p.ids = const_cast<uint32_t *>(ids);
    p.weights = const_cast<float *>(weights);
    p.d_weights = d_weights;
    p.d_logits = d_logits;
    p.ld_logits = ld_logits;
    p.ld_d_logits = ld_d_logits;
    p.m = m;
    p.n_experts = n_experts;
    p.top_k = top_k;
    p.selected = !all;
    return finish_launch(launch_moe_route_backward(dt, p, cuda_stream(stream)), fn, cuda_stream(stream));
}

gbmm_status gbmm_moe_sort_scratch_bytes(uint32_t m, uint32_t top_k, uint32_t n_experts, uint64_t *bytes) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_moe_sort_scratch_bytes";
    gbmm_status st = check_slots(fn, m, top_k, n_experts);
    if (st != GBMM_OK) return st;
    if (bytes == nullptr) return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: null output", fn);
    *bytes = moe_sort_scratch_words(static_cast<uint64_t>(m) * top_k, n_experts) * 4;
    return GBMM_OK;
}

gbmm_status gbmm_moe_sort(uint32_t m, uint32_t top_k, uint32_t n_experts, const uint32_t *ids, uint32_t *offsets,
                          uint32_t *order, uint32_t *position, void *scratch, uint64_t scratch_bytes,
                          gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_moe_sort";
    gbmm_status st = check_slots(fn, m, top_k, n_experts);
    if (st != GBMM_OK) return st;
    const uint64_t rows = static_cast<uint64_t>(m) * top_k;
    const uint64_t need = moe_sort_scratch_words(rows, n_experts) * 4;
    if (scratch_bytes < need || (need != 0 && scratch == nullptr))
        return fail(GBMM_ERR_SCRATCH, "%s: requires %llu bytes of scratch, got %llu", fn, (unsigned long long)need,
                    (unsigned long long)(scratch ? scratch_bytes : 0));
    const Operand ops[] = {{"ids", ids, rows * 4, 4, false},
                           {"offsets", offsets, (n_experts + 1ull) * 4, 4, true},
                           {"order", order, rows * 4, 4, true},
                           {"position", position, rows * 4, 4, true},
                           {"scratch", scratch, need, 4, true}};
    st = check_operands(fn, ops, 5);
    if (st != GBMM_OK) return st;
    if (!resolve_kernel(fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    MoeSortParams p{};
    p.ids = ids;
    p.offsets = offsets;
    p.order = order;
    p.position = position;
    p.scratch = static_cast<uint32_t *>(scratch);
    p.rows = static_cast<uint32_t>(rows);
    p.n_experts = n_experts;
    const int launches = moe_sort_launches(rows);
    // whatever can fail ahead of the last launch does so ahead of the first
    if (launches > 1 && !resolve_kernel("gbmm_moe_sort_place")) return GBMM_ERR_KERNEL_UNAVAILABLE;
    const cudaError_t prepared = prepare_moe_sort(rows);
    if (prepared != cudaSuccess) return finish_launch(prepared, fn, cuda_stream(stream));
    for (int step = 0; step < launches; ++step) {
        st = finish_launch(launch_moe_sort(step, p, cuda_stream(stream)), fn, cuda_stream(stream));
        if (st != GBMM_OK) return st;
    }
    return GBMM_OK;
}

gbmm_status gbmm_moe_dispatch(gbmm_dtype dt, uint32_t m, uint32_t top_k, uint32_t n_experts, int64_t n, const void *x,
                              int64_t ldx, const uint32_t *position, const uint32_t *offsets, void *xs, int64_t ldxs,
                              gbmm_stream stream) {
    record_error(GBMM_OK, "");
    RowsCall c{"gbmm_moe_dispatch", dt, m, top_k, n_experts, n, "x", "xs", nullptr};
    c.tok = x;
    c.ld_tok = ldx;
    c.row = xs;
    c.ld_row = ldxs;
    c.row_output = true;
    c.position = position;
    c.offsets = offsets;
    bool empty;
    gbmm_status st = check_rows(c, &empty);
    if (st != GBMM_OK || empty) return st;
    if (!resolve_kernel(c.fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    MoeRowsParams p = rows_params(c);
    p.tok_in = x;
    p.ld_tok_in = ldx;
    p.row_out = xs;
    p.ld_row_out = ldxs;
    return finish_launch(launch_moe_dispatch(dt, p, cuda_stream(stream)), c.fn, cuda_stream(stream));
}

gbmm_status gbmm_moe_dispatch_backward(gbmm_dtype dt, uint32_t m, uint32_t top_k, uint32_t n_experts, int64_t n,
                                       const void *d_xs, int64_t ld_dxs, const uint32_t *position,
                                       const uint32_t *offsets, void *d_x, int64_t ld_dx, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    RowsCall c{"gbmm_moe_dispatch_backward", dt, m, top_k, n_experts, n, "d_x", "d_xs", nullptr};
    c.tok = d_x;
    c.ld_tok = ld_dx;
    c.tok_output = true;
    c.row = d_xs;
    c.ld_row = ld_dxs;
    c.position = position;
    c.offsets = offsets;
    bool empty;
    gbmm_status st = check_rows(c, &empty);
    if (st != GBMM_OK || empty) return st;
    if (!resolve_kernel(c.fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    MoeRowsParams p = rows_params(c);
    p.tok_out = d_x;
    p.ld_tok_out = ld_dx;
    p.row_in = d_xs;
    p.ld_row_in = ld_dxs;
    return finish_launch(launch_moe_combine(dt, p, cuda_stream(stream)), c.fn, cuda_stream(stream));
}

gbmm_status gbmm_moe_combine(gbmm_dtype dt, uint32_t m, uint32_t top_k, uint32_t n_experts, int64_t n, const void *ys,
                             int64_t ldys, const float *weights, const uint32_t *position, const uint32_t *offsets,
                             void *y, int64_t ldy, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    RowsCall c{"gbmm_moe_combine", dt, m, top_k, n_experts, n, "y", "ys", nullptr};
    c.tok = y;
    c.ld_tok = ldy;
    c.tok_output = true;
    c.row = ys;
    c.ld_row = ldys;
    c.has_weights = true;
    c.weights = weights;
    c.position = position;
    c.offsets = offsets;
    bool empty;
    gbmm_status st = check_rows(c, &empty);
    if (st != GBMM_OK || empty) return st;
    if (!resolve_kernel(c.fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    MoeRowsParams p = rows_params(c);
    p.tok_out = y;
    p.ld_tok_out = ldy;
    p.row_in = ys;
    p.ld_row_in = ldys;
    return finish_launch(launch_moe_combine(dt, p, cuda_stream(stream)), c.fn, cuda_stream(stream));
}

gbmm_status gbmm_moe_combine_backward(gbmm_dtype dt, uint32_t m, uint32_t top_k, uint32_t n_experts, int64_t n,
                                      const void *ys, int64_t ldys, const float *weights, const uint32_t *position,
                                      const uint32_t *offsets, const void *d_y, int64_t ld_dy, void *d_ys,
                                      int64_t ld_dys, float *d_weights, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    RowsCall c{"gbmm_moe_combine_backward", dt, m, top_k, n_experts, n, "d_y", "ys", "d_ys"};
    c.tok = d_y;
    c.ld_tok = ld_dy;
    c.row = ys;
    c.ld_row = ldys;
    c.row2 = d_ys;
    c.ld_row2 = ld_dys;
    c.has_weights = c.has_d_weights = true;
    c.weights = weights;
    c.d_weights = d_weights;
    c.position = position;
    c.offsets = offsets;
    bool empty;
    gbmm_status st = check_rows(c, &empty);
    if (st != GBMM_OK || empty) return st;
    if (!resolve_kernel(c.fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    MoeRowsParams p = rows_params(c);
    p.tok_in = d_y;
    p.ld_tok_in = ld_dy;
    p.row_in = ys;
    p.ld_row_in = ldys;
    p.row_out = d_ys;
    p.ld_row_out = ld_dys;
    p.d_weights = d_weights;
    return finish_launch(launch_moe_combine_backward(dt, p, cuda_stream(stream)), c.fn, cuda_stream(stream));
}

gbmm_status gbmm_gemv_q4(gbmm_dtype dt, uint32_t m, int64_t n, int64_t k, uint32_t group, const void *q,
                         int64_t ldq_bytes, const void *scales, gbmm_dtype scale_dt, const uint8_t *zeros,
                         const void *x, int64_t ldx, void *y, int64_t ldy, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_gemv_q4";
    Q4Params p{};
    uint64_t q_bytes;
    gbmm_status st = check_q4(fn, dt, n, k, group, ldq_bytes, scale_dt, &p, &q_bytes);
    if (st != GBMM_OK) return st;
    if (ldx < k || ldy < n || m > INT32_MAX)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: ldx %lld < k, ldy %lld < n, or m %u >= 2^31", fn, (long long)ldx,
                    (long long)ldy, m);
    if (m == 0 || n == 0) return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt)), ssize = static_cast<uint32_t>(dtype_size(scale_dt));
    uint64_t x_bytes, y_bytes;
    if (!span(m, k, ldx, size, &x_bytes) || !span(m, n, ldy, size, &y_bytes))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const uint64_t cells = static_cast<uint64_t>(n) * static_cast<uint64_t>(p.groups);
    const Operand ops[] = {{"q", q, q_bytes, 1, false},
                           {"scales", scales, cells * ssize, ssize, false},
                           {"zeros", zeros, zeros ? cells : 0, 1, false},
                           {"x", x, x_bytes, size, false},
                           {"y", y, y_bytes, size, true}};
    st = check_operands(fn, ops, 5);
    if (st != GBMM_OK) return st;
    p.q = static_cast<const uint8_t *>(q);
    p.scales = scales;
    p.zeros = zeros;
    p.x = x;
    p.out = y;
    p.ldx = ldx;
    p.ldo = ldy;
    p.rows = m;
    p.top_k = 1;
    p.n_experts = 1;
    return launch_q4(fn, dt, p, cuda_stream(stream));
}

gbmm_status gbmm_matmul_id_q4(gbmm_dtype dt, uint32_t m, int64_t n, int64_t k, uint32_t top_k, uint32_t n_experts,
                              uint32_t input_layout, uint32_t group, const void *q, int64_t ldq_bytes,
                              int64_t expert_stride_bytes, const void *scales, gbmm_dtype scale_dt,
                              const uint8_t *zeros, const void *x, const uint32_t *ids, void *out,
                              gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_matmul_id_q4";
    Q4Params p{};
    uint64_t matrix_bytes;
    gbmm_status st = check_q4(fn, dt, n, k, group, ldq_bytes, scale_dt, &p, &matrix_bytes);
    if (st != GBMM_OK) return st;
    st = check_slots(fn, m, top_k, n_experts);
    if (st != GBMM_OK) return st;
    if (input_layout > GBMM_INPUT_SLOTTED)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: unknown input layout %u", fn, input_layout);
    if (expert_stride_bytes < 0 || static_cast<uint64_t>(expert_stride_bytes) < matrix_bytes)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: expert stride %lld is smaller than one %llu-byte matrix", fn,
                    (long long)expert_stride_bytes, (unsigned long long)matrix_bytes);
    if (m == 0 || n == 0) return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt)), ssize = static_cast<uint32_t>(dtype_size(scale_dt));
    const uint64_t rows = static_cast<uint64_t>(m) * top_k;
    const uint64_t x_rows = input_layout == GBMM_INPUT_SHARED_PER_TOKEN ? m : rows;
    uint64_t q_bytes, x_bytes, out_bytes, cells;
    if (!span(n_experts, static_cast<int64_t>(matrix_bytes), expert_stride_bytes, 1, &q_bytes) ||
        !span(static_cast<uint64_t>(n_experts) * n, p.groups, p.groups, ssize, &cells) ||
        !span(x_rows, k, k, size, &x_bytes) || !span(rows, n, n, size, &out_bytes))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const Operand ops[] = {{"q", q, q_bytes, 1, false},
                           {"scales", scales, cells, ssize, false},
                           {"zeros", zeros, zeros ? cells / ssize : 0, 1, false},
                           {"x", x, x_bytes, size, false},
                           {"expert IDs", ids, rows * 4, 4, false},
                           {"output", out, out_bytes, size, true}};
    st = check_operands(fn, ops, 6);
    if (st != GBMM_OK) return st;
    p.q = static_cast<const uint8_t *>(q);
    p.expert_stride = expert_stride_bytes;
    p.scales = scales;
    p.zeros = zeros;
    p.x = x;
    p.out = out;
    p.ids = ids;
    p.ldx = input_layout == GBMM_INPUT_SHARED_PER_TOKEN ? k : k * static_cast<int64_t>(top_k);
    p.x_slot_stride = input_layout == GBMM_INPUT_SHARED_PER_TOKEN ? 0 : k;
    p.ldo = n;
    p.rows = static_cast<uint32_t>(rows);
    p.top_k = top_k;
    p.n_experts = n_experts;
    return launch_q4(fn, dt, p, cuda_stream(stream));
}

}  // extern "C"
