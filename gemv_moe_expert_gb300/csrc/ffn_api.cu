// ffn_api.cu -- the extern "C" entry points of the gated projection
// (gbmm_gated*) and of the 8-bit integer product (gbmm_quantize_i8,
// gbmm_gemm_i8): argument checks, all of them before the first launch, then
// the choice of kernels.
#include "api_checks.h"
#include "kernel_params.h"

using namespace gbmm;

namespace {

constexpr int64_t kAlign = 256;  // of each part of a scratch buffer

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

bool in_range(int64_t v) { return v >= 0 && v <= INT32_MAX; }

// The parts that a call takes from its scratch, one behind the other, each on a multiple of
// kAlign bytes from a base that is rounded up to one.
struct Parts {
    uint64_t bytes = kAlign;
    bool ok = true;  // false: more bytes than an int64 counts
    uint64_t add(int64_t rows, int64_t ld, int size) {
        const uint64_t at = bytes;
        const unsigned __int128 more = static_cast<unsigned __int128>(rows) * static_cast<uint64_t>(ld) * size;
        ok = ok && more < (1ull << 62) && bytes < (1ull << 62);
        if (ok) bytes += static_cast<uint64_t>(round_up(static_cast<int64_t>(more), kAlign));
        return at;
    }
    uint64_t needed() const { return bytes > kAlign ? bytes : 0; }
    static char *base(void *scratch) {
        return reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(scratch) + kAlign - 1) / kAlign * kAlign) - kAlign;
    }
};

gbmm_status too_large(const char *fn) { return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: scratch extent overflows", fn); }

Operand matrix(const char *label, const void *p, uint64_t bytes, int64_t cols, int64_t ld, uint32_t size, bool output) {
    return {label, p, bytes, size, output, static_cast<uint64_t>(cols) * size, static_cast<uint64_t>(ld) * size};
}

bool rows16(const void *p, int64_t ld_bytes) { return rows_on(p, ld_bytes, 16); }
// Few rows run as dot products, a warp for each column or two; more run as tiles.
constexpr int64_t kDotRows = 8;

// A 16-bit matrix as TMA reads it: in place (to null), or laid out again in a part of the scratch.
struct Laid {
    const void *from;
    void *to;
    int64_t rows, cols, from_ld, ld;
    const void *p() const { return to != nullptr ? to : from; }
};
Laid lay(const void *p, int64_t rows, int64_t cols, int64_t ld, void *scratch, Parts *parts) {
    Laid l{p, nullptr, rows, cols, ld, ld};
    if (rows16(p, ld * 2)) return l;
    l.ld = round_up(cols, 8);
    l.to = Parts::base(scratch) + parts->add(rows, l.ld, 2);
    return l;
}
// x and both weights, of the same columns, in one launch.
gbmm_status lay_again(const char *fn, const Laid &x, const Laid (&w)[2], cudaStream_t s) {
    const Laid *const all[3] = {&x, &w[0], &w[1]};
    RepackParams r[3];
    bool any = false;
    for (int i = 0; i < 3; ++i) {
        const Laid &l = *all[i];
        const bool laid = l.to != nullptr;
        r[i] = {l.from, l.to, laid ? l.rows : 0, l.cols, l.from_ld, round_up(l.cols, 8), 2};
        any = any || (laid && l.rows > 0);
    }
    return any ? finish_launch(launch_repack16(r, s), fn, s) : GBMM_OK;
}

// what the tensor-core products share
bool pair_params(PairTcParams *p, PairTcMaps *maps, int dt, void *c, int64_t ldc, int64_t m, int64_t n, int64_t k) {
    *p = PairTcParams{};
    p->c = c;
    p->ldc = ldc;
    p->m = static_cast<int32_t>(m);
    p->n = static_cast<int32_t>(n);
    p->k = static_cast<int32_t>(k);
    p->c_tma = encode_store32(&maps->out[0], dt, c, n, m, ldc);
    p->err = device_error_word();
    p->wait_limit_ns = kWaitLimitNs;
    return p->err != nullptr;
}

// whether m rows run as dot products: at most kDotRows, and rows beyond the first times weights up to `most`
bool few_rows(int64_t m, int64_t n, int64_t k, int64_t most) {
    return m <= kDotRows && (k == 0 || (m - 1) * n <= most / k);
}

// 16-bit rows go to the tensor cores as soon as the dot products, 0.04 us for each row and MB of weights beyond the first
// row, cost more than that way's additional 5 us (11008 x 4096: 26.9 us for one row, 35, 48 and 81 for 2, 4 and 8 against
// 31 to 32; 1408 x 2048: 3 to 4.5 us against 6.5); rows that start anywhere once they pay for being laid out again, too
// (4096 x 4096: 18, 24, 49 and 111 us for 1, 2, 4 and 8 rows against 37).
bool gated_dot(int64_t m, int64_t n, int64_t k, bool aligned) {
    return few_rows(m, n, k, aligned ? 32LL << 20 : 48LL << 20);
}

void few_params(FewTcParams *p, void *c, int64_t ldc, int64_t m, int64_t n, int64_t k) {
    p->c = c;
    p->ldc = ldc;
    p->m = static_cast<int32_t>(m);
    p->n = static_cast<int32_t>(n);
    p->k = static_cast<int32_t>(k);
    p->err = device_error_word();
    p->wait_limit_ns = kWaitLimitNs;
}

// How an 8-bit product runs: dot products of bytes; bytes that become f16 inside the kernel, those of a as f16 from
// the scratch once there are many tokens; or both operands as f16 in the scratch.  What is laid out again there: 0
// nothing, 1 bytes (rows that TMA cannot read), 2 f16.
struct I8Plan {
    enum { kDot, kFew, kTiles } route;
    int a_size, b_size;
};
I8Plan i8_plan(int64_t m, int64_t n, int64_t k, bool a_aligned, bool b_aligned) {
    // Dot products cost 0.06 us for each row and MB of weights beyond the first row (0.3 where rows start anywhere), the
    // tensor cores' way about 5 us more than reading the weights (and writing and reading them again): 11008 x 4096
    // 9.1, 12.8, 19 and 30 us for 1, 2, 4 and 8 rows against 15; 4096 x 4096 in odd rows 6.7 and 43 for 1 and 8 against 15.
    const bool dot = few_rows(m, n, k, a_aligned && b_aligned ? 85LL << 20 : 24LL << 20);
    if (dot || n == 0 || k == 0) return {I8Plan::kDot, 0, 0};
    if (!few_tc_takes(true, m, n, k)) return {I8Plan::kTiles, 2, 2};
    return {I8Plan::kFew, few_tc_half_tokens(m) ? 2 : a_aligned ? 0 : 1, b_aligned ? 0 : 1};
}

gbmm_status check_gated(const char *fn, gbmm_dtype dt, uint32_t activation, int64_t m, int64_t n, int64_t k) {
    if (!known_dtype(dt))
        return fail(GBMM_ERR_UNSUPPORTED_DTYPE, "%s: dtype %d is not f32, f16 or bf16", fn, (int)dt);
    if (activation > GBMM_GATE_RELU)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: unknown activation %u", fn, activation);
    if (!in_range(m) || !in_range(n) || !in_range(k))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: m, n and k must lie in [0, 2^31)", fn);
    return GBMM_OK;
}

}  // namespace

extern "C" {

gbmm_status gbmm_gated_scratch_bytes(gbmm_dtype dt, int64_t m, int64_t n, int64_t k, int aligned, uint64_t *bytes) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_gated_scratch_bytes";
    const gbmm_status st = check_gated(fn, dt, 0, m, n, k);
    if (st != GBMM_OK) return st;
    if (bytes == nullptr) return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: bytes is null", fn);
    *bytes = 0;
    if (dt == GBMM_F32 || aligned || gated_dot(m, n, k, false) || m == 0 || n == 0 || k == 0) return GBMM_OK;
    Parts parts;
    parts.add(m, round_up(k, 8), 2);
    parts.add(n, round_up(k, 8), 2);
    parts.add(n, round_up(k, 8), 2);
    if (!parts.ok) return too_large(fn);
    *bytes = parts.needed();
    return GBMM_OK;
}

gbmm_status gbmm_gated(gbmm_dtype dt, uint32_t activation, int64_t m, int64_t n, int64_t k, const void *x, int64_t ldx,
                       const void *w_gate, const void *w_up, int64_t ldw, void *h, int64_t ldh, void *gate, void *up,
                       int64_t ld_saved, void *scratch, uint64_t scratch_bytes, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_gated";
    gbmm_status st = check_gated(fn, dt, activation, m, n, k);
    if (st != GBMM_OK) return st;
    if ((gate == nullptr) != (up == nullptr))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: gate and up come together or not at all", fn);
    if (ldx < k || ldw < k || ldh < n || (gate != nullptr && ld_saved < n))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: a leading dimension is smaller than its row", fn);
    if (m == 0 || n == 0) return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt));
    uint64_t xb, wb, hb, sb = 0;
    if (!span(m, k, ldx, size, &xb) || !span(n, k, ldw, size, &wb) || !span(m, n, ldh, size, &hb) ||
        (gate != nullptr && !span(m, n, ld_saved, size, &sb)))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const Operand ops[] = {matrix("x", x, xb, k, ldx, size, false),       matrix("w_gate", w_gate, wb, k, ldw, size, false),
                           matrix("w_up", w_up, wb, k, ldw, size, false), matrix("h", h, hb, n, ldh, size, true),
                           matrix("gate", gate, sb, n, ld_saved, size, true), matrix("up", up, sb, n, ld_saved, size, true),
                           {"scratch", scratch, scratch ? scratch_bytes : 0, 1, true}};
    st = check_operands(fn, ops, 7);
    if (st != GBMM_OK) return st;
    const bool aligned = rows16(x, ldx * 2) && rows16(w_gate, ldw * 2) && rows16(w_up, ldw * 2);
    const bool dot = gated_dot(m, n, k, aligned) || (m <= kDotRows && !aligned && scratch == nullptr);
    const bool tiles16 = dt != GBMM_F32 && !dot && k > 0;
    Parts parts;
    Laid lx{}, lw[2] = {};
    if (tiles16) {
        lx = lay(x, m, k, ldx, scratch, &parts);
        lw[0] = lay(w_gate, n, k, ldw, scratch, &parts);
        lw[1] = lay(w_up, n, k, ldw, scratch, &parts);
    }
    const uint64_t need = parts.needed();
    if (!parts.ok) return too_large(fn);
    if (need > 0 && scratch != nullptr && scratch_bytes < need)
        return fail(GBMM_ERR_SCRATCH, "%s: needs %llu bytes of scratch for this layout (got %llu)", fn,
                    (unsigned long long)need, (unsigned long long)scratch_bytes);
    if (!resolve_kernel(fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    cudaStream_t s = cuda_stream(stream);
    if (tiles16 && (need == 0 || scratch != nullptr)) {
        const bool few = few_tc_takes(false, m, n, k);
        FewTcMaps few_maps{};
        FewTcParams fp{};
        PairTcMaps maps{};
        PairTcParams q{};
        uint32_t tokens = 0;
        bool ok;
        if (few) {
            few_params(&fp, h, ldh, m, n, k);
            tokens = static_cast<uint32_t>(few_tc_plan(false, m, n, k, device_sm_count(), &fp));
            const uint32_t rows = static_cast<uint32_t>(few_tc_rows(false));
            ok = fp.err != nullptr && encode_matrix16(&few_maps.x[0], dt, lx.p(), k, m, lx.ld, tokens) &&
                 encode_matrix16(&few_maps.w[0], dt, lw[0].p(), k, n, lw[0].ld, rows) &&
                 encode_matrix16(&few_maps.w[1], dt, lw[1].p(), k, n, lw[1].ld, rows);
            fp.saved[0] = gate;
            fp.saved[1] = up;
            fp.ld_saved = ld_saved;
            fp.act = static_cast<int32_t>(activation);
        } else {
            const uint32_t rows = static_cast<uint32_t>(pair_tc_rows());
            ok = pair_params(&q, &maps, dt, h, ldh, m, n, k) && encode_matrix16(&maps.a[0], dt, lx.p(), k, m, lx.ld, rows) &&
                 encode_matrix16(&maps.b[0], dt, lw[0].p(), k, n, lw[0].ld, rows) &&
                 encode_matrix16(&maps.b[1], dt, lw[1].p(), k, n, lw[1].ld, rows);
            maps.a[1] = maps.a[0];
            q.saved[0] = gate;
            q.saved[1] = up;
            q.ld_saved = ld_saved;
            q.saved_tma = gate != nullptr && encode_store32(&maps.out[1], dt, gate, n, m, ld_saved) &&
                          encode_store32(&maps.out[2], dt, up, n, m, ld_saved);
            q.act = static_cast<int32_t>(activation);
        }
        if (!ok) return fail(GBMM_ERR_CUDA, "%s: tensor maps or the device error word are unavailable", fn);
        st = lay_again(fn, lx, lw, s);
        if (st != GBMM_OK) return st;
        return finish_launch(few ? launch_gated_few(dt, static_cast<int>(tokens), few_maps, fp, s)
                                 : launch_gated_tc(dt, maps, q, device_sm_count(), s),
                             fn, s);
    }
    GatedParams p{};
    p.x = x;
    p.w[0] = w_gate;
    p.w[1] = w_up;
    p.h = h;
    p.saved[0] = gate;
    p.saved[1] = up;
    p.m = m;
    p.n = n;
    p.k = k;
    p.ldx = ldx;
    p.ldw = ldw;
    p.ldh = ldh;
    p.ld_saved = ld_saved;
    p.act = static_cast<int32_t>(activation);
    return finish_launch(m <= kDotRows ? launch_gated_rowdot(dt, p, s) : launch_gated_simt(dt, p, s), fn, s);
}

gbmm_status gbmm_gated_backward_scratch_bytes(gbmm_dtype dt, int64_t m, int64_t n, int64_t k, int aligned,
                                              uint64_t *bytes) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_gated_backward_scratch_bytes";
    const gbmm_status st = check_gated(fn, dt, 0, m, n, k);
    if (st != GBMM_OK) return st;
    if (bytes == nullptr) return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: bytes is null", fn);
    const int size = dtype_size(dt);
    Parts parts;
    parts.add(m, round_up(n, 16 / size), size);
    parts.add(m, round_up(n, 16 / size), size);
    if (dt != GBMM_F32 && !aligned) {
        if (m > gated_few_tokens()) parts.add(m, round_up(k, 8), 2);  // few tokens' x is read as it lies
        parts.add(n, round_up(k, 8), 2);
        parts.add(n, round_up(k, 8), 2);
    }
    if (!parts.ok) return too_large(fn);
    *bytes = parts.needed();
    return GBMM_OK;
}

gbmm_status gbmm_gated_backward(gbmm_dtype dt, uint32_t activation, int64_t m, int64_t n, int64_t k, const void *x,
                                int64_t ldx, const void *w_gate, const void *w_up, int64_t ldw, const void *gate,
                                const void *up, int64_t ld_saved, const void *d_h, int64_t ld_dh, void *d_x,
                                int64_t ld_dx, void *d_w_gate, void *d_w_up, int64_t ld_dw, void *scratch,
                                uint64_t scratch_bytes, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_gated_backward";
    gbmm_status st = check_gated(fn, dt, activation, m, n, k);
    if (st != GBMM_OK) return st;
    if ((d_w_gate == nullptr) != (d_w_up == nullptr))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: d_w_gate and d_w_up come together or not at all", fn);
    const bool need_x = d_x != nullptr, need_w = d_w_gate != nullptr;
    if ((need_w && ldx < k) || (need_x && ldw < k) || ld_saved < n || ld_dh < n || (need_x && ld_dx < k) ||
        (need_w && ld_dw < k))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: a leading dimension is smaller than its row", fn);
    if (k == 0 || (!need_x && !need_w) || (m == 0 && !need_w) || (n == 0 && !need_x) || (m == 0 && n == 0))
        return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt));
    uint64_t xb, wb, sb, hb, dxb = 0, dwb = 0;
    if (!span(m, k, ldx, size, &xb) || !span(n, k, ldw, size, &wb) || !span(m, n, ld_saved, size, &sb) ||
        !span(m, n, ld_dh, size, &hb) || (need_x && !span(m, k, ld_dx, size, &dxb)) ||
        (need_w && !span(n, k, ld_dw, size, &dwb)))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const bool empty = m == 0 || n == 0;  // what is left to do is writing zeros
    // the weights' gradients of few tokens take no tiles (gated.cu)
    const bool outer_few = dt != GBMM_F32 && need_w && m <= gated_few_tokens();
    if (empty || !need_w) xb = 0;
    if (empty || !need_x) wb = 0;
    Parts parts;
    const int64_t ldd = round_up(n, 16 / static_cast<int>(size));
    const uint64_t d_at[2] = {parts.add(m, ldd, static_cast<int>(size)), parts.add(m, ldd, static_cast<int>(size))};
    Laid lx{x, nullptr, m, k, ldx, ldx}, lw[2] = {{w_gate, nullptr, n, k, ldw, ldw}, {w_up, nullptr, n, k, ldw, ldw}};
    if (dt != GBMM_F32 && !empty) {
        if (need_w && !outer_few) lx = lay(x, m, k, ldx, scratch, &parts);
        if (need_x) {
            lw[0] = lay(w_gate, n, k, ldw, scratch, &parts);
            lw[1] = lay(w_up, n, k, ldw, scratch, &parts);
        }
    }
    if (!parts.ok) return too_large(fn);
    const Operand ops[] = {matrix("x", x, xb, k, ldx, size, false),
                           matrix("w_gate", w_gate, wb, k, ldw, size, false),
                           matrix("w_up", w_up, wb, k, ldw, size, false),
                           matrix("gate", gate, sb, n, ld_saved, size, false),
                           matrix("up", up, sb, n, ld_saved, size, false),
                           matrix("d_h", d_h, hb, n, ld_dh, size, false),
                           matrix("d_x", d_x, dxb, k, ld_dx, size, true),
                           matrix("d_w_gate", d_w_gate, dwb, k, ld_dw, size, true),
                           matrix("d_w_up", d_w_up, dwb, k, ld_dw, size, true),
                           {"scratch", scratch, scratch ? scratch_bytes : 0, 1, true}};
    st = check_operands(fn, ops, 10);
    if (st != GBMM_OK) return st;
    if (!empty && (scratch == nullptr || scratch_bytes < parts.bytes))
        return fail(GBMM_ERR_SCRATCH, "%s: needs %llu bytes of scratch (got %llu)", fn, (unsigned long long)parts.bytes,
                    (unsigned long long)(scratch ? scratch_bytes : 0));
    // the kernels are asked for before the first launch, so that nothing runs where one is missing
    if (!resolve_kernel(fn) || !resolve_kernel("gbmm_fill_zero")) return GBMM_ERR_KERNEL_UNAVAILABLE;
    cudaStream_t s = cuda_stream(stream);
    if (empty) {
        if (m == 0) {
            st = finish_launch(launch_fill_zero(dt, d_w_gate, 1, n, k, ld_dw, 0, s), fn, s);
            if (st == GBMM_OK) st = finish_launch(launch_fill_zero(dt, d_w_up, 1, n, k, ld_dw, 0, s), fn, s);
        } else {
            st = finish_launch(launch_fill_zero(dt, d_x, 1, m, k, ld_dx, 0, s), fn, s);
        }
        return st;
    }
    char *const base = Parts::base(scratch);
    GatedGradParams g{};
    g.gate = gate;
    g.up = up;
    g.d_h = d_h;
    for (int i = 0; i < 2; ++i) g.d[i] = base + d_at[i];
    g.m = m;
    g.n = n;
    g.ld_saved = ld_saved;
    g.ld_dh = ld_dh;
    g.ldd = ldd;
    g.act = static_cast<int32_t>(activation);
    void *const dw[2] = {d_w_gate, d_w_up};
    PairTcMaps maps{};
    PairTcParams q{};
    FewTcMaps few_maps{};
    FewTcParams fp{};
    const bool few = dt != GBMM_F32 && need_x && few_tc_takes_sum(m, n, k, need_w && !outer_few, device_sm_count());
    int tokens = 0;
    if (dt != GBMM_F32) {
        const uint32_t rows = static_cast<uint32_t>(pair_tc_rows()), box = static_cast<uint32_t>(pair_tc_block_k());
        bool ok = pair_params(&q, &maps, dt, d_x, ld_dx, m, k, n);
        if (few) {
            few_params(&fp, d_x, ld_dx, m, k, n);
            tokens = few_tc_plan_sum(m, n, k, device_sm_count(), &fp);
        }
        q.need_c = need_x && !few;
        q.need_dw = need_w && !outer_few;
        q.ld_dw = ld_dw;
        q.dw_tma = 1;
        for (int i = 0; i < 2 && ok; ++i) {
            if (few)
                ok = encode_matrix16(&few_maps.x[i], dt, g.d[i], n, m, ldd, static_cast<uint32_t>(tokens)) &&
                     encode_matrix16(&few_maps.w[i], dt, lw[i].p(), k, n, lw[i].ld, static_cast<uint32_t>(few_tc_block_k()));
            else if (need_x)
                ok = encode_matrix16(&maps.a[i], dt, g.d[i], n, m, ldd, rows) &&
                     encode_matrix16(&maps.b[i], dt, lw[i].p(), k, n, lw[i].ld, box);
            if (q.need_dw && ok) {
                ok = encode_matrix16(&maps.dw_a[i], dt, g.d[i], n, m, ldd, box) &&
                     encode_matrix16(&maps.dw_b, dt, lx.p(), k, m, lx.ld, box);
                q.dw[i] = dw[i];
                if (!encode_store32(&maps.out[1 + i], dt, dw[i], k, n, ld_dw)) q.dw_tma = 0;
            }
        }
        if (!ok) return fail(GBMM_ERR_CUDA, "%s: tensor maps or the device error word are unavailable", fn);
    }
    st = lay_again(fn, lx, lw, s);
    if (st != GBMM_OK) return st;
    if (outer_few) {
        if (!need_x) g.d[0] = g.d[1] = nullptr;
        const OuterGemmParams pw{x, {nullptr, nullptr}, {dw[0], dw[1]}, m, n, k, ldx, ldd, ld_dw};
        st = finish_launch(launch_gated_outer_few(dt, g, pw, s), fn, s);
    } else {
        st = finish_launch(launch_gated_grad(dt, g, s), fn, s);
    }
    if (st != GBMM_OK) return st;
    if (dt == GBMM_F32) {
        const SumGemmParams px{{g.d[0], g.d[1]}, {w_gate, w_up}, d_x, m, k, n, ldd, ldw, ld_dx};
        const OuterGemmParams pw{x, {g.d[0], g.d[1]}, {dw[0], dw[1]}, m, n, k, ldx, ldd, ld_dw};
        return finish_launch(launch_gated_products_simt(need_x ? &px : nullptr, need_w ? &pw : nullptr, s), fn, s);
    }
    if (few) st = finish_launch(launch_sum_few(dt, tokens, few_maps, fp, s), fn, s);
    if (st != GBMM_OK || !(q.need_c || q.need_dw)) return st;
    return finish_launch(launch_gated_products_tc(dt, maps, q, device_sm_count(), s), fn, s);
}

gbmm_status gbmm_quantize_i8(gbmm_dtype dt, int64_t m, int64_t k, const void *x, int64_t ldx, int8_t *q, int64_t ldq,
                             float *scale, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_quantize_i8";
    if (!known_dtype(dt))
        return fail(GBMM_ERR_UNSUPPORTED_DTYPE, "%s: dtype %d is not f32, f16 or bf16", fn, (int)dt);
    if (!in_range(m) || !in_range(k))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: m and k must lie in [0, 2^31)", fn);
    if (ldx < k || ldq < k)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: a leading dimension is smaller than the row length %lld", fn,
                    (long long)k);
    if (m == 0) return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt));
    uint64_t xb, qb;
    if (!span(m, k, ldx, size, &xb) || !span(m, k, ldq, 1, &qb))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const Operand ops[] = {matrix("x", x, xb, k, ldx, size, false), matrix("q", q, qb, k, ldq, 1, true),
                           {"scale", scale, static_cast<uint64_t>(m) * 4, 4, true}};
    const gbmm_status st = check_operands(fn, ops, 3);
    if (st != GBMM_OK) return st;
    if (!resolve_kernel(fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    const QuantizeParams p{x, q, scale, m, k, ldx, ldq};
    return finish_launch(launch_quantize_i8(dt, p, cuda_stream(stream)), fn, cuda_stream(stream));
}

gbmm_status gbmm_gemm_i8_scratch_bytes(int64_t m, int64_t n, int64_t k, int aligned, uint64_t *bytes) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_gemm_i8_scratch_bytes";
    if (!in_range(m) || !in_range(n) || k < 0 || k > GBMM_I8_MAX_K)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: m and n must lie in [0, 2^31), k in [0, %d]", fn, GBMM_I8_MAX_K);
    if (bytes == nullptr) return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: bytes is null", fn);
    *bytes = 0;
    const I8Plan plan = i8_plan(m, n, k, aligned != 0, aligned != 0);
    if (plan.a_size == 0 && plan.b_size == 0) return GBMM_OK;
    Parts parts;
    if (plan.a_size) parts.add(m, round_up(k, 16), plan.a_size);
    if (plan.b_size) parts.add(n, round_up(k, 16), plan.b_size);
    if (!parts.ok) return too_large(fn);
    *bytes = parts.needed();
    return GBMM_OK;
}

gbmm_status gbmm_gemm_i8(gbmm_dtype dt, int64_t m, int64_t n, int64_t k, const int8_t *a, int64_t lda,
                         const float *scale_a, const int8_t *b, int64_t ldb, const float *scale_b, void *c, int64_t ldc,
                         void *scratch, uint64_t scratch_bytes, gbmm_stream stream) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_gemm_i8";
    if (!known_dtype(dt))
        return fail(GBMM_ERR_UNSUPPORTED_DTYPE, "%s: dtype %d is not f32, f16 or bf16", fn, (int)dt);
    if (!in_range(m) || !in_range(n) || k < 0 || k > GBMM_I8_MAX_K)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: m and n must lie in [0, 2^31), k in [0, %d]", fn, GBMM_I8_MAX_K);
    if (lda < k || ldb < k || ldc < n)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: a leading dimension is smaller than its row", fn);
    if (m == 0 || n == 0) return GBMM_OK;
    const uint32_t size = static_cast<uint32_t>(dtype_size(dt));
    uint64_t ab, bb, cb;
    if (!span(m, k, lda, 1, &ab) || !span(n, k, ldb, 1, &bb) || !span(m, n, ldc, size, &cb))
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: operand extent overflows", fn);
    const I8Plan plan = i8_plan(m, n, k, rows16(a, lda), rows16(b, ldb));
    const int64_t lda2 = plan.a_size ? round_up(k, 16) : lda, ldb2 = plan.b_size ? round_up(k, 16) : ldb;
    Parts parts;
    const uint64_t a_at = plan.a_size ? parts.add(m, lda2, plan.a_size) : 0, b_at = plan.b_size ? parts.add(n, ldb2, plan.b_size) : 0;
    const uint64_t need = parts.needed();
    if (!parts.ok) return too_large(fn);
    const Operand ops[] = {matrix("a", a, ab, k, lda, 1, false),
                           {"scale_a", scale_a, scale_a ? static_cast<uint64_t>(m) * 4 : 0, 4, false},
                           matrix("b", b, bb, k, ldb, 1, false),
                           {"scale_b", scale_b, scale_b ? static_cast<uint64_t>(n) * 4 : 0, 4, false},
                           matrix("c", c, cb, n, ldc, size, true),
                           {"scratch", scratch, scratch ? scratch_bytes : 0, 1, true}};
    gbmm_status st = check_operands(fn, ops, 6);
    if (st != GBMM_OK) return st;
    if (need > 0 && (scratch == nullptr || scratch_bytes < need))
        return fail(GBMM_ERR_SCRATCH, "%s: needs %llu bytes of scratch (got %llu)", fn, (unsigned long long)need,
                    (unsigned long long)(scratch ? scratch_bytes : 0));
    if (!resolve_kernel(fn)) return GBMM_ERR_KERNEL_UNAVAILABLE;
    cudaStream_t s = cuda_stream(stream);
    if (plan.route == I8Plan::kDot) {
        const GemmI8Params p{a, b, scale_a, scale_b, c, m, n, k, lda, ldb, ldc};
        return finish_launch(launch_gemm_i8_dot(dt, p, s), fn, s);
    }
    const void *const a2 = plan.a_size ? Parts::base(scratch) + a_at : static_cast<const void *>(a);
    const void *const b2 = plan.b_size ? Parts::base(scratch) + b_at : static_cast<const void *>(b);
    FewTcMaps few{};
    FewTcParams fp{};
    PairTcMaps maps{};
    PairTcParams q{};
    uint32_t tokens = 0;
    bool ok;
    if (plan.route == I8Plan::kFew) {
        few_params(&fp, c, ldc, m, n, k);
        fp.scale_a = scale_a;
        fp.scale_b = scale_b;
        tokens = static_cast<uint32_t>(few_tc_plan(true, m, n, k, device_sm_count(), &fp));
        ok = fp.err != nullptr && encode_matrix8(&few.w[0], b2, k, n, ldb2, static_cast<uint32_t>(few_tc_rows(true))) &&
             (plan.a_size == 2 ? encode_matrix16(&few.x[0], GBMM_F16, a2, k, m, lda2, tokens)
                               : encode_matrix8(&few.x[0], a2, k, m, lda2, tokens));
        few.w[1] = few.w[0];
    } else {
        const uint32_t rows = static_cast<uint32_t>(pair_tc_rows());
        ok = pair_params(&q, &maps, dt, c, ldc, m, n, k) && encode_matrix16(&maps.a[0], GBMM_F16, a2, k, m, lda2, rows) &&
             encode_matrix16(&maps.b[0], GBMM_F16, b2, k, n, ldb2, rows);
        maps.a[1] = maps.a[0];
        maps.b[1] = maps.b[0];
        q.scale_a = scale_a;
        q.scale_b = scale_b;
    }
    if (!ok) return fail(GBMM_ERR_CUDA, "%s: tensor maps or the device error word are unavailable", fn);
    if (need > 0) {
        const RepackParams ra{a, const_cast<void *>(a2), plan.a_size ? m : 0, k, lda, lda2, plan.a_size};
        const RepackParams rb{b, const_cast<void *>(b2), plan.b_size ? n : 0, k, ldb, ldb2, plan.b_size};
        st = finish_launch(launch_lay_out_codes(ra, rb, s), fn, s);
        if (st != GBMM_OK) return st;
    }
    return finish_launch(plan.route == I8Plan::kFew ? launch_gemm_i8_few(dt, static_cast<int>(tokens), few, fp, s)
                                                    : launch_gemm_i8_tc(dt, maps, q, device_sm_count(), s),
                         fn, s);
}

gbmm_status gbmm_test_few_plan(int form, int64_t m, int64_t n, int64_t k, int32_t sms, int32_t plan[4]) {
    record_error(GBMM_OK, "");
    const char *fn = "gbmm_test_few_plan";
    if (form < 0 || form > 2 || m < 1 || n < 1 || k < 1 || !in_range(m) || !in_range(n) || !in_range(k) || sms < 1 ||
        plan == nullptr)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: unknown form, size out of range, or plan is null", fn);
    for (int i = 0; i < 4; ++i) plan[i] = 0;
    const bool codes = form == 1;
    if (codes ? k > GBMM_I8_MAX_K || i8_plan(m, n, k, true, true).route != I8Plan::kFew
              : form == 0 && (gated_dot(m, n, k, true) || !few_tc_takes(false, m, n, k)))
        return GBMM_OK;
    FewTcParams p{};
    plan[0] = form == 2 ? few_tc_plan_sum(m, n, k, sms, &p) : few_tc_plan(codes, m, n, k, sms, &p);
    plan[1] = p.ksplit;
    plan[2] = static_cast<int32_t>(p.tmem_cols);
    plan[3] = few_tc_ctas_per_sm(codes, plan[0]);
    return GBMM_OK;
}

gbmm_status gbmm_test_gradient_plan(int64_t m, int64_t n, int64_t k, int need_x, int need_w, int32_t sms,
                                    int32_t plan[4]) {
    record_error(GBMM_OK, "");
    if (m < 1 || n < 1 || k < 1 || !in_range(m) || !in_range(n) || !in_range(k) || (!need_x && !need_w) || sms < 1 ||
        plan == nullptr)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "gbmm_test_gradient_plan: nothing asked for, size out of range, or plan is null");
    gated_products_simt_plan(m, n, k, need_x != 0, need_w != 0, sms, plan);
    return GBMM_OK;
}

gbmm_status gbmm_test_gated_plan(int64_t m, int64_t n, int64_t k, int32_t sms, int32_t plan[2]) {
    record_error(GBMM_OK, "");
    if (m <= kDotRows || n < 1 || k < 0 || !in_range(m) || !in_range(n) || !in_range(k) || sms < 1 || plan == nullptr)
        return fail(GBMM_ERR_INVALID_ARGUMENT, "gbmm_test_gated_plan: size out of range, or plan is null");
    gated_simt_plan(m, n, k, sms, plan);
    return GBMM_OK;
}

}  // extern "C"
