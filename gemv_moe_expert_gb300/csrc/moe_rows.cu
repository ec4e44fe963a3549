// moe_rows.cu -- rows of a mixture-of-experts layer into expert order and back:
// dispatch (copy), combine (weighted sum over a token's slots; with weights of 1
// the gradient of the dispatch) and the gradient of combine.
//
// All three are bound by HBM: a row of x or y and top_k rows of xs or ys per
// token, a few operations an element.  Every kernel works in token order, so a
// token's row is read or written once and its top_k rows in expert order, each
// a contiguous run of n elements, are addressed through position; working in
// expert order would read the token's row once per slot.  Rows whose position is
// at or past *valid have no expert.  Measured on 4096 tokens x 8 slots of 4096
// elements (us, and GB/s; a plain copy reaches 6790): dispatch f32 100 (6030), bf16 50;
// combine 95 (6350), 51; the gradient of dispatch 94 (6400), 50.5, of combine 176 (6470), 92;
// 4 tokens x 8 slots of 2048 5.1 to 6.4 each, a launch and two trips to memory.
//
// A block is a grid of tx x ty threads: tx along the row (one access of VB bytes
// a thread and step), ty tokens.  Slots are taken in batches of B, all of a batch's
// loads issued before the first is used.  The blocks of combine and of its gradient stay
// and walk over the tokens: the places of the next token's slots are loaded while the
// current token's rows are in flight.  A dispatch has a block for every ty tokens.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 256;
constexpr int B = 4;
// Blocks an SM (the registers they may use follow).  4-byte elements need fewer
// registers for the same bytes in flight.  Measured on 4096 tokens x 8 slots of
// 4096 elements: combine f32 95 us with 4 and 97 us with 5, bf16 52 and 51 us; its
// gradient f32 177 us with 3 and 190 us with 4, bf16 97 and 92 us.  Shifted rows need
// twice the registers for a piece: bf16 combine 83 us with 3 and 113 with 4; its gradient 172
// with 4, 195 with 3 and 200 with 5 (with 4 it spills 112 to 120 bytes a thread).
template <typename T, bool SHIFT> struct Resident {
    static constexpr int kDispatch = 4;
    static constexpr int kCombine = SHIFT ? 3 : sizeof(T) == 4 ? 4 : 5;
    static constexpr int kBackward = SHIFT ? 4 : sizeof(T) == 4 ? 3 : 4;
};
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kNowhere = 0xffffffffu;

template <int VB> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <typename T, int VB>
__device__ __forceinline__ typename Raw<VB>::type load_raw(const T *p) {
    return __ldg(reinterpret_cast<const typename Raw<VB>::type *>(p));
}
template <typename T, int VB>
__device__ __forceinline__ void store_raw(T *p, const typename Raw<VB>::type &r) {
    *reinterpret_cast<typename Raw<VB>::type *>(p) = r;
}

// 16 bytes at any element: the two aligned chunks that cover them, and how many bytes of
// the first come before.
struct Chunks {
    uint4 a, b;
    uint32_t off;
};
template <typename T> __device__ __forceinline__ Chunks load_chunks(const T *p) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - off);
    return Chunks{__ldg(q), __ldg(q + 1), off};
}
__device__ __forceinline__ uint4 shifted(const Chunks &c) {
    const bool two = c.off & 8u, one = c.off & 4u;
    const uint32_t bits = 8 * (c.off & 3u);
    uint32_t w[8] = {c.a.x, c.a.y, c.a.z, c.a.w, c.b.x, c.b.y, c.b.z, c.b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = two ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = one ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int V, typename R>
__device__ __forceinline__ void unpack(const R &r, float (&f)[V]) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = Elem<T>::to_f(e[j]);
}

template <typename T, int V, typename R>
__device__ __forceinline__ R pack(const float (&f)[V]) {
    R r;
    T *e = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = Elem<T>::from_f(f[j]);
    return r;
}

__device__ __forceinline__ uint32_t valid_rows(const MoeRowsParams &p) {
    const uint32_t rows = p.m * p.top_k;
    return p.valid != nullptr ? min(__ldg(p.valid), rows) : rows;
}

// Places and weights of a batch of slots of token t: slot s0 + b in lane b of the
// token's warps; kNowhere past the token's slots and past the last token, weight 0
// where there is no expert.  One load for the batch, handed out by shuffles, so
// that the rows' loads wait for one latency and not for one a slot.
struct Slots {
    uint32_t at;
    float w;
    __device__ __forceinline__ void load(const MoeRowsParams &p, uint32_t valid, uint64_t t, uint32_t s0) {
        const uint32_t s = s0 + (threadIdx.x & 31);
        at = kNowhere;
        w = 0.f;
        if (t < p.m && s < s0 + B && s < p.top_k) {
            const uint32_t r = static_cast<uint32_t>(t) * p.top_k + s;
            w = p.weights != nullptr ? __ldg(p.weights + r) : 1.f;
            at = p.position != nullptr ? __ldg(p.position + r) : r;
            if (at >= valid) w = 0.f;
        }
    }
    __device__ __forceinline__ uint32_t place(int b) const { return __shfl_sync(kFull, at, b); }
    __device__ __forceinline__ float weight(int b) const { return __shfl_sync(kFull, w, b); }
};

// V elements as loaded: with one access, or (SHIFT) as the two chunks that cover them.
template <typename R, bool SHIFT> struct Piece {
    R r;
    __device__ __forceinline__ void clear() { r = R{}; }
    template <typename T> __device__ __forceinline__ void load(const T *p) { r = load_raw<T, sizeof(R)>(p); }
    __device__ __forceinline__ R get() const { return r; }
};
template <typename R> struct Piece<R, true> {
    Chunks c;
    __device__ __forceinline__ void clear() { c = Chunks{}; }
    template <typename T> __device__ __forceinline__ void load(const T *p) { c = load_chunks<T>(p); }
    __device__ __forceinline__ R get() const { return shifted(c); }
};

// Columns of a row are dealt to threads in steps that all threads of a warp take
// together (the shuffles need the whole warp; a thread past the end idles): first
// the columns that divide into accesses of VB bytes, then the rest one by one.  The
// two are separate calls so that every access in them is one predicated instruction
// (with the choice inside the loop each load sat behind its own branch and the
// loads of a batch no longer overlapped).
//
// Rows that do not all start on multiples of 16 bytes (SHIFT) are still written 16 bytes
// at a time: every row that is written has its own first whole access, `head` elements
// in and one access further (so that what covers a piece of a row that is read never
// starts before that row), its last one ends an access before the row does, and the
// elements before and behind them are the rest.  4096 tokens x 8 slots x 4097 (in brackets
// one element an access): dispatch bf16 59 us (102), f32 104 (162); combine 83 (177), 130
// (214); its gradient 172 (285), 274 (424).

struct Columns {
    int64_t from, to, step;  // elements
};
template <int V>
__device__ __forceinline__ Columns whole_columns(const MoeRowsParams &p, bool shift) {
    return Columns{(static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V, shift ? p.n : p.n / V * V,
                   static_cast<int64_t>(gridDim.y) * blockDim.x * V};
}
template <int V>
__device__ __forceinline__ Columns rest_columns(const MoeRowsParams &p, bool shift) {
    return Columns{(shift ? 0 : p.n / V * V) + threadIdx.x,
                   blockIdx.y != 0 ? 0 : shift ? min(p.n, static_cast<int64_t>(5 * V)) : p.n,
                   static_cast<int64_t>(blockDim.x)};
}

// Element of a row, written at `row`, that column i means, and whether there is one.
struct Place {
    int64_t i;
    bool in;
};
template <typename T, int VB, bool SHIFT>
__device__ __forceinline__ Place place_of(const MoeRowsParams &p, const Columns &c, int64_t i, const T *row) {
    if (!SHIFT) return Place{i, i < c.to};
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const uint32_t past = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u;
    const int64_t first = V + (16u - past) % 16u / static_cast<uint32_t>(sizeof(T));
    if (VB == 16) return Place{first + i, first + i + 2 * V <= p.n};
    const int64_t whole = p.n - 2 * V >= first ? (p.n - 2 * V - first) / V * V + V : 0;
    return Place{i < first ? i : i + whole, i < p.n - whole};
}

template <typename T, int VB, bool SHIFT>
__device__ __forceinline__ void dispatch_columns(const MoeRowsParams &p, const Slots &slots, uint32_t valid,
                                                 const T *x, const Columns &c) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t rows = p.m * p.top_k;
    const int lane = threadIdx.x & 31;
    T *out = static_cast<T *>(p.row_out);
    for (int64_t i = c.from; i - lane * V < c.to; i += c.step) {
        if constexpr (SHIFT) {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t at = slots.place(b);
                T *row = out + static_cast<int64_t>(at) * p.ld_row_out;
                const Place to = place_of<T, VB, SHIFT>(p, c, i, row);
                if (to.in && at < rows) {
                    R v;
                    if constexpr (VB == 16)
                        v = shifted(load_chunks<T>(x + to.i));
                    else
                        v = load_raw<T, VB>(x + to.i);
                    store_raw<T, VB>(row + to.i, at < valid ? v : R{});
                }
            }
        } else {
            const bool in = i < c.to;
            R v{};
            if (in) v = load_raw<T, VB>(x + i);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t at = slots.place(b);
                if (in && at < rows)
                    store_raw<T, VB>(out + static_cast<int64_t>(at) * p.ld_row_out + i, at < valid ? v : R{});
            }
        }
    }
}

template <typename T, int VB, bool SHIFT>
__global__ void __launch_bounds__(kThreads, Resident<T, SHIFT>::kDispatch)
    moe_dispatch_kernel(const __grid_constant__ MoeRowsParams p) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    grid_dep_begin();
    const uint32_t valid = valid_rows(p);
    // One turn, as there is a block for every ty tokens (written without the loop, rows that start
    // anywhere took 5 % longer: 59.8 us for 57.0, bf16, 4096 tokens x 8 slots x 4097).
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.y;
    uint64_t t = static_cast<uint64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    Slots slots, next;
    slots.load(p, valid, t, 0);
    for (; t < p.m; t += step) {
        next.load(p, valid, t + step, 0);
        const T *x = static_cast<const T *>(p.tok_in) + static_cast<int64_t>(t) * p.ld_tok_in;
        for (uint32_t s0 = 0; s0 < p.top_k; s0 += B) {
            if (s0 != 0) slots.load(p, valid, t, s0);
            dispatch_columns<T, VB, SHIFT>(p, slots, valid, x, whole_columns<V>(p, SHIFT));
            if (V > 1) dispatch_columns<T, sizeof(T), SHIFT>(p, slots, valid, x, rest_columns<V>(p, SHIFT));
        }
        slots = next;
    }
}

// A slot without an expert adds 0 * 0.
template <typename T, int VB, bool SHIFT>
__device__ __forceinline__ void combine_columns(const MoeRowsParams &p, uint32_t t, Slots slots, uint32_t valid,
                                                const Columns &c) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const int lane = threadIdx.x & 31;
    const T *in_rows = static_cast<const T *>(p.row_in);
    T *y = static_cast<T *>(p.tok_out) + static_cast<int64_t>(t) * p.ld_tok_out;
    for (int64_t step = c.from; step - lane * V < c.to; step += c.step) {
        const auto [i, in] = place_of<T, VB, SHIFT>(p, c, step, y);
        float acc[V];
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
        for (uint32_t s0 = 0; s0 < p.top_k; s0 += B) {
            if (p.top_k > B) slots.load(p, valid, t, s0);
            Piece<R, SHIFT && VB == 16> v[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t at = slots.place(b);
                v[b].clear();
                if (in && at < valid) v[b].load(in_rows + static_cast<int64_t>(at) * p.ld_row_in + i);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const float w = slots.weight(b);
                float f[V];
                unpack<T, V>(v[b].get(), f);
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = fmaf(w, f[j], acc[j]);
            }
        }
        if (in) store_raw<T, VB>(y + i, pack<T, V, R>(acc));
    }
}

template <typename T, int VB, bool SHIFT>
__global__ void __launch_bounds__(kThreads, Resident<T, SHIFT>::kCombine)
    moe_combine_kernel(const __grid_constant__ MoeRowsParams p) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    grid_dep_begin();
    const uint32_t valid = valid_rows(p);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.y;
    uint64_t t = static_cast<uint64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    Slots slots, next;
    slots.load(p, valid, t, 0);
    for (; t < p.m; t += step) {
        next.load(p, valid, t + step, 0);
        const uint32_t token = static_cast<uint32_t>(t);
        combine_columns<T, VB, SHIFT>(p, token, slots, valid, whole_columns<V>(p, SHIFT));
        if (V > 1) combine_columns<T, sizeof(T), SHIFT>(p, token, slots, valid, rest_columns<V>(p, SHIFT));
        slots = next;
    }
}

// Sums each v[b] over the warp; lane l returns the sum of v[l / (32 / B)]: each of
// the first log2 B steps halves the values a lane carries, so 4 sums take 6
// shuffles instead of 20.
__device__ __forceinline__ float warp_sums(float (&v)[B]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int half = B / 2; half > 0; half /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = up ? v[i + half] : v[i], give = up ? v[i] : v[i + half];
            v[i] = keep + __shfl_xor_sync(kFull, give, o);
        }
    }
#pragma unroll
    for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(kFull, v[0], o);
    return v[0];
}

// one slot's part of combine_backward_columns: d_ys, and the dot product's terms
template <typename T, int V, typename R>
__device__ __forceinline__ R backward_piece(const R &y, const float (&g)[V], float w, float &dot) {
    float f[V], wg[V];
    unpack<T, V>(y, f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        dot = fmaf(g[j], f[j], dot);
        wg[j] = w * g[j];
    }
    return pack<T, V, R>(wg);
}

template <typename T, int VB, bool SHIFT>
__device__ __forceinline__ void combine_backward_columns(const MoeRowsParams &p, const Slots &slots, uint32_t valid,
                                                         const T *dy, const Columns &c, float (&dot)[B]) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t rows = p.m * p.top_k;
    const int lane = threadIdx.x & 31;
    const T *in_rows = static_cast<const T *>(p.row_in);
    T *out = static_cast<T *>(p.row_out);
    for (int64_t step = c.from; step - lane * V < c.to; step += c.step) {
        float g[V];
        if constexpr (SHIFT) {
            // each slot has its own piece of dy: two slots at once, and more blocks an SM
            constexpr int kBatch = 2;
#pragma unroll
            for (int b0 = 0; b0 < B; b0 += kBatch) {
                Piece<R, VB == 16> v[kBatch], graw[kBatch];
                Place place[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const uint32_t at = slots.place(b0 + u);
                    place[u] = place_of<T, VB, SHIFT>(p, c, step, out + static_cast<int64_t>(at) * p.ld_row_out);
                    v[u].clear();
                    graw[u].clear();
                    if (place[u].in && at < valid) {
                        v[u].load(in_rows + static_cast<int64_t>(at) * p.ld_row_in + place[u].i);
                        graw[u].load(dy + place[u].i);
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const uint32_t at = slots.place(b0 + u);
                    unpack<T, V>(graw[u].get(), g);
                    const R d = backward_piece<T, V>(v[u].get(), g, slots.weight(b0 + u), dot[b0 + u]);
                    if (place[u].in && at < rows)
                        store_raw<T, VB>(out + static_cast<int64_t>(at) * p.ld_row_out + place[u].i,
                                         at < valid ? d : R{});
                }
            }
        } else {
            const bool in = step < c.to;
            R v[B], graw{};
            if (in) graw = load_raw<T, VB>(dy + step);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t at = slots.place(b);
                v[b] = R{};
                if (in && at < valid) v[b] = load_raw<T, VB>(in_rows + static_cast<int64_t>(at) * p.ld_row_in + step);
            }
            unpack<T, V>(graw, g);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t at = slots.place(b);
                const R d = backward_piece<T, V>(v[b], g, slots.weight(b), dot[b]);
                if (in && at < rows)
                    store_raw<T, VB>(out + static_cast<int64_t>(at) * p.ld_row_out + step, at < valid ? d : R{});
            }
        }
    }
}

// The grid's y extent is 1: a block sees a token's whole row, for the dot products.
template <typename T, int VB, bool SHIFT>
__global__ void __launch_bounds__(kThreads, Resident<T, SHIFT>::kBackward)
    moe_combine_backward_kernel(const __grid_constant__ MoeRowsParams p) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    __shared__ float part[2][kThreads / 32][B];
    const int lane = threadIdx.x & 31;
    grid_dep_begin();
    const uint32_t valid = valid_rows(p);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.y;
    const int warps = blockDim.x / 32, first_warp = threadIdx.y * warps, warp = first_warp + threadIdx.x / 32;
    int turn = 0;
    uint64_t t = static_cast<uint64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    Slots slots, next;
    slots.load(p, valid, t, 0);
    // every thread of the block takes the same number of turns (they meet at barriers)
    for (uint64_t t_block = static_cast<uint64_t>(blockIdx.x) * blockDim.y; t_block < p.m; t_block += step, t += step) {
        next.load(p, valid, t + step, 0);
        const bool live = t < p.m;
        const T *dy = static_cast<const T *>(p.tok_in) + static_cast<int64_t>(live ? t : 0) * p.ld_tok_in;
        for (uint32_t s0 = 0; s0 < p.top_k; s0 += B) {
            if (s0 != 0) slots.load(p, valid, t, s0);
            float dot[B];
#pragma unroll
            for (int b = 0; b < B; ++b) dot[b] = 0.f;
            if (live) {
                combine_backward_columns<T, VB, SHIFT>(p, slots, valid, dy, whole_columns<V>(p, SHIFT), dot);
                if (V > 1)
                    combine_backward_columns<T, sizeof(T), SHIFT>(p, slots, valid, dy, rest_columns<V>(p, SHIFT), dot);
            }
            // a slot without an expert has met zeros only, unless d_y is not finite
            const float sum = warp_sums(dot);
            constexpr int kLanes = 32 / B;  // that hold the same sum
            if (warps == 1) {
                const uint32_t s = s0 + lane / kLanes;
                const uint32_t at = __shfl_sync(kFull, slots.at, lane / kLanes);
                if (lane % kLanes == 0 && live && s < p.top_k)
                    p.d_weights[t * p.top_k + s] = at < valid ? sum : 0.f;
                continue;
            }
            // the warps of a token add up in order of their number; two buffers, so that
            // one barrier a turn keeps the sums of the turn before from being overwritten
            if (lane % kLanes == 0) part[turn][warp][lane / kLanes] = sum;
            __syncthreads();
            if (threadIdx.x < B && live && s0 + threadIdx.x < p.top_k) {
                float total = 0.f;
                for (int q = 0; q < warps; ++q) total += part[turn][first_warp + q][threadIdx.x];
                p.d_weights[t * p.top_k + s0 + threadIdx.x] = slots.at < valid ? total : 0.f;
            }
            turn ^= 1;
        }
        slots = next;
    }
}

// whether every row starts on a multiple of 16 bytes
template <typename T> bool aligned_rows(const MoeRowsParams &p) {
    const void *ptrs[4] = {p.tok_in, p.tok_out, p.row_in, p.row_out};
    const int64_t lds[4] = {p.ld_tok_in, p.ld_tok_out, p.ld_row_in, p.ld_row_out};
    uint64_t bits = 0;
    for (int i = 0; i < 4; ++i)
        if (ptrs[i] != nullptr)
            bits |= reinterpret_cast<uintptr_t>(ptrs[i]) | static_cast<uint64_t>(lds[i]) * sizeof(T);
    return bits % 16 == 0;
}

struct Shape {
    dim3 grid, block;
};

// tx covers a row of nvec accesses if it can, or half of it where that still gives
// every SM its `resident` blocks (two steps a thread: 8192 tokens x 8 slots of 2048
// bf16, gradient of combine, 91 us against 97 us).  `stays`: no more blocks than
// that; they walk over the tokens (combine of the same rows 51 us, 54 us with a
// block for each token).  A dispatch is mostly stores and is faster with a block for
// each token (49 us against 56 us).  Along the row there are further blocks when there
// are few tokens and a block need not see a whole row.
Shape shape_of(const MoeRowsParams &p, int V, int resident, bool stays, bool rows_whole) {
    const int64_t nvec = (p.n + V - 1) / V;
    const int64_t most = static_cast<int64_t>(resident) * device_sm_count();
    unsigned tx = 32;
    while (tx < static_cast<unsigned>(kThreads) &&
           tx * (static_cast<int64_t>(p.m) * tx * 2 >= most * kThreads ? 2 : 1) < nvec)
        tx *= 2;
    const unsigned ty = kThreads / tx;
    int64_t gx = (static_cast<int64_t>(p.m) + ty - 1) / ty, gy = 1;
    if (stays && gx > most) gx = most;
    while (!rows_whole && gx * gy * 2 <= most && gy * tx < nvec) gy *= 2;
    return Shape{dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(tx, ty)};
}

enum Which { kDispatch, kCombine, kCombineBackward };

// Started early: dispatch after the sort 52.6 us a pair for 54.8 (4096 tokens x 8 slots x 4096
// bf16), the gradients of combine and dispatch 143.6 for 146.1 (8192 tokens x 8 slots x 2048 bf16).
template <typename T, int VB, bool SHIFT>
cudaError_t launch_vb(Which which, const MoeRowsParams &p, cudaStream_t s) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    using Blocks = Resident<T, SHIFT>;
    if (which == kDispatch) {
        const Shape h = shape_of(p, V, Blocks::kDispatch, false, false);
        return launch_early(moe_dispatch_kernel<T, VB, SHIFT>, h.grid, h.block, 0, s, p);
    } else if (which == kCombine) {
        const Shape h = shape_of(p, V, Blocks::kCombine, true, false);
        return launch_early(moe_combine_kernel<T, VB, SHIFT>, h.grid, h.block, 0, s, p);
    } else {
        const Shape h = shape_of(p, V, Blocks::kBackward, true, true);
        return launch_early(moe_combine_backward_kernel<T, VB, SHIFT>, h.grid, h.block, 0, s, p);
    }
}

// 16 bytes an access; rows that start anywhere are shifted into place unless they are so short
// that much of them lies outside the whole accesses (bf16, 31057 tokens x 3 slots x 73: dispatch
// 26 us shifted, 14 one element an access, combine 24 and 18, its gradient 58 and 37; 20000 x 4 x 131
// 19 and 17.6, 18.5 and 22.7, 43 and 50).
template <typename T>
cudaError_t launch_t(Which which, const MoeRowsParams &p, cudaStream_t s) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    if (aligned_rows<T>(p)) return launch_vb<T, 16, false>(which, p, s);
    if (p.n >= 16 * V) return launch_vb<T, 16, true>(which, p, s);
    return launch_vb<T, static_cast<int>(sizeof(T)), false>(which, p, s);
}

cudaError_t launch_dt(int dt, Which which, const MoeRowsParams &p, cudaStream_t s) {
    switch (dt) {
    case kF32: return launch_t<float>(which, p, s);
    case kF16: return launch_t<__half>(which, p, s);
    case kBF16: return launch_t<__nv_bfloat16>(which, p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_moe_dispatch(int dt, const MoeRowsParams &p, cudaStream_t s) {
    return launch_dt(dt, kDispatch, p, s);
}
cudaError_t launch_moe_combine(int dt, const MoeRowsParams &p, cudaStream_t s) { return launch_dt(dt, kCombine, p, s); }
cudaError_t launch_moe_combine_backward(int dt, const MoeRowsParams &p, cudaStream_t s) {
    return launch_dt(dt, kCombineBackward, p, s);
}

}  // namespace gbmm
