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
// a thread and step), ty tokens.  Slots are taken in batches of B (4, or 8 for more
// than 4 slots), all of a batch's loads issued before the first is used.  Blocks
// stay and walk over the tokens: the places of the next token's slots are loaded
// while the current token's rows are in flight.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 256;
constexpr int B = 4;
// Blocks an SM (the registers they may use follow).  4-byte elements need fewer
// registers for the same bytes in flight.  Measured on 4096 tokens x 8 slots of
// 4096 elements: combine f32 95 us with 4 and 97 us with 5, bf16 52 and 51 us; its
// gradient f32 177 us with 3 and 190 us with 4, bf16 97 and 92 us.
template <typename T> struct Resident {
    static constexpr int kCombine = sizeof(T) == 4 ? 4 : 5;
    static constexpr int kBackward = sizeof(T) == 4 ? 3 : 4;
};
constexpr int kDispatchBlocks = 4;
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
// that the rows' loads wait for one latency and not for eight.
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

// Columns of a row are dealt to threads in steps that all threads of a warp take
// together (the shuffles need the whole warp; a thread past the end idles): first
// the columns that divide into accesses of VB bytes, then the rest one by one.  The
// two are separate calls so that every access in them is one predicated instruction
// (with the choice inside the loop each load sat behind its own branch and the
// loads of a batch no longer overlapped).

struct Columns {
    int64_t from, to, step;  // elements
};
template <int V>
__device__ __forceinline__ Columns whole_columns(const MoeRowsParams &p) {
    return Columns{(static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V, p.n / V * V,
                   static_cast<int64_t>(gridDim.y) * blockDim.x * V};
}
template <int V>
__device__ __forceinline__ Columns rest_columns(const MoeRowsParams &p) {
    return Columns{p.n / V * V + threadIdx.x, blockIdx.y == 0 ? p.n : 0, static_cast<int64_t>(blockDim.x)};
}

template <typename T, int VB>
__device__ __forceinline__ void dispatch_columns(const MoeRowsParams &p, const Slots &slots, uint32_t valid,
                                                 const T *x, const Columns &c) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t rows = p.m * p.top_k;
    const int lane = threadIdx.x & 31;
    T *out = static_cast<T *>(p.row_out);
    for (int64_t i = c.from; i - lane * V < c.to; i += c.step) {
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

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads, kDispatchBlocks)
    moe_dispatch_kernel(const __grid_constant__ MoeRowsParams p) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t valid = valid_rows(p);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.y;
    uint64_t t = static_cast<uint64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    Slots slots, next;
    slots.load(p, valid, t, 0);
    for (; t < p.m; t += step) {
        next.load(p, valid, t + step, 0);
        const T *x = static_cast<const T *>(p.tok_in) + static_cast<int64_t>(t) * p.ld_tok_in;
        for (uint32_t s0 = 0; s0 < p.top_k; s0 += B) {
            if (s0 != 0) slots.load(p, valid, t, s0);
            dispatch_columns<T, VB>(p, slots, valid, x, whole_columns<V>(p));
            if (V > 1) dispatch_columns<T, sizeof(T)>(p, slots, valid, x, rest_columns<V>(p));
        }
        slots = next;
    }
}

// A slot without an expert adds 0 * 0.
template <typename T, int VB>
__device__ __forceinline__ void combine_columns(const MoeRowsParams &p, uint32_t t, Slots slots, uint32_t valid,
                                                const Columns &c) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const int lane = threadIdx.x & 31;
    const T *in_rows = static_cast<const T *>(p.row_in);
    T *y = static_cast<T *>(p.tok_out) + static_cast<int64_t>(t) * p.ld_tok_out;
    for (int64_t i = c.from; i - lane * V < c.to; i += c.step) {
        const bool in = i < c.to;
        float acc[V];
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
        for (uint32_t s0 = 0; s0 < p.top_k; s0 += B) {
            if (p.top_k > B) slots.load(p, valid, t, s0);
            R v[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint32_t at = slots.place(b);
                v[b] = R{};
                if (in && at < valid) v[b] = load_raw<T, VB>(in_rows + static_cast<int64_t>(at) * p.ld_row_in + i);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const float w = slots.weight(b);
                float f[V];
                unpack<T, V>(v[b], f);
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = fmaf(w, f[j], acc[j]);
            }
        }
        if (in) store_raw<T, VB>(y + i, pack<T, V, R>(acc));
    }
}

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads, Resident<T>::kCombine)
    moe_combine_kernel(const __grid_constant__ MoeRowsParams p) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t valid = valid_rows(p);
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.y;
    uint64_t t = static_cast<uint64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    Slots slots, next;
    slots.load(p, valid, t, 0);
    for (; t < p.m; t += step) {
        next.load(p, valid, t + step, 0);
        combine_columns<T, VB>(p, static_cast<uint32_t>(t), slots, valid, whole_columns<V>(p));
        if (V > 1) combine_columns<T, sizeof(T)>(p, static_cast<uint32_t>(t), slots, valid, rest_columns<V>(p));
        slots = next;
    }
}

// Sums each v[b] over the warp; lane l returns the sum of v[l / (32 / B)]: each of
// the first log2 B steps halves the values a lane carries, so 8 sums take 9
// shuffles instead of 40.
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

template <typename T, int VB>
__device__ __forceinline__ void combine_backward_columns(const MoeRowsParams &p, const Slots &slots, uint32_t valid,
                                                         const T *dy, const Columns &c, float (&dot)[B]) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t rows = p.m * p.top_k;
    const int lane = threadIdx.x & 31;
    const T *in_rows = static_cast<const T *>(p.row_in);
    T *out = static_cast<T *>(p.row_out);
    for (int64_t i = c.from; i - lane * V < c.to; i += c.step) {
        const bool in = i < c.to;
        R v[B], graw{};
        if (in) graw = load_raw<T, VB>(dy + i);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const uint32_t at = slots.place(b);
            v[b] = R{};
            if (in && at < valid) v[b] = load_raw<T, VB>(in_rows + static_cast<int64_t>(at) * p.ld_row_in + i);
        }
        float g[V];
        unpack<T, V>(graw, g);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const uint32_t at = slots.place(b);
            const float w = slots.weight(b);
            float f[V], wg[V];
            unpack<T, V>(v[b], f);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                dot[b] = fmaf(g[j], f[j], dot[b]);
                wg[j] = w * g[j];
            }
            const R d = pack<T, V, R>(wg);
            if (in && at < rows)
                store_raw<T, VB>(out + static_cast<int64_t>(at) * p.ld_row_out + i, at < valid ? d : R{});
        }
    }
}

// The grid's y extent is 1: a block sees a token's whole row, for the dot products.
template <typename T, int VB>
__global__ void __launch_bounds__(kThreads, Resident<T>::kBackward)
    moe_combine_backward_kernel(const __grid_constant__ MoeRowsParams p) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    __shared__ float part[2][kThreads / 32][B];
    const int lane = threadIdx.x & 31;
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
                combine_backward_columns<T, VB>(p, slots, valid, dy, whole_columns<V>(p), dot);
                if (V > 1) combine_backward_columns<T, sizeof(T)>(p, slots, valid, dy, rest_columns<V>(p), dot);
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

// Bytes of an access that every row start allows: 16, else 4, else one element.
template <typename T>
int access_bytes(const MoeRowsParams &p) {
    const void *ptrs[4] = {p.tok_in, p.tok_out, p.row_in, p.row_out};
    const int64_t lds[4] = {p.ld_tok_in, p.ld_tok_out, p.ld_row_in, p.ld_row_out};
    uint64_t bits = 0;
    for (int i = 0; i < 4; ++i)
        if (ptrs[i] != nullptr)
            bits |= reinterpret_cast<uintptr_t>(ptrs[i]) | static_cast<uint64_t>(lds[i]) * sizeof(T);
    return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : static_cast<int>(sizeof(T));
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

template <typename T, int VB>
cudaError_t launch_vb(Which which, const MoeRowsParams &p, cudaStream_t s) {
    constexpr int V = VB / static_cast<int>(sizeof(T));
    if (which == kDispatch) {
        const Shape h = shape_of(p, V, kDispatchBlocks, false, false);
        moe_dispatch_kernel<T, VB><<<h.grid, h.block, 0, s>>>(p);
    } else if (which == kCombine) {
        const Shape h = shape_of(p, V, Resident<T>::kCombine, true, false);
        moe_combine_kernel<T, VB><<<h.grid, h.block, 0, s>>>(p);
    } else {
        const Shape h = shape_of(p, V, Resident<T>::kBackward, true, true);
        moe_combine_backward_kernel<T, VB><<<h.grid, h.block, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(Which which, const MoeRowsParams &p, cudaStream_t s) {
    switch (access_bytes<T>(p)) {
    case 16: return launch_vb<T, 16>(which, p, s);
    case 4: return launch_vb<T, 4>(which, p, s);
    default: return launch_vb<T, static_cast<int>(sizeof(T))>(which, p, s);
    }
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
