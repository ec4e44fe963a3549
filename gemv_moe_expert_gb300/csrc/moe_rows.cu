// moe_rows.cu -- rows of a mixture-of-experts layer into expert order and back:
// dispatch (copy), combine (weighted sum over a token's slots; with weights of 1
// the gradient of the dispatch) and the gradient of combine.
//
// All three are bound by HBM: a row of x or y and top_k rows of xs or ys per
// token, a few operations an element.  Every kernel works in token order, so a
// token's row is read or written once and its top_k rows in expert order, each
// a contiguous run of n elements, are addressed through position; working in
// expert order would read the token's row once per slot.  Rows whose position is
// at or past *valid have no expert.
//
// A block is a grid of tx x ty threads: tx along the row (one access of VB bytes
// a thread and step), ty tokens.  Slots are taken in batches of kBatch, all of a
// batch's loads issued before the first is used.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kNowhere = 0xffffffffu;

template <int VB> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

// V elements of a row starting at element i, zeros past its end
template <typename T, int VB>
__device__ __forceinline__ typename Raw<VB>::type load_raw(const T *row, int64_t i, int64_t n) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    if (V == 1 || i + V <= n) return __ldg(reinterpret_cast<const R *>(row + i));
    R r{};
    T *e = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (i + j < n) e[j] = row[i + j];
    return r;
}

template <typename T, int VB>
__device__ __forceinline__ void store_raw(T *row, int64_t i, int64_t n, const typename Raw<VB>::type &r) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    if (V == 1 || i + V <= n) {
        *reinterpret_cast<R *>(row + i) = r;
        return;
    }
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (i + j < n) row[i + j] = e[j];
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
// place of slot s of token t, kNowhere past the token's slots
__device__ __forceinline__ uint32_t place_of(const MoeRowsParams &p, uint32_t t, uint32_t s) {
    if (s >= p.top_k) return kNowhere;
    const uint32_t r = t * p.top_k + s;
    return p.position != nullptr ? __ldg(p.position + r) : r;
}

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads) moe_dispatch_kernel(MoeRowsParams p) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.m) return;
    const uint32_t rows = p.m * p.top_k, valid = valid_rows(p);
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.x * V;
    const T *x = static_cast<const T *>(p.tok_in) + static_cast<int64_t>(t) * p.ld_tok_in;
    T *out = static_cast<T *>(p.row_out);
    for (uint32_t s0 = 0; s0 < p.top_k; s0 += kBatch) {
        uint32_t at[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) at[b] = place_of(p, t, s0 + b);
        for (int64_t i = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V; i < p.n; i += step) {
            const R v = load_raw<T, VB>(x, i, p.n);
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (at[b] < rows)
                    store_raw<T, VB>(out + static_cast<int64_t>(at[b]) * p.ld_row_out, i, p.n, at[b] < valid ? v : R{});
        }
    }
}

template <typename T, int VB>
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(MoeRowsParams p) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.m) return;
    const uint32_t valid = valid_rows(p);
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.x * V;
    const T *in = static_cast<const T *>(p.row_in);
    T *y = static_cast<T *>(p.tok_out) + static_cast<int64_t>(t) * p.ld_tok_out;
    for (int64_t i = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V; i < p.n; i += step) {
        float acc[V];
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
        for (uint32_t s0 = 0; s0 < p.top_k; s0 += kBatch) {
            R v[kBatch];
            float w[kBatch];
            bool has[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const uint32_t at = place_of(p, t, s0 + b);
                has[b] = at < valid;
                if (has[b]) {
                    v[b] = load_raw<T, VB>(in + static_cast<int64_t>(at) * p.ld_row_in, i, p.n);
                    w[b] = p.weights != nullptr ? __ldg(p.weights + t * p.top_k + s0 + b) : 1.f;
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (has[b]) {
                    float f[V];
                    unpack<T, V>(v[b], f);
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = fmaf(w[b], f[j], acc[j]);
                }
            }
        }
        store_raw<T, VB>(y, i, p.n, pack<T, V, R>(acc));
    }
}

// Sums v[b] over the warp; lane l returns the sum of v[l / 4] (8 values, 9
// shuffles: each of the first three steps halves the values a lane carries).
__device__ __forceinline__ float warp_sum8(const float (&v)[kBatch], int lane) {
    static_assert(kBatch == 8, "written for batches of 8");
    float a[4], b[2], c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 16;
        const float keep = up ? v[i + 4] : v[i], give = up ? v[i] : v[i + 4];
        a[i] = keep + __shfl_xor_sync(kFull, give, 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool up = lane & 8;
        const float keep = up ? a[i + 2] : a[i], give = up ? a[i] : a[i + 2];
        b[i] = keep + __shfl_xor_sync(kFull, give, 8);
    }
    {
        const bool up = lane & 4;
        const float keep = up ? b[1] : b[0], give = up ? b[0] : b[1];
        c = keep + __shfl_xor_sync(kFull, give, 4);
    }
    c += __shfl_xor_sync(kFull, c, 2);
    c += __shfl_xor_sync(kFull, c, 1);
    return c;
}

// blockDim.x is a multiple of 32, so a warp belongs to one token; the grid's y
// extent is 1 (a block sees a token's whole row, for the dot products).
template <typename T, int VB>
__global__ void __launch_bounds__(kThreads) moe_combine_backward_kernel(MoeRowsParams p) {
    using R = typename Raw<VB>::type;
    constexpr int V = VB / static_cast<int>(sizeof(T));
    __shared__ float part[kThreads / 32][kBatch];
    const int lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < p.m;
    const uint32_t rows = p.m * p.top_k, valid = valid_rows(p);
    const T *in = static_cast<const T *>(p.row_in);
    T *out = static_cast<T *>(p.row_out);
    const T *dy = static_cast<const T *>(p.tok_in) + static_cast<int64_t>(live ? t : 0) * p.ld_tok_in;
    for (uint32_t s0 = 0; s0 < p.top_k; s0 += kBatch) {
        uint32_t at[kBatch];
        float w[kBatch], dot[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            at[b] = live ? place_of(p, t, s0 + b) : kNowhere;
            w[b] = at[b] < valid ? __ldg(p.weights + t * p.top_k + s0 + b) : 0.f;
            dot[b] = 0.f;
        }
        for (int64_t i = static_cast<int64_t>(threadIdx.x) * V; i < p.n; i += static_cast<int64_t>(blockDim.x) * V) {
            if (!live) break;
            R v[kBatch];
            const R graw = load_raw<T, VB>(dy, i, p.n);
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (at[b] < valid) v[b] = load_raw<T, VB>(in + static_cast<int64_t>(at[b]) * p.ld_row_in, i, p.n);
            float g[V];
            unpack<T, V>(graw, g);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (at[b] >= rows) continue;
                R d{};
                if (at[b] < valid) {
                    float f[V], wg[V];
                    unpack<T, V>(v[b], f);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        dot[b] = fmaf(g[j], f[j], dot[b]);
                        wg[j] = w[b] * g[j];
                    }
                    d = pack<T, V, R>(wg);
                }
                store_raw<T, VB>(out + static_cast<int64_t>(at[b]) * p.ld_row_out, i, p.n, d);
            }
        }
        // the warps of a token add up in order of their number
        const float sum = warp_sum8(dot, lane);
        const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5;
        if ((lane & 3) == 0) part[warp][lane >> 2] = sum;
        __syncthreads();
        if (threadIdx.x < kBatch && live && s0 + threadIdx.x < p.top_k) {
            float total = 0.f;
            for (int q = 0; q < static_cast<int>(blockDim.x) / 32; ++q) total += part[warp + q][threadIdx.x];
            p.d_weights[t * p.top_k + s0 + threadIdx.x] = total;
        }
        __syncthreads();
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

// tx covers a row of nvec accesses if it can; rows_whole: a block must see the
// whole row.
Shape shape_of(const MoeRowsParams &p, int V, bool rows_whole) {
    const int64_t nvec = (p.n + V - 1) / V;
    unsigned tx = 32;
    while (tx < static_cast<unsigned>(kThreads) && tx < nvec) tx *= 2;
    const unsigned ty = kThreads / tx;
    int64_t gy = rows_whole ? 1 : (nvec + tx - 1) / tx;
    if (gy > 65535) gy = 65535;
    if (gy < 1) gy = 1;
    return Shape{dim3((p.m + ty - 1) / ty, static_cast<unsigned>(gy)), dim3(tx, ty)};
}

enum Which { kDispatch, kCombine, kCombineBackward };

template <typename T, int VB>
cudaError_t launch_vb(Which which, const MoeRowsParams &p, cudaStream_t s) {
    const Shape h = shape_of(p, VB / static_cast<int>(sizeof(T)), which == kCombineBackward);
    if (which == kDispatch)
        moe_dispatch_kernel<T, VB><<<h.grid, h.block, 0, s>>>(p);
    else if (which == kCombine)
        moe_combine_kernel<T, VB><<<h.grid, h.block, 0, s>>>(p);
    else
        moe_combine_backward_kernel<T, VB><<<h.grid, h.block, 0, s>>>(p);
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
