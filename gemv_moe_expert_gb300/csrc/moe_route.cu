// moe_route.cu -- top-k softmax router of a mixture-of-experts layer, forward
// and backward.
//
// One warp owns a token and keeps its logits in registers, V a lane, so every
// logit is read once (twice over a training step) with one access of W = min(V, 4)
// elements.  The selection compares integer keys that order as the scores do:
// each of the top_k steps is one maximum and one minimum over the warp (the
// largest key, then the lowest expert that has it).  The softmax subtracts the
// maximum and sums in f32.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Integer that orders as the score does, 0 for a score that is not greater
// than -inf.  Adding +0 turns -0 into +0, so the two compare equal.
__device__ __forceinline__ uint32_t score_key(float score) {
    if (!(score > neg_inf())) return 0u;
    const uint32_t u = __float_as_uint(score + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// largest value of the warp; there are no NaN among them
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// Lane `lane` holds experts expert_of(lane, 0..V-1), increasing: runs of W
// neighbours, 32 W apart.
template <int V> struct Lanes {
    static constexpr int W = V < 4 ? V : 4;
    __device__ static __forceinline__ uint32_t expert_of(int lane, int j) {
        return static_cast<uint32_t>(j / W * 32 * W + lane * W + j % W);
    }
};

template <typename T, int W> struct alignas(sizeof(T) * W) Run {
    T v[W];
};

// row[expert_of(lane, j)] for every j, `fill` past the row's E elements; vec: whole runs can be read
template <typename T, int V>
__device__ __forceinline__ void load_lanes(const T *row, uint32_t E, int lane, bool vec, float fill, float (&out)[V]) {
    constexpr int W = Lanes<V>::W;
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        const uint32_t e = Lanes<V>::expert_of(lane, c * W);
        if (vec) {
            Run<T, W> r;
            if (e < E) r = *reinterpret_cast<const Run<T, W> *>(row + e);
#pragma unroll
            for (int i = 0; i < W; ++i) out[c * W + i] = e < E ? Elem<T>::to_f(r.v[i]) : fill;
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) out[c * W + i] = e + i < E ? Elem<T>::to_f(row[e + i]) : fill;
        }
    }
}

// The token's logits, -inf for experts that are not live, and their keys.
template <typename T, int V>
__device__ __forceinline__ void load_row(const MoeRouteParams &p, uint32_t t, int lane, float (&l)[V],
                                         uint32_t (&key)[V]) {
    load_lanes<T, V>(static_cast<const T *>(p.logits) + static_cast<int64_t>(t) * p.ld_logits, p.n_experts, lane,
                     p.logits_vec != 0, neg_inf(), l);
    if (p.bias != nullptr) {
        float b[V];
        load_lanes<float, V>(p.bias, p.n_experts, lane, p.bias_vec != 0, 0.f, b);
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = score_key(l[j] + b[j]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = score_key(l[j]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (key[j] == 0u) l[j] = neg_inf();
}

// exp(l - max) in place (0 for experts that are not live), and their sum
template <int V>
__device__ __forceinline__ float softmax_terms(float (&l)[V], const uint32_t (&key)[V], float *top_out) {
    float top = l[0], sum = 0.f;
#pragma unroll
    for (int j = 1; j < V; ++j) top = fmaxf(top, l[j]);
    top = warp_max(top);
    *top_out = top;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        l[j] = key[j] != 0u ? expf(l[j] - top) : 0.f;
        sum += l[j];
    }
    return warp_sum(sum);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(MoeRouteParams p) {
    const int lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= p.m) return;
    float l[V];
    uint32_t key[V];
    load_row<T, V>(p, t, lane, l, key);

    float top = neg_inf(), sum = 0.f;
    if (!p.selected) sum = softmax_terms<V>(l, key, &top);

    // Slot s ends up in lane s.  With few experts a lane the keys are put in
    // descending order first (neighbours are exchanged only when the later one is
    // larger, so equals keep the lowest expert first) and each step looks at the
    // lane's head alone; sorting more than 4 costs more than looking at all of them.
    uint32_t my_id = p.n_experts;
    if (V <= 4) {
        uint32_t at[V];
#pragma unroll
        for (int j = 0; j < V; ++j) at[j] = Lanes<V>::expert_of(lane, j);
#pragma unroll
        for (int end = V - 1; end > 0; --end) {
#pragma unroll
            for (int j = 0; j < end; ++j) {
                const bool swap = key[j + 1] > key[j];
                const uint32_t k0 = key[j], a0 = at[j];
                key[j] = swap ? key[j + 1] : k0;
                at[j] = swap ? at[j + 1] : a0;
                key[j + 1] = swap ? k0 : key[j + 1];
                at[j + 1] = swap ? a0 : at[j + 1];
            }
        }
        for (uint32_t s = 0; s < p.top_k; ++s) {
            const uint32_t most = __reduce_max_sync(kFull, key[0]);
            if (most == 0u) break;  // fewer live experts than slots
            const uint32_t e = __reduce_min_sync(kFull, key[0] == most ? at[0] : kFull);
            if (lane == static_cast<int>(s)) my_id = e;
            if (at[0] == e) {
#pragma unroll
                for (int j = 0; j + 1 < V; ++j) {
                    key[j] = key[j + 1];
                    at[j] = at[j + 1];
                }
                key[V - 1] = 0u;
            }
        }
    } else {
        for (uint32_t s = 0; s < p.top_k; ++s) {
            uint32_t best = 0u, at = 0u;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (key[j] > best) {
                    best = key[j];
                    at = j;
                }
            }
            const uint32_t most = __reduce_max_sync(kFull, best);
            if (most == 0u) break;
            const uint32_t mine = static_cast<uint32_t>(Lanes<V>::expert_of(lane, 0)) + at / 4 * 128 + at % 4;
            const uint32_t e = __reduce_min_sync(kFull, best == most ? mine : kFull);
            if (lane == static_cast<int>(s)) my_id = e;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (Lanes<V>::expert_of(lane, j) == e) key[j] = 0u;
        }
    }

    const bool chosen = my_id < p.n_experts;
    float my_l = neg_inf();
    if (chosen)
        my_l = Elem<T>::to_f(static_cast<const T *>(p.logits)[static_cast<int64_t>(t) * p.ld_logits + my_id]);
    if (p.selected) top = warp_max(my_l);
    const float w = chosen ? expf(my_l - top) : 0.f;
    if (p.selected) sum = warp_sum(w);
    if (lane < static_cast<int>(p.top_k)) {
        const int64_t r = static_cast<int64_t>(t) * p.top_k + lane;
        p.ids[r] = my_id;
        p.weights[r] = chosen ? w / sum : 0.f;
    }
}

// The slots' gradients reach the lanes that own their experts through a row of
// shared memory for each warp: V / W accesses instead of top_k * V comparisons.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) moe_route_backward_kernel(MoeRouteParams p) {
    constexpr int W = Lanes<V>::W;
    __shared__ __align__(16) float rows[kWarps][32 * V];
    const int lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    float *mine = rows[threadIdx.x >> 5];
    if (t >= p.m) return;
    // slot s in lane s
    uint32_t id = p.n_experts;
    float w = 0.f, d = 0.f;
    if (lane < static_cast<int>(p.top_k)) {
        const int64_t r = static_cast<int64_t>(t) * p.top_k + lane;
        id = p.ids[r];
        if (id < p.n_experts) {
            w = p.weights[r];
            d = p.d_weights[r];
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) mine[j * 32 + lane] = 0.f;
    float l[V];
    uint32_t key[V];
    if (!p.selected) load_row<T, V>(p, t, lane, l, key);
    const float dot = warp_sum(w * d);  // also orders the zeros before what follows
    __syncwarp();
    if (id < p.n_experts) mine[id] = p.selected ? w * (d - dot) : d;
    __syncwarp();
    float g[V];
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        const Run<float, W> r = *reinterpret_cast<const Run<float, W> *>(mine + Lanes<V>::expert_of(lane, c * W));
#pragma unroll
        for (int i = 0; i < W; ++i) g[c * W + i] = r.v[i];
    }
    if (!p.selected) {
        float top;
        const float inv = 1.f / softmax_terms<V>(l, key, &top);
#pragma unroll
        for (int j = 0; j < V; ++j) g[j] = key[j] != 0u ? l[j] * inv * (g[j] - dot) : 0.f;
    }
    T *row = static_cast<T *>(p.d_logits) + static_cast<int64_t>(t) * p.ld_d_logits;
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        const uint32_t e = Lanes<V>::expert_of(lane, c * W);
        if (p.d_logits_vec) {
            Run<T, W> r;
#pragma unroll
            for (int i = 0; i < W; ++i) r.v[i] = Elem<T>::from_f(g[c * W + i]);
            if (e < p.n_experts) *reinterpret_cast<Run<T, W> *>(row + e) = r;
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                if (e + i < p.n_experts) row[e + i] = Elem<T>::from_f(g[c * W + i]);
        }
    }
}

// whether rows ld elements apart, and E elements long, divide into aligned runs of W
bool runs_fit(const void *ptr, int64_t ld, uint32_t E, int W, int size) {
    return reinterpret_cast<uintptr_t>(ptr) % (W * size) == 0 && ld % W == 0 && E % W == 0;
}

template <typename T, int V>
cudaError_t launch_v(bool backward, MoeRouteParams p, cudaStream_t s) {
    constexpr int W = Lanes<V>::W;
    const unsigned grid = (p.m + kWarps - 1) / kWarps;
    p.logits_vec = runs_fit(p.logits, p.ld_logits, p.n_experts, W, sizeof(T));
    p.bias_vec = runs_fit(p.bias, W, p.n_experts, W, sizeof(float));
    p.d_logits_vec = runs_fit(p.d_logits, p.ld_d_logits, p.n_experts, W, sizeof(T));
    if (backward)
        moe_route_backward_kernel<T, V><<<grid, kThreads, 0, s>>>(p);
    else
        moe_route_kernel<T, V><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(bool backward, const MoeRouteParams &p, cudaStream_t s) {
    if (p.n_experts <= 32) return launch_v<T, 1>(backward, p, s);
    if (p.n_experts <= 64) return launch_v<T, 2>(backward, p, s);
    if (p.n_experts <= 128) return launch_v<T, 4>(backward, p, s);
    if (p.n_experts <= 256) return launch_v<T, 8>(backward, p, s);
    if (p.n_experts <= 512) return launch_v<T, 16>(backward, p, s);
    return launch_v<T, 32>(backward, p, s);
}

cudaError_t launch_dt(int dt, bool backward, const MoeRouteParams &p, cudaStream_t s) {
    switch (dt) {
    case kF32: return launch_t<float>(backward, p, s);
    case kF16: return launch_t<__half>(backward, p, s);
    case kBF16: return launch_t<__nv_bfloat16>(backward, p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_moe_route(int dt, const MoeRouteParams &p, cudaStream_t s) { return launch_dt(dt, false, p, s); }
cudaError_t launch_moe_route_backward(int dt, const MoeRouteParams &p, cudaStream_t s) {
    return launch_dt(dt, true, p, s);
}

}  // namespace gbmm
