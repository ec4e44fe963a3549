// moe_route.cu -- top-k softmax router of a mixture-of-experts layer, forward
// and backward.
//
// One warp owns a token: its logits live in registers (expert j * 32 + lane in
// register j), so every logit is read once.  The selection compares integer
// keys that order as the scores do; the softmax subtracts the maximum.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Integer that orders as the score does, 0 for a score that is not greater
// than -inf.  Adding +0 turns -0 into +0, so the two compare equal.
__device__ __forceinline__ uint32_t score_key(float score) {
    if (!(score > neg_inf())) return 0u;
    const uint32_t u = __float_as_uint(score + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// The token's logits, -inf for experts that are not live, and their keys.
template <typename T, int V>
__device__ __forceinline__ void load_row(const MoeRouteParams &p, uint32_t t, int lane, float (&l)[V],
                                         uint32_t (&key)[V]) {
    const T *row = static_cast<const T *>(p.logits) + static_cast<int64_t>(t) * p.ld_logits;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t e = j * 32 + lane;
        l[j] = e < p.n_experts ? Elem<T>::to_f(row[e]) : neg_inf();
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t e = j * 32 + lane;
        const float score = p.bias != nullptr && e < p.n_experts ? l[j] + p.bias[e] : l[j];
        key[j] = score_key(score);
        if (key[j] == 0u) l[j] = neg_inf();
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(MoeRouteParams p) {
    const int lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.m) return;
    float l[V];
    uint32_t key[V];
    load_row<T, V>(p, t, lane, l, key);

    float top = neg_inf(), sum = 0.f;
    if (!p.selected) {
#pragma unroll
        for (int j = 0; j < V; ++j) top = fmaxf(top, l[j]);
        top = warp_max(top);
        if (top > neg_inf()) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += key[j] != 0u ? expf(l[j] - top) : 0.f;
        }
        sum = warp_sum(sum);
    }

    // slot s ends up in lane s
    uint32_t my_id = p.n_experts;
    float my_l = neg_inf();
    for (uint32_t s = 0; s < p.top_k; ++s) {
        uint32_t best = 0u, at = 0u;
        float best_l = neg_inf();
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (key[j] > best) {
                best = key[j];
                at = j;
                best_l = l[j];
            }
        }
        const uint32_t most = __reduce_max_sync(kFull, best);
        if (most == 0u) break;  // fewer live experts than slots
        const uint32_t e = __reduce_min_sync(kFull, best == most ? at * 32 + lane : kFull);
        const float el = __shfl_sync(kFull, best_l, e & 31);
        if (lane == static_cast<int>(s)) {
            my_id = e;
            my_l = el;
        }
        if (lane == static_cast<int>(e & 31)) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j == static_cast<int>(e >> 5)) key[j] = 0u;
        }
    }

    const bool chosen = my_id < p.n_experts;
    if (p.selected) top = warp_max(my_l);
    float w = chosen ? expf(my_l - top) : 0.f;
    if (p.selected) sum = warp_sum(w);
    if (lane < static_cast<int>(p.top_k)) {
        const int64_t r = static_cast<int64_t>(t) * p.top_k + lane;
        p.ids[r] = my_id;
        p.weights[r] = chosen ? w / sum : 0.f;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) moe_route_backward_kernel(MoeRouteParams p) {
    const int lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
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
    const float dot = warp_sum(w * d);

    float out[V];
    if (p.selected) {
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = 0.f;
        const float mine = w * (d - dot);
        for (uint32_t s = 0; s < p.top_k; ++s) {
            const uint32_t e = __shfl_sync(kFull, id, s);
            const float v = __shfl_sync(kFull, mine, s);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e == static_cast<uint32_t>(j * 32 + lane)) out[j] = v;
        }
    } else {
        float l[V], g[V];
        uint32_t key[V];
        load_row<T, V>(p, t, lane, l, key);
        float top = neg_inf(), sum = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            top = fmaxf(top, l[j]);
            g[j] = 0.f;
        }
        top = warp_max(top);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            l[j] = key[j] != 0u ? expf(l[j] - top) : 0.f;
            sum += l[j];
        }
        sum = warp_sum(sum);
        for (uint32_t s = 0; s < p.top_k; ++s) {
            const uint32_t e = __shfl_sync(kFull, id, s);
            const float v = __shfl_sync(kFull, d, s);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (e == static_cast<uint32_t>(j * 32 + lane)) g[j] = v;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = key[j] != 0u ? l[j] / sum * (g[j] - dot) : 0.f;
    }
    T *row = static_cast<T *>(p.d_logits) + static_cast<int64_t>(t) * p.ld_d_logits;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t e = j * 32 + lane;
        if (e < p.n_experts) row[e] = Elem<T>::from_f(out[j]);
    }
}

template <typename T, int V>
cudaError_t launch_v(bool backward, const MoeRouteParams &p, cudaStream_t s) {
    const unsigned grid = (p.m + kThreads / 32 - 1) / (kThreads / 32);
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
