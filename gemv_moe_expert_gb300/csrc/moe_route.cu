// moe_route.cu -- top-k softmax router of a mixture-of-experts layer, forward
// and backward.
//
// A warp keeps the logits of its tokens in registers, V a lane, so every logit is
// read once (twice over a training step) with one access of W = min(V, 4) elements.  The
// selection compares integer keys that order as the scores do: each of the top_k steps
// is one maximum over the warp and one ballot for the first lane that has it.  The
// softmax subtracts the maximum and sums in f32.
//
// In this layout the selection serves one token at a time with a whole warp, and with many tokens the
// kernel is bound by instruction issue (80 % of the cycles in which an SM has work forward, 68 %
// backward), so it saves instructions: a lane's keys are sorted once, into a list in shared memory from which
// the lane of a step's maximum alone takes its next; the weights come from the terms
// of the softmax, left in shared memory, in place of the logits again; and with many tokens
// a warp takes several of them, so that what concerns the slots is done for all at once.
//
// Measured (us forward / backward): 65536 tokens, 8 of 128 experts, f32, softmax over all
// 20.0 (288 instructions a token; the bytes take 5.6) / 14.8 (155; 10.8); one token a warp 23.0 /
// 21.2; and with registers moved up in place of lists, two reductions a step and the logits read
// again 27 / 20.5.  The same with bf16, a bias and softmax over the chosen 18.2 / 7.3; 2 of 64 experts
// 9.8 / 9.5; 32768 tokens, 8 of 256 experts, bf16 16.8 / 7.3; 15762 tokens, 15 of 512 23.9 / 15.4;
// 2048 tokens, 8 of 64 2.4 / 1.9.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 128;
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

// Lane `lane` holds experts expert_of(lane, 0..V-1), increasing: V neighbours where lists
// of sorted keys are made (an earlier lane's experts lie before a later one's), else runs
// of W neighbours, 32 W apart.
template <int V, bool LISTS> struct Lanes {
    static constexpr int W = V < 4 ? V : 4;
    __device__ static __forceinline__ uint32_t expert_of(int lane, int j) {
        return static_cast<uint32_t>(LISTS ? lane * V + j : j / W * 32 * W + lane * W + j % W);
    }
};

template <typename T, int W> struct alignas(sizeof(T) * W) Run {
    T v[W];
};

// row[expert_of(lane, j)] for every j, `fill` past the row's E elements; vec: whole runs can be read
template <bool LISTS, typename T, int V>
__device__ __forceinline__ void load_lanes(const T *row, uint32_t E, int lane, bool vec, float fill, float (&out)[V]) {
    constexpr int W = Lanes<V, false>::W;
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        const uint32_t e = Lanes<V, LISTS>::expert_of(lane, c * W);
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

// row[expert_of(lane, j)] = v[j], in shared memory
template <bool LISTS, int V> __device__ __forceinline__ void store_lanes(float *row, int lane, const float (&v)[V]) {
    constexpr int W = Lanes<V, false>::W;
#pragma unroll
    for (int c = 0; c < V / W; ++c) {
        Run<float, W> r;
#pragma unroll
        for (int i = 0; i < W; ++i) r.v[i] = v[c * W + i];
        *reinterpret_cast<Run<float, W> *>(row + Lanes<V, LISTS>::expert_of(lane, c * W)) = r;
    }
}

// Keys of a token's scores (b: the bias); l becomes -inf for experts that are not live.
template <int V>
__device__ __forceinline__ void keys_of(float (&l)[V], const float (&b)[V], uint32_t (&key)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        key[j] = score_key(l[j] + b[j]);
        if (key[j] == 0u) l[j] = neg_inf();
    }
}

// l becomes exp(l - max), 0 for experts that are not live; returns the lane's sum
template <int V> __device__ __forceinline__ float softmax_terms(float (&l)[V]) {
    float top = l[0], sum = 0.f;
#pragma unroll
    for (int j = 1; j < V; ++j) top = fmaxf(top, l[j]);
    top = warp_max(top);
    if (top == neg_inf()) top = 0.f;  // none is live: exp(-inf) is 0
#pragma unroll
    for (int j = 0; j < V; ++j) {
        l[j] = expf(l[j] - top);
        sum += l[j];
    }
    return sum;
}

// Sums of s[0 .. N-1] over the warp's lanes, sum n in the n-th group of 32 / N lanes.
template <int N> __device__ __forceinline__ float scatter_sum(float (&s)[N], int lane) {
#pragma unroll
    for (int half = N / 2, o = 16; half > 0; half /= 2, o /= 2) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = upper ? s[i + half] : s[i], send = upper ? s[i] : s[i + half];
            s[i] = keep + __shfl_xor_sync(kFull, send, o);
        }
    }
#pragma unroll
    for (int o = 16 / N; o > 0; o /= 2) s[0] += __shfl_xor_sync(kFull, s[0], o);
    return s[0];
}

template <int N> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = 16 / N; o > 0; o /= 2) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <int N> __device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = 16 / N; o > 0; o /= 2) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// slot[0 .. top_k - 1] of a token become its experts, best first; left alone where
// fewer are live.
template <int V>
__device__ __forceinline__ void select(const uint32_t (&key)[V], uint2 (*list)[32], uint32_t top_k, int lane,
                                       uint32_t *slot) {
    // the lane's keys in descending order; of equals the lowest expert comes first
    uint32_t rank[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rank[j] = 0u;
#pragma unroll
    for (int i = 1; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < i; ++j) {
            if (key[i] > key[j])
                ++rank[j];
            else
                ++rank[i];
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) list[rank[j]][lane] = make_uint2(key[j], Lanes<V, true>::expert_of(lane, j));
    // one step: the largest head wins, and its lane moves on
    const uint32_t before = (1u << lane) - 1u;
    const uint2 *head = &list[0][lane];
    uint2 h = *head;
#pragma unroll 8
    for (uint32_t s = 0; s < top_k; ++s) {
        const uint32_t most = __reduce_max_sync(kFull, h.x);
        // of equals the first lane's: a lane's experts lie before the next one's
        const bool equal = h.x == most && most != 0u;
        if ((__ballot_sync(kFull, equal) & before) == 0u && equal) {
            slot[s] = h.y;
            head += 32;
            h = *head;
        }
    }
    __syncwarp();
}

// The same by a look at all of a lane's experts in each step (with 8 experts a lane 29.7 us for
// 19.7 for 32768 tokens).
template <int V>
__device__ __forceinline__ void select_scan(uint32_t (&key)[V], uint32_t top_k, int lane, uint32_t *slot) {
    for (uint32_t s = 0; s < top_k; ++s) {
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
        const uint32_t own = static_cast<uint32_t>(Lanes<V, false>::expert_of(lane, 0)) + at / 4 * 128 + at % 4;
        const uint32_t e = __reduce_min_sync(kFull, best == most ? own : kFull);
        if (lane == 0) slot[s] = e;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (Lanes<V, false>::expert_of(lane, j) == e) key[j] = 0u;
    }
    __syncwarp();
}

// A warp takes N tokens; what is done for each slot is done for all of them at once,
// slot s of the n-th token in lane s of the n-th group of 32 / N lanes.
template <typename T, int V, int N, bool LISTS>
__global__ void __launch_bounds__(kThreads) moe_route_kernel(MoeRouteParams p) {
    constexpr int kGroup = 32 / N;
    __shared__ __align__(16) float rows[kWarps][N][32 * V];  // what the weights are made of
    __shared__ uint2 lists[LISTS ? kWarps : 1][LISTS ? V + 1 : 1][32];
    __shared__ uint32_t slots[kWarps][N][kGroup];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, own = lane / kGroup;
    const uint32_t t0 = (blockIdx.x * kWarps + warp) * N;
    grid_dep_begin();
    if (t0 >= p.m) return;
    float l[N][V], b[V], sums[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t t = min(t0 + n, p.m - 1);
        load_lanes<LISTS, T, V>(static_cast<const T *>(p.logits) + static_cast<int64_t>(t) * p.ld_logits, p.n_experts,
                                lane, p.logits_vec != 0, neg_inf(), l[n]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = 0.f;
    if (p.bias != nullptr) load_lanes<LISTS, float, V>(p.bias, p.n_experts, lane, p.bias_vec != 0, 0.f, b);
    slots[warp][own][lane % kGroup] = p.n_experts;
    if (LISTS) lists[warp][V][lane] = make_uint2(0u, 0u);
    __syncwarp();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t key[V];
        keys_of<V>(l[n], b, key);
        if (!p.selected) sums[n] = softmax_terms<V>(l[n]);
        store_lanes<LISTS, V>(rows[warp][n], lane, l[n]);
        if constexpr (LISTS)
            select<V>(key, lists[warp], p.top_k, lane, slots[warp][n]);
        else
            select_scan<V>(key, p.top_k, lane, slots[warp][n]);
    }

    const uint32_t id = slots[warp][own][lane % kGroup];
    const bool chosen = id < p.n_experts;
    float w = chosen ? rows[warp][own][id] : p.selected ? neg_inf() : 0.f, sum;
    if (!p.selected) {
        sum = scatter_sum<N>(sums, lane);
    } else {
        const float top = group_max<N>(w);
        w = chosen ? expf(w - top) : 0.f;
        sum = group_sum<N>(w);
    }
    const uint32_t t = t0 + own, s = lane % kGroup;
    if (s < p.top_k && t < p.m) {
        const int64_t r = static_cast<int64_t>(t) * p.top_k + s;
        p.ids[r] = id;
        p.weights[r] = chosen ? w / sum : 0.f;
    }
}

// The slots' gradients reach the lanes that own their experts through a row of
// shared memory for each token: V / W accesses instead of top_k * V comparisons.
// (32 registers with up to 4 experts a lane: 8.1 us for 7.0 with more; 65536 tokens of bf16)
template <typename T, int V, int N>
__global__ void __launch_bounds__(kThreads, V <= 4 ? 2048 / kThreads : 0) moe_route_backward_kernel(MoeRouteParams p) {
    constexpr int W = Lanes<V, false>::W, kGroup = 32 / N;
    __shared__ __align__(16) float rows[kWarps][N][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, own = lane / kGroup;
    const uint32_t t0 = (blockIdx.x * kWarps + warp) * N;
    grid_dep_begin();
    if (t0 >= p.m) return;
    // slot s of the n-th token in lane s of the n-th group
    const uint32_t slot = lane % kGroup;
    uint32_t id = p.n_experts;
    float w = 0.f, d = 0.f;
    if (slot < p.top_k && t0 + own < p.m) {
        const int64_t r = static_cast<int64_t>(t0 + own) * p.top_k + slot;
        id = p.ids[r];
        if (id < p.n_experts) {
            w = p.weights[r];
            d = p.d_weights[r];
        }
    }
    static_assert(N * V <= 32, "a bit for each expert of a lane");
    float l[N][V], sums[N];
    uint32_t dead = 0u;  // experts that are not live
    if (!p.selected) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t t = min(t0 + n, p.m - 1);
            const T *row = static_cast<const T *>(p.logits) + static_cast<int64_t>(t) * p.ld_logits;
            load_lanes<false, T, V>(row, p.n_experts, lane, p.logits_vec != 0, neg_inf(), l[n]);
        }
    }
    float zeros[V];
#pragma unroll
    for (int j = 0; j < V; ++j) zeros[j] = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) store_lanes<false, V>(rows[warp][n], lane, zeros);
    const float dot = group_sum<N>(w * d);
    __syncwarp();
    if (id < p.n_experts) rows[warp][own][id] = p.selected ? w * (d - dot) : d;
    __syncwarp();
    if (!p.selected) {
        float b[V];
#pragma unroll
        for (int j = 0; j < V; ++j) b[j] = 0.f;
        if (p.bias != nullptr) load_lanes<false, float, V>(p.bias, p.n_experts, lane, p.bias_vec != 0, 0.f, b);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint32_t key[V];
            keys_of<V>(l[n], b, key);
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (key[j] == 0u) dead |= 1u << (n * V + j);
            sums[n] = softmax_terms<V>(l[n]);
        }
    }
    const float inv = p.selected ? 1.f : 1.f / scatter_sum<N>(sums, lane);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float dot_n = __shfl_sync(kFull, dot, n * kGroup), inv_n = __shfl_sync(kFull, inv, n * kGroup);
        if (t0 + n >= p.m) break;
        T *row = static_cast<T *>(p.d_logits) + static_cast<int64_t>(t0 + n) * p.ld_d_logits;
#pragma unroll
        for (int c = 0; c < V / W; ++c) {
            const uint32_t e = Lanes<V, false>::expert_of(lane, c * W);
            const Run<float, W> r = *reinterpret_cast<const Run<float, W> *>(rows[warp][n] + e);
            float g[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if (p.selected)
                    g[i] = r.v[i];
                else
                    g[i] = dead >> (n * V + c * W + i) & 1u ? 0.f : l[n][c * W + i] * inv_n * (r.v[i] - dot_n);
            }
            if (p.d_logits_vec) {
                Run<T, W> out;
#pragma unroll
                for (int i = 0; i < W; ++i) out.v[i] = Elem<T>::from_f(g[i]);
                if (e < p.n_experts) *reinterpret_cast<Run<T, W> *>(row + e) = out;
            } else {
#pragma unroll
                for (int i = 0; i < W; ++i)
                    if (e + i < p.n_experts) row[e + i] = Elem<T>::from_f(g[i]);
            }
        }
    }
}

// whether rows ld elements apart, and E elements long, divide into aligned runs of W
bool runs_fit(const void *ptr, int64_t ld, uint32_t E, int W, int size) {
    return reinterpret_cast<uintptr_t>(ptr) % (W * size) == 0 && ld % W == 0 && E % W == 0;
}

template <typename T, int V, int N>
cudaError_t launch_n(bool backward, const MoeRouteParams &p, cudaStream_t s) {
    const unsigned grid = (p.m + kWarps * N - 1) / (kWarps * N);
    // Started early when there are many waves of blocks (128 experts, both ways, early and not: 65536
    // tokens 31.7 us and 32.6; 16384 16.0 and 12.5, as blocks that come early crowd a few SMs).
    const bool early = p.m >= 256u * static_cast<uint32_t>(device_sm_count());
    auto start = [&](void (*kernel)(MoeRouteParams)) {
        if (early) return launch_early(kernel, grid, kThreads, 0, s, p);
        kernel<<<grid, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    };
    if (backward) return start(moe_route_backward_kernel<T, V, N>);
    // Sorted lists with up to 8 experts a lane; with 16 they cost more than a look at all of them
    // in each step does until there are some steps (15762 tokens, 512 experts: 2 slots 20.7 us
    // and 13.8, 8 slots 21.9 and 26.8, 15 slots 23.8 and 42.4).
    if constexpr (V <= 8) return start(moe_route_kernel<T, V, N, true>);
    if constexpr (V == 16) {
        if (p.top_k > 5) return start(moe_route_kernel<T, V, N, true>);
    }
    if constexpr (V > 8) return start(moe_route_kernel<T, V, N, false>);
}

template <typename T, int V>
cudaError_t launch_v(bool backward, MoeRouteParams p, cudaStream_t s) {
    constexpr int W = Lanes<V, false>::W;
    p.logits_vec = runs_fit(p.logits, p.ld_logits, p.n_experts, W, sizeof(T));
    p.bias_vec = runs_fit(p.bias, W, p.n_experts, W, sizeof(float));
    p.d_logits_vec = runs_fit(p.d_logits, p.ld_d_logits, p.n_experts, W, sizeof(T));
    // Several tokens a warp, as long as their slots fit into its lanes and there are 64 tokens an
    // SM: 8 of 128 experts, four a warp and one, forward: 2048 tokens 3.6 and 2.4 us, 8192
    // 5.0 and 4.3, 16384 6.8 and 6.8 (backward 5.7 and 7.0), 65536 20.5 and 23.0.  8 of 256
    // experts, 32768 tokens: two a warp 17.1, one 19.7, four 17.8; 16 of 128 experts, 65536 tokens, two
    // 26.5 (backward 17.1), one 28.3 (21.5).
    if constexpr (V <= 8) {
        const bool many = p.m >= 64u * static_cast<uint32_t>(device_sm_count());
        if (V <= 4 && p.top_k <= 8 && many) return launch_n<T, V, 4>(backward, p, s);
        if (p.top_k <= 16 && many) return launch_n<T, V, 2>(backward, p, s);
    }
    return launch_n<T, V, 1>(backward, p, s);
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
