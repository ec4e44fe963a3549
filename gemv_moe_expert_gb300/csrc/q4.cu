// q4.cu -- matrix-vector products with 4-bit weights and group scales, dense or
// per expert id.
//
// One warp computes one output row j for one row of x: lanes stride over the
// packed bytes, the integer products of a group are scaled as they are summed.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_scale(const Q4Params &p, int64_t at) {
    switch (p.scale_dtype) {
    case kF32: return static_cast<const float *>(p.scales)[at];
    case kF16: return __half2float(static_cast<const __half *>(p.scales)[at]);
    default: return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.scales)[at]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) q4_kernel(Q4Params p) {
    const int lane = threadIdx.x & 31;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (j >= p.n) return;
    for (uint32_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        T *out = static_cast<T *>(p.out) + static_cast<int64_t>(r) * p.ldo + j;
        const uint32_t e = p.ids != nullptr ? p.ids[r] : 0u;
        float acc = 0.f;
        if (e < p.n_experts) {
            const uint8_t *q = p.q + static_cast<int64_t>(e) * p.expert_stride + j * p.ldq;
            const int64_t cell = (static_cast<int64_t>(e) * p.n + j) * p.groups;
            const T *x = static_cast<const T *>(p.x) + static_cast<int64_t>(r / p.top_k) * p.ldx +
                         static_cast<int64_t>(r % p.top_k) * p.x_slot_stride;
            for (int64_t i = lane; i < (p.k + 1) / 2; i += 32) {
                const int64_t g = 2 * i / p.group;
                const uint32_t b = q[i];
                const float z = p.zeros != nullptr ? static_cast<float>(p.zeros[cell + g]) : 8.f;
                float v = (static_cast<float>(b & 15u) - z) * Elem<T>::to_f(x[2 * i]);
                if (2 * i + 1 < p.k) v = fmaf(static_cast<float>(b >> 4) - z, Elem<T>::to_f(x[2 * i + 1]), v);
                acc = fmaf(load_scale(p, cell + g), v, acc);
            }
        }
        acc = warp_sum(acc);
        if (lane == 0) *out = Elem<T>::from_f(acc);
    }
}

template <typename T>
cudaError_t launch_t(const Q4Params &p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.n + kThreads / 32 - 1) / (kThreads / 32)),
                    p.rows < 65535u ? p.rows : 65535u);
    q4_kernel<T><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_q4(int dt, const Q4Params &p, cudaStream_t s) {
    switch (dt) {
    case kF32: return launch_t<float>(p, s);
    case kF16: return launch_t<__half>(p, s);
    case kBF16: return launch_t<__nv_bfloat16>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gbmm
