// moe_rows.cu -- rows of a mixture-of-experts layer into expert order and back:
// dispatch (copy), combine (weighted sum over a token's slots; with weights of 1
// the gradient of the dispatch) and the gradient of combine.
//
// Every kernel works in token order: a token's row is read or written once and
// its top_k rows in expert order are addressed through position.  Rows whose
// position is at or past *valid have no expert.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t valid_rows(const MoeRowsParams &p) {
    return p.valid != nullptr ? *p.valid : p.m * p.top_k;
}
__device__ __forceinline__ uint32_t place_of(const MoeRowsParams &p, uint32_t r) {
    return p.position != nullptr ? p.position[r] : r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) moe_dispatch_kernel(MoeRowsParams p) {
    const uint32_t t = blockIdx.x, rows = p.m * p.top_k, valid = valid_rows(p);
    const T *x = static_cast<const T *>(p.tok_in) + static_cast<int64_t>(t) * p.ld_tok_in;
    for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
        const T v = x[i];
        for (uint32_t s = 0; s < p.top_k; ++s) {
            const uint32_t at = place_of(p, t * p.top_k + s);
            if (at < rows)
                static_cast<T *>(p.row_out)[static_cast<int64_t>(at) * p.ld_row_out + i] =
                    at < valid ? v : Elem<T>::from_f(0.f);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) moe_combine_kernel(MoeRowsParams p) {
    const uint32_t t = blockIdx.x, rows = p.m * p.top_k, valid = min(valid_rows(p), rows);
    for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
        float acc = 0.f;
        for (uint32_t s = 0; s < p.top_k; ++s) {
            const uint32_t r = t * p.top_k + s, at = place_of(p, r);
            if (at >= valid) continue;
            const float v =
                Elem<T>::to_f(static_cast<const T *>(p.row_in)[static_cast<int64_t>(at) * p.ld_row_in + i]);
            acc = p.weights != nullptr ? fmaf(p.weights[r], v, acc) : acc + v;
        }
        static_cast<T *>(p.tok_out)[static_cast<int64_t>(t) * p.ld_tok_out + i] = Elem<T>::from_f(acc);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) moe_combine_backward_kernel(MoeRowsParams p) {
    __shared__ float part[kThreads / 32];
    const uint32_t t = blockIdx.x, rows = p.m * p.top_k, valid = valid_rows(p);
    const T *dy = static_cast<const T *>(p.tok_in) + static_cast<int64_t>(t) * p.ld_tok_in;
    for (uint32_t s = 0; s < p.top_k; ++s) {
        const uint32_t r = t * p.top_k + s, at = place_of(p, r);
        float dot = 0.f;
        if (at < rows) {
            const T *y = static_cast<const T *>(p.row_in) + static_cast<int64_t>(at) * p.ld_row_in;
            T *d = static_cast<T *>(p.row_out) + static_cast<int64_t>(at) * p.ld_row_out;
            const float w = p.weights[r];
            for (int64_t i = threadIdx.x; i < p.n; i += kThreads) {
                if (at < valid) {
                    const float g = Elem<T>::to_f(dy[i]);
                    dot = fmaf(g, Elem<T>::to_f(y[i]), dot);
                    d[i] = Elem<T>::from_f(w * g);
                } else {
                    d[i] = Elem<T>::from_f(0.f);
                }
            }
        }
        dot = warp_sum(dot);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            float sum = 0.f;
            for (int w = 0; w < kThreads / 32; ++w) sum += part[w];
            p.d_weights[r] = sum;
        }
        __syncthreads();
    }
}

}  // namespace

#define GBMM_LAUNCH_ROWS(kernel)                                                           \
    switch (dt) {                                                                          \
    case kF32: kernel<float><<<p.m, kThreads, 0, s>>>(p); return cudaGetLastError();       \
    case kF16: kernel<__half><<<p.m, kThreads, 0, s>>>(p); return cudaGetLastError();      \
    case kBF16: kernel<__nv_bfloat16><<<p.m, kThreads, 0, s>>>(p); return cudaGetLastError(); \
    default: return cudaErrorInvalidValue;                                                 \
    }

cudaError_t launch_moe_dispatch(int dt, const MoeRowsParams &p, cudaStream_t s) {
    GBMM_LAUNCH_ROWS(moe_dispatch_kernel)
}
cudaError_t launch_moe_combine(int dt, const MoeRowsParams &p, cudaStream_t s) { GBMM_LAUNCH_ROWS(moe_combine_kernel) }
cudaError_t launch_moe_combine_backward(int dt, const MoeRowsParams &p, cudaStream_t s) {
    GBMM_LAUNCH_ROWS(moe_combine_backward_kernel)
}

}  // namespace gbmm
