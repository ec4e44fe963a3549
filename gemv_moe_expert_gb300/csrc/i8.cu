// i8.cu -- rows of values to 8-bit codes with a scale each, and the product of
// such codes for few rows, c[i, j] = (sum_x a[i, x] b[j, x]) scale_a[i] scale_b[j],
// the sum in 32-bit integers.
#include "device_common.cuh"

namespace gbmm {

namespace {

bool rows_on(const void *p, int64_t ld_bytes, int unit) {
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && ld_bytes % unit == 0;
}

// ---------------------------------------------------------------------------
// quantisation: scale = max |x| * f32(1 / 127), code = the integer nearest to x / scale, ties to even
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The integer nearest to x / s for |x| <= 127 s (1 + 2^-22), ties to even.  rint(x * inv) is that
// integer or, next to the middle of two, its neighbour; the remainder x - n s is exact in one fma (it
// is a multiple of the smaller of x's and s's last places and below s), and says which.
__device__ __forceinline__ int nearest_code(float x, float s, float inv) {
    float n = rintf(s < 1e-30f ? x / s : x * inv);
    const float r = fmaf(-n, s, x), twice = 2.f * fabsf(r);
    if (twice > s || (twice == s && (static_cast<int>(n) & 1))) n += r > 0.f ? 1.f : -1.f;
    return static_cast<int>(fminf(fmaxf(n, -127.f), 127.f));
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantizeParams p) {
    constexpr int kN = Elem<T>::kVec;
    __shared__ uint32_t warp_max[8];
    const int64_t i = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + i * p.ldx;
    int8_t *q = p.q + i * p.ldq;
    // infinities and NaN are above every finite value in the order of the absolute value's bits
    uint32_t most = 0;
    int64_t at = threadIdx.x * kN;
    if (kVec) {
        for (; at + kN <= p.k; at += 256 * kN) {
            float v[kN];
            unpack16<T>(ld_cached16(x + at), v);
#pragma unroll
            for (int e = 0; e < kN; ++e) most = max(most, abs_bits(v[e]));
        }
        for (int e = 0; e < kN && at + e < p.k; ++e) most = max(most, abs_bits(Elem<T>::to_f(x[at + e])));
    } else {
        for (int64_t c = threadIdx.x; c < p.k; c += 256) most = max(most, abs_bits(Elem<T>::to_f(x[c])));
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) most = max(most, warp_max[w]);
    const bool finite = most < 0x7f800000u;
    const float s = finite ? __uint_as_float(most) * (1.f / 127.f) : __uint_as_float(0x7fc00000u);
    if (threadIdx.x == 0) p.scale[i] = s;
    const bool live = finite && s > 0.f;
    const float inv = 1.f / s;
    if (kVec) {
        for (at = threadIdx.x * kN; at < p.k; at += 256 * kN) {
            if (at + kN <= p.k) {
                float v[kN];
                unpack16<T>(ld_cached16(x + at), v);
                uint32_t w[kN / 4];
#pragma unroll
                for (int g = 0; g < kN / 4; ++g) {
                    w[g] = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[g] |= (static_cast<uint32_t>(live ? nearest_code(v[4 * g + e], s, inv) : 0) & 255u) << (8 * e);
                }
                if constexpr (kN == 8) *reinterpret_cast<uint2 *>(q + at) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint32_t *>(q + at) = w[0];
            } else {
                for (int e = 0; at + e < p.k; ++e)
                    q[at + e] = static_cast<int8_t>(live ? nearest_code(Elem<T>::to_f(x[at + e]), s, inv) : 0);
            }
        }
    } else {
        for (int64_t c = threadIdx.x; c < p.k; c += 256)
            q[c] = static_cast<int8_t>(live ? nearest_code(Elem<T>::to_f(x[c]), s, inv) : 0);
    }
}

template <typename T>
cudaError_t quantize_t(const QuantizeParams &p, cudaStream_t s) {
    const bool vec = rows_on(p.x, p.ldx * static_cast<int64_t>(sizeof(T)), 16) && rows_on(p.q, p.ldq, Elem<T>::kVec);
    if (vec) quantize_kernel<T, true><<<static_cast<unsigned>(p.m), 256, 0, s>>>(p);
    else quantize_kernel<T, false><<<static_cast<unsigned>(p.m), 256, 0, s>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// the product for few rows: a warp takes kR columns j and kM rows i, its lanes divide k
// ---------------------------------------------------------------------------

constexpr int kDotWarps = 4;
constexpr int kR = 2;

template <typename T, int kM, int kUnit>
__global__ void __launch_bounds__(32 * kDotWarps) gemm_i8_dot_kernel(const GemmI8Params p) {
    const int lane = threadIdx.x & 31;
    const int64_t j0 = (static_cast<int64_t>(blockIdx.x) * kDotWarps + (threadIdx.x >> 5)) * kR;
    if (j0 >= p.n) return;
    const int8_t *b[kR];
#pragma unroll
    for (int c = 0; c < kR; ++c) b[c] = p.b + min(j0 + c, p.n - 1) * p.ldb;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.y) * kM; i0 < p.m; i0 += static_cast<int64_t>(gridDim.y) * kM) {
        const int8_t *a = p.a + i0 * p.lda;
        int acc[kM][kR];
#pragma unroll
        for (int r = 0; r < kM; ++r)
#pragma unroll
            for (int c = 0; c < kR; ++c) acc[r][c] = 0;
        int64_t at = lane * kUnit;
        if (kUnit == 16) {
            constexpr int kU = 4;
            for (; at + (kU - 1) * 512 + 16 <= p.k; at += kU * 512) {
                uint4 w[kU][kR];
#pragma unroll
                for (int q = 0; q < kU; ++q)
#pragma unroll
                    for (int c = 0; c < kR; ++c) w[q][c] = ld_stream16(b[c] + at + q * 512);
#pragma unroll
                for (int q = 0; q < kU; ++q)
#pragma unroll
                    for (int r = 0; r < kM; ++r) {
                        if (i0 + r >= p.m) break;
                        const uint4 v = ld_cached16(a + r * p.lda + at + q * 512);
#pragma unroll
                        for (int c = 0; c < kR; ++c) {
                            acc[r][c] = __dp4a(static_cast<int>(w[q][c].x), static_cast<int>(v.x), acc[r][c]);
                            acc[r][c] = __dp4a(static_cast<int>(w[q][c].y), static_cast<int>(v.y), acc[r][c]);
                            acc[r][c] = __dp4a(static_cast<int>(w[q][c].z), static_cast<int>(v.z), acc[r][c]);
                            acc[r][c] = __dp4a(static_cast<int>(w[q][c].w), static_cast<int>(v.w), acc[r][c]);
                        }
                    }
            }
        }
        if (kUnit >= 4) {
            for (; at + kUnit <= p.k; at += 32 * kUnit)
#pragma unroll
                for (int g = 0; g < kUnit; g += 4) {
                    int w[kR];
#pragma unroll
                    for (int c = 0; c < kR; ++c) w[c] = *reinterpret_cast<const int *>(b[c] + at + g);
#pragma unroll
                    for (int r = 0; r < kM; ++r) {
                        if (i0 + r >= p.m) break;
                        const int v = *reinterpret_cast<const int *>(a + r * p.lda + at + g);
#pragma unroll
                        for (int c = 0; c < kR; ++c) acc[r][c] = __dp4a(w[c], v, acc[r][c]);
                    }
                }
        }
        // what is left of a row: less than a unit (one lane), or all of it where rows start anywhere
        for (; at < p.k; at += 32 * kUnit)
            for (int e = 0; e < kUnit && at + e < p.k; ++e) {
#pragma unroll
                for (int r = 0; r < kM; ++r) {
                    if (i0 + r >= p.m) break;
                    const int v = a[r * p.lda + at + e];
#pragma unroll
                    for (int c = 0; c < kR; ++c) acc[r][c] += v * static_cast<int>(b[c][at + e]);
                }
            }
#pragma unroll
        for (int r = 0; r < kM; ++r)
#pragma unroll
            for (int c = 0; c < kR; ++c) acc[r][c] = __reduce_add_sync(0xffffffffu, acc[r][c]);
#pragma unroll
        for (int r = 0; r < kM; ++r)
#pragma unroll
            for (int c = 0; c < kR; ++c) {
                if (lane != r * kR + c || i0 + r >= p.m || j0 + c >= p.n) continue;
                const float sa = p.scale_a != nullptr ? p.scale_a[i0 + r] : 1.f;
                const float sb = p.scale_b != nullptr ? p.scale_b[j0 + c] : 1.f;
                static_cast<T *>(p.c)[(i0 + r) * p.ldc + j0 + c] =
                    Elem<T>::from_f(static_cast<float>(acc[r][c]) * sa * sb);
            }
    }
}

template <typename T, int kM>
cudaError_t dot_m(const GemmI8Params &p, cudaStream_t s) {
    const int64_t across = (p.n + kDotWarps * kR - 1) / (kDotWarps * kR), down = (p.m + kM - 1) / kM;
    const dim3 grid(static_cast<unsigned>(across), static_cast<unsigned>(down < 65535 ? down : 65535));
    if (rows_on(p.a, p.lda, 16) && rows_on(p.b, p.ldb, 16))
        gemm_i8_dot_kernel<T, kM, 16><<<grid, 32 * kDotWarps, 0, s>>>(p);
    else if (rows_on(p.a, p.lda, 4) && rows_on(p.b, p.ldb, 4))
        gemm_i8_dot_kernel<T, kM, 4><<<grid, 32 * kDotWarps, 0, s>>>(p);
    else
        gemm_i8_dot_kernel<T, kM, 1><<<grid, 32 * kDotWarps, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dot_t(const GemmI8Params &p, cudaStream_t s) {
    if (p.m == 1) return dot_m<T, 1>(p, s);
    if (p.m == 2) return dot_m<T, 2>(p, s);
    if (p.m <= 4) return dot_m<T, 4>(p, s);
    return dot_m<T, 8>(p, s);
}

}  // namespace

cudaError_t launch_quantize_i8(int dt, const QuantizeParams &p, cudaStream_t s) {
    switch (dt) {
    case kF32: return quantize_t<float>(p, s);
    case kF16: return quantize_t<__half>(p, s);
    case kBF16: return quantize_t<__nv_bfloat16>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gemm_i8_dot(int dt, const GemmI8Params &p, cudaStream_t s) {
    switch (dt) {
    case kF32: return dot_t<float>(p, s);
    case kF16: return dot_t<__half>(p, s);
    case kBF16: return dot_t<__nv_bfloat16>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gbmm
