// i8.cu -- rows of values to 8-bit codes with a scale each, and the product of
// such codes for few rows, c[i, j] = (sum_x a[i, x] b[j, x]) scale_a[i] scale_b[j],
// the sum in 32-bit integers.
#include "device_common.cuh"

namespace gbmm {

namespace {

template <typename T> struct Pair;
template <> struct Pair<__half> { using type = __half2; };
template <> struct Pair<__nv_bfloat16> { using type = __nv_bfloat162; };

// ---------------------------------------------------------------------------
// quantisation: scale = max |x| * f32(1 / 127), code = the integer nearest to x / scale, ties to even
//
// A row is read once, into registers, by 32 or 256 threads (more for rows that these do not hold; a row longer than
// 1024 threads hold is read again).  8192 x 11008 bf16: 45 us, 6.0 TB/s; 63 us while a value within 2^-12 of a
// middle, one of 2000, sent its thread to work all of its codes out exactly.  Bound by HBM, 3 bytes an element of 16 bits, so what each element costs
// in instructions matters: fma(x, 1 / scale, 1.5 * 2^23) leaves the code in its low byte, and the distance to it tells
// whether the quotient may lie on the other side of a middle; only such a thread works its codes out exactly.
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The integer nearest to x / s for |x| <= 127 s (1 + 2^-22), ties to even.  rint(x / s) in f32 is that
// integer or, next to the middle of two, its neighbour; the remainder x - n s is exact in one fma (it
// is a multiple of the smaller of x's and s's last places and below s), and says which.
__device__ __forceinline__ int nearest_code(float x, float s) {
    float n = rintf(x / s);
    const float r = fmaf(-n, s, x), twice = 2.f * fabsf(r);
    if (twice > s || (twice == s && (static_cast<int>(n) & 1))) n += r > 0.f ? 1.f : -1.f;
    return static_cast<int>(fminf(fmaxf(n, -127.f), 127.f));
}

// What a row's scale gives: inv = 1 / scale; live: false where every code is 0 (scale 0 or NaN); exact: true for scales
// below 1e-30, far above the 3e-39 below which 1 / scale leaves f32's range: no inv there, every code is worked out exactly.
struct RowScale {
    float s, inv;
    bool live, exact;
};
__device__ __forceinline__ RowScale row_scale(uint32_t most) {
    RowScale r;
    // infinities and NaN are above every finite value in the order of the absolute value's bits
    const bool finite = most < 0x7f800000u;
    r.s = finite ? __uint_as_float(most) * (1.f / 127.f) : __uint_as_float(0x7fc00000u);
    r.live = finite && r.s > 0.f;
    r.exact = r.live && r.s < 1e-30f;
    r.inv = r.live && !r.exact ? 1.f / r.s : 0.f;
    return r;
}

// Codes of four values of a live row, one a byte.  x * inv is off by 3 * 2^-24 of itself, 2^-15.3 at most: a quotient
// that is further than 2^-15 from a middle is rounded to the side that it lies on.  far: the largest distance from
// a code so far; above kNear some code has to be worked out exactly (6 values in 100000).
constexpr float kNear = 0.5f - 0x1p-15f;
__device__ __forceinline__ uint32_t codes4(const float *v, float inv, float &far) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: what is added to it is rounded to an integer
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float t = fmaf(v[e], inv, kMagic);
        far = fmaxf(far, fabsf(fmaf(v[e], inv, kMagic - t)));
        w[e] = __float_as_uint(t);
    }
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

template <int kT>
__device__ __forceinline__ uint32_t row_max(uint32_t most) {
    most = __reduce_max_sync(0xffffffffu, most);
    if (kT > 32) {
        __shared__ uint32_t warp_max[32];
        const int lane = threadIdx.x & 31;
        if (lane == 0) warp_max[threadIdx.x >> 5] = most;
        __syncthreads();
        most = __reduce_max_sync(0xffffffffu, warp_max[lane % (kT / 32)]);
    }
    return most;
}

// the largest absolute value of a piece, as bits of an f32; a NaN gives a NaN
template <typename T>
__device__ __forceinline__ uint32_t piece_max(const uint4 &v) {
    if constexpr (sizeof(T) == 4) {
        return max(max(v.x & 0x7fffffffu, v.y & 0x7fffffffu), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
    } else {
        using T2 = typename Pair<T>::type;
        const T2 *h = reinterpret_cast<const T2 *>(&v);
        const T2 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
        return max(abs_bits(Elem<T>::to_f(m.x)), abs_bits(Elem<T>::to_f(m.y)));
    }
}

// writes the codes of a piece; true if some of them have to be worked out exactly
template <typename T>
__device__ __forceinline__ bool store_codes(const uint4 &v, const RowScale &r, int8_t *q) {
    constexpr int kN = Elem<T>::kVec;
    float f[kN], far = 0.f;
    unpack16<T>(v, f);
    if constexpr (kN == 8) *reinterpret_cast<uint2 *>(q) = make_uint2(codes4(f, r.inv, far), codes4(f + 4, r.inv, far));
    else *reinterpret_cast<uint32_t *>(q) = codes4(f, r.inv, far);
    return far > kNear || r.exact;
}

// the codes of n values, worked out exactly
template <typename T>
__device__ __noinline__ void exact_codes(const T *x, int8_t *q, int n, float s) {
    for (int e = 0; e < n; ++e) q[e] = static_cast<int8_t>(nearest_code(Elem<T>::to_f(x[e]), s));
}

// kT threads a row, kP pieces of 16 bytes a thread; kP == 0: any length, read twice
template <typename T, int kT, int kP>
__global__ void __launch_bounds__(kT < 256 ? 256 : kT, kT <= 256 && kP <= 6 ? 5 : kT == 512 ? 2 : 1) quantize_kernel(const QuantizeParams p) {
    constexpr int kN = Elem<T>::kVec;
    grid_dep_begin();
    const int64_t i = kT < 256 ? static_cast<int64_t>(blockIdx.x) * (256 / kT) + threadIdx.x / kT : blockIdx.x;
    if (kT == 32 && i >= p.m) return;
    const int t = threadIdx.x % kT;
    const T *x = static_cast<const T *>(p.x) + i * p.ldx;
    int8_t *q = p.q + i * p.ldq;
    const int64_t pieces = p.k / kN;
    // the last, partial piece belongs to one thread
    const int rest = static_cast<int>(p.k % kN);
    const bool has_rest = rest != 0 && t == static_cast<int>(pieces % kT);
    uint32_t most = 0;
    if (has_rest)
        for (int e = 0; e < rest; ++e) most = max(most, abs_bits(Elem<T>::to_f(x[pieces * kN + e])));
    uint4 v[kP > 0 ? kP : 1];
    if constexpr (kP > 0) {
#pragma unroll
        for (int c = 0; c < kP; ++c) {
            const int64_t at = t + c * kT;
            v[c] = at < pieces ? ld_stream16(x + at * kN) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < kP; ++c) most = max(most, piece_max<T>(v[c]));
    } else {
#pragma unroll 4
        for (int64_t at = t; at < pieces; at += kT) most = max(most, piece_max<T>(ld_cached16(x + at * kN)));
    }
    const RowScale r = row_scale(row_max<kT>(most));
    if (t == 0) p.scale[i] = r.s;
    if constexpr (kP > 0) {
        uint32_t redo = 0;
#pragma unroll
        for (int c = 0; c < kP; ++c) {
            const int64_t at = t + c * kT;
            if (!r.live) v[c] = make_uint4(0, 0, 0, 0);  // no NaN or infinity
            if (at < pieces && store_codes<T>(v[c], r, q + at * kN)) redo |= 1u << c;
        }
        for (; redo != 0; redo &= redo - 1) {
            const int64_t at = (t + (__ffs(redo) - 1) * kT) * kN;
            exact_codes<T>(x + at, q + at, kN, r.s);
        }
    } else {
        for (int64_t at = t; at < pieces; at += kT) {
            const uint4 w = r.live ? ld_cached16(x + at * kN) : make_uint4(0, 0, 0, 0);
            if (store_codes<T>(w, r, q + at * kN)) exact_codes<T>(x + at * kN, q + at * kN, kN, r.s);
        }
    }
    if (has_rest)
        for (int e = 0; e < rest; ++e) {
            const int64_t at = pieces * kN + e;
            q[at] = static_cast<int8_t>(r.live ? nearest_code(Elem<T>::to_f(x[at]), r.s) : 0);
        }
}

// rows that start anywhere: one element an access, eight in flight
template <typename T>
__global__ void __launch_bounds__(256) quantize_any_kernel(const QuantizeParams p) {
    grid_dep_begin();
    const int64_t i = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + i * p.ldx;
    int8_t *q = p.q + i * p.ldq;
    uint32_t most = 0;
#pragma unroll 8
    for (int64_t c = threadIdx.x; c < p.k; c += 256) most = max(most, abs_bits(Elem<T>::to_f(x[c])));
    const RowScale r = row_scale(row_max<256>(most));
    if (threadIdx.x == 0) p.scale[i] = r.s;
    for (int64_t c = threadIdx.x; c < p.k; c += 8 * 256) {
        float v[8], far = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = r.live && c + 256 * e < p.k ? Elem<T>::to_f(x[c + 256 * e]) : 0.f;
        const uint32_t w[2] = {codes4(v, r.inv, far), codes4(v + 4, r.inv, far)};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + 256 * e < p.k) q[c + 256 * e] = static_cast<int8_t>(w[e / 4] >> (8 * (e % 4)));
        if (far > kNear || r.exact)
            for (int64_t at = c; at < c + 8 * 256 && at < p.k; at += 256) exact_codes<T>(x + at, q + at, 1, r.s);
    }
}

template <typename T, int kT, int kP>
cudaError_t quantize_p(const QuantizeParams &p, cudaStream_t s) {
    const int64_t blocks = kT < 256 ? (p.m + 256 / kT - 1) / (256 / kT) : p.m;
    return launch_early(quantize_kernel<T, kT, kP>, dim3(static_cast<unsigned>(blocks)), dim3(kT < 256 ? 256 : kT), 0, s, p);
}

template <typename T>
cudaError_t quantize_t(const QuantizeParams &p, cudaStream_t s) {
    if (!rows_on(p.x, p.ldx * static_cast<int64_t>(sizeof(T)), 16) || !rows_on(p.q, p.ldq, Elem<T>::kVec))
        return launch_early(quantize_any_kernel<T>, dim3(static_cast<unsigned>(p.m)), dim3(256), 0, s, p);
    const int64_t pieces = p.k / Elem<T>::kVec;
    if (pieces <= 64) return quantize_p<T, 32, 2>(p, s);
    if (pieces <= 256) return quantize_p<T, 256, 1>(p, s);
    if (pieces <= 512) return quantize_p<T, 256, 2>(p, s);
    if (pieces <= 1024) return quantize_p<T, 256, 4>(p, s);
    if (pieces <= 1536) return quantize_p<T, 256, 6>(p, s);
    if (pieces <= 2048) return quantize_p<T, 256, 8>(p, s);
    if (pieces <= 3584) return quantize_p<T, 512, 7>(p, s);
    if (pieces <= 4096) return quantize_p<T, 512, 8>(p, s);
    if (pieces <= 8192) return quantize_p<T, 1024, 8>(p, s);
    return quantize_p<T, 1024, 0>(p, s);
}

// ---------------------------------------------------------------------------
// the product for few rows: a warp takes a column j and kM rows i, its lanes divide k.  Bound by reading b: a lane
// asks for kU units of its column before it uses the first.  A unit is 16 or 4 bytes where all rows allow that;
// rows that start anywhere are read as the aligned words around each group of four, shifted into place.
// ---------------------------------------------------------------------------

constexpr int kDotWarps = 4;

// the four codes at row + 4 g; the row has k codes, and what lies past them counts as 0
__device__ __forceinline__ uint32_t any4(const int8_t *row, int64_t g, int64_t k) {
    if (4 * g >= k) return 0;
    const int8_t *at = row + 4 * g;
    const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 3u);
    const uint32_t *word = reinterpret_cast<const uint32_t *>(at - shift);
    if (g > 0 && 4 * g + 8 <= k) return __funnelshift_r(__ldg(word), __ldg(word + 1), 8 * shift);
    uint32_t v = 0;  // at a row's ends only its own bytes are read
    for (int e = 0; e < 4; ++e)
        if (4 * g + e < k) v |= static_cast<uint32_t>(static_cast<uint8_t>(at[e])) << (8 * e);
    return v;
}

template <int kUnit> struct Codes;
template <> struct Codes<16> {
    uint4 v;
    __device__ __forceinline__ int dot(const Codes &o, int s) const {
        s = __dp4a(static_cast<int>(v.x), static_cast<int>(o.v.x), s);
        s = __dp4a(static_cast<int>(v.y), static_cast<int>(o.v.y), s);
        s = __dp4a(static_cast<int>(v.z), static_cast<int>(o.v.z), s);
        return __dp4a(static_cast<int>(v.w), static_cast<int>(o.v.w), s);
    }
    static __device__ __forceinline__ Codes stream(const int8_t *row, int64_t u, int64_t) { return {ld_stream16(row + 16 * u)}; }
    static __device__ __forceinline__ Codes cached(const int8_t *row, int64_t u, int64_t) { return {ld_cached16(row + 16 * u)}; }
};
template <> struct Codes<4> {
    uint32_t v;
    __device__ __forceinline__ int dot(const Codes &o, int s) const {
        return __dp4a(static_cast<int>(v), static_cast<int>(o.v), s);
    }
    static __device__ __forceinline__ Codes stream(const int8_t *row, int64_t u, int64_t) { return cached(row, u, 0); }
    static __device__ __forceinline__ Codes cached(const int8_t *row, int64_t u, int64_t) {
        return {__ldg(reinterpret_cast<const uint32_t *>(row) + u)};
    }
};
template <> struct Codes<1> {
    uint32_t v;
    __device__ __forceinline__ int dot(const Codes &o, int s) const {
        return __dp4a(static_cast<int>(v), static_cast<int>(o.v), s);
    }
    static __device__ __forceinline__ Codes stream(const int8_t *row, int64_t u, int64_t k) { return {any4(row, u, k)}; }
    static __device__ __forceinline__ Codes cached(const int8_t *row, int64_t u, int64_t k) { return {any4(row, u, k)}; }
};

// kShare: warps of a column (1, or all of a block where there are few columns)
template <typename T, int kM, int kUnit, int kShare>
__global__ void __launch_bounds__(32 * kDotWarps) gemm_i8_dot_kernel(const GemmI8Params p) {
    constexpr int kU = kShare > 1 ? 2 : 4;
    constexpr int kLanes = 32 * kShare;
    constexpr int kStep = kUnit == 16 ? 16 : 4;  // codes in a unit
    grid_dep_begin();
    const int lane = threadIdx.x & 31, share = kShare > 1 ? threadIdx.x >> 5 : 0;
    const int64_t j = kShare > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kDotWarps + (threadIdx.x >> 5);
    if (j >= p.n) return;
    const int8_t *b = p.b + j * p.ldb;
    // units that are whole; rows that start anywhere have one more, whose missing codes are 0
    const int64_t units = kUnit == 1 ? (p.k + 3) / 4 : p.k / kStep;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.y) * kM; i0 < p.m; i0 += static_cast<int64_t>(gridDim.y) * kM) {
        const int8_t *a = p.a + i0 * p.lda;
        const int rows = static_cast<int>(p.m - i0 < kM ? p.m - i0 : kM);
        int acc[kM];
#pragma unroll
        for (int r = 0; r < kM; ++r) acc[r] = 0;
        for (int64_t at = 32 * share + lane; at < units; at += kU * kLanes) {
            Codes<kUnit> w[kU];
#pragma unroll
            for (int q = 0; q < kU; ++q) {
                if (at + q * kLanes >= units) break;
                w[q] = Codes<kUnit>::stream(b, at + q * kLanes, p.k);
            }
#pragma unroll
            for (int q = 0; q < kU; ++q) {
                if (at + q * kLanes >= units) break;
#pragma unroll
                for (int r = 0; r < kM; ++r) {
                    if (r >= rows) break;
                    acc[r] = w[q].dot(Codes<kUnit>::cached(a + r * p.lda, at + q * kLanes, p.k), acc[r]);
                }
            }
        }
        const int64_t e = units * kStep + lane;  // less than a unit is left at the end of a row
        if (share == 0 && e < p.k) {
#pragma unroll
            for (int r = 0; r < kM; ++r) {
                if (r >= rows) break;
                acc[r] += static_cast<int>(a[r * p.lda + e]) * static_cast<int>(b[e]);
            }
        }
#pragma unroll
        for (int r = 0; r < kM; ++r) acc[r] = __reduce_add_sync(0xffffffffu, acc[r]);
        if constexpr (kShare > 1) {
            __shared__ int part[kShare][kM];
            __syncthreads();  // what an earlier turn left has been read
            if (lane == 0) {
#pragma unroll
                for (int r = 0; r < kM; ++r) part[share][r] = acc[r];
            }
            __syncthreads();
            if (share != 0) continue;
#pragma unroll
            for (int q = 1; q < kShare; ++q)
#pragma unroll
                for (int r = 0; r < kM; ++r) acc[r] += part[q][r];
        }
#pragma unroll
        for (int r = 0; r < kM; ++r) {
            if (lane != r || r >= rows) continue;
            const float sa = p.scale_a != nullptr ? p.scale_a[i0 + r] : 1.f;
            const float sb = p.scale_b != nullptr ? p.scale_b[j] : 1.f;
            static_cast<T *>(p.c)[(i0 + r) * p.ldc + j] = Elem<T>::from_f(static_cast<float>(acc[r]) * sa * sb);
        }
    }
}

template <typename T, int kM, int kUnit>
cudaError_t dot_unit(const GemmI8Params &p, cudaStream_t s) {
    const int64_t down = (p.m + kM - 1) / kM;
    const dim3 block(32 * kDotWarps);
    const unsigned y = static_cast<unsigned>(down < 65535 ? down : 65535);
    const int64_t apart = (p.n + kDotWarps - 1) / kDotWarps;
    // A block's four warps share a column once each lane has four units of it (or of several rows' sums) to add up:
    // 4096 columns of 11008 codes 9.2 against 10.2 us, 11008 of 4096 11.7 against 9.1.
    const int64_t units = p.k / (kUnit == 16 ? 16 : 4);
    if (units >= 16 * 32 || (p.m > 1 && units >= 4 * 32))
        return launch_early(gemm_i8_dot_kernel<T, kM, kUnit, kDotWarps>, dim3(static_cast<unsigned>(p.n), y), block, 0, s, p);
    return launch_early(gemm_i8_dot_kernel<T, kM, kUnit, 1>, dim3(static_cast<unsigned>(apart), y), block, 0, s, p);
}

template <typename T, int kM>
cudaError_t dot_m(const GemmI8Params &p, cudaStream_t s) {
    if (rows_on(p.a, p.lda, 16) && rows_on(p.b, p.ldb, 16)) return dot_unit<T, kM, 16>(p, s);
    if (rows_on(p.a, p.lda, 4) && rows_on(p.b, p.ldb, 4)) return dot_unit<T, kM, 4>(p, s);
    return dot_unit<T, kM, 1>(p, s);
}

template <typename T>
cudaError_t dot_t(const GemmI8Params &p, cudaStream_t s) {
    if (p.m == 1) return dot_m<T, 1>(p, s);
    if (p.m == 2) return dot_m<T, 2>(p, s);
    if (p.m <= 4) return dot_m<T, 4>(p, s);
    return dot_m<T, 8>(p, s);
}

// ---------------------------------------------------------------------------
// codes laid out again, as bytes or as f16; both operands of a product in one launch
// ---------------------------------------------------------------------------

// The codes of a row from column j0 on, 2048 for a warp: 16 a lane and access where rows allow it, else 4.
__device__ __forceinline__ void lay_out_part(const RepackParams &p, bool aligned, int64_t i, int64_t j0, int lane) {
    const int8_t *row = static_cast<const int8_t *>(p.src) + i * p.lds;
    if (aligned) {
        constexpr int kU = 4;
        uint4 v[kU];
#pragma unroll
        for (int q = 0; q < kU; ++q) {
            const int64_t j = j0 + 16 * (lane + 32 * q);
            if (j + 16 <= p.cols) v[q] = ld_stream16(row + j);
            else v[q] = make_uint4(any4(row, j / 4, p.cols), any4(row, j / 4 + 1, p.cols), any4(row, j / 4 + 2, p.cols),
                                   any4(row, j / 4 + 3, p.cols));
        }
#pragma unroll
        for (int q = 0; q < kU; ++q) {
            const int64_t j = j0 + 16 * (lane + 32 * q);
            if (j >= p.ldd) break;
            if (p.to_size == 1) {
                *reinterpret_cast<uint4 *>(static_cast<int8_t *>(p.dst) + i * p.ldd + j) = v[q];
                continue;
            }
            const uint2 w0 = codes_to_half(v[q].x), w1 = codes_to_half(v[q].y), w2 = codes_to_half(v[q].z),
                        w3 = codes_to_half(v[q].w);
            // one store of a whole sector: two of 16 bytes each wrote half of every sector twice
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             static_cast<uint16_t *>(p.dst) + i * p.ldd + j),
                         "r"(w0.x), "r"(w0.y), "r"(w1.x), "r"(w1.y), "r"(w2.x), "r"(w2.y), "r"(w3.x), "r"(w3.y)
                         : "memory");
        }
        return;
    }
    constexpr int kU = 8;
#pragma unroll 1
    for (int64_t j1 = j0; j1 < j0 + 2048 && j1 < p.ldd; j1 += 128 * kU) {
        uint32_t v[kU];
        shifted_words<1, kU>(reinterpret_cast<const uint8_t *>(row), j1 / 4, p.cols, lane, v);
#pragma unroll
        for (int q = 0; q < kU; ++q) {
            const int64_t j = j1 + 4 * (lane + 32 * q);
            if (j >= p.ldd) break;
            if (p.to_size == 1) *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(p.dst) + i * p.ldd + j) = v[q];
            else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.dst) + i * p.ldd + j) = codes_to_half(v[q]);
        }
    }
}

__global__ void __launch_bounds__(256) lay_out_codes_kernel(const RepackParams a, const RepackParams b, int a_aligned,
                                                            int b_aligned, int64_t parts) {
    grid_dep_begin();
    const int lane = threadIdx.x & 31;
    const int64_t items = (a.rows + b.rows) * parts, warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; at < items; at += warps) {
        const int64_t i = at / parts, j0 = (at - i * parts) * 2048;
        if (i < a.rows) lay_out_part(a, a_aligned, i, j0, lane);
        else lay_out_part(b, b_aligned, i - a.rows, j0, lane);
    }
}

}  // namespace

cudaError_t launch_lay_out_codes(const RepackParams &a, const RepackParams &b, cudaStream_t s) {
    const int64_t widest = a.ldd > b.ldd ? a.ldd : b.ldd, parts = (widest + 2047) / 2048;
    const int64_t blocks = ((a.rows + b.rows) * parts + 7) / 8, most = 16LL * device_sm_count();
    if (blocks == 0) return cudaSuccess;
    return launch_early(lay_out_codes_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, s, a,
                        b, static_cast<int>(rows_on(a.src, a.lds, 16)), static_cast<int>(rows_on(b.src, b.lds, 16)), parts);
}

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
