// gated.cu -- the gated projection h = act(x Wg^T) * (x Wu^T) on the FFMA pipe,
// the gradients of its two projections, and rows laid out again for TMA.
//
// Every kernel here takes any strides and alignment; the tensor-core forms are
// chosen by the entry points (ffn_api.cu) where types and layouts allow.
#include "gated.cuh"

namespace gbmm {

namespace {

constexpr int kLanes = 32;

// N consecutive elements starting at p as f32; `whole`: one access, else the first `left`
template <typename T, int N>
__device__ __forceinline__ void load_f(const T *p, bool whole, int64_t left, float (&v)[N]) {
    static_assert(N * sizeof(T) == 16 || N * sizeof(T) == 8, "one 8- or 16-byte access");
    if (whole) {
        T t[N];
        if (N * sizeof(T) == 16) *reinterpret_cast<uint4 *>(t) = *reinterpret_cast<const uint4 *>(p);
        else *reinterpret_cast<uint2 *>(t) = *reinterpret_cast<const uint2 *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = Elem<T>::to_f(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < left ? Elem<T>::to_f(p[i]) : 0.f;
    }
}
template <typename T, int N>
__device__ __forceinline__ void store_f(T *p, bool whole, int64_t left, const float (&v)[N]) {
    T t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = Elem<T>::from_f(v[i]);
    if (whole) {
        if (N * sizeof(T) == 16) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(t);
        else *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(t);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = t[i];
    }
}

// ---------------------------------------------------------------------------
// few rows: one warp computes column j of both projections for kM rows of x.  Bound by reading the weights: a lane
// asks for kU units of both weight rows before it uses the first.  A unit is the widest access (16 to 2 bytes) that
// every row allows.
// ---------------------------------------------------------------------------

constexpr int kDotWarps = 4;

template <int kBytes>
struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <typename T, typename R>
__device__ __forceinline__ void unpack(const R &raw, float (&v)[sizeof(R) / sizeof(T)]) {
    if constexpr (sizeof(R) == 16) {
        unpack16<T>(raw, v);
    } else {
        T t[sizeof(R) / sizeof(T)];
        memcpy(t, &raw, sizeof(R));
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(R) / sizeof(T)); ++i) v[i] = Elem<T>::to_f(t[i]);
    }
}
template <typename R>
__device__ __forceinline__ R load_weights(const void *p) {
    if constexpr (sizeof(R) == 16) return ld_stream16(p);
    else return __ldg(static_cast<const R *>(p));
}

template <typename T, int kM, int kBytes>
__global__ void __launch_bounds__(32 * kDotWarps) gated_rowdot_kernel(const GatedParams p) {
    using R = typename Raw<kBytes>::type;
    constexpr int kN = kBytes / sizeof(T);
    constexpr int kU = kBytes == 16 && kM > 2 ? 4 : 8;
    grid_dep_begin();
    const int lane = threadIdx.x & 31;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kDotWarps + (threadIdx.x >> 5);
    if (j >= p.n) return;
    const T *x = static_cast<const T *>(p.x);
    const T *w0 = static_cast<const T *>(p.w[0]) + j * p.ldw;
    const T *w1 = static_cast<const T *>(p.w[1]) + j * p.ldw;
    const int rows = static_cast<int>(p.m);
    float g[kM], u[kM];
#pragma unroll
    for (int r = 0; r < kM; ++r) g[r] = u[r] = 0.f;
    const int64_t units = p.k / kN;
    for (int64_t at = lane; at < units; at += kU * kLanes) {
        R a[kU], b[kU];
#pragma unroll
        for (int q = 0; q < kU; ++q) {
            if (at + q * kLanes >= units) break;
            a[q] = load_weights<R>(w0 + (at + q * kLanes) * kN);
            b[q] = load_weights<R>(w1 + (at + q * kLanes) * kN);
        }
#pragma unroll
        for (int q = 0; q < kU; ++q) {
            if (at + q * kLanes >= units) break;
            float wa[kN], wb[kN], xv[kN];
            unpack<T>(a[q], wa);
            unpack<T>(b[q], wb);
#pragma unroll
            for (int r = 0; r < kM; ++r) {
                if (r >= rows) break;
                unpack<T>(__ldg(reinterpret_cast<const R *>(x + r * p.ldx + (at + q * kLanes) * kN)), xv);
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    g[r] = fmaf(wa[e], xv[e], g[r]);
                    u[r] = fmaf(wb[e], xv[e], u[r]);
                }
            }
        }
    }
    // less than a unit is left at the end of a row
    const int64_t e = units * kN + lane;
    if (e < p.k) {
        const float wa = Elem<T>::to_f(w0[e]), wb = Elem<T>::to_f(w1[e]);
#pragma unroll
        for (int r = 0; r < kM; ++r) {
            if (r >= rows) break;
            const float xv = Elem<T>::to_f(x[r * p.ldx + e]);
            g[r] = fmaf(wa, xv, g[r]);
            u[r] = fmaf(wb, xv, u[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kM; ++r) {
        g[r] = warp_sum(g[r]);
        u[r] = warp_sum(u[r]);
    }
#pragma unroll
    for (int r = 0; r < kM; ++r) {
        if (lane != r || r >= rows) continue;
        static_cast<T *>(p.h)[r * p.ldh + j] = Elem<T>::from_f(gate_act(p.act, g[r]) * u[r]);
        if (p.saved[0] != nullptr) {
            static_cast<T *>(p.saved[0])[r * p.ld_saved + j] = Elem<T>::from_f(g[r]);
            static_cast<T *>(p.saved[1])[r * p.ld_saved + j] = Elem<T>::from_f(u[r]);
        }
    }
}

bool rows_on(const void *p, int64_t ld_bytes, int unit) {
    return reinterpret_cast<uintptr_t>(p) % unit == 0 && ld_bytes % unit == 0;
}
bool rows16(const void *p, int64_t ld, size_t size) { return rows_on(p, ld * static_cast<int64_t>(size), 16); }

template <typename T, int kM>
cudaError_t rowdot_m(const GatedParams &p, cudaStream_t s) {
    constexpr int64_t size = sizeof(T);
    int unit = 16;
    while (unit > size && !(rows_on(p.x, p.ldx * size, unit) && rows_on(p.w[0], p.ldw * size, unit) &&
                            rows_on(p.w[1], p.ldw * size, unit)))
        unit /= 2;
    const dim3 grid(static_cast<unsigned>((p.n + kDotWarps - 1) / kDotWarps)), block(32 * kDotWarps);
    switch (unit) {
    case 16: return launch_early(gated_rowdot_kernel<T, kM, 16>, grid, block, 0, s, p);
    case 8: return launch_early(gated_rowdot_kernel<T, kM, 8>, grid, block, 0, s, p);
    case 4: return launch_early(gated_rowdot_kernel<T, kM, 4>, grid, block, 0, s, p);
    default:
        if constexpr (sizeof(T) == 2) return launch_early(gated_rowdot_kernel<T, kM, 2>, grid, block, 0, s, p);
        return cudaErrorInvalidValue;
    }
}

template <typename T>
cudaError_t rowdot_t(const GatedParams &p, cudaStream_t s) {
    if (p.m == 1) return rowdot_m<T, 1>(p, s);
    if (p.m == 2) return rowdot_m<T, 2>(p, s);
    if (p.m <= 4) return rowdot_m<T, 4>(p, s);
    return p.m <= 8 ? rowdot_m<T, 8>(p, s) : cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// FFMA tiles: two products in one pass.  kSum == false: c0 = a b0^T and c1 = a b1^T, b [n, k]
// (the gated projection, two accumulators); kSum == true: c = a0 b0 + a1 b1, b [k, n] (the
// gradient of x, one accumulator, the contraction over both sources).  16 kTM x 16 kTN tiles,
// kTM x kTN outputs a thread and product, 16 deep, the next step's loads in registers while the
// current one is multiplied.
// ---------------------------------------------------------------------------

struct TileArgs {
    const void *a[2], *b[2];
    int64_t m, n, k, lda, ldb;
    int32_t a_vec, b_vec;  // groups of four elements can be read in one access
    int64_t tiles_n;
};

constexpr int kTK = 16;

template <typename T, bool kSum, int kTM, int kTN>
struct TileProduct {
    static constexpr int kBM = 16 * kTM, kBN = 16 * kTN, kProducts = kSum ? 1 : 2;
    static constexpr int kAPieces = kBM * kTK / 4, kBPieces = kBN * kTK / 4;
    static constexpr int kA = (kAPieces + 255) / 256, kB = (kBPieces + 255) / 256;
    struct Smem {
        float a[2][kTK][kBM + 4];
        float b[2][kProducts][kTK][kBN + 4];
    };
    float acc[kProducts][kTM][kTN];

    __device__ __forceinline__ void run(const TileArgs &t, int64_t m0, int64_t n0, Smem &sm) {
        const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
#pragma unroll
        for (int q = 0; q < kProducts; ++q)
#pragma unroll
            for (int r = 0; r < kTM; ++r)
#pragma unroll
                for (int c = 0; c < kTN; ++c) acc[q][r][c] = 0.f;
        float ra[kA][4], rb[kProducts][kB][4];
        const int64_t steps1 = (t.k + kTK - 1) / kTK, steps = kSum ? 2 * steps1 : steps1;
        auto load = [&](int64_t step) {
            const int src = kSum && step >= steps1 ? 1 : 0;
            const int64_t k0 = (step - src * steps1) * kTK;
            const T *A = static_cast<const T *>(t.a[src]);
#pragma unroll
            for (int e = 0; e < kA; ++e) {  // piece: row q / 4, k 4 (q % 4)
                const int q = tid + 256 * e;
                const int64_t i = m0 + q / 4, x = k0 + 4 * (q % 4);
                const bool ok = (kAPieces % 256 == 0 || q < kAPieces) && i < t.m && x < t.k;
                load_part(A + i * t.lda + x, ok, t.a_vec, t.k - x, ra[e]);
            }
#pragma unroll
            for (int pr = 0; pr < kProducts; ++pr) {
                const T *B = static_cast<const T *>(t.b[kSum ? src : pr]);
#pragma unroll
                for (int e = 0; e < kB; ++e) {
                    const int q = tid + 256 * e;
                    const bool in = kBPieces % 256 == 0 || q < kBPieces;
                    if (kSum) {  // piece: k q / (kBN / 4), columns 4 (q % (kBN / 4))
                        const int64_t y = k0 + q / (kBN / 4), j = n0 + 4 * (q % (kBN / 4));
                        load_part(B + y * t.ldb + j, in && y < t.k && j < t.n, t.b_vec, t.n - j, rb[pr][e]);
                    } else {     // piece: column q / 4, k 4 (q % 4)
                        const int64_t j = n0 + q / 4, x = k0 + 4 * (q % 4);
                        load_part(B + j * t.ldb + x, in && j < t.n && x < t.k, t.b_vec, t.k - x, rb[pr][e]);
                    }
                }
            }
        };
        auto store = [&](int buf) {
#pragma unroll
            for (int e = 0; e < kA; ++e) {
                const int q = tid + 256 * e;
                if (kAPieces % 256 == 0 || q < kAPieces)
#pragma unroll
                    for (int c = 0; c < 4; ++c) sm.a[buf][4 * (q % 4) + c][q / 4] = ra[e][c];
            }
#pragma unroll
            for (int pr = 0; pr < kProducts; ++pr)
#pragma unroll
                for (int e = 0; e < kB; ++e) {
                    const int q = tid + 256 * e;
                    if (kBPieces % 256 != 0 && q >= kBPieces) continue;
                    if (kSum) {
                        *reinterpret_cast<float4 *>(&sm.b[buf][pr][q / (kBN / 4)][4 * (q % (kBN / 4))]) =
                            make_float4(rb[pr][e][0], rb[pr][e][1], rb[pr][e][2], rb[pr][e][3]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c) sm.b[buf][pr][4 * (q % 4) + c][q / 4] = rb[pr][e][c];
                    }
                }
        };
        if (steps > 0) {
            load(0);
            store(0);
        }
        __syncthreads();
        int cur = 0;
        for (int64_t step = 0; step < steps; ++step) {
            const bool more = step + 1 < steps;
            if (more) load(step + 1);
#pragma unroll
            for (int kk = 0; kk < kTK; ++kk) {
                float av[kTM], bv[kProducts][kTN];
                fetch<kTM>(sm.a[cur][kk], ty, av);
#pragma unroll
                for (int pr = 0; pr < kProducts; ++pr) fetch<kTN>(sm.b[cur][pr][kk], tx, bv[pr]);
#pragma unroll
                for (int pr = 0; pr < kProducts; ++pr)
#pragma unroll
                    for (int r = 0; r < kTM; ++r)
#pragma unroll
                        for (int c = 0; c < kTN; ++c) acc[pr][r][c] = fmaf(av[r], bv[pr][c], acc[pr][r][c]);
            }
            if (more) store(cur ^ 1);
            __syncthreads();
            cur ^= 1;
        }
    }

    // thread t's outputs of a dimension: kN == 2: 2t..; 4: 4t..; 8: 4t.. and 64 + 4t..
    template <int kN>
    static __device__ __forceinline__ int place(int t, int i) {
        return kN == 2 ? 2 * t + i : (i < 4 ? 4 * t + i : 60 + 4 * t + i);
    }
    template <int kN>
    static __device__ __forceinline__ void fetch(const float *row, int t, float (&v)[kN]) {
        if constexpr (kN == 2) {
            const float2 f = *reinterpret_cast<const float2 *>(row + 2 * t);
            v[0] = f.x, v[1] = f.y;
        } else {
#pragma unroll
            for (int h = 0; h < kN / 4; ++h) {
                const float4 f = *reinterpret_cast<const float4 *>(row + 64 * h + 4 * t);
                v[4 * h] = f.x, v[4 * h + 1] = f.y, v[4 * h + 2] = f.z, v[4 * h + 3] = f.w;
            }
        }
    }
    static __device__ __forceinline__ void load_part(const T *p, bool ok, bool vec, int64_t left, float (&v)[4]) {
        if (!ok) {
            v[0] = v[1] = v[2] = v[3] = 0.f;
        } else if (vec && left >= 4) {
            if constexpr (sizeof(T) == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(p);
                v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(p);
                const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = Elem<T>::to_f(e[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = i < left ? Elem<T>::to_f(p[i]) : 0.f;
        }
    }
};

template <typename T, int kTM, int kTN>
__global__ void __launch_bounds__(256, 2) gated_simt_kernel(const TileArgs t, const GatedParams p) {
    using Tile = TileProduct<T, false, kTM, kTN>;
    __shared__ __align__(16) typename Tile::Smem sm;
    Tile tile;
    const int64_t m0 = blockIdx.x / t.tiles_n * Tile::kBM, n0 = blockIdx.x % t.tiles_n * Tile::kBN;
    tile.run(t, m0, n0, sm);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int r = 0; r < kTM; ++r) {
        const int64_t i = m0 + Tile::template place<kTM>(ty, r);
        if (i >= p.m) continue;
#pragma unroll
        for (int c = 0; c < kTN; ++c) {
            const int64_t j = n0 + Tile::template place<kTN>(tx, c);
            if (j >= p.n) continue;
            const float g = tile.acc[0][r][c], u = tile.acc[1][r][c];
            static_cast<T *>(p.h)[i * p.ldh + j] = Elem<T>::from_f(gate_act(p.act, g) * u);
            if (p.saved[0] != nullptr) {
                static_cast<T *>(p.saved[0])[i * p.ld_saved + j] = Elem<T>::from_f(g);
                static_cast<T *>(p.saved[1])[i * p.ld_saved + j] = Elem<T>::from_f(u);
            }
        }
    }
}

template <typename T, int kTM, int kTN>
__global__ void __launch_bounds__(256, 2) sum_gemm_simt_kernel(const TileArgs t, T *c_out, int64_t ldc) {
    using Tile = TileProduct<T, true, kTM, kTN>;
    __shared__ __align__(16) typename Tile::Smem sm;
    Tile tile;
    const int64_t m0 = blockIdx.x / t.tiles_n * Tile::kBM, n0 = blockIdx.x % t.tiles_n * Tile::kBN;
    tile.run(t, m0, n0, sm);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int r = 0; r < kTM; ++r) {
        const int64_t i = m0 + Tile::template place<kTM>(ty, r);
        if (i >= t.m) continue;
#pragma unroll
        for (int c = 0; c < kTN; ++c) {
            const int64_t j = n0 + Tile::template place<kTN>(tx, c);
            if (j < t.n) c_out[i * ldc + j] = Elem<T>::from_f(tile.acc[0][r][c]);
        }
    }
}

bool groups_of_4(const void *p, int64_t ld, size_t size) {
    return reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && ld % 4 == 0;
}

// blocks for tiles of bm x bn, and the tiles across a row; 0 where there are too many
unsigned tile_grid(int64_t m, int64_t n, int bm, int bn, TileArgs *t) {
    t->tiles_n = (n + bn - 1) / bn;
    const unsigned __int128 blocks = static_cast<unsigned __int128>((m + bm - 1) / bm) * t->tiles_n;
    return blocks > INT32_MAX ? 0 : static_cast<unsigned>(blocks);
}

template <typename T>
cudaError_t gated_simt_t(const GatedParams &p, cudaStream_t s) {
    TileArgs t{{p.x, p.x}, {p.w[0], p.w[1]}, p.m, p.n, p.k, p.ldx, p.ldw, 0, 0, 0};
    t.a_vec = groups_of_4(p.x, p.ldx, sizeof(T));
    t.b_vec = groups_of_4(p.w[0], p.ldw, sizeof(T)) && groups_of_4(p.w[1], p.ldw, sizeof(T));
    unsigned blocks = tile_grid(p.m, p.n, 128, 64, &t);
    if (blocks >= static_cast<unsigned>(device_sm_count())) {
        gated_simt_kernel<T, 8, 4><<<blocks, 256, 0, s>>>(t, p);
    } else {
        blocks = tile_grid(p.m, p.n, 64, 32, &t);
        if (blocks == 0) return cudaErrorInvalidConfiguration;
        gated_simt_kernel<T, 4, 2><<<blocks, 256, 0, s>>>(t, p);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t sum_gemm_t(const SumGemmParams &p, cudaStream_t s) {
    TileArgs t{{p.a[0], p.a[1]}, {p.b[0], p.b[1]}, p.m, p.n, p.k, p.lda, p.ldb, 0, 0, 0};
    t.a_vec = groups_of_4(p.a[0], p.lda, sizeof(T)) && groups_of_4(p.a[1], p.lda, sizeof(T));
    t.b_vec = groups_of_4(p.b[0], p.ldb, sizeof(T)) && groups_of_4(p.b[1], p.ldb, sizeof(T));
    unsigned blocks = tile_grid(p.m, p.n, 128, 128, &t);
    if (blocks >= static_cast<unsigned>(device_sm_count())) {
        sum_gemm_simt_kernel<T, 8, 8><<<blocks, 256, 0, s>>>(t, static_cast<T *>(p.c), p.ldc);
    } else {
        blocks = tile_grid(p.m, p.n, 64, 64, &t);
        if (blocks == 0) return cudaErrorInvalidConfiguration;
        sum_gemm_simt_kernel<T, 4, 4><<<blocks, 256, 0, s>>>(t, static_cast<T *>(p.c), p.ldc);
    }
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// d_gate = d_h * up * act'(gate), d_up = d_h * act(gate): one pass, 16 bytes an access
// ---------------------------------------------------------------------------

template <typename T>
__global__ void __launch_bounds__(256) gated_grad_kernel(const GatedGradParams p, int vec) {
    constexpr int kN = Elem<T>::kVec;
    grid_dep_begin();
    const int64_t pieces = (p.n + kN - 1) / kN, total = pieces * p.m;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < total;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t i = at / pieces, j = (at - i * pieces) * kN, left = p.n - j;
        const bool whole = vec && left >= kN;
        float g[kN], u[kN], d[kN], dg[kN], du[kN];
        load_f<T, kN>(static_cast<const T *>(p.gate) + i * p.ld_saved + j, whole, left, g);
        load_f<T, kN>(static_cast<const T *>(p.up) + i * p.ld_saved + j, whole, left, u);
        load_f<T, kN>(static_cast<const T *>(p.d_h) + i * p.ld_dh + j, whole, left, d);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
            float slope;
            const float a = gate_act_slope(p.act, g[e], &slope);
            dg[e] = d[e] * u[e] * slope;
            du[e] = d[e] * a;
        }
        store_f<T, kN>(static_cast<T *>(p.d[0]) + i * p.ldd + j, left >= kN, left, dg);
        store_f<T, kN>(static_cast<T *>(p.d[1]) + i * p.ldd + j, left >= kN, left, du);
    }
}

template <typename T>
cudaError_t gated_grad_t(const GatedGradParams &p, cudaStream_t s) {
    const int vec = rows16(p.gate, p.ld_saved, sizeof(T)) && rows16(p.up, p.ld_saved, sizeof(T)) &&
                    rows16(p.d_h, p.ld_dh, sizeof(T));
    const int64_t blocks = (p.m * ((p.n + Elem<T>::kVec - 1) / Elem<T>::kVec) + 255) / 256;
    const int64_t most = 16LL * device_sm_count();
    return launch_early(gated_grad_kernel<T>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, s,
                        p, vec);
}

// ---------------------------------------------------------------------------
// rows that TMA cannot read (or that hold 8-bit codes), written 16 bytes at a time into rows that
// it can
// ---------------------------------------------------------------------------

struct alignas(16) Halves {
    uint16_t v[8];
};

__device__ __forceinline__ uint16_t as_bits(uint16_t v) { return v; }
__device__ __forceinline__ uint16_t as_bits(int8_t v) { return __half_as_ushort(__int2half_rn(v)); }

template <typename S>
__global__ void __launch_bounds__(256) repack_kernel(const RepackParams p) {
    grid_dep_begin();
    const int64_t pieces = p.ldd / 8, total = pieces * p.rows;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < total;
         at += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t i = at / pieces, j = (at - i * pieces) * 8;
        const S *src = static_cast<const S *>(p.src) + i * p.lds + j;
        Halves h;
#pragma unroll
        for (int e = 0; e < 8; ++e) h.v[e] = j + e < p.cols ? as_bits(src[e]) : uint16_t{0};
        *reinterpret_cast<Halves *>(static_cast<uint16_t *>(p.dst) + i * p.ldd + j) = h;
    }
}

template <typename S>
cudaError_t repack_t(const RepackParams &p, cudaStream_t s) {
    const int64_t blocks = (p.rows * (p.ldd / 8) + 255) / 256, most = 16LL * device_sm_count();
    if (blocks == 0) return cudaSuccess;
    return launch_early(repack_kernel<S>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, s, p);
}

}  // namespace

#define GBMM_BY_TYPE(dt, call)                    \
    switch (dt) {                                 \
    case kF32: return call<float>(p, s);          \
    case kF16: return call<__half>(p, s);         \
    case kBF16: return call<__nv_bfloat16>(p, s); \
    default: return cudaErrorInvalidValue;        \
    }

cudaError_t launch_gated_rowdot(int dt, const GatedParams &p, cudaStream_t s) { GBMM_BY_TYPE(dt, rowdot_t) }
cudaError_t launch_gated_simt(int dt, const GatedParams &p, cudaStream_t s) { GBMM_BY_TYPE(dt, gated_simt_t) }
cudaError_t launch_gated_grad(int dt, const GatedGradParams &p, cudaStream_t s) { GBMM_BY_TYPE(dt, gated_grad_t) }
cudaError_t launch_sum_gemm_simt(int dt, const SumGemmParams &p, cudaStream_t s) { GBMM_BY_TYPE(dt, sum_gemm_t) }
cudaError_t launch_repack16(const RepackParams &p, cudaStream_t s) { return repack_t<uint16_t>(p, s); }
cudaError_t launch_codes_to_f16(const RepackParams &p, cudaStream_t s) { return repack_t<int8_t>(p, s); }

}  // namespace gbmm
