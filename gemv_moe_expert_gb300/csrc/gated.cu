// gated.cu -- the gated projection h = act(x Wg^T) * (x Wu^T) on the FFMA pipe,
// the gradients of its two projections, and rows laid out again for TMA.
//
// Every kernel here takes any strides and alignment; the tensor-core forms are
// chosen by the entry points (ffn_api.cu) where types and layouts allow.
#include <cooperative_groups.h>

#include <algorithm>

#include "gated.cuh"

namespace cg = cooperative_groups;

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

// Sums of N values over a warp: lanes trade halves of what they hold, so that N + log2(32 / N) exchanges do in place of
// 5 N.  v[0] of lane l is then the sum of value l / (32 / N).
template <int N>
__device__ __forceinline__ void reduce_scatter(float (&v)[N], int lane) {
    int bit = kLanes / 2;
#pragma unroll
    for (int half = N / 2; half >= 1; half /= 2, bit /= 2) {
        const bool high = (lane & bit) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = high ? v[half + i] : v[i], send = high ? v[i] : v[half + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    }
#pragma unroll
    for (; bit >= 1; bit /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
}

// kShare: warps of a column (1, or all of a block)
template <typename T, int kM, int kBytes, int kShare>
__global__ void __launch_bounds__(32 * kDotWarps) gated_rowdot_kernel(const GatedParams p) {
    using R = typename Raw<kBytes>::type;
    constexpr int kN = kBytes / sizeof(T);
    constexpr int kU = kShare > 1 ? 2 : 4;
    constexpr int kStep = kLanes * kShare;
    grid_dep_begin();
    const int lane = threadIdx.x & 31, share = kShare > 1 ? threadIdx.x >> 5 : 0;
    const int64_t j = kShare > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kDotWarps + (threadIdx.x >> 5);
    if (j >= p.n) return;
    const T *x = static_cast<const T *>(p.x);
    const T *w0 = static_cast<const T *>(p.w[0]) + j * p.ldw;
    const T *w1 = static_cast<const T *>(p.w[1]) + j * p.ldw;
    const int rows = static_cast<int>(p.m);
    float g[kM], u[kM];
#pragma unroll
    for (int r = 0; r < kM; ++r) g[r] = u[r] = 0.f;
    const int64_t units = p.k / kN;
    for (int64_t at = share * kLanes + lane; at < units; at += kU * kStep) {
        R a[kU], b[kU];
#pragma unroll
        for (int q = 0; q < kU; ++q) {
            if (at + q * kStep >= units) break;
            a[q] = load_weights<R>(w0 + (at + q * kStep) * kN);
            b[q] = load_weights<R>(w1 + (at + q * kStep) * kN);
        }
#pragma unroll
        for (int q = 0; q < kU; ++q) {
            if (at + q * kStep >= units) break;
            float wa[kN], wb[kN], xv[kN];
            unpack<T>(a[q], wa);
            unpack<T>(b[q], wb);
#pragma unroll
            for (int r = 0; r < kM; ++r) {
                if (r >= rows) break;
                unpack<T>(__ldg(reinterpret_cast<const R *>(x + r * p.ldx + (at + q * kStep) * kN)), xv);
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
    if (share == 0 && e < p.k) {
        const float wa = Elem<T>::to_f(w0[e]), wb = Elem<T>::to_f(w1[e]);
#pragma unroll
        for (int r = 0; r < kM; ++r) {
            if (r >= rows) break;
            const float xv = Elem<T>::to_f(x[r * p.ldx + e]);
            g[r] = fmaf(wa, xv, g[r]);
            u[r] = fmaf(wb, xv, u[r]);
        }
    }
    float v[2 * kM];
#pragma unroll
    for (int r = 0; r < kM; ++r) v[r] = g[r], v[kM + r] = u[r];
    // value `which` of the warp's sums lies in v[0]; the gate's kM values come before the up projection's
    reduce_scatter<2 * kM>(v, lane);
    constexpr int kCopies = kLanes / (2 * kM);  // lanes that hold the same value
    const int which = lane / kCopies;
    float sum = v[0];
    if constexpr (kShare > 1) {
        __shared__ float part[kShare][2 * kM];
        if (lane % kCopies == 0) part[share][which] = sum;
        __syncthreads();
        if (share != 0) return;
        sum = 0.f;
#pragma unroll
        for (int q = 0; q < kShare; ++q) sum += part[q][which];
    }
    const float other = __shfl_down_sync(0xffffffffu, sum, kM * kCopies);  // the up projection's value
    if (lane % kCopies == 0 && which < rows) {
        const int64_t r = which;
        if (which < kM) {
            static_cast<T *>(p.h)[r * p.ldh + j] = Elem<T>::from_f(gate_act(p.act, sum) * other);
            if (p.saved[0] != nullptr) {
                static_cast<T *>(p.saved[0])[r * p.ld_saved + j] = Elem<T>::from_f(sum);
                static_cast<T *>(p.saved[1])[r * p.ld_saved + j] = Elem<T>::from_f(other);
            }
        }
    }
}

bool rows16(const void *p, int64_t ld, size_t size) { return rows_on(p, ld * static_cast<int64_t>(size), 16); }

template <typename T, int kM, int kBytes>
cudaError_t rowdot_unit(const GatedParams &p, cudaStream_t s) {
    const dim3 block(32 * kDotWarps);
    // The block's four warps share a column once each lane has a unit of it: 11008 columns of 4096 bf16 values 26.9 us
    // against 29.1, 1408 of 2048 2.9 against 3.9.
    if (p.k / (kBytes / static_cast<int64_t>(sizeof(T))) >= kDotWarps * kLanes)
        return launch_early(gated_rowdot_kernel<T, kM, kBytes, kDotWarps>, dim3(static_cast<unsigned>(p.n)), block, 0, s, p);
    const dim3 grid(static_cast<unsigned>((p.n + kDotWarps - 1) / kDotWarps));
    return launch_early(gated_rowdot_kernel<T, kM, kBytes, 1>, grid, block, 0, s, p);
}

template <typename T, int kM>
cudaError_t rowdot_m(const GatedParams &p, cudaStream_t s) {
    constexpr int64_t size = sizeof(T);
    int unit = 16;
    while (unit > size && !(rows_on(p.x, p.ldx * size, unit) && rows_on(p.w[0], p.ldw * size, unit) &&
                            rows_on(p.w[1], p.ldw * size, unit)))
        unit /= 2;
    switch (unit) {
    case 16: return rowdot_unit<T, kM, 16>(p, s);
    case 8: return rowdot_unit<T, kM, 8>(p, s);
    case 4: return rowdot_unit<T, kM, 4>(p, s);
    default:
        if constexpr (sizeof(T) == 2) return rowdot_unit<T, kM, 2>(p, s);
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
// FFMA tiles: two products in one pass.
//   kGated  c0 = a b0^T, c1 = a b1^T    a [m, k], b [n, k]    the gated projection; two accumulators
//   kSum    c = a0 b0 + a1 b1           a [m, k], b [k, n]    the gradient of x; one accumulator, the contraction
//                                                             runs over the first source and then the second
//   kOuter  c0 = b0^T a, c1 = b1^T a    a [k, m], b [k, n]    the weights' gradients; two accumulators, rows of c
//                                                             along n
// 16 kTM x 16 kTN tiles, kTM x kTN outputs a thread and product, 16 deep, the next step's loads in registers while the
// current one is multiplied.  Two neighbouring outputs share an instruction (fma.rn.f32x2), which leaves issue slots
// for the shared-memory reads.
// ---------------------------------------------------------------------------

enum TileMode { kGated, kSum, kOuter };

struct TileArgs {
    const void *a[2], *b[2];
    int64_t m, n, k, lda, ldb;
    int32_t a_vec, b_vec;  // groups of four elements can be read in one access
    int64_t tiles_n;
    uint32_t parts = 1;    // CTAs that share a tile
    int32_t fold = 0;      // 1: a long contraction, the sums of kFold steps each are added up in shared memory
};

constexpr int kTK = 16;

// Steps of the contraction whose sums stay in one register.  Normal products summed one after the other end 4e-7 of the
// sum's own size off (rms) after 512, 1.2e-6 after 4096 and 3.3e-6 after 32768, the rounding of each addition growing with
// the sum so far; in runs of 512 whose sums are then added, 32768 stay at 5e-7.
constexpr int64_t kFold = 32;

__device__ __forceinline__ uint64_t both(float v) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(v));
    return d;
}
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ float half_of(uint64_t v, int i) {
    return __uint_as_float(static_cast<uint32_t>(i == 0 ? v : v >> 32));
}

template <typename T, int kMode, int kTM, int kTN>
struct TileProduct {
    static constexpr int kBM = 16 * kTM, kBN = 16 * kTN, kProducts = kMode == kSum ? 1 : 2;
    // operands whose rows run along k are transposed on their way into shared memory
    static constexpr bool kAK = kMode != kOuter, kBK = kMode == kGated;
    static constexpr int kAPieces = kBM * kTK / 4, kBPieces = kBN * kTK / 4;
    static constexpr int kA = (kAPieces + 255) / 256, kB = (kBPieces + 255) / 256;
    struct Smem {
        float a[2][kTK][kBM + 4];
        float b[2][kProducts][kTK][kBN + 4];
    };
    uint64_t acc[kProducts][kTM][kTN / 2];

    static constexpr uint32_t kFoldBytes = kProducts * kTM * kTN * 256 * sizeof(float);

    __device__ __forceinline__ float at(int pr, int r, int c) const { return half_of(acc[pr][r][c / 2], c & 1); }

    // adds what is stored to the sums (unless they are the first) and stores them again (unless they are the last); each
    // thread its own
    __device__ __forceinline__ void fold(uint64_t *sums, bool first, bool last) {
        int i = threadIdx.x;
#pragma unroll
        for (int pr = 0; pr < kProducts; ++pr)
#pragma unroll
            for (int r = 0; r < kTM; ++r)
#pragma unroll
                for (int c = 0; c < kTN / 2; ++c, i += 256) {
                    uint64_t &v = acc[pr][r][c];
                    if (!first) {
                        const uint64_t w = sums[i];
                        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
                    }
                    if (!last) {
                        sums[i] = v;
                        v = 0;
                    }
                }
    }

    // part of parts: the share of the contraction (kSum: of both sources) that this block takes
    __device__ __forceinline__ void run(const TileArgs &t, int64_t m0, int64_t n0, Smem &sm, int part = 0, int parts = 1) {
        extern __shared__ __align__(16) uint64_t sums[];
        bool folded = false;
        const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
        for (int q = 0; q < kProducts; ++q)
#pragma unroll
            for (int r = 0; r < kTM; ++r)
#pragma unroll
                for (int c = 0; c < kTN / 2; ++c) acc[q][r][c] = 0;
        float ra[kA][4], rb[kProducts][kB][4];
        const int64_t steps1 = (t.k + kTK - 1) / kTK, all = (kMode == kSum ? 2 : 1) * steps1;
        const int64_t begin = all * part / parts, end = all * (part + 1) / parts;
        auto load = [&](int64_t step) {
            const int64_t k0 = (kMode == kSum && step >= steps1 ? step - steps1 : step) * kTK;
            const int src = kMode == kSum && step >= steps1 ? 1 : 0;
            load_tile<kAK, kBM, kA>(static_cast<const T *>(src ? t.a[1] : t.a[0]), t.lda, m0, t.m, k0, t.k, t.a_vec, ra);
#pragma unroll
            for (int pr = 0; pr < kProducts; ++pr)
                load_tile<kBK, kBN, kB>(static_cast<const T *>((kMode == kSum ? src : pr) ? t.b[1] : t.b[0]), t.ldb, n0, t.n, k0, t.k,
                                        t.b_vec, rb[pr]);
        };
        auto store = [&](int buf) {
            store_tile<kAK, kBM, kA>(sm.a[buf], ra);
#pragma unroll
            for (int pr = 0; pr < kProducts; ++pr) store_tile<kBK, kBN, kB>(sm.b[buf][pr], rb[pr]);
        };
        if (begin < end) {
            load(begin);
            store(0);
        }
        __syncthreads();
        int cur = 0;
        for (int64_t step = begin; step < end; ++step) {
            const bool more = step + 1 < end;
            if (more) load(step + 1);
            // the next k's values are read while this one's are multiplied
            float av[2][kTM];
            uint64_t bv[2][kProducts][kTN / 2];
            fetch(sm, cur, 0, ty, tx, av[0], bv[0]);
#pragma unroll
            for (int kk = 0; kk < kTK; ++kk) {
                if (kk + 1 < kTK) fetch(sm, cur, kk + 1, ty, tx, av[(kk + 1) & 1], bv[(kk + 1) & 1]);
#pragma unroll
                for (int r = 0; r < kTM; ++r) {
                    const uint64_t a2 = both(av[kk & 1][r]);
#pragma unroll
                    for (int pr = 0; pr < kProducts; ++pr)
#pragma unroll
                        for (int c = 0; c < kTN / 2; ++c) fma2(acc[pr][r][c], a2, bv[kk & 1][pr][c]);
                }
            }
            if (more) store(cur ^ 1);
            if (t.fold && more && (step - begin + 1) % kFold == 0) {
                fold(sums, !folded, false);
                folded = true;
            }
            __syncthreads();
            cur ^= 1;
        }
        if (folded) fold(sums, false, true);
    }

    // The cluster's other CTAs hand their sums to the first one through shared memory, two rows a thread at a time;
    // it adds them in the order of their ranks.
    __device__ __forceinline__ void reduce_cluster(Smem &sm, int rank, int parts) {
        cg::cluster_group cluster = cg::this_cluster();
        uint64_t *mine = reinterpret_cast<uint64_t *>(&sm);
        static_assert(256 * kTN * sizeof(uint64_t) <= sizeof(Smem), "two rows a thread");
#pragma unroll
        for (int pr = 0; pr < kProducts; ++pr)
#pragma unroll
            for (int r = 0; r < kTM; r += 2) {
                if (rank != 0)
#pragma unroll
                    for (int e = 0; e < kTN; ++e)
                        mine[e * 256 + threadIdx.x] = acc[pr][r + e / (kTN / 2)][e % (kTN / 2)];
                cluster.sync();
                if (rank == 0)
                    for (int q = 1; q < parts; ++q) {
                        const uint64_t *other = cluster.map_shared_rank(mine, q);
#pragma unroll
                        for (int e = 0; e < kTN; ++e) {
                            uint64_t &v = acc[pr][r + e / (kTN / 2)][e % (kTN / 2)];
                            const uint64_t w = other[e * 256 + threadIdx.x];
                            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(w));
                        }
                    }
                cluster.sync();
            }
    }

    static __device__ __forceinline__ void fetch(const Smem &sm, int cur, int kk, int ty, int tx, float (&av)[kTM],
                                                 uint64_t (&bv)[kProducts][kTN / 2]) {
#pragma unroll
        for (int h = 0; h < kTM / 4; ++h) {
            const float4 f = *reinterpret_cast<const float4 *>(&sm.a[cur][kk][64 * h + 4 * ty]);
            av[4 * h] = f.x, av[4 * h + 1] = f.y, av[4 * h + 2] = f.z, av[4 * h + 3] = f.w;
        }
#pragma unroll
        for (int pr = 0; pr < kProducts; ++pr)
#pragma unroll
            for (int h = 0; h < kTN / 4; ++h) {
                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(&sm.b[cur][pr][kk][64 * h + 4 * tx]);
                bv[pr][2 * h] = f.x, bv[pr][2 * h + 1] = f.y;
            }
    }

    // where output i of thread t lies in its dimension: 4 t .., and 64 + 4 t .. from the fifth on
    static __device__ __forceinline__ int place(int t, int i) { return i < 4 ? 4 * t + i : 60 + 4 * t + i; }

    // Pieces of four elements along the rows: K-major (rows of kLong along k) piece q is row q / 4, k 4 (q % 4); else
    // k q / (kLong / 4), places 4 (q % (kLong / 4)).
    template <bool kKMajor, int kLong, int kPieces>
    static __device__ __forceinline__ void load_tile(const T *src, int64_t ld, int64_t o0, int64_t o_end, int64_t k0,
                                                     int64_t k_end, bool vec, float (&v)[kPieces][4]) {
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
            const int q = threadIdx.x + 256 * e;
            const bool in = kLong * kTK / 4 % 256 == 0 || q < kLong * kTK / 4;
            const int64_t o = o0 + (kKMajor ? q / 4 : 4 * (q % (kLong / 4)));
            const int64_t x = k0 + (kKMajor ? 4 * (q % 4) : q / (kLong / 4));
            load_part(src + (kKMajor ? o * ld + x : x * ld + o), in && o < o_end && x < k_end, vec,
                      kKMajor ? k_end - x : o_end - o, v[e]);
        }
    }
    template <bool kKMajor, int kLong, int kPieces>
    static __device__ __forceinline__ void store_tile(float (&dst)[kTK][kLong + 4], const float (&v)[kPieces][4]) {
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
            const int q = threadIdx.x + 256 * e;
            if (kLong * kTK / 4 % 256 != 0 && q >= kLong * kTK / 4) continue;
            if (kKMajor) {
#pragma unroll
                for (int c = 0; c < 4; ++c) dst[4 * (q % 4) + c][q / 4] = v[e][c];
            } else {
                *reinterpret_cast<float4 *>(&dst[q / (kLong / 4)][4 * (q % (kLong / 4))]) =
                    make_float4(v[e][0], v[e][1], v[e][2], v[e][3]);
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

// kSplit: a cluster of t.parts CTAs a tile, a share of the contraction each
template <typename T, int kTM, int kTN, bool kSplit>
__global__ void __launch_bounds__(256, 2) gated_simt_kernel(const TileArgs t, const GatedParams p) {
    using Tile = TileProduct<T, kGated, kTM, kTN>;
    __shared__ __align__(16) typename Tile::Smem sm;
    Tile tile;
    const unsigned parts = kSplit ? t.parts : 1, block = blockIdx.x / parts;
    const int64_t m0 = block / t.tiles_n * Tile::kBM, n0 = block % t.tiles_n * Tile::kBN;
    if constexpr (kSplit) {
        const int rank = static_cast<int>(blockIdx.x % parts);  // in the cluster, too
        tile.run(t, m0, n0, sm, rank, static_cast<int>(parts));
        tile.reduce_cluster(sm, rank, static_cast<int>(parts));
        if (rank != 0) return;
    } else {
        tile.run(t, m0, n0, sm);
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int r = 0; r < kTM; ++r) {
        const int64_t i = m0 + Tile::place(ty, r);
        if (i >= p.m) continue;
#pragma unroll
        for (int c = 0; c < kTN; ++c) {
            const int64_t j = n0 + Tile::place(tx, c);
            if (j >= p.n) continue;
            const float g = tile.at(0, r, c), u = tile.at(1, r, c);
            static_cast<T *>(p.h)[i * p.ldh + j] = Elem<T>::from_f(gate_act(p.act, g) * u);
            if (p.saved[0] != nullptr) {
                static_cast<T *>(p.saved[0])[i * p.ld_saved + j] = Elem<T>::from_f(g);
                static_cast<T *>(p.saved[1])[i * p.ld_saved + j] = Elem<T>::from_f(u);
            }
        }
    }
}

// One tile of the gradient of x.  kSplit: a cluster of `parts` CTAs a tile (two: one source each).
template <int kTM, int kTN, bool kSplit>
__device__ __forceinline__ void sum_tile(const TileArgs &t, float *out, int64_t ldc, int64_t block, int rank, int parts,
                                         typename TileProduct<float, kSum, kTM, kTN>::Smem &sm) {
    using Tile = TileProduct<float, kSum, kTM, kTN>;
    Tile tile;
    const int64_t m0 = block / t.tiles_n * Tile::kBM, n0 = block % t.tiles_n * Tile::kBN;
    if constexpr (kSplit) {
        tile.run(t, m0, n0, sm, rank, parts);
        tile.reduce_cluster(sm, rank, parts);
        if (rank != 0) return;
    } else {
        tile.run(t, m0, n0, sm);
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int r = 0; r < kTM; ++r) {
        const int64_t i = m0 + Tile::place(ty, r);
        if (i >= t.m) continue;
#pragma unroll
        for (int c = 0; c < kTN; ++c) {
            const int64_t j = n0 + Tile::place(tx, c);
            if (j < t.n) out[i * ldc + j] = tile.at(0, r, c);
        }
    }
}

// One tile of the gradients of the weights; here t.m runs along the columns of the outputs and t.n along their rows.
struct OuterOut {
    float *c[2];
    int64_t ldc;
    int32_t vec;
};
template <int kTM, int kTN, bool kSplit>
__device__ __forceinline__ void outer_tile(const TileArgs &t, const OuterOut &o, int64_t block, int rank, int parts,
                                           typename TileProduct<float, kOuter, kTM, kTN>::Smem &sm) {
    using Tile = TileProduct<float, kOuter, kTM, kTN>;
    Tile tile;
    const int64_t m0 = block / t.tiles_n * Tile::kBM, n0 = block % t.tiles_n * Tile::kBN;
    if constexpr (kSplit) {
        tile.run(t, m0, n0, sm, rank, parts);
        tile.reduce_cluster(sm, rank, parts);
        if (rank != 0) return;
    } else {
        tile.run(t, m0, n0, sm);
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int pr = 0; pr < 2; ++pr)
#pragma unroll
        for (int c = 0; c < kTN; ++c) {
            const int64_t row = n0 + Tile::place(tx, c);
            if (row >= t.n) continue;
            float *dst = (pr == 0 ? o.c[0] : o.c[1]) + row * o.ldc;
#pragma unroll
            for (int h = 0; h < kTM; h += 4) {
                const int64_t col = m0 + Tile::place(ty, h);
                if (o.vec && col + 4 <= t.m) {
                    *reinterpret_cast<float4 *>(dst + col) = make_float4(tile.at(pr, h, c), tile.at(pr, h + 1, c),
                                                                         tile.at(pr, h + 2, c), tile.at(pr, h + 3, c));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < t.m) dst[col + e] = tile.at(pr, h + e, c);
                }
            }
        }
}

// Both gradients in one grid, so that the tiles of one fill the places that the other's leave.  Clusters of `parts` divide
// the contraction of one tile (x_split, w_split) or take a tile each; the side with the longer chains comes first.
struct GradGrid {
    unsigned x_tiles, w_tiles, parts, x_blocks, w_blocks;
    int32_t x_split, w_split, w_first;
};
template <int kXM, int kXN, int kWM, int kWN>
__global__ void __launch_bounds__(256, 2)
gradients_simt_kernel(const TileArgs tx, float *out, int64_t ldc, const TileArgs tw, const OuterOut o, const GradGrid g) {
    __shared__ __align__(16) union {
        typename TileProduct<float, kSum, kXM, kXN>::Smem x;
        typename TileProduct<float, kOuter, kWM, kWN>::Smem w;
    } sm;
    const unsigned first = g.w_first ? g.w_blocks : g.x_blocks;
    const bool is_x = (blockIdx.x < first) != (g.w_first != 0);
    const unsigned block = blockIdx.x < first ? blockIdx.x : blockIdx.x - first;
    const bool split = is_x ? g.x_split : g.w_split;
    const unsigned tile = split ? block / g.parts : block;
    const int rank = split ? static_cast<int>(block % g.parts) : 0, parts = static_cast<int>(g.parts);
    if (tile >= (is_x ? g.x_tiles : g.w_tiles)) return;
    if (is_x) {
        if (split) sum_tile<kXM, kXN, true>(tx, out, ldc, tile, rank, parts, sm.x);
        else sum_tile<kXM, kXN, false>(tx, out, ldc, tile, 0, 1, sm.x);
    } else {
        if (split) outer_tile<kWM, kWN, true>(tw, o, tile, rank, parts, sm.w);
        else outer_tile<kWM, kWN, false>(tw, o, tile, 0, 1, sm.w);
    }
}

// Not started early behind the kernel before it: blocks that take places as they come free gather on a few SMs, and a
// grid of about one block an SM then takes twice as long (512 x 1408 x 2048 gradients: 412 against 300 us).
// cluster: CTAs of a cluster; fold_bytes: the shared memory of sums of sums, 0 for short contractions.
template <typename... Params, typename... Args>
cudaError_t launch_whole(void (*kernel)(Params...), unsigned blocks, unsigned cluster, uint32_t fold_bytes, cudaStream_t s,
                         const Args &...args) {
    if (fold_bytes > 0) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(fold_bytes));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = fold_bytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// 1 where a contraction of k (of `sources`, divided over `parts`) is long: from one and a half runs
int32_t folds(int64_t k, int sources, int64_t parts) {
    return (k + kTK - 1) / kTK * sources / parts > kFold * 3 / 2;
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

// The ways to divide the tiles of both gradients: clusters of one to eight CTAs, either or both kinds divided.  Calls
// time(grid, steps of a block of x, of w) for each, and returns the grid of the least.
template <typename Time>
GradGrid least_grid(unsigned x_tiles, unsigned w_tiles, int64_t x_steps, int64_t w_steps, int64_t x_join, int64_t w_join,
                    int64_t *least, Time time) {
    GradGrid best{};
    *least = -1;
    for (unsigned parts = 1; parts <= 8; ++parts)
        for (int split = parts > 1 ? 1 : 0; split < (parts > 1 ? 4 : 1); ++split) {
            const int xs = split & 1, ws = split >> 1;
            if ((xs && x_tiles == 0) || (ws && w_tiles == 0)) continue;
            auto blocks = [&](unsigned tiles, int divided) {
                return divided ? static_cast<int64_t>(tiles) * parts
                               : (static_cast<int64_t>(tiles) + parts - 1) / parts * parts;
            };
            const int64_t xb = blocks(x_tiles, xs), wb = blocks(w_tiles, ws);
            if (xb + wb > INT32_MAX) continue;
            GradGrid g{x_tiles, w_tiles, parts, static_cast<unsigned>(xb), static_cast<unsigned>(wb), xs, ws, 0};
            const int64_t t = time(g, x_tiles == 0 ? 0 : xs ? (x_steps + parts - 1) / parts + x_join : x_steps,
                                   w_tiles == 0 ? 0 : ws ? (w_steps + parts - 1) / parts + w_join : w_steps);
            if (*least < 0 || t < *least) {
                *least = t;
                best = g;
            }
        }
    return best;
}

// Few tiles: what counts is the longest chain of steps (0.3 us each) of any block, the exchange in a cluster as kJoin
// steps.  Blocks beyond two an SM (an eighth fewer in large clusters, which lie within groups of 16 to 20 SMs) wait for a
// place, as long as an average one.  m x n x k 21 x 640 x 64: 13.9 us, and 57 undivided; 4000 x 128 x 256: 47 and 267;
// 256 x 512 x 512: 25 and 63.
GradGrid few_tiles_grid(unsigned x_tiles, unsigned w_tiles, int64_t x_steps, int64_t w_steps, int64_t sms) {
    constexpr int64_t kJoin = 8;
    int64_t least;
    return least_grid(x_tiles, w_tiles, x_steps, w_steps, kJoin, kJoin, &least, [&](GradGrid &g, int64_t xc, int64_t wc) {
        const int64_t places = (g.parts > 4 ? 14 : 16) * sms / 8;
        const int64_t count = static_cast<int64_t>(g.x_blocks) + g.w_blocks, all = g.x_blocks * xc + g.w_blocks * wc;
        g.w_first = wc > xc;
        return std::max(xc, wc) + (count > places ? all / count * ((count - 1) / places) : 0);
    });
}

// What a tile's step of the contraction takes of an SM in ns (8 to 16 tiles of one kind an SM), and the exchange in a
// cluster in such steps.
struct StepCost {
    int64_t x, w, x_join, w_join;
};
constexpr StepCost kLargeSteps{1577, 1394, 3, 4}, kSmallSteps{554, 819, 3, 5};

// Many tiles: the longer chains begin, one after the other on each SM (two at once take twice as long), and the others go
// wherever an SM is done first.  m x n x k, against pairs on the gradient of x and the weights' undivided behind it: 26 x
// 9664 x 384 107 us and 1008; 6605 x 192 x 320 105 and 699; 2346 x 892 x 686 307 and 522; 7297 x 256 x 2944 825 and 1762;
// 512 x 1408 x 2048, where the two are the same, 238.
GradGrid many_tiles_grid(unsigned x_tiles, unsigned w_tiles, int64_t x_steps, int64_t w_steps, const StepCost &cost,
                         int64_t sms, int64_t *least) {
    return least_grid(x_tiles, w_tiles, x_steps, w_steps, cost.x_join, cost.w_join, least,
                      [&](GradGrid &g, int64_t x_chain, int64_t w_chain) {
        // a block's time, with a step for its beginning and end
        const int64_t xc = x_tiles ? cost.x * (x_chain + 1) : 0, wc = w_tiles ? cost.w * (w_chain + 1) : 0;
        g.w_first = wc > xc;
        const int64_t count = static_cast<int64_t>(g.x_blocks) + g.w_blocks, n1 = g.w_first ? g.w_blocks : g.x_blocks;
        const int64_t n2 = count - n1, c1 = std::max(xc, wc), c2 = std::min(xc, wc);
        const int64_t over = n1 % sms, low = n1 / sms * c1, high = low + (over > 0 ? c1 : 0);
        int64_t t = high;
        if (n2 > 0) {
            auto ended = [&](int64_t at) {
                return (sms - over) * ((at - low) / c2) + over * (at > high ? (at - high) / c2 : 0);
            };
            t = std::max(t, low + c2);
            while (ended(t) < n2) t += std::max(c2 / 2, (n2 - ended(t)) / sms * c2);
        }
        // One CTA alone does not use an SM up, and clusters of more than four lie two to an SM.  Where the grid is more
        // than the SMs hold, clusters wait for as many places at once: the odd sizes the longest.
        t = std::max(t, c1 * (g.parts > 4 ? 17 : 12) / 10);
        if (4 * count > 7 * sms) t = t * (g.parts <= 2 ? 100 : g.parts == 4 || g.parts == 8 ? 105 : 112) / 100;
        return t;
    });
}

// The launch of the gradients' products by tiles of one size; x null or w null where one of them is not asked for.
template <int kXM, int kXN, int kWM, int kWN>
struct GradTiles {
    TileArgs tx, tw;
    unsigned x_tiles = 0, w_tiles = 0;
    int64_t x_steps = 0, w_steps = 0;
    bool fits = true;
    GradGrid grid{};
    GradTiles(const SumGemmParams *x, const OuterGemmParams *w, const TileArgs &x_args, const TileArgs &w_args)
        : tx(x_args), tw(w_args) {
        if (x != nullptr) {
            x_tiles = tile_grid(x->m, x->n, 16 * kXM, 16 * kXN, &tx);
            x_steps = 2 * ((x->k + kTK - 1) / kTK);
        }
        if (w != nullptr) {
            w_tiles = tile_grid(tw.m, tw.n, 16 * kWM, 16 * kWN, &tw);
            w_steps = (w->m + kTK - 1) / kTK;
        }
        fits = (x == nullptr || x_tiles > 0) && (w == nullptr || w_tiles > 0);
    }
    // sets the grid; its time, or -1 where the tiles are too many
    int64_t plan(const StepCost &cost, int64_t sms) {
        int64_t time = -1;
        if (fits) grid = many_tiles_grid(x_tiles, w_tiles, x_steps, w_steps, cost, sms, &time);
        return time;
    }
    cudaError_t launch(float *c, int64_t ldc, const OuterOut &o, cudaStream_t s) {
        constexpr uint32_t kX = TileProduct<float, kSum, kXM, kXN>::kFoldBytes;
        constexpr uint32_t kW = TileProduct<float, kOuter, kWM, kWN>::kFoldBytes;
        if (x_tiles) tx.fold = folds(tx.k, 2, grid.x_split ? grid.parts : 1);
        if (w_tiles) tw.fold = folds(tw.k, 1, grid.w_split ? grid.parts : 1);
        return launch_whole(gradients_simt_kernel<kXM, kXN, kWM, kWN>, grid.x_blocks + grid.w_blocks, grid.parts,
                            (tx.fold | tw.fold) * std::max(kX, kW), s, tx, c, ldc, tw, o, grid);
    }
};

// Clusters lie within groups of SMs: CTAs in clusters of 1 to 8 that run at once, of two and of one for each SM, in
// percent (cudaOccupancyMaxActiveClusters).
constexpr int kPairPlaces[9] = {0, 100, 100, 95, 97, 95, 90, 87, 94}, kSinglePlaces[9] = {0, 100, 100, 90, 94, 92, 90, 69, 78};

// How many CTAs share a tile of a gated projection, and the time that comes to in ns.  step: what a step of the contraction
// takes of an SM; join: steps of the exchange in a cluster, beside half a step for each CTA.
struct GatedGrid {
    int64_t time = -1;
    unsigned parts = 1;
};
GatedGrid gated_grid(unsigned tiles, int64_t steps, int64_t step, int64_t join, int64_t sms) {
    GatedGrid best;
    for (unsigned parts = 1; parts <= 8 && tiles > 0; ++parts) {
        const int64_t count = static_cast<int64_t>(tiles) * parts;
        if (count > INT32_MAX) break;
        const int64_t pairs = 2 * sms * kPairPlaces[parts] / 100, singles = sms * kSinglePlaces[parts] / 100;
        // where CTAs wait for a place, half of an exchange runs under another tile
        const int64_t exchange = parts > 1 ? (2 * join + parts) / (count > pairs ? 4 : 2) : 0;
        const int64_t chain = step * (1 + (steps + parts - 1) / parts + exchange);
        // in fifths of a chain: one CTA alone does not use an SM up, two beside each other take twice as long
        auto round = [&](int64_t blocks) { return blocks <= singles ? 6 : 10; };
        int64_t t;
        if (count <= pairs) {
            t = chain * round(count) / 5;
        } else if (count <= 3 * sms) {
            t = chain * (10 + round(count - pairs)) / 5;
        } else {
            // after four rounds the SMs are apart enough for half of the last one to be filled
            t = chain * ((count + sms - 1) / sms);
            if (count > 4 * sms) t = std::min(t, chain * count / sms + chain / 2);
            if (parts == 3 || (parts > 4 && parts < 8)) t = t * 112 / 100;  // which find as many places at once rarely
        }
        if (best.time < 0 || t < best.time) best = GatedGrid{t, parts};
    }
    return best;
}

// Tiles 128 rows high or 64, and the CTAs that share one; blocks: 0 where there are too many.  m x n x k, against tiles
// that were divided only where they were at most one an SM: 10 x 5795 x 2512 198 -> 100 us, 512 x 1408 x 2048 178 -> 137,
// 512 x 2816 x 2048 367 -> 253, 6469 x 231 x 7616 1383 -> 1070, 454 x 145 x 25 9.5 -> 6.5.
struct GatedPlan {
    bool high = true;
    unsigned parts = 1, blocks = 0;
    GatedPlan(int64_t m, int64_t n, int64_t k, int64_t sms) {
        TileArgs t{};
        const unsigned large = tile_grid(m, n, 128, 64, &t), small = tile_grid(m, n, 64, 64, &t);
        const int64_t steps = (k + kTK - 1) / kTK;
        // two products of 128 x 64 or 64 x 64 outputs, like the weights' gradients
        const GatedGrid by_large = gated_grid(large, steps, kLargeSteps.w, 4, sms);
        const GatedGrid by_small = gated_grid(small, steps, kSmallSteps.w, 2, sms);
        if (by_large.time < 0) return;
        high = by_small.time < 0 || by_large.time <= by_small.time;
        parts = high ? by_large.parts : by_small.parts;
        blocks = parts * (high ? large : small);
    }
};

template <typename T>
cudaError_t gated_simt_t(const GatedParams &p, cudaStream_t s) {
    TileArgs t{{p.x, p.x}, {p.w[0], p.w[1]}, p.m, p.n, p.k, p.ldx, p.ldw, 0, 0, 0};
    t.a_vec = groups_of_4(p.x, p.ldx, sizeof(T));
    t.b_vec = groups_of_4(p.w[0], p.ldw, sizeof(T)) && groups_of_4(p.w[1], p.ldw, sizeof(T));
    t.tiles_n = (p.n + 63) / 64;
    const GatedPlan plan(p.m, p.n, p.k, device_sm_count());
    if (plan.blocks == 0) return cudaErrorInvalidConfiguration;
    t.parts = plan.parts;
    t.fold = folds(p.k, 1, t.parts);
    const uint32_t bytes =
        t.fold * (plan.high ? TileProduct<T, kGated, 8, 4>::kFoldBytes : TileProduct<T, kGated, 4, 4>::kFoldBytes);
    if (t.parts > 1)
        return plan.high ? launch_whole(gated_simt_kernel<T, 8, 4, true>, plan.blocks, t.parts, bytes, s, t, p)
                         : launch_whole(gated_simt_kernel<T, 4, 4, true>, plan.blocks, t.parts, bytes, s, t, p);
    return plan.high ? launch_whole(gated_simt_kernel<T, 8, 4, false>, plan.blocks, 1, bytes, s, t, p)
                     : launch_whole(gated_simt_kernel<T, 4, 4, false>, plan.blocks, 1, bytes, s, t, p);
}

// ---------------------------------------------------------------------------
// d_gate = d_h * up * act'(gate), d_up = d_h * act(gate): one pass, 16 bytes an access; bound by HBM (4096 x 5504 bf16:
// 225 MB in 40 us).  Both are rounded to the tensors' type, which is what the tensor cores multiply: half a step
// between the inputs and a gradient, beside the half step of the gradient itself.
// ---------------------------------------------------------------------------

template <typename T, int kAct>
__device__ __forceinline__ void grad_piece(const GatedGradParams &p, int vec, int64_t i, int64_t j) {
    constexpr int kN = Elem<T>::kVec;
    const int64_t left = p.n - j;
    const bool whole = vec && left >= kN;
    float g[kN], u[kN], d[kN], dg[kN], du[kN];
    load_f<T, kN>(static_cast<const T *>(p.gate) + i * p.ld_saved + j, whole, left, g);
    load_f<T, kN>(static_cast<const T *>(p.up) + i * p.ld_saved + j, whole, left, u);
    load_f<T, kN>(static_cast<const T *>(p.d_h) + i * p.ld_dh + j, whole, left, d);
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        float slope;
        const float a = sizeof(T) == 2 ? gate_act_slope_16(kAct, g[e], &slope) : gate_act_slope(kAct, g[e], &slope);
        dg[e] = d[e] * u[e] * slope;
        du[e] = d[e] * a;
    }
    store_f<T, kN>(static_cast<T *>(p.d[0]) + i * p.ldd + j, left >= kN, left, dg);
    store_f<T, kN>(static_cast<T *>(p.d[1]) + i * p.ldd + j, left >= kN, left, du);
}

// blocks walk over the pieces; the row and the place in it advance without a division
template <typename T, int kAct>
__global__ void __launch_bounds__(256) gated_grad_kernel(const GatedGradParams p, int vec) {
    constexpr int kN = Elem<T>::kVec;
    grid_dep_begin();
    const int64_t pieces = (p.n + kN - 1) / kN, stride = static_cast<int64_t>(gridDim.x) * 256;
    const int64_t down = stride / pieces, across = stride - down * pieces;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    int64_t i = at / pieces, j = at - i * pieces;
    while (i < p.m) {
        grad_piece<T, kAct>(p, vec, i, j * kN);
        i += down;
        j += across;
        if (j >= pieces) {
            j -= pieces;
            ++i;
        }
    }
}

template <typename T>
cudaError_t gated_grad_t(const GatedGradParams &p, cudaStream_t s) {
    const int vec = rows16(p.gate, p.ld_saved, sizeof(T)) && rows16(p.up, p.ld_saved, sizeof(T)) &&
                    rows16(p.d_h, p.ld_dh, sizeof(T));
    const int64_t blocks = (p.m * ((p.n + Elem<T>::kVec - 1) / Elem<T>::kVec) + 255) / 256;
    const int64_t most = 16LL * device_sm_count();
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most)), block(256);
    switch (p.act) {
    case GBMM_GATE_SILU: return launch_early(gated_grad_kernel<T, GBMM_GATE_SILU>, grid, block, 0, s, p, vec);
    case GBMM_GATE_GELU: return launch_early(gated_grad_kernel<T, GBMM_GATE_GELU>, grid, block, 0, s, p, vec);
    case GBMM_GATE_GELU_TANH: return launch_early(gated_grad_kernel<T, GBMM_GATE_GELU_TANH>, grid, block, 0, s, p, vec);
    default: return launch_early(gated_grad_kernel<T, GBMM_GATE_RELU>, grid, block, 0, s, p, vec);
    }
}

// ---------------------------------------------------------------------------
// the weights' gradients of up to four tokens: d_w[i, :] = sum over the tokens of d[token, i] x[token, :], bound by writing
// them.  A block takes 32 rows of both weights and 256 columns: it evaluates d_gate and d_up of its rows into shared memory
// (f32, nothing is rounded on the way into the sums), then a warp takes every eighth row and a lane eight columns of it,
// whose values of x it holds in registers.  Blocks of the first columns also write d_gate and d_up, rounded, for d_x.
// Against tiles of the tensor cores, with d_x: 4 tokens 5504 x 2048 21.6 us and 31.6, 1408 x 2048 11.4 and 16.4; with 8
// tokens, whose values of x take 64 registers, 35.9 and 32.0.
// ---------------------------------------------------------------------------

constexpr int kFewRows = 32, kFewCols = 256, kFewTokens = 4;

// kVec: a lane's eight columns lie together and are one access; else every 32nd
template <typename T, int kAct, bool kVec>
__global__ void __launch_bounds__(256) outer_few_kernel(const GatedGradParams p, const OuterGemmParams w) {
    __shared__ __align__(16) float sd[2][kFewRows][kFewTokens];
    grid_dep_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t chunks = (w.k + kFewCols - 1) / kFewCols;
    const int64_t i0 = blockIdx.x / chunks * kFewRows, j0 = blockIdx.x % chunks * kFewCols;
    const int tokens = static_cast<int>(p.m);
    if (warp < kFewTokens) {
        const int64_t i = i0 + lane;  // this thread's row; its token is `warp`
        float dg = 0.f, du = 0.f;
        if (warp < tokens && i < p.n) {
            const float g = Elem<T>::to_f(static_cast<const T *>(p.gate)[warp * p.ld_saved + i]);
            const float u = Elem<T>::to_f(static_cast<const T *>(p.up)[warp * p.ld_saved + i]);
            const float d = Elem<T>::to_f(static_cast<const T *>(p.d_h)[warp * p.ld_dh + i]);
            float slope;
            const float a = gate_act_slope_16(kAct, g, &slope);
            dg = d * u * slope;
            du = d * a;
            if (j0 == 0 && p.d[0] != nullptr) {
                static_cast<T *>(p.d[0])[warp * p.ldd + i] = Elem<T>::from_f(dg);
                static_cast<T *>(p.d[1])[warp * p.ldd + i] = Elem<T>::from_f(du);
            }
        }
        sd[0][lane][warp] = dg;
        sd[1][lane][warp] = du;
    }
    auto column = [&](int e) { return kVec ? j0 + 8 * lane + e : j0 + lane + 32 * e; };
    const int64_t left = w.k - column(0);
    float x[kFewTokens][8];
#pragma unroll
    for (int t = 0; t < kFewTokens; ++t) {
        const T *from = static_cast<const T *>(w.x) + t * w.ldx;
        if (kVec) {
            if (t < tokens && left > 0) {
                load_f<T, 8>(from + column(0), left >= 8, left, x[t]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[t][e] = 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[t][e] = t < tokens && column(e) < w.k ? Elem<T>::to_f(from[column(e)]) : 0.f;
        }
    }
    __syncthreads();
    for (int r = warp; r < kFewRows && i0 + r < p.n; r += 8) {
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
            float d[kFewTokens], v[8];
#pragma unroll
            for (int q = 0; q < kFewTokens / 4; ++q) {
                const float4 f = *reinterpret_cast<const float4 *>(&sd[pr][r][4 * q]);
                d[4 * q] = f.x, d[4 * q + 1] = f.y, d[4 * q + 2] = f.z, d[4 * q + 3] = f.w;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
            for (int t = 0; t < kFewTokens; ++t) {
                if (t >= tokens) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fmaf(d[t], x[t][e], v[e]);
            }
            T *to = static_cast<T *>(pr == 0 ? w.c[0] : w.c[1]) + (i0 + r) * w.ldc;
            if (kVec) {
                if (left > 0) store_f<T, 8>(to + column(0), left >= 8, left, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (column(e) < w.k) to[column(e)] = Elem<T>::from_f(v[e]);
            }
        }
    }
}

template <typename T, bool kVec>
cudaError_t outer_few_v(const GatedGradParams &p, const OuterGemmParams &w, cudaStream_t s) {
    const int64_t blocks = (p.n + kFewRows - 1) / kFewRows * ((w.k + kFewCols - 1) / kFewCols);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks)), block(256);
    switch (p.act) {
    case GBMM_GATE_SILU: return launch_early(outer_few_kernel<T, GBMM_GATE_SILU, kVec>, grid, block, 0, s, p, w);
    case GBMM_GATE_GELU: return launch_early(outer_few_kernel<T, GBMM_GATE_GELU, kVec>, grid, block, 0, s, p, w);
    case GBMM_GATE_GELU_TANH: return launch_early(outer_few_kernel<T, GBMM_GATE_GELU_TANH, kVec>, grid, block, 0, s, p, w);
    default: return launch_early(outer_few_kernel<T, GBMM_GATE_RELU, kVec>, grid, block, 0, s, p, w);
    }
}
template <typename T>
cudaError_t outer_few_t(const GatedGradParams &p, const OuterGemmParams &w, cudaStream_t s) {
    const bool vec = rows16(w.x, w.ldx, 2) && rows16(w.c[0], w.ldc, 2) && rows16(w.c[1], w.ldc, 2);
    return vec ? outer_few_v<T, true>(p, w, s) : outer_few_v<T, false>(p, w, s);
}

// ---------------------------------------------------------------------------
// 16-bit rows that TMA cannot read, written again into rows that it can
// ---------------------------------------------------------------------------

// a warp takes 512 values of a row at a time, of up to three matrices of as many columns
__global__ void __launch_bounds__(256)
repack16_kernel(const RepackParams first, const RepackParams second, const RepackParams third, int64_t parts) {
    constexpr int kU = 8;
    grid_dep_begin();
    const int lane = threadIdx.x & 31;
    const int64_t items = (first.rows + second.rows + third.rows) * parts, warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; at < items; at += warps) {
        const int64_t row = at / parts, o0 = (at - row * parts) * (32 * kU);  // words of two values
        const bool in_first = row < first.rows, in_second = row < first.rows + second.rows;
        const RepackParams &p = in_first ? first : in_second ? second : third;
        const int64_t i = in_first ? row : in_second ? row - first.rows : row - first.rows - second.rows;
        const uint8_t *src = static_cast<const uint8_t *>(p.src) + 2 * i * p.lds;
        uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.dst) + i * p.ldd);
        uint32_t v[kU];
        shifted_words<2, kU>(src, o0, 2 * p.cols, lane, v);
#pragma unroll
        for (int q = 0; q < kU; ++q)
            if (2 * (o0 + 32 * q + lane) < p.ldd) dst[o0 + 32 * q + lane] = v[q];
    }
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

// The weights' gradients of at most gated_few_tokens() tokens, 16-bit types; p.d null: d_gate and d_up are not written.
int gated_few_tokens() { return kFewTokens; }
cudaError_t launch_gated_outer_few(int dt, const GatedGradParams &p, const OuterGemmParams &w, cudaStream_t s) {
    return dt == kF16 ? outer_few_t<__half>(p, w, s) : outer_few_t<__nv_bfloat16>(p, w, s);
}

namespace {

// The gradients of f32 blocks: x null or w null where one of them is not asked for.
struct GradPlan {
    GradTiles<8, 8, 8, 4> large;
    GradTiles<4, 4, 4, 4> small;
    bool take_small = false;
    GradPlan(const SumGemmParams *x, const OuterGemmParams *w, const TileArgs &tx, const TileArgs &tw, int64_t sms)
        : large(x, w, tx, tw), small(x, w, tx, tw) {
        // fewer large tiles, those of x in pairs, than SMs
        if (large.fits && small.fits && 2 * static_cast<int64_t>(large.x_tiles) + large.w_tiles < sms) {
            small.grid = few_tiles_grid(small.x_tiles, small.w_tiles, small.x_steps, small.w_steps, sms);
            take_small = true;
        } else {
            const int64_t time_large = large.plan(kLargeSteps, sms), time_small = small.plan(kSmallSteps, sms);
            take_small = time_small >= 0 && time_small < time_large;
            large.fits = time_large >= 0;
        }
    }
};
TileArgs x_args(const SumGemmParams &x) {
    TileArgs t{{x.a[0], x.a[1]}, {x.b[0], x.b[1]}, x.m, x.n, x.k, x.lda, x.ldb, 0, 0, 0};
    t.a_vec = groups_of_4(x.a[0], x.lda, 4) && groups_of_4(x.a[1], x.lda, 4);
    t.b_vec = groups_of_4(x.b[0], x.ldb, 4) && groups_of_4(x.b[1], x.ldb, 4);
    return t;
}
TileArgs w_args(const OuterGemmParams &w) {
    TileArgs t{{w.x, w.x}, {w.d[0], w.d[1]}, w.k, w.n, w.m, w.ldx, w.ldd, 0, 0, 0};
    t.a_vec = groups_of_4(w.x, w.ldx, 4);
    t.b_vec = groups_of_4(w.d[0], w.ldd, 4) && groups_of_4(w.d[1], w.ldd, 4);
    return t;
}

}  // namespace

cudaError_t launch_gated_products_simt(const SumGemmParams *x, const OuterGemmParams *w, cudaStream_t s) {
    GradPlan plan(x, w, x != nullptr ? x_args(*x) : TileArgs{}, w != nullptr ? w_args(*w) : TileArgs{}, device_sm_count());
    if (!plan.large.fits) return cudaErrorInvalidConfiguration;
    OuterOut o{};
    if (w != nullptr)
        o = OuterOut{{static_cast<float *>(w->c[0]), static_cast<float *>(w->c[1])},
                     w->ldc,
                     groups_of_4(w->c[0], w->ldc, 4) && groups_of_4(w->c[1], w->ldc, 4)};
    float *const c = x != nullptr ? static_cast<float *>(x->c) : nullptr;
    const int64_t ldc = x != nullptr ? x->ldc : 0;
    return plan.take_small ? plan.small.launch(c, ldc, o, s) : plan.large.launch(c, ldc, o, s);
}

// the height of a tile of a gated projection on the FFMA pipe and the CTAs that share one; zeros where there are too many
void gated_simt_plan(int64_t m, int64_t n, int64_t k, int64_t sms, int32_t plan[2]) {
    const GatedPlan p(m, n, k, sms);
    plan[0] = p.blocks == 0 ? 0 : p.high ? 128 : 64;
    plan[1] = p.blocks == 0 ? 0 : static_cast<int32_t>(p.parts);
}
// tile: the edge of a tile of x (weights: as many columns, and 64 rows); grid: CTAs that divide a tile of x, of the weights
// (1: undivided), whether the weights' come first
void gated_products_simt_plan(int64_t m, int64_t n, int64_t k, bool need_x, bool need_w, int64_t sms, int32_t plan[4]) {
    SumGemmParams x{};
    OuterGemmParams w{};
    x.m = w.m = m;
    x.n = w.k = k;
    x.k = w.n = n;
    const GradPlan p(need_x ? &x : nullptr, need_w ? &w : nullptr, x_args(x), w_args(w), sms);
    const GradGrid &g = p.take_small ? p.small.grid : p.large.grid;
    plan[0] = p.take_small ? 64 : 128;
    plan[1] = g.x_split ? static_cast<int32_t>(g.parts) : 1;
    plan[2] = g.w_split ? static_cast<int32_t>(g.parts) : 1;
    plan[3] = g.w_first;
}

// ldd and cols the same in all three; rows 0: nothing to do
cudaError_t launch_repack16(const RepackParams (&p)[3], cudaStream_t s) {
    const int64_t parts = (p[0].ldd + 511) / 512, most = 32LL * device_sm_count();
    const int64_t blocks = ((p[0].rows + p[1].rows + p[2].rows) * parts + 7) / 8;
    if (blocks == 0) return cudaSuccess;
    return launch_early(repack16_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, s, p[0],
                        p[1], p[2], parts);
}

}  // namespace gbmm
