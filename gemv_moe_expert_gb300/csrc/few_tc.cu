// few_tc.cu -- products of the feed-forward block for some tens of tokens, on the tensor cores as
// y^T = W x^T: the weights' rows are the MMA's M side (128 a tile), the tokens its N side (kN).
//   gated   h = act(x Wg^T) * (x Wu^T): 64 rows of Wg and the same 64 of Wu share a tile, so an output's two
//           projections lie 64 rows apart
//   codes   c = (a b^T) scale_a scale_b for 8-bit codes: the weights' codes reach shared memory as bytes, and eight
//           warps write them as f16 (exact) into tensor memory, from where the MMAs take their A operand; the
//           tokens' codes become f16 in shared memory, or come as f16 from 64 tokens on.  Each 1024 of k has an
//           accumulator of its own: sums of products of two codes are exact up to there (2^24), and the accumulators are
//           added as integers at the end.
//   sum     d_x = d_gate Wg + d_up Wu, the gradient of x: the weights' columns are the M side (128 a tile, in boxes of 64 x
//           64), the contraction runs over the rows of Wg and then of Wu
// Every weight byte is read once (per kN tokens), and the kernel is bound by that stream; two CTAs share an SM
// where the ring allows, and the contraction is split over a thread-block cluster of up to eight CTAs where the tiles
// are few.  Each CTA leaves its partial sums in its own (by then idle) ring, and after a cluster barrier every CTA adds
// up its share of the tokens, in the order of the ranks, through distributed shared memory.
//   warp 0      TMA
//   warp 1      tensor memory, MMAs
//   warps 2..5  (codes: 2..9, bytes to f16) the epilogue
// Every mbarrier wait is bounded; on a timeout the kernel records it in the device error word.  Whatever role gave up,
// the CTA waits (bounded) for its own copies and MMAs, still takes part in the cluster barriers, releases its TMEM and
// returns.
#include <cooperative_groups.h>

#include <type_traits>

#include "gated.cuh"

namespace cg = cooperative_groups;

namespace gbmm {

namespace {

constexpr int kBM = 128;
constexpr int kMaxSplit = 8;
constexpr uint32_t kWBytes = kBM * 128;  // 128 rows of 128 bytes: 64 16-bit values or 128 codes
constexpr int kChunk = 8;                // code blocks (of 128) whose sums stay exact: 1024 of k

enum Kind { kGated, kCodes8, kSum };

// CTAs that an SM holds at once.  Together they never ask for more than its kTmemCols columns of tensor memory: a CTA
// that waited for columns would wait without a limit, and for one that may itself be waiting in a cluster barrier.
constexpr int ctas_per_sm(bool codes, int tokens) { return codes && tokens == 128 ? 1 : 2; }
constexpr uint32_t kTmemCols = 512;

template <int kKind, int kN>
struct Ring {
    static constexpr bool kCodes = kKind == kCodes8;
    static constexpr int kWarps = kCodes ? 8 : 4;  // behind the TMA and MMA warps
    static constexpr int kThreads = 64 + 32 * kWarps;
    static constexpr bool kHalfX = kCodes && kN >= 64;  // the tokens' codes come as f16
    static constexpr uint32_t kXBytes = kN * 128;       // 64 16-bit values or 128 codes of each token
    // a stage: a k-block as TMA brings it
    static constexpr uint32_t kStageBytes = kWBytes + (kHalfX ? 2 : 1) * kXBytes;
    static constexpr int kStages = kCodes ? (kN <= 16 ? 5 : kN <= 32 ? 4 : kN == 64 ? 3 : 4)
                                          : (kN <= 16 ? 6 : kN == 32 ? 5 : kN == 64 ? 4 : 3);
    // codes: slots for a k-block in f16, the weights' kSlotCols columns of tensor memory, the tokens' kSlotBytes
    static constexpr int kSlots = kCodes ? 2 : 0;
    static constexpr uint32_t kSlotCols = 64;
    static constexpr uint32_t kSlotBytes = kHalfX ? 0 : 2 * kXBytes;
    static constexpr uint32_t kSlot0 = kStages * kStageBytes;
    static constexpr uint32_t kRingBytes = kSlot0 + kSlots * kSlotBytes;
    static constexpr uint32_t kBarBytes = 256;
    static constexpr uint32_t kSmemBytes = kRingBytes + kBarBytes + 1024;
    static_assert(kSlots * kSlotCols == (kCodes ? 128 : 0), "few_tc_plan() counts them");
    static_assert(kStageBytes % 1024 == 0 && kSlotBytes % 1024 == 0, "swizzled tiles need 1024-byte alignment");
    static_assert(kBM * kN * 4 <= kRingBytes, "the partial sums are parked in the ring");
    static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");
    static_assert(228 * 1024 / (kSmemBytes + 1024) == ctas_per_sm(kCodes, kN), "CTAs that shared memory lets an SM hold");
    static_assert(8 * (2 * (kStages + kSlots) + 2) + 8 <= kBarBytes, "barriers");
};

__device__ __forceinline__ void load16(uint32_t at, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}

// The 128 codes of each of kRows tokens at `raw`, as f16 in two tiles of 64 at `dst`; all 128-byte swizzled.
// Thread t of 128 takes rows t % kRows, so that eight neighbours' 16-byte accesses fall into different banks.
template <int kRows>
__device__ __forceinline__ void convert_tokens(uint32_t raw, uint32_t dst, int t) {
    static_assert(kRows * 8 % 128 == 0, "whole turns");
#pragma unroll
    for (int i = 0; i < kRows * 8 / 128; ++i) {
        const int row = (t + 128 * i) % kRows, c = (t + 128 * i) / kRows;
        uint32_t v[4];
        load16(raw + row * 128 + ((c ^ (row & 7)) << 4), v);
        const uint32_t to = dst + (c >> 2) * (kRows * 128) + row * 128;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint2 a = codes_to_half(v[2 * e]), b = codes_to_half(v[2 * e + 1]);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((2 * (c & 3) + e) ^ (row & 7)) << 4)),
                         "r"(a.x), "r"(a.y), "r"(b.x), "r"(b.y)
                         : "memory");
        }
    }
}

template <typename TC, uint32_t kFmt, int kKind, int kN>
__global__ void __launch_bounds__(Ring<kKind, kN>::kThreads)
few_tc_kernel(const __grid_constant__ FewTcMaps maps, const FewTcParams p) {
    using R = Ring<kKind, kN>;
    constexpr bool kCodes = R::kCodes;
    constexpr int kStages = R::kStages, kSlots = R::kSlots, kWarps = R::kWarps;
    constexpr int kRows = kKind == kGated ? kBM / 2 : kBM;  // outputs across a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t s0 = raw_addr + pad;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + R::kRingBytes);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };                       // bytes of stage s have landed
    auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };          // ... are used up
    auto slot_full = [&](int s) { return bar0 + 8u * (2 * kStages + s); };      // codes: slot s holds f16
    auto slot_empty = [&](int s) { return bar0 + 8u * (2 * kStages + kSlots + s); };
    const uint32_t tfull_bar = bar0 + 8u * (2 * (kStages + kSlots));
    const uint32_t drain_bar = tfull_bar + 8u;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * (kStages + kSlots) + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ksplit = p.ksplit;
    const int rank = static_cast<int>(blockIdx.x) % ksplit;  // == rank in the cluster
    const int tile = static_cast<int>(blockIdx.x) / ksplit;
    const int n0 = tile / p.token_blocks * kRows, t0 = tile % p.token_blocks * kN;
    const uint64_t lim = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), kCodes && !R::kHalfX ? kWarps / 2 : 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(slot_full(s), kWarps / 2);
            mbar_init(slot_empty(s), 1);
        }
        mbar_init(tfull_bar, 1);
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.x[0]);
        tma_prefetch_desc(&maps.w[0]);
        if (!kCodes) tma_prefetch_desc(&maps.w[1]);
        if (kKind == kSum) tma_prefetch_desc(&maps.x[1]);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot, acc_base = tmem_base + kSlots * R::kSlotCols;
    grid_dep_begin();
    // this CTA's share of the k-blocks (128 bytes of a row each)
    constexpr int kBlock = kCodes ? 128 : 64;
    const int blocks1 = p.k / kBlock + (p.k % kBlock != 0);  // of a source
    const int kb_total = kKind == kSum ? 2 * blocks1 : blocks1;
    const int kb0 = static_cast<int>(static_cast<int64_t>(kb_total) * rank / ksplit);
    const int kblocks = static_cast<int>(static_cast<int64_t>(kb_total) * (rank + 1) / ksplit) - kb0;

    auto fail = [&]() {
        *abort_flag = 1;
        report_device_error(p.err, kKidFewTc);
    };

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            const uint64_t pol = p.token_blocks == 1 ? policy_evict_first() : policy_evict_normal();
            uint32_t issued = 0;
            bool ok = true;
            for (int kb = 0; kb < kblocks; ++kb) {
                const int stage = kb % kStages;
                const uint32_t use = static_cast<uint32_t>(kb / kStages);
                if (use > 0 && !mbar_wait_bounded(empty_bar(stage), (use - 1u) & 1u, lim, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t sw = s0 + stage * R::kStageBytes;
                const bool second = kKind == kSum && kb0 + kb >= blocks1;
                const int k0 = (second ? kb0 + kb - blocks1 : kb0 + kb) * kBlock;
                const CUtensorMap *const x = second ? &maps.x[1] : &maps.x[0];
                mbar_arrive_expect_tx(full_bar(stage), R::kStageBytes);
                if constexpr (kKind == kSum) {
                    const CUtensorMap *const w = second ? &maps.w[1] : &maps.w[0];
                    tma_load_3d_hint(sw, w, full_bar(stage), n0, k0, 0, pol);
                    tma_load_3d_hint(sw + kWBytes / 2, w, full_bar(stage), n0 + 64, k0, 0, pol);
                } else {
                    tma_load_3d_hint(sw, &maps.w[0], full_bar(stage), k0, n0, 0, pol);
                    if (!kCodes) tma_load_3d_hint(sw + kWBytes / 2, &maps.w[1], full_bar(stage), k0, n0, 0, pol);
                }
                tma_load_3d(sw + kWBytes, x, full_bar(stage), k0, t0, 0);
                if (R::kHalfX) tma_load_3d(sw + kWBytes + R::kXBytes, x, full_bar(stage), k0 + 64, t0, 0);
                ++issued;
            }
            if (!ok) fail();
            // This CTA's copies have landed before it goes on to use the ring for something else, also where another role
            // gave up after the last of them was issued.
            for (int s = 0; s < kStages; ++s) {
                const uint32_t n_s = issued / kStages + (static_cast<uint32_t>(s) < issued % kStages ? 1u : 0u);
                if (n_s > 0 && !mbar_wait_bounded(full_bar(s), (n_s - 1u) & 1u, lim, nullptr)) fail();
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            constexpr uint32_t kIdesc = idesc_f16(kFmt, kBM, kN, kKind == kSum ? 1u : 0u);
            bool ok = true;
            for (int kb = 0; kb < kblocks; ++kb) {
                const int stage = kb % kStages;
                const uint32_t stage_at = s0 + stage * R::kStageBytes;
                if (!kCodes || R::kHalfX)
                    ok = mbar_wait_bounded(full_bar(stage), static_cast<uint32_t>(kb / kStages) & 1u, lim, abort_flag);
                if constexpr (kCodes) {
                    const int slot = kb % kSlots;
                    ok = ok && mbar_wait_bounded(slot_full(slot), static_cast<uint32_t>(kb / kSlots) & 1u, lim, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = acc_base + static_cast<uint32_t>(kb / kChunk * kN);
                    const uint32_t sx = R::kHalfX ? stage_at + kWBytes : s0 + R::kSlot0 + slot * R::kSlotBytes;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_f16_ts(d, tmem_base + slot * R::kSlotCols + kk * 8,
                                    sdesc_kmajor_sw128(sx + (kk >> 2) * R::kXBytes + (kk & 3) * 32), kIdesc,
                                    kb % kChunk == 0 && kk == 0 ? 0u : 1u);
                    umma_commit(slot_empty(slot));
                    if (R::kHalfX) umma_commit(empty_bar(stage));
                } else {
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16_ss(acc_base,
                                    kKind == kSum ? sdesc_mnmajor_sw128(stage_at + kk * 2048, kWBytes / 2)
                                                  : sdesc_kmajor_sw128(stage_at + kk * 32),
                                    sdesc_kmajor_sw128(stage_at + kWBytes + kk * 32), kIdesc, kb == 0 && kk == 0 ? 0u : 1u);
                    umma_commit(empty_bar(stage));
                }
            }
            if (ok) umma_commit(tfull_bar);
            else fail();
            // every MMA this thread issued has completed once this arrives
            umma_commit(drain_bar);
            mbar_wait_bounded(drain_bar, 0, lim, nullptr);
        }
    } else if constexpr (kCodes) {
        // ---------------- codes to f16 ----------------
        // Two groups of four warps take every other k-block, each with a slot of its own: while one waits for its bytes or
        // for its stores to tensor memory, the other converts.
        const int group = (warp - 2) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const int t = (threadIdx.x - 64) & 127;
        for (int kb = group; kb < kblocks; kb += 2) {
            const int stage = kb % kStages, slot = group;
            const uint32_t phase = static_cast<uint32_t>(kb / kStages) & 1u, use = static_cast<uint32_t>(kb / kSlots);
            int ready = 1;
            if (lane == 0) ready = mbar_wait_bounded(full_bar(stage), phase, lim, abort_flag);
            ready = __shfl_sync(0xffffffffu, ready, 0);
            // every lane orders the bytes that TMA wrote before its own reads
            if (ready && lane != 0) mbar_try_wait(full_bar(stage), phase);
            const uint32_t from = s0 + stage * R::kStageBytes + row * 128;
            const uint32_t to = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + slot * R::kSlotCols;
            uint32_t v[8][4];
            if (ready) {
#pragma unroll
                for (int c = 0; c < 8; ++c) load16(from + ((c ^ (row & 7)) << 4), v[c]);
                if (lane == 0 && use > 0) ready = mbar_wait_bounded(slot_empty(slot), (use - 1u) & 1u, lim, abort_flag);
            }
            ready = __shfl_sync(0xffffffffu, ready, 0);
            if (!ready) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint2 f = codes_to_half(v[4 * h + (i >> 2)][i & 3]);
                    w[2 * i] = f.x;
                    w[2 * i + 1] = f.y;
                }
                tmem_st32(to + h * 32, w);
            }
            if constexpr (!R::kHalfX) {
                convert_tokens<kN>(s0 + stage * R::kStageBytes + kWBytes, s0 + R::kSlot0 + slot * R::kSlotBytes, t);
                fence_async_smem();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(slot_full(slot));
                if (!R::kHalfX) mbar_arrive(empty_bar(stage));
            }
        }
    }
    // the ring is idle from here on: copies have landed, conversions and MMAs are done or given up
    __syncwarp();
    __syncthreads();

    // ---------------- epilogue: partial sums to shared memory, [token][row] ----------------
    using Sum = typename std::conditional<kCodes, int, float>::type;
    Sum *part = reinterpret_cast<Sum *>(smem);
    const int tokens = min(kN, p.m - t0);
    if (warp >= 2) {
        const int quarter = warp & 3;  // TMEM lanes 32 * quarter .. + 31
        int ready = 0;
        if (lane == 0) ready = mbar_wait_bounded(tfull_bar, 0, lim, abort_flag);
        ready = __shfl_sync(0xffffffffu, ready, 0);
        __syncwarp();
        if (!ready && lane == 0) fail();
        if (ready) tc_fence_after();
        const int chunks = !ready || kblocks == 0 ? 0 : kCodes ? (kblocks + kChunk - 1) / kChunk : 1;
        const int row = quarter * 32 + lane;
        // two warps a quarter take every other 16 tokens
        for (int j = 16 * ((warp - 2) >> 2); j < tokens; j += 4 * kWarps) {
            Sum v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0;
            for (int c = 0; c < chunks; ++c) {
                uint32_t r[16];
                tmem_ld16(acc_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(c * kN + j), r);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if constexpr (kCodes) v[e] += __float2int_rn(__uint_as_float(r[e]));
                    else v[e] = __uint_as_float(r[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) part[(j + e) * kBM + row] = v[e];
        }
    }
    cg::cluster_group cluster = cg::this_cluster();
    // every thread of the cluster reaches both barriers, on every path
    if (ksplit > 1) cluster.sync();
    else __syncthreads();
    if (warp >= 2) {
        const int t = threadIdx.x - 64;
        // a thread's column, and which of the tokens that run at once is its own
        constexpr int kAcross = kRows, kDown = 32 * kWarps / kAcross;
        const int col = t % kAcross, first = t / kAcross;
        const int64_t j = static_cast<int64_t>(n0) + col;
        if (j < p.n) {
            const float sb = kCodes && p.scale_b != nullptr ? __ldg(p.scale_b + j) : 1.f;
            // several tokens at a time, so that as many reads of other CTAs' sums are under way
            constexpr int kB = 4;
            for (int tk0 = kDown * rank + first; tk0 < tokens; tk0 += kB * kDown * ksplit) {
                Sum g[kB], u[kB];
#pragma unroll
                for (int e = 0; e < kB; ++e) g[e] = u[e] = 0;
#pragma unroll 4
                for (int q = 0; q < ksplit; ++q) {
                    const Sum *from = (ksplit > 1 ? cluster.map_shared_rank(part, q) : part) + col;
#pragma unroll
                    for (int e = 0; e < kB; ++e) {
                        const int tk = min(tk0 + e * kDown * ksplit, tokens - 1);
                        g[e] += from[tk * kBM];
                        if constexpr (kKind == kGated) u[e] += from[tk * kBM + 64];
                    }
                }
#pragma unroll
                for (int e = 0; e < kB; ++e) {
                    const int tk = tk0 + e * kDown * ksplit;
                    if (tk >= tokens) break;
                    const int64_t i = t0 + tk;
                    TC *const out = static_cast<TC *>(p.c) + i * p.ldc + j;
                    if constexpr (kCodes) {
                        const float sa = p.scale_a != nullptr ? __ldg(p.scale_a + i) : 1.f;
                        *out = Elem<TC>::from_f(static_cast<float>(g[e]) * sa * sb);
                    } else if constexpr (kKind == kSum) {
                        *out = Elem<TC>::from_f(g[e]);
                    } else {
                        *out = Elem<TC>::from_f(gate_act_16(p.act, g[e]) * u[e]);
                        if (p.saved[0] != nullptr) {
                            static_cast<TC *>(p.saved[0])[i * p.ld_saved + j] = Elem<TC>::from_f(g[e]);
                            static_cast<TC *>(p.saved[1])[i * p.ld_saved + j] = Elem<TC>::from_f(u[e]);
                        }
                    }
                }
            }
        }
    }
    if (ksplit > 1) cluster.sync();  // every rank's shared memory lives until all have read it

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, p.tmem_cols);
    }
}

template <typename TC, uint32_t kFmt, int kKind, int kN>
cudaError_t few_n(const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s) {
    using R = Ring<kKind, kN>;
    static DeviceBits attr_set{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(attr_set & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(few_tc_kernel<TC, kFmt, kKind, kN>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set |= bit;
    }
    const int rows = kKind == kGated ? kBM / 2 : kBM;
    const int64_t blocks = (static_cast<int64_t>(p.n) + rows - 1) / rows * p.token_blocks * p.ksplit;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(R::kThreads);
    cfg.dynamicSmemBytes = R::kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.ksplit);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_tc_kernel<TC, kFmt, kKind, kN>, maps, p);
}

template <typename TC, uint32_t kFmt, int kKind>
cudaError_t few_t(int tokens, const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s) {
    if (p.ksplit < 1 || p.ksplit > kMaxSplit || ctas_per_sm(kKind == kCodes8, tokens) * p.tmem_cols > kTmemCols)
        return cudaErrorInvalidValue;
    switch (tokens) {
    case 16: return few_n<TC, kFmt, kKind, 16>(maps, p, s);
    case 32: return few_n<TC, kFmt, kKind, 32>(maps, p, s);
    case 64: return few_n<TC, kFmt, kKind, 64>(maps, p, s);
    case 128: return few_n<TC, kFmt, kKind, 128>(maps, p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

int few_tc_rows(bool codes) { return codes ? kBM : kBM / 2; }
int few_tc_block_k() { return 64; }
int few_tc_ctas_per_sm(bool codes, int tokens) { return ctas_per_sm(codes, tokens); }

namespace {
constexpr int kCodeCols = 128;  // columns of tensor memory that hold weights
// code blocks that one CTA's accumulators take
int64_t code_blocks(int tokens) {
    return (static_cast<int>(kTmemCols) / ctas_per_sm(true, tokens) - kCodeCols) / tokens * kChunk;
}

struct Split {
    int64_t ctas, split;
};
Split split_for(int kind, int tokens, int64_t m, int64_t n, int64_t k, int num_sms) {
    const bool codes = kind == kCodes8;
    const int64_t rows = few_tc_rows(kind != kGated), tiles = (n + rows - 1) / rows * ((m + tokens - 1) / tokens);
    const int64_t kb = codes ? (k + 127) / 128 : (k + 63) / 64 * (kind == kSum ? 2 : 1);
    int64_t split = 1;
    // as many CTAs as the SMs hold at once (a cluster lies within a group of 16 to 20 SMs, so that an eighth of
    // the places may not be used), each with a few blocks of its own (1408 x 2048 bf16, 16 tokens: 9.0, 7.1 and
    // 8.5 us with at least 4, 8 and 16; 8-bit codes, 64 tokens: 8.3, 10.5 and 13.2 us with 2, 4 and 8)
    while (split < kMaxSplit && 8 * tiles * (split + 1) <= 7LL * ctas_per_sm(codes, tokens) * num_sms &&
           kb >= (codes ? 2 : 8) * (split + 1))
        ++split;
    if (codes)
        while (split < kMaxSplit && (kb + split - 1) / split > code_blocks(tokens)) ++split;
    return {tiles * split, split};
}
}  // namespace

// Up to 128 tokens; codes up to 256, and up to 512 where both operands' f16 form would fill few of the 256 x 256 tiles
// (1408 x 2048, 512 tokens: 15 us here, 19 there; 11008 x 4096: 104 and 77).
bool few_tc_takes(bool codes, int64_t m, int64_t n, int64_t k) {
    if (!codes) return m <= 128;
    if (m > 256 && (m > 512 || m * n > (1 << 20))) return false;
    return (k + 127) / 128 <= kMaxSplit * code_blocks(m <= 16 ? 16 : m <= 32 ? 32 : 128);
}
// whether the tokens' codes come as f16, in boxes of 64 k, rather than as bytes
bool few_tc_half_tokens(int64_t m) { return m > 32; }

// The tokens of a tile; sets the CTAs that share its contraction and the columns of tensor memory.
int few_tc_plan(bool codes, int64_t m, int64_t n, int64_t k, int num_sms, FewTcParams *p) {
    int tokens = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 || codes ? 64 : 128;
    Split s = split_for(codes ? kCodes8 : kGated, tokens, m, n, k, num_sms);
    if (codes && m > 32) {
        // Tiles of 128 tokens read the weights once, but have an SM to themselves: taken where they fill the SMs once
        // (128 tokens: 4096 x 11008 26.5 us against 38 with 64 a tile, 11008 x 4096 42.7 against 37.7), or where 64 leave
        // no room for the accumulators of so long a sum.
        const Split wide = split_for(kCodes8, 128, m, n, k, num_sms);
        const int64_t kb = (k + 127) / 128;
        const bool fills = m > 64 && m <= 128 && wide.ctas <= num_sms && 4 * wide.ctas >= 3LL * num_sms;
        if (fills || kb > s.split * code_blocks(64)) {
            tokens = 128;
            s = wide;
        }
    }
    p->token_blocks = static_cast<int32_t>((m + tokens - 1) / tokens);
    p->ksplit = static_cast<int32_t>(s.split);
    int64_t cols = tokens;
    if (codes) cols = kCodeCols + (((k + 127) / 128 + s.split - 1) / s.split + kChunk - 1) / kChunk * tokens;
    p->tmem_cols = 32;
    while (p->tmem_cols < cols) p->tmem_cols *= 2;
    return tokens;
}

// The gradient of x, m tokens of k columns from n rows of both weights, in a launch of its own.  In the other way,
// 256 x 256 tiles among those of the weights' gradients (pair_tc.cu), one tile runs through the whole contraction: taken
// here where that chain of k-blocks (0.6 of them for half tiles) is by half longer than all work over all pairs, and long
// enough to be worth a launch.  bf16, here and there: 1 token, 5504 x 2048 31 and 66 us; 16, 1408 x 2048 17 and 19; 256,
// 5504 x 2048 48 and 59; 1024, 11008 x 704 90 and 124; but 16, 704 x 512 13 and 12, 128, 1408 x 2048 24 and 19.  Where the
// weights' gradients are not in that grid any chain will do (4 tokens, 704 x 512 9.0 and 12.7; 1, 200 x 200 6.6 and 8.1).
bool few_tc_takes_sum(int64_t m, int64_t n, int64_t k, bool need_w, int num_sms) {
    const int64_t chain = 2 * ((n + 63) / 64), across = (k + 255) / 256, tiles = (m + 255) / 256 * across;
    const int64_t pairs = num_sms / 2;
    if (chain < (m > 64 ? 100 : need_w ? 40 : 0)) return false;
    const int64_t work = tiles * chain + (need_w ? 2 * ((n + 255) / 256) * across * ((m + 63) / 64) : 0);
    return (2 * tiles <= pairs ? 0.6 : 1.0) * static_cast<double>(chain) * static_cast<double>(pairs) >=
           1.5 * static_cast<double>(work);
}
int few_tc_plan_sum(int64_t m, int64_t n, int64_t k, int num_sms, FewTcParams *p) {
    const int tokens = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
    p->token_blocks = static_cast<int32_t>((m + tokens - 1) / tokens);
    p->ksplit = static_cast<int32_t>(split_for(kSum, tokens, m, k, n, num_sms).split);
    p->tmem_cols = tokens < 32 ? 32 : tokens;
    return tokens;
}

cudaError_t launch_gated_few(int dt, int tokens, const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s) {
    return dt == kF16 ? few_t<__half, 0, kGated>(tokens, maps, p, s) : few_t<__nv_bfloat16, 1, kGated>(tokens, maps, p, s);
}
cudaError_t launch_sum_few(int dt, int tokens, const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s) {
    return dt == kF16 ? few_t<__half, 0, kSum>(tokens, maps, p, s) : few_t<__nv_bfloat16, 1, kSum>(tokens, maps, p, s);
}
cudaError_t launch_gemm_i8_few(int dt, int tokens, const FewTcMaps &maps, const FewTcParams &p, cudaStream_t s) {
    switch (dt) {
    case kF32: return few_t<float, 0, kCodes8>(tokens, maps, p, s);
    case kF16: return few_t<__half, 0, kCodes8>(tokens, maps, p, s);
    case kBF16: return few_t<__nv_bfloat16, 0, kCodes8>(tokens, maps, p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace gbmm
