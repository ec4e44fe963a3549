// pair_tc.cu -- products of the feed-forward block on the tensor cores, 256 x 256
// accumulators on CTA pairs (tcgen05.mma.cta_group::2, M = 256, N = 256, K = 16):
//   kGated  h = act(x Wg^T) * (x Wu^T): the pair's even CTA loads 128 rows of Wg, its odd CTA
//           the same 128 rows of Wu, so columns 0..127 of each CTA's accumulator hold the gate
//           and 128..255 the up projection of the same outputs; one thread has both
//   kGrads  the gradients of x and of both weights from those of both projections, in one grid:
//           c = a0 b0 + a1 b1, the contraction running over the first source and then the
//           second, and dw_i = a_i^T x.  The tiles of c are the long ones; they come first, and
//           those of dw level the pairs out (Walk)
//   kCodes  c = (a b^T) scale_a scale_b for 8-bit codes held as f16: a product of two codes, and
//           any sum of them below 2^24, is exact in the f32 accumulator; after each 1024 of k (at
//           most 2^24) the epilogue adds the accumulator to 32-bit integers in registers
// The tensor core has no fast 8-bit integer form on sm_103a, so codes run at the 16-bit rate.
//
// Roles and buffers are those of the CTA-pair GEMM (gemm_tc.cu): per CTA and k-block of 64 a 128 x
// 64 piece of A and of B in a six-deep ring, two accumulators in tensor memory, so that a tile's
// epilogue runs under the next tile's MMAs, a grouped raster of tiles, and the last round's tiles
// as two halves where it would leave half of the pairs idle.  Eight epilogue warps a CTA: a lane
// quarter and half of the columns each, since both projections' activation (or the integer
// conversion) costs more than rounding.
//   warp 0      TMA (both CTAs), completion counted on the even CTA's barrier
//   warp 1      tensor memory; in the even CTA one thread issues the pair's MMAs
//   warps 2..9  epilogue (both CTAs)
// Every wait is bounded; a timeout raises both CTAs' abort flags and the device error word.
#include <algorithm>

#include "gated.cuh"

namespace gbmm {

namespace {

constexpr int kBM = 128;  // rows of A and of B in one CTA
constexpr int kBN = 256;  // accumulator columns
constexpr int kBK = 64;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kGroupM = 8;
constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr uint32_t kStageBytes = 2 * kABytes;
constexpr uint32_t kMNBox = 64 * kBK * 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOutBytes = 4096;  // of each epilogue warp
constexpr uint32_t kSmemBytes = kStages * kStageBytes + kEpiWarps * kOutBytes + 256 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");
constexpr uint64_t kBlockLimitNs = 4000;  // what a k-block may add to a wait for all of a unit's
constexpr int kExactBlocks = 1024 / kBK;  // k-blocks whose sum of products of two codes stays within 2^24

enum Mode { kGated, kGrads, kCodes };

template <int kMode>
struct Shape {
    static constexpr int kTileN = kMode == kGated ? kBN / 2 : kBN;  // outputs across a tile
};

__host__ __device__ constexpr int blocks_for(int k) { return k / kBK + (k % kBK != 0); }

struct Unit {
    int mb, nb;
    int h;       // half of the tile's columns that a half unit computes
    int halves;  // 2: whole tile, 1: half unit h, 0: nothing (half past n)
    int dw;      // -1: c; 0, 1: that weight's gradient
};

// Units [0, split_from) are whole tiles; every tile from there on is two half units.
__host__ __device__ __forceinline__ Unit decode(int u, int split_from, int tile_n, int tiles_m, const PairTcParams &p) {
    Unit t;
    const bool half = u >= split_from;
    int tile = half ? split_from + (u - split_from) / 2 : u;
    const int weight = tiles_m * p.tiles_n;
    const int which = tile >= weight ? 1 : 0;  // c has no tiles beyond these
    tile -= which * weight;
    t.dw = which;
    const int first_m = tile / (kGroupM * p.tiles_n) * kGroupM;
    const int gm = kGroupM < tiles_m - first_m ? kGroupM : tiles_m - first_m;
    const int local = tile % (kGroupM * p.tiles_n);
    t.mb = first_m + local % gm;
    t.nb = local / gm;
    t.h = half ? (u - split_from) & 1 : 0;
    t.halves = !half ? 2 : (static_cast<int64_t>(t.nb) * tile_n + t.h * (tile_n / 2) < p.n ? 1 : 0);
    return t;
}

// The units of one pair, the same for all its warps.  Units of c (of the only output, where there is one) go round
// the pairs; where the last round leaves some pairs without, those first take `early` units of the weights'
// gradients each, and what is left of these goes round all pairs again, beginning with pair `behind`.
template <int kMode>
struct Walk {
    const PairTcParams &p;
    const int pair;
    int i = 0;
    __host__ __device__ __forceinline__ Walk(const PairTcParams &params, int own) : p(params), pair(own) {}
    __host__ __device__ __forceinline__ bool next(Unit *t) {
        for (;;) {
            if (!any(t)) return false;
            if (t->halves != 0) return true;
        }
    }

  private:
    __host__ __device__ __forceinline__ bool any(Unit *t) {
        int j = i++;
        const int u = pair + j * p.pairs;
        if (u < p.c_units) {
            *t = decode(u, p.c_split, Shape<kMode>::kTileN, p.tiles_m, p);
            t->dw = -1;
            return true;
        }
        if constexpr (kMode != kGrads) return false;
        j -= p.c_units > pair ? (p.c_units - pair + p.pairs - 1) / p.pairs : 0;
        const int over = p.c_units % p.pairs, without = p.pairs - over;
        const int taken = p.early * without < p.dw_units ? p.early * without : p.dw_units;
        int w;
        if (pair >= over && j < p.early) {
            w = pair - over + j * without;
            if (w >= taken) return false;  // all are taken
        } else {
            if (pair >= over) j -= p.early;
            w = taken + (pair - p.behind + p.pairs) % p.pairs + j * p.pairs;
            if (w >= p.dw_units) return false;
        }
        *t = decode(w, p.dw_split, Shape<kMode>::kTileN, p.dw_tiles_m, p);
        return true;
    }
};

template <typename TC>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A warp's way out for 32 x 32 outputs, one row a lane: through shared memory (swizzled, so that no two
// lanes meet in a bank) and one TMA store, which writes whole row segments and leaves what is outside the matrix
// alone; where TMA cannot write the rows, a row at a time.  Direct 32-byte stores, every lane its own row, held a warp
// for about 700 cycles each.
// Every write commits one bulk group, an empty one where it needs no TMA store: the groups count the writes, so that
// the newest one may be open when the other buffer is written again.
template <typename TC>
struct Writer {
    static constexpr int kBufs = sizeof(TC) == 4 ? 1 : 2;
    uint32_t base;  // 4 KB of shared memory
    int next = 0;

    // where 16-byte piece i of row r lies
    static __device__ __forceinline__ uint32_t piece(int r, int i) {
        return sizeof(TC) == 4 ? r * 128 + ((i ^ (r & 7)) << 4) : r * 64 + ((i ^ ((r >> 1) & 3)) << 4);
    }

    __device__ __forceinline__ void write(const float (&v)[32], const CUtensorMap *map, bool tma, TC *c, int64_t ld,
                                          int64_t row0, int64_t col, int64_t m, int64_t n, int lane) {
        if (row0 >= m || col >= n) return;
        const uint32_t buf = base + static_cast<uint32_t>(next) * (4096 / kBufs);
        next = (next + 1) % kBufs;
        if (lane == 0) bulk_store_read<kBufs - 1>();
        __syncwarp();
        constexpr int kPieces = 32 * sizeof(TC) / 16, kPer = 16 / sizeof(TC);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            uint32_t w[4];
            if constexpr (sizeof(TC) == 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[4 * i + e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack2<TC>(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + piece(lane, i)), "r"(w[0]), "r"(w[1]),
                         "r"(w[2]), "r"(w[3])
                         : "memory");
        }
        // a TMA store writes whole groups of 16 bytes, past the last column where that does not end one
        if (tma && (col + 32 <= n || n * sizeof(TC) % 16 == 0)) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, buf, static_cast<int32_t>(col), static_cast<int32_t>(row0));
                bulk_commit();
            }
            return;
        }
        // rows that TMA cannot write: a row an access, a lane a column
        __syncwarp();
        const int rows = static_cast<int>(m - row0 < 32 ? m - row0 : 32);
        TC *dst = c + row0 * ld + col + lane;
        const bool live = col + lane < n;
#pragma unroll 8
        for (int r = 0; r < rows; ++r, dst += ld) {
            const uint32_t at = buf + piece(r, lane / kPer) + lane % kPer * sizeof(TC);
            if constexpr (sizeof(TC) == 4) {
                uint32_t e;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(e) : "r"(at) : "memory");
                if (live) *reinterpret_cast<uint32_t *>(dst) = e;
            } else {
                uint16_t e;
                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(e) : "r"(at) : "memory");
                if (live) *reinterpret_cast<uint16_t *>(dst) = e;
            }
        }
        if (lane == 0) bulk_commit();
        __syncwarp();
    }
    __device__ __forceinline__ void finish(int lane) const {
        if (lane == 0) bulk_store_done();
    }
};

template <int kAct>
__device__ __forceinline__ void gate32(const uint32_t (&g)[32], const uint32_t (&u)[32], float (&h)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) h[i] = gate_act_16(kAct, __uint_as_float(g[i])) * __uint_as_float(u[i]);
}

template <typename TC, uint32_t kFmt, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
pair_tc_kernel(const __grid_constant__ PairTcMaps maps, const PairTcParams p) {
    constexpr int kTileN = Shape<kMode>::kTileN;
    constexpr bool kBMN = kMode == kGrads;  // B stored [k, n]
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t s0 = raw_addr + pad;  // stage s: A at s0 + s * kStageBytes, B kABytes after it
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes + kEpiWarps * kOutBytes);
    const uint32_t bar0 = smem_addr(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * kStages + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * kStages + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kStages + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();  // 0 issues the MMAs
    const bool leader = rank == 0;
    const uint64_t lim = p.wait_limit_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);   // the even CTA's producer arrive + both CTAs' bytes
            mbar_init(empty_bar(s), 1);  // the pair MMAs' commit
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 2 * kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        // only maps that the call has encoded
        if (kMode != kGrads || p.need_c) {
            tma_prefetch_desc(&maps.a[0]);
            tma_prefetch_desc(&maps.b[0]);
            if (kMode != kCodes) tma_prefetch_desc(&maps.b[1]);
            if (kMode == kGrads) tma_prefetch_desc(&maps.a[1]);
        }
        if (kMode == kGrads && p.need_dw) {
            tma_prefetch_desc(&maps.dw_a[0]);
            tma_prefetch_desc(&maps.dw_a[1]);
            tma_prefetch_desc(&maps.dw_b);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    // both CTAs' barriers exist before any copy, commit or arrival can reach them
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dep_begin();
    const int blocks1 = blocks_for(p.k);  // k-blocks of a source
    // k-blocks of a unit, and how many go into one accumulator
    auto blocks_of = [&](const Unit &t) {
        return kMode != kGrads ? blocks1 : t.dw < 0 ? 2 * blocks1 : blocks_for(p.m);
    };
    const int pair = static_cast<int>(blockIdx.x) >> 1;
    // a timeout stops both CTAs of the pair
    const uint32_t peer_abort = mapa_shared(smem_addr(const_cast<int *>(abort_flag)), rank ^ 1u);
    auto raise_abort = [&]() {
        *abort_flag = 1;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_abort), "r"(1) : "memory");
        report_device_error(p.err, kKidPairTc);
    };

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            Walk<kMode> walk(p, pair);
            for (Unit t; ok && walk.next(&t);) {
                const int kblocks = blocks_of(t);
                const int arow = t.mb * 2 * kBM + static_cast<int>(rank) * kBM;
                // a half unit uses the first 64 of the 128 B rows that each CTA loads
                const int brow = kMode == kGated ? t.nb * kTileN + t.h * (kTileN / 2)
                                 : t.halves == 2 ? t.nb * kTileN + static_cast<int>(rank) * kBM
                                                 : t.nb * kTileN + t.h * (kTileN / 2) + static_cast<int>(rank) * (kBM / 2);
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait_bounded_cluster(empty_bar(stage), phase ^ 1u, lim, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (leader) mbar_arrive_expect_tx(full_bar(stage), 2 * kStageBytes);
                    const uint32_t sa = s0 + stage * kStageBytes, sb = sa + kABytes;
                    const uint32_t fb = mapa_shared(full_bar(stage), 0);
                    const bool outer = kMode == kGrads && t.dw >= 0;
                    const bool second = kMode == kGrads && !outer && kb >= blocks1;
                    const int k0 = (second ? kb - blocks1 : kb) * kBK;
                    if (outer) {
                        const CUtensorMap *ma = t.dw == 1 ? &maps.dw_a[1] : &maps.dw_a[0];
                        tma_load_3d_pair(sa, ma, fb, arow, k0, 0);
                        tma_load_3d_pair(sa + kMNBox, ma, fb, arow + 64, k0, 0);
                    } else {
                        tma_load_3d_pair(sa, second ? &maps.a[1] : &maps.a[0], fb, k0, arow, 0);
                    }
                    if (kBMN) {
                        const CUtensorMap *mb = outer ? &maps.dw_b : second ? &maps.b[1] : &maps.b[0];
                        tma_load_3d_pair(sb, mb, fb, brow, k0, 0);
                        tma_load_3d_pair(sb + kMNBox, mb, fb, brow + 64, k0, 0);
                    } else {
                        tma_load_3d_pair(sb, kMode == kGated && !leader ? &maps.b[1] : &maps.b[0], fb, k0, brow, 0);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // Every stage has been used up before this CTA goes on to its end; a role that gave up after the last copies were
            // issued shows here.
            for (int s = 0; ok && s < kStages; ++s) {
                ok = mbar_wait_bounded_cluster(empty_bar(stage), phase ^ 1u, lim, abort_flag);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {
                raise_abort();
                // copies still in flight land within microseconds; give them 200 us
                const uint64_t t0 = global_ns();
                while (global_ns() - t0 < 200000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ---------------- pair MMA issuer (even CTA) ----------------
            constexpr uint32_t kIdesc = idesc_f16(kFmt, 2 * kBM, kBN, 0u, kBMN ? 1u : 0u);
            constexpr uint32_t kIdescHalf = idesc_f16(kFmt, 2 * kBM, kBN / 2, 0u, kBMN ? 1u : 0u);
            constexpr uint32_t kAColumns = idesc_f16(kFmt, 2 * kBM, kBN, 1u) & ~idesc_f16(kFmt, 2 * kBM, kBN);  // A stored [k, m]
            int stage = 0;
            uint32_t phase = 0;
            uint32_t acc_phase[2] = {0u, 0u};
            bool ok = true;
            int local = 0;
            Walk<kMode> walk(p, pair);
            for (Unit t; ok && walk.next(&t);) {
                const int kblocks = blocks_of(t), chunk = kMode == kCodes ? kExactBlocks : kblocks;
                const bool outer = kMode == kGrads && t.dw >= 0;
                const uint32_t idesc = (t.halves == 2 ? kIdesc : kIdescHalf) | (outer ? kAColumns : 0u);
                for (int c0 = 0; c0 < kblocks && ok; c0 += chunk) {
                    const int a = local++ & 1;
                    // both CTAs' epilogues have read what this accumulator held
                    if (!mbar_wait_bounded_cluster(tempty_bar(a), acc_phase[a] ^ 1u, lim, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(a * kBN);
                    const int c1 = min(c0 + chunk, kblocks);
                    for (int kb = c0; kb < c1; ++kb) {
                        if (!mbar_wait_bounded_cluster(full_bar(stage), phase, lim, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sa = s0 + stage * kStageBytes, sb = sa + kABytes;
#pragma unroll
                        for (int kk = 0; kk < kBK / 16; ++kk) {
                            const uint64_t da = outer ? sdesc_mnmajor_sw128(sa + kk * 2048, kMNBox)
                                                      : sdesc_kmajor_sw128(sa + kk * 32);
                            const uint64_t db = kBMN ? sdesc_mnmajor_sw128(sb + kk * 2048, kMNBox)
                                                     : sdesc_kmajor_sw128(sb + kk * 32);
                            umma_f16_ss_pair(d_tmem, da, db, idesc, kb != c0 || kk != 0 ? 1u : 0u);
                        }
                        umma_commit_pair_mc(empty_bar(stage), 0x3);  // the stage is free in both CTAs
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit_pair_mc(tfull_bar(a), 0x3);
                    acc_phase[a] ^= 1u;
                }
            }
            if (!ok) raise_abort();
            umma_commit_pair_mc(drain_bar, 0x1);
            mbar_wait_bounded(drain_bar, 0, lim, nullptr);
        }
    } else {
        // ---------------- epilogue (warps 2..9, both CTAs) ----------------
        const int quarter = warp & 3;        // TMEM lanes 32 * quarter .. + 31
        const int side = (warp - 2) >> 2;    // which half of a unit's outputs
        uint32_t tphase[2] = {0u, 0u};
        int local = 0;
        bool ok = true;
        Writer<TC> out;
        out.base = s0 + kStages * kStageBytes + static_cast<uint32_t>(warp - 2) * kOutBytes;
        Walk<kMode> walk(p, pair);
        for (Unit t; ok && walk.next(&t);) {
            const int kblocks = blocks_of(t), chunk = kMode == kCodes ? kExactBlocks : kblocks;
            const int64_t row0 = static_cast<int64_t>(t.mb) * 2 * kBM + static_cast<int64_t>(rank) * kBM + quarter * 32;
            const int width = t.halves * (kTileN / 2);  // outputs across this unit
            const int mine = width / 2;                 // and this warp's share of them
            const int64_t col0 = static_cast<int64_t>(t.nb) * kTileN + t.h * (kTileN / 2) + side * mine;
            TC *const c = static_cast<TC *>(p.c);
            // codes: scales of this lane's row and of column lane of each 32
            float sa = 1.f, sb[kMode == kCodes ? 4 : 1];
            if constexpr (kMode == kCodes) {
                if (p.scale_a != nullptr && row0 + lane < p.m) sa = __ldg(p.scale_a + row0 + lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sb[i] = p.scale_b != nullptr && col0 + 32 * i + lane < p.n ? __ldg(p.scale_b + col0 + 32 * i + lane) : 1.f;
            }
            int sum[kMode == kCodes ? kBN / 2 : 1];
            if constexpr (kMode == kCodes) {
#pragma unroll
                for (int i = 0; i < kBN / 2; ++i) sum[i] = 0;
            }
            for (int c0 = 0; c0 < kblocks; c0 += chunk) {
                const int a = local++ & 1;
                int ready = 0;
                // a whole chain of k-blocks (0.28 us each) lies between two arrivals: more than `lim` where m is 2^28
                const uint64_t chain = static_cast<uint64_t>(min(chunk, kblocks - c0)) * kBlockLimitNs;
                if (lane == 0) ready = mbar_wait_bounded_cluster(tfull_bar(a), tphase[a], lim + chain, abort_flag);
                ready = __shfl_sync(0xffffffffu, ready, 0);
                if (!ready) {
                    if (lane == 0) raise_abort();
                    ok = false;
                    break;
                }
                __syncwarp();
                tc_fence_after();
                const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                        static_cast<uint32_t>(a * kBN + side * mine);
                if constexpr (kMode == kCodes) {
#pragma unroll
                    for (int i = 0; i < kBN / 2; i += 16) {
                        if (i >= mine) break;
                        uint32_t r[16];
                        tmem_ld16(t_addr + i, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum[i + e] += __float2int_rn(__uint_as_float(r[e]));
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < mine; i += 32) {
                        uint32_t r[32];
                        float v[32];
                        tmem_ld32(t_addr + i, r);
                        const int64_t col = col0 + i;
                        if constexpr (kMode == kGated) {
                            uint32_t q[32];
                            tmem_ld32(t_addr + width + i, q);
                            tmem_ld_wait();
                            switch (p.act) {
                            case GBMM_GATE_SILU: gate32<GBMM_GATE_SILU>(r, q, v); break;
                            case GBMM_GATE_GELU: gate32<GBMM_GATE_GELU>(r, q, v); break;
                            case GBMM_GATE_GELU_TANH: gate32<GBMM_GATE_GELU_TANH>(r, q, v); break;
                            default: gate32<GBMM_GATE_RELU>(r, q, v);
                            }
                            out.write(v, &maps.out[0], p.c_tma, c, p.ldc, row0, col, p.m, p.n, lane);
                            if (p.saved[0] != nullptr) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
                                out.write(v, &maps.out[1], p.saved_tma, static_cast<TC *>(p.saved[0]), p.ld_saved, row0,
                                          col, p.m, p.n, lane);
#pragma unroll
                                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(q[e]);
                                out.write(v, &maps.out[2], p.saved_tma, static_cast<TC *>(p.saved[1]), p.ld_saved, row0,
                                          col, p.m, p.n, lane);
                            }
                        } else {
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
                            if (kMode == kGrads && t.dw >= 0)
                                out.write(v, t.dw == 0 ? &maps.out[1] : &maps.out[2], p.dw_tma,
                                          static_cast<TC *>(t.dw == 0 ? p.dw[0] : p.dw[1]), p.ld_dw, row0, col, p.k, p.n,
                                          lane);
                            else
                                out.write(v, &maps.out[0], p.c_tma, c, p.ldc, row0, col, p.m, p.n, lane);
                        }
                    }
                }
                // this CTA's rows of the accumulator are read: hand it back to the even CTA's issuer
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(tempty_bar(a), 0));
                tphase[a] ^= 1u;
            }
            if constexpr (kMode == kCodes) {
                if (ok) {
#pragma unroll
                    for (int i = 0; i < kBN / 2; i += 32) {
                        if (i >= mine) break;
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = static_cast<float>(sum[i + e]) * sa * __shfl_sync(0xffffffffu, sb[i / 32], e);
                        out.write(v, &maps.out[0], p.c_tma, c, p.ldc, row0, col0 + i, p.m, p.n, lane);
                    }
                }
            }
        }
        out.finish(lane);
    }

    tc_fence_before();
    __syncthreads();
    // every pair MMA has completed (the even CTA waited for its drain) and both CTAs' epilogues are
    // done before either CTA releases the columns
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

// Tiles of the last round become half units where that round would leave half of the pairs idle: of `tiles` on
// `pairs`, as many as this.
int last_tiles(int tiles, int pairs) {
    const int last = tiles > pairs ? tiles % pairs : (2 * tiles <= pairs ? tiles : 0);
    return 2 * last <= pairs ? last : 0;
}

// Sets the units and how Walk deals them out.  With both outputs: the division, of the few that there are, whose
// busiest pair has the least to do, in k-blocks of `c_cost` and `dw_cost` a tile.
void plan_units(PairTcParams *p, int c_tiles, int dw_tiles, int c_cost, int dw_cost) {
    const int pairs = p->pairs;
    auto units = [](int tiles, int halved, int32_t *count, int32_t *split) {
        *split = tiles - halved;
        *count = tiles + halved;
    };
    p->early = p->behind = 0;
    units(c_tiles, dw_tiles == 0 ? last_tiles(c_tiles, pairs) : 0, &p->c_units, &p->c_split);
    units(dw_tiles, c_tiles == 0 ? last_tiles(dw_tiles, pairs) : 0, &p->dw_units, &p->dw_split);
    if (c_tiles == 0 || dw_tiles == 0) return;
    constexpr double kHalf = 0.6;  // of a tile's time for half of it: A is read as often
    double best = -1;
    const PairTcParams whole = *p;
    for (int halve = 0; halve < (last_tiles(c_tiles, pairs) > 0 ? 2 : 1); ++halve) {
        PairTcParams q = whole;
        units(c_tiles, halve ? last_tiles(c_tiles, pairs) : 0, &q.c_units, &q.c_split);
        const int over = q.c_units % pairs, without = pairs - over, rounds = q.c_units / pairs;
        const double last = halve ? kHalf * c_cost : c_cost;  // what the pairs before `over` have more
        // whole rounds of c (halved tiles begin a round or are all there is)
        const double base = halve && q.c_split == 0 && rounds > 0 ? kHalf * c_cost * rounds : 1.0 * c_cost * rounds;
        for (int up = 0; up < (over > 0 ? 2 : 1); ++up) {
            q.early = over > 0 ? static_cast<int>(last / dw_cost) + up : 0;
            if (q.early > dw_tiles) q.early = dw_tiles;
            const int taken = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(q.early) * without, dw_tiles));
            const int rest = dw_tiles - taken;
            const bool first_without = over > 0 && q.early * dw_cost < last;  // whose turn it is then
            q.behind = first_without ? over : 0;
            for (int h = 0; h < 2; ++h) {
                const int halved = h ? last_tiles(rest, pairs) : 0;
                if (h && halved == 0) break;
                units(dw_tiles, halved, &q.dw_units, &q.dw_split);
                const int left = rest + halved, every = left / pairs, more = left % pairs;
                // units of the last round weigh `unit` each
                const double unit = halved ? kHalf * dw_cost : dw_cost;
                double most = 0;
                for (int c = 0; c < pairs; ++c) {
                    const bool without_one = c >= over;
                    double load = base + (without_one ? 0 : last);
                    if (without_one && q.early > 0) {
                        const int own = c - over < taken ? (taken - 1 - (c - over)) / without + 1 : 0;
                        load += static_cast<double>(own) * dw_cost;
                    }
                    load += static_cast<double>(every) * (halved && rest < pairs ? unit : dw_cost);
                    if ((c - q.behind + pairs) % pairs < more) load += unit;
                    most = std::max(most, load);
                }
                if (best < 0 || most < best) {
                    best = most;
                    *p = q;
                }
            }
        }
    }
}

template <typename TC, uint32_t kFmt, int kMode>
cudaError_t pair_t(const PairTcMaps &maps, PairTcParams p, int num_sms, cudaStream_t s) {
    constexpr int kTileN = Shape<kMode>::kTileN;
    static DeviceBits attr_set{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(attr_set & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(pair_tc_kernel<TC, kFmt, kMode>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_set |= bit;
    }
    const int pairs = num_sms / 2;
    const int64_t tn = (static_cast<int64_t>(p.n) + kTileN - 1) / kTileN, tm = (static_cast<int64_t>(p.m) + 2 * kBM - 1) / (2 * kBM);
    const int64_t wm = (static_cast<int64_t>(p.k) + 2 * kBM - 1) / (2 * kBM);
    const int64_t c_tiles = kMode == kGrads && !p.need_c ? 0 : tm * tn;
    const int64_t dw_tiles = kMode == kGrads && p.need_dw ? 2 * wm * tn : 0;
    if (pairs < 1 || c_tiles + dw_tiles < 1 || c_tiles > INT32_MAX / 4 || dw_tiles > INT32_MAX / 4)
        return cudaErrorInvalidConfiguration;
    p.tiles_m = static_cast<int32_t>(tm);
    p.dw_tiles_m = static_cast<int32_t>(wm);
    p.tiles_n = static_cast<int32_t>(tn);
    p.pairs = pairs;
    plan_units(&p, static_cast<int>(c_tiles), static_cast<int>(dw_tiles), 2 * blocks_for(p.k),
               blocks_for(p.m));
    const int units = p.c_units + p.dw_units;
    // the first pairs have all units where there are fewer of them than pairs
    const int clusters = units < pairs && (p.c_units == 0 || p.dw_units == 0 || p.early > 0) ? units : pairs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, pair_tc_kernel<TC, kFmt, kMode>, maps, p);
}

}  // namespace

cudaError_t launch_gated_tc(int dt, const PairTcMaps &maps, const PairTcParams &p, int num_sms, cudaStream_t s) {
    return dt == kF16 ? pair_t<__half, 0, kGated>(maps, p, num_sms, s)
                      : pair_t<__nv_bfloat16, 1, kGated>(maps, p, num_sms, s);
}
cudaError_t launch_gated_products_tc(int dt, const PairTcMaps &maps, const PairTcParams &p, int num_sms, cudaStream_t s) {
    return dt == kF16 ? pair_t<__half, 0, kGrads>(maps, p, num_sms, s)
                      : pair_t<__nv_bfloat16, 1, kGrads>(maps, p, num_sms, s);
}
cudaError_t launch_gemm_i8_tc(int dt, const PairTcMaps &maps, const PairTcParams &p, int num_sms, cudaStream_t s) {
    switch (dt) {
    case kF32: return pair_t<float, 0, kCodes>(maps, p, num_sms, s);
    case kF16: return pair_t<__half, 0, kCodes>(maps, p, num_sms, s);
    case kBF16: return pair_t<__nv_bfloat16, 0, kCodes>(maps, p, num_sms, s);
    default: return cudaErrorInvalidValue;
    }
}

int pair_tc_rows() { return kBM; }
int pair_tc_block_k() { return kBK; }

}  // namespace gbmm
