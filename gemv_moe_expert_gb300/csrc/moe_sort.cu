// moe_sort.cu -- stable counting sort of routed rows by expert.
//
// key[r] = min(ids[r], n_experts).  A CTA ranks a tile of rows: each warp holds P
// runs of 32 consecutive rows, a run's lanes with equal keys find each other
// through a bit mask of the key in shared memory (one OR a lane; the mask holds
// the lanes whatever the order of the ORs), and the first of them advances the
// warp's count of the key; scans over the warps, over the tiles and over the keys
// then give every row its place.  No atomics decide an order, so the result is
// exactly the stable one.
//
// Up to kClusterTiles small tiles run as one launch: one cluster with a CTA for
// each tile.  More rows take three launches of larger tiles (count, scan along the
// tiles, place) and scratch for the counts of every tile.  Bound by latency: a few
// bytes a row, and a chain of loads, shared-memory passes and barriers (32768 rows
// of 128 experts 6.2 us, 524288 rows 10.3 us; with match.any in place of the masks
// and eight tiles of 4096 rows 10.3 us, without the early start 18.5 us).
#include <cooperative_groups.h>

#include "device_common.cuh"

namespace cg = cooperative_groups;

namespace gbmm {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterP = 2, kLargeP = 4;  // rows a thread
// The largest cluster; a GB300 has room for one with the shared memory that 1024 experts take (226 KB
// a CTA, one CTA an SM).
constexpr int kClusterTiles = 16;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kMaxKeys = 1025;
constexpr uint32_t kPitch = kWarps + 1;  // counts[key][warp]: an odd pitch spreads the keys over the banks

constexpr uint64_t tiles_of(uint64_t rows, int P) {
    const uint64_t tile = static_cast<uint64_t>(kThreads) * P;
    return rows == 0 ? 1 : (rows + tile - 1) / tile;
}

// shared memory of a tile: masks[warp][key], then counts[key][warp]
constexpr size_t tile_bytes(uint32_t keys) { return (static_cast<size_t>(keys) * (2 * kWarps + kPitch) + 7) / 8 * 16; }

__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// One tile's rows, in the registers of the CTA's threads.
template <int P> struct Tile {
    uint32_t key[P];   // kFull past the end
    uint32_t rank[P];  // among the warp's earlier rows of the same key
    int64_t row;       // of j = 0; run j is 32 j further
    uint16_t *counts;  // [key][kPitch]

    // Loads tile `index`, ranks its rows within their warps and scans the warps: counts
    // becomes, for each key, the number of rows of the warps before; total their sum.
    __device__ __forceinline__ void load(const MoeSortParams &p, uint32_t index, uint32_t *smem, uint32_t *total) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const uint32_t keys = p.n_experts + 1;
        row = static_cast<int64_t>(index) * (kThreads * P) + warp * (32 * P) + lane;
#pragma unroll
        for (int j = 0; j < P; ++j)
            key[j] = row + 32 * j < p.rows ? min(__ldg(p.ids + row + 32 * j), p.n_experts) : kFull;
        uint32_t *masks = smem + warp * keys;
        counts = reinterpret_cast<uint16_t *>(smem + kWarps * keys);
        for (uint32_t i = threadIdx.x; i < tile_bytes(keys) / 16; i += kThreads)
            reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const bool has = key[j] != kFull;
            if (has) atomicOr(masks + key[j], 1u << lane);
            __syncwarp();
            const uint32_t same = has ? masks[key[j]] : 0u;
            uint16_t *mine = counts + key[j] * kPitch + warp;
            const uint32_t before = has ? *mine : 0u;
            rank[j] = before + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (has && lane == __ffs(same) - 1) {
                *mine = static_cast<uint16_t>(before + __popc(same));
                masks[key[j]] = 0u;
            }
            __syncwarp();
        }
        __syncthreads();
        for (uint32_t e = threadIdx.x; e < keys; e += kThreads) {
            uint16_t *c = counts + e * kPitch;
            uint32_t run = 0;
#pragma unroll
            for (int w0 = 0; w0 < kWarps; w0 += 8) {
                uint32_t n[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) n[w] = c[w0 + w];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    c[w0 + w] = static_cast<uint16_t>(run);
                    run += n[w];
                }
            }
            total[e] = run;
        }
        __syncthreads();
    }

    __device__ __forceinline__ void place(const MoeSortParams &p, const uint32_t *first) const {
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            if (key[j] == kFull) continue;
            const uint32_t r = static_cast<uint32_t>(row + 32 * j);
            const uint32_t at = first[key[j]] + counts[key[j] * kPitch + warp] + rank[j];
            p.position[r] = at;
            p.order[at] = r;
        }
    }
};

// Exclusive scan over the keys, two to a thread: c0 and c1 are the counts of
// keys 2 tid and 2 tid + 1.  Returns the first place of key 2 tid.
__device__ __forceinline__ uint32_t scan_keys(uint32_t c0, uint32_t c1, uint32_t *warp_sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t inc = warp_inclusive(c0 + c1, lane);
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    const uint32_t s = warp_sums[lane];
    const uint32_t below = __shfl_sync(kFull, warp_inclusive(s, lane) - s, warp);
    return below + inc - c0 - c1;
}

// ---- one launch: a cluster whose CTA c owns tile c ----
//
// Each CTA writes its totals into every CTA's shared memory (stores need no answer;
// reading the others' totals would wait for each of them in turn), and one cluster
// barrier makes them visible.
__global__ void __launch_bounds__(kThreads, 1) moe_sort_cluster_kernel(const __grid_constant__ MoeSortParams p) {
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ __align__(4) uint16_t all[kClusterTiles][kMaxKeys + 1];  // [tile][key]
    __shared__ uint32_t warp_sums[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t keys = p.n_experts + 1, rank = cluster.block_rank(), tiles = cluster.num_blocks();
    uint32_t *total = smem, *first = smem + keys;  // over the masks, which are done with by then
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    grid_dep_begin();
    Tile<kClusterP> tile;
    tile.load(p, rank, smem, total);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA runs: its shared memory can be written
    for (uint32_t e = 2 * threadIdx.x; e < keys; e += 2 * kThreads) {
        const uint32_t pair = total[e] | (e + 1 < keys ? total[e + 1] << 16 : 0u);
        uint32_t *to = reinterpret_cast<uint32_t *>(&all[rank][e]);
        for (uint32_t b = 0; b < tiles; ++b) *cluster.map_shared_rank(to, b) = pair;
    }
    cluster.sync();  // every tile's totals have arrived
    uint32_t c[2], below[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t e = 2 * threadIdx.x + i;
        c[i] = below[i] = 0;
        if (e < keys) {
#pragma unroll
            for (uint32_t b = 0; b < kClusterTiles; ++b) {
                const uint32_t n = b < tiles ? all[b][e] : 0u;
                c[i] += n;
                if (b < rank) below[i] += n;
            }
        }
    }
    uint32_t start = scan_keys(c[0], c[1], warp_sums);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t e = 2 * threadIdx.x + i;
        if (e < keys) {
            first[e] = start + below[i];
            if (rank == 0) p.offsets[e] = start;
        }
        start += c[i];
    }
    __syncthreads();
    tile.place(p, first);
}

// ---- three launches; scratch: counts[key][tile], then totals[key] ----
//
// The second and third start while the one before them runs (programmatic
// dependent launch) and wait for it before they touch scratch: the third ranks its
// tile meanwhile.

__global__ void __launch_bounds__(kThreads) moe_sort_count_kernel(MoeSortParams p) {
    __shared__ uint32_t hist[kMaxKeys];
    const uint32_t keys = p.n_experts + 1, tiles = gridDim.x;
    grid_dep_launch_dependents();
    for (uint32_t e = threadIdx.x; e < keys; e += kThreads) hist[e] = 0u;
    __syncthreads();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads * kLargeP);
#pragma unroll
    for (int j = 0; j < kLargeP; ++j) {
        const int64_t r = base + j * kThreads + threadIdx.x;
        if (r < p.rows) atomicAdd(&hist[min(p.ids[r], p.n_experts)], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < keys; e += kThreads)
        p.scratch[static_cast<int64_t>(e) * tiles + blockIdx.x] = hist[e];
}

__global__ void __launch_bounds__(256) moe_sort_scan_kernel(MoeSortParams p, uint32_t tiles) {
    const uint32_t keys = p.n_experts + 1;
    const uint32_t e = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    grid_dep_launch_dependents();
    if (e >= keys) return;
    grid_dep_wait();
    uint32_t *row = p.scratch + static_cast<int64_t>(e) * tiles;
    uint32_t run = 0;
    for (uint32_t t0 = 0; t0 < tiles; t0 += 32) {
        const uint32_t c = t0 + lane < tiles ? row[t0 + lane] : 0u;
        const uint32_t inc = warp_inclusive(c, lane);
        if (t0 + lane < tiles) row[t0 + lane] = run + inc - c;
        run += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) p.scratch[static_cast<int64_t>(keys) * tiles + e] = run;
}

__global__ void __launch_bounds__(kThreads, 1) moe_sort_place_kernel(MoeSortParams p) {
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ uint32_t warp_sums[kWarps];
    const uint32_t keys = p.n_experts + 1, tiles = gridDim.x;
    uint32_t *total = smem, *first = smem + keys;  // over the masks, which are done with by then
    grid_dep_launch_dependents();
    Tile<kLargeP> tile;
    tile.load(p, blockIdx.x, smem, total);
    grid_dep_wait();
    const uint32_t *totals = p.scratch + static_cast<int64_t>(keys) * tiles;
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = 2 * threadIdx.x + i < keys ? totals[2 * threadIdx.x + i] : 0u;
    uint32_t start = scan_keys(c[0], c[1], warp_sums);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t e = 2 * threadIdx.x + i;
        if (e < keys) {
            first[e] = start + p.scratch[static_cast<int64_t>(e) * tiles + blockIdx.x];
            if (blockIdx.x == 0) p.offsets[e] = start;
        }
        start += c[i];
    }
    __syncthreads();
    tile.place(p, first);
}

// once for each device: the kernel may use the shared memory of kMaxKeys keys, and
// clusters of more than 8 CTAs
template <typename K>
cudaError_t allow(K *kernel, bool cluster, DeviceBits *done) {
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (*done & bit) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(tile_bytes(kMaxKeys)));
    if (e == cudaSuccess && cluster) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) *done |= bit;
    return e;
}

}  // namespace

uint64_t moe_sort_scratch_words(uint64_t rows, uint32_t n_experts) {
    return tiles_of(rows, kClusterP) <= kClusterTiles ? 0 : (tiles_of(rows, kLargeP) + 1) * (n_experts + 1ull);
}

int moe_sort_launches(uint64_t rows) { return tiles_of(rows, kClusterP) <= kClusterTiles ? 1 : 3; }

cudaError_t prepare_moe_sort(uint64_t rows) {
    static DeviceBits cluster_done{0}, place_done{0};
    if (moe_sort_launches(rows) == 1) return allow(moe_sort_cluster_kernel, true, &cluster_done);
    return allow(moe_sort_place_kernel, false, &place_done);
}

cudaError_t launch_moe_sort(int step, const MoeSortParams &p, cudaStream_t s) {
    const uint32_t keys = p.n_experts + 1;
    const size_t smem = tile_bytes(keys);
    if (moe_sort_launches(p.rows) == 1) {
        const unsigned tiles = static_cast<unsigned>(tiles_of(p.rows, kClusterP));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(tiles, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = tiles;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, moe_sort_cluster_kernel, p);
    }
    const unsigned tiles = static_cast<unsigned>(tiles_of(p.rows, kLargeP));
    if (step == 0) {
        // not early: the kernel two launches on reads the ids before it waits
        moe_sort_count_kernel<<<tiles, kThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    if (step == 1) return launch_early(moe_sort_scan_kernel, (keys + 7) / 8, 256, 0, s, p, tiles);
    return launch_early(moe_sort_place_kernel, tiles, kThreads, smem, s, p);
}

}  // namespace gbmm
