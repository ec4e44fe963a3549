// moe_sort.cu -- stable counting sort of routed rows by expert.
//
// key[r] = min(ids[r], n_experts).  A CTA ranks a tile of kTile rows: each warp
// holds kPerThread runs of 32 consecutive rows, lanes with equal keys find each
// other with one match instruction, and one of them advances the warp's count
// of that key in shared memory; scans over the warps, over the tiles and over
// the keys then give every row its place.  No atomics decide an order, so the
// result is exactly the stable one.
//
// Up to kClusterTiles tiles run as one launch: one cluster with a CTA for each
// tile, which read each other's counts through distributed shared memory.  More
// tiles take three launches (count, scan along the tiles, place) and scratch for
// the counts of every tile.
#include <cooperative_groups.h>

#include "device_common.cuh"

namespace cg = cooperative_groups;

namespace gbmm {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 4;
constexpr int kTile = kThreads * kPerThread;
constexpr int kClusterTiles = 8;  // portable cluster size
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kMaxKeys = 1025;
constexpr uint32_t kPitch = kWarps + 1;  // counts[key][warp]: an odd pitch spreads the keys over the banks

__host__ __device__ __forceinline__ uint32_t tiles_of(uint64_t rows) {
    return rows == 0 ? 1u : static_cast<uint32_t>((rows + kTile - 1) / kTile);
}

__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// One tile's rows, in the registers of the CTA's threads.
struct Tile {
    uint32_t key[kPerThread];   // kFull past the end
    uint32_t rank[kPerThread];  // among the warp's earlier rows of the same key
    int64_t row;                // of j = 0; run j is 32 j further

    // loads tile `index`, ranks its rows within their warps; counts is left with
    // the number of rows of each (key, warp)
    __device__ __forceinline__ void load(const MoeSortParams &p, uint32_t index, uint16_t *counts) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const uint32_t keys = p.n_experts + 1;
        row = static_cast<int64_t>(index) * kTile + warp * (32 * kPerThread) + lane;
#pragma unroll
        for (int j = 0; j < kPerThread; ++j)
            key[j] = row + 32 * j < p.rows ? min(__ldg(p.ids + row + 32 * j), p.n_experts) : kFull;
        uint32_t *words = reinterpret_cast<uint32_t *>(counts);
        for (uint32_t i = threadIdx.x; i < (keys * kPitch + 1) / 2; i += kThreads) words[i] = 0u;
        unsigned same[kPerThread];
#pragma unroll
        for (int j = 0; j < kPerThread; ++j) same[j] = __match_any_sync(kFull, key[j]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPerThread; ++j) {
            uint16_t *mine = counts + key[j] * kPitch + warp;
            const bool has = key[j] != kFull;
            const uint32_t before = has ? *mine : 0u;
            rank[j] = before + __popc(same[j] & ((1u << lane) - 1u));
            __syncwarp();
            if (has && lane == __ffs(same[j]) - 1) *mine = static_cast<uint16_t>(before + __popc(same[j]));
            __syncwarp();
        }
        __syncthreads();
    }

    __device__ __forceinline__ void place(const MoeSortParams &p, const uint16_t *counts, const uint32_t *first) const {
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int j = 0; j < kPerThread; ++j) {
            if (key[j] == kFull) continue;
            const uint32_t r = static_cast<uint32_t>(row + 32 * j);
            const uint32_t at = first[key[j]] + counts[key[j] * kPitch + warp] + rank[j];
            p.position[r] = at;
            p.order[at] = r;
        }
    }
};

// counts[key][*] become exclusive prefixes over the warps (warp w in lane w), total[key] their sum
__device__ __forceinline__ void scan_warps(uint32_t keys, uint16_t *counts, uint32_t *total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (uint32_t e = warp; e < keys; e += kWarps) {
        const uint32_t c = counts[e * kPitch + lane];
        const uint32_t inc = warp_inclusive(c, lane);
        counts[e * kPitch + lane] = static_cast<uint16_t>(inc - c);
        if (lane == 31) total[e] = inc;
    }
}

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
    extern __shared__ __align__(16) uint16_t counts[];  // [keys][kPitch]
    __shared__ uint32_t total[kMaxKeys], first[kMaxKeys], all[kClusterTiles][kMaxKeys], warp_sums[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t keys = p.n_experts + 1, rank = cluster.block_rank(), tiles = cluster.num_blocks();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    Tile tile;
    tile.load(p, rank, counts);
    scan_warps(keys, counts, total);
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA runs: its shared memory can be written
    for (uint32_t e = threadIdx.x; e < keys; e += kThreads) {
        const uint32_t n = total[e];
        for (uint32_t b = 0; b < tiles; ++b) *cluster.map_shared_rank(&all[rank][e], b) = n;
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
    tile.place(p, counts, first);
}

// ---- three launches; scratch: counts[key][tile], then totals[key] ----

__global__ void __launch_bounds__(kThreads) moe_sort_count_kernel(MoeSortParams p) {
    __shared__ uint32_t hist[kMaxKeys];
    const uint32_t keys = p.n_experts + 1, tiles = gridDim.x;
    for (uint32_t e = threadIdx.x; e < keys; e += kThreads) hist[e] = 0u;
    __syncthreads();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
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
    if (e >= keys) return;
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
    extern __shared__ __align__(16) uint16_t counts[];  // [keys][kPitch]
    __shared__ uint32_t total[kMaxKeys], first[kMaxKeys], warp_sums[kWarps];
    const uint32_t keys = p.n_experts + 1, tiles = gridDim.x;
    Tile tile;
    tile.load(p, blockIdx.x, counts);
    scan_warps(keys, counts, total);
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
    tile.place(p, counts, first);
}

template <typename K>
cudaError_t allow_smem(K *kernel, unsigned long long *done) {
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (*done & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((kMaxKeys * kPitch + 1) / 2 * 4));
    if (e == cudaSuccess) *done |= bit;
    return e;
}

}  // namespace

uint64_t moe_sort_scratch_words(uint64_t rows, uint32_t n_experts) {
    const uint64_t tiles = tiles_of(rows);
    return tiles <= kClusterTiles ? 0 : (tiles + 1) * (n_experts + 1ull);
}

int moe_sort_launches(uint64_t rows) { return tiles_of(rows) <= kClusterTiles ? 1 : 3; }

cudaError_t launch_moe_sort(int step, const MoeSortParams &p, cudaStream_t s) {
    static unsigned long long cluster_done = 0, place_done = 0;
    const uint32_t keys = p.n_experts + 1, tiles = tiles_of(p.rows);
    const size_t smem = (static_cast<size_t>(keys) * kPitch + 1) / 2 * 4;
    if (tiles <= kClusterTiles) {
        const cudaError_t e = allow_smem(moe_sort_cluster_kernel, &cluster_done);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(tiles, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = tiles;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, moe_sort_cluster_kernel, p);
    }
    if (step == 0) {
        moe_sort_count_kernel<<<tiles, kThreads, 0, s>>>(p);
    } else if (step == 1) {
        moe_sort_scan_kernel<<<(keys + 7) / 8, 256, 0, s>>>(p, tiles);
    } else {
        const cudaError_t e = allow_smem(moe_sort_place_kernel, &place_done);
        if (e != cudaSuccess) return e;
        moe_sort_place_kernel<<<tiles, kThreads, smem, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace gbmm
