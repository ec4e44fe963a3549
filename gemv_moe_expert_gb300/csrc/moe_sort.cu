// moe_sort.cu -- stable counting sort of routed rows by expert.
//
// key[r] = min(ids[r], n_experts).  Three launches: (0) each CTA counts its
// tile of kTile rows per key; (1) one warp per key turns the tiles' counts into
// an exclusive prefix along the tiles and a total; (2) each CTA scans the totals
// into the keys' first places, ranks its rows within the tile (rows of one
// warp in order, matched lanes by lane number) and writes both permutations.
// No atomics decide an order, so the result is exactly the stable one.
#include "device_common.cuh"

namespace gbmm {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 4;
constexpr int kTile = kThreads * kPerThread;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kMaxKeys = 1025;

__host__ __device__ __forceinline__ uint32_t tiles_of(uint64_t rows) {
    return rows == 0 ? 1u : static_cast<uint32_t>((rows + kTile - 1) / kTile);
}

// scratch: counts[key][tile], then totals[key]
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
        uint32_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += v;
        }
        if (t0 + lane < tiles) row[t0 + lane] = run + inc - c;
        run += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0) p.scratch[static_cast<int64_t>(keys) * tiles + e] = run;
}

__global__ void __launch_bounds__(kThreads) moe_sort_place_kernel(MoeSortParams p) {
    extern __shared__ uint16_t counts[];  // [kWarps][keys]
    __shared__ uint32_t first[kMaxKeys];  // place of the tile's first row of each key
    __shared__ uint32_t warp_sums[kWarps];
    const uint32_t keys = p.n_experts + 1, tiles = gridDim.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint16_t *mine = counts + static_cast<uint32_t>(warp) * keys;
    for (uint32_t e = lane; e < keys; e += 32) mine[e] = 0;
    __syncwarp();

    // this warp's rows: kPerThread runs of 32 in order
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile + static_cast<int64_t>(warp) * 32 * kPerThread;
    uint32_t key[kPerThread];
    uint16_t rank[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        const int64_t r = base + j * 32 + lane;
        key[j] = r < p.rows ? min(p.ids[r], p.n_experts) : kFull;
    }
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        const unsigned same = __match_any_sync(kFull, key[j]);
        rank[j] = 0;
        if (key[j] != kFull) rank[j] = mine[key[j]] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (key[j] != kFull && lane == __ffs(same) - 1) mine[key[j]] += __popc(same);
        __syncwarp();
    }

    // exclusive scan of the totals over the keys (two per thread)
    const uint32_t *totals = p.scratch + static_cast<int64_t>(keys) * tiles;
    const uint32_t e0 = 2 * tid, e1 = e0 + 1;
    const uint32_t c0 = e0 < keys ? totals[e0] : 0u, c1 = e1 < keys ? totals[e1] : 0u;
    uint32_t inc = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    uint32_t below = 0;
    for (int w = 0; w < warp; ++w) below += warp_sums[w];
    const uint32_t start0 = below + inc - c0 - c1, start1 = start0 + c0;
    if (e0 < keys) first[e0] = start0 + p.scratch[static_cast<int64_t>(e0) * tiles + blockIdx.x];
    if (e1 < keys) first[e1] = start1 + p.scratch[static_cast<int64_t>(e1) * tiles + blockIdx.x];
    if (blockIdx.x == 0) {
        if (e0 < keys) p.offsets[e0] = start0;
        if (e1 < keys) p.offsets[e1] = start1;
    }
    // exclusive scan of the warps' counts for each key
    for (uint32_t e = tid; e < keys; e += kThreads) {
        uint32_t run = 0;
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = counts[static_cast<uint32_t>(w) * keys + e];
            counts[static_cast<uint32_t>(w) * keys + e] = static_cast<uint16_t>(run);
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
        if (key[j] == kFull) continue;
        const uint32_t r = static_cast<uint32_t>(base + j * 32 + lane);
        const uint32_t at = first[key[j]] + mine[key[j]] + rank[j];
        p.position[r] = at;
        p.order[at] = r;
    }
}

}  // namespace

uint64_t moe_sort_scratch_words(uint64_t rows, uint32_t n_experts) {
    return (static_cast<uint64_t>(tiles_of(rows)) + 1) * (n_experts + 1ull);
}

int moe_sort_launches(uint64_t, uint32_t) { return 3; }

cudaError_t launch_moe_sort(int step, const MoeSortParams &p, cudaStream_t s) {
    const uint32_t keys = p.n_experts + 1, tiles = tiles_of(p.rows);
    if (step == 0) {
        moe_sort_count_kernel<<<tiles, kThreads, 0, s>>>(p);
    } else if (step == 1) {
        moe_sort_scan_kernel<<<(keys + 7) / 8, 256, 0, s>>>(p, tiles);
    } else {
        const size_t smem = static_cast<size_t>(kWarps) * keys * sizeof(uint16_t);
        static unsigned long long attr_set = 0;
        int dev = 0;
        cudaGetDevice(&dev);
        const unsigned long long bit = 1ull << (dev & 63);
        if (!(attr_set & bit)) {
            cudaError_t e = cudaFuncSetAttribute(moe_sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kWarps * kMaxKeys * static_cast<int>(sizeof(uint16_t)));
            if (e != cudaSuccess) return e;
            attr_set |= bit;
        }
        moe_sort_place_kernel<<<tiles, kThreads, smem, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace gbmm
