// q4.cuh -- matrix-vector products with 4-bit weights and group scales, dense or
// per expert id: the kernel, instantiated for one type of x in each q4_*.cu.
//
//   y[i, j] = sum over groups g of s[j,g] * sum over x in g of (q[j,x] - z[j,g]) x[i,x]
//
// The weights are read once from HBM and have to become multiplier operands: the
// kernel is bound by that stream, and next by the instructions that unpack it.
// So the products run on the tensor cores straight from registers (mma m16n8k16:
// 16 weight rows x 16 columns against 8 columns of x): a thread masks two codes
// at a time into 16-bit floats whose mantissa holds the code, subtracts the zero
// point (exactly: the codes are small integers) and has half an A register; a
// product in f32 registers would also have to widen every code and multiply it
// once per row of x.  The sum of a group is an f32 accumulator, scaled into the
// result by one f32 multiply-add a group.
//
// The order of a contraction is free, so a thread keeps the 16 bytes it loads
// (32 neighbouring codes of a row) and x is stored in shared memory in the order
// in which those codes come out of the words: with groups of 128 columns a quad of
// lanes covers one group; for groups of 64 and 32 the lanes of a quad first
// exchange words, so that one mma never mixes two groups.
//
// x in f32 is split exactly into three bf16 terms (8 significant bits each) that
// take three columns of the mma's eight; the f32 sum of the three products is
// exact up to the accumulator's rounding.
//
// A CTA has kWarps warps: wk of them split the columns (chunks of 128, one after
// the other) of the same 16 rows, and kWarps / wk take different rows.  Each warp
// keeps kDepth chunks of weights in flight in registers.
#pragma once

#include "device_common.cuh"

namespace gbmm {
namespace q4 {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kWindow = 1024;  // routed rows that a CTA searches for its expert's
constexpr uint32_t kFull = 0xffffffffu;

enum Kind { kHalf, kBfloat, kFloat };  // type of x

// NT column tiles of 8: chunks in flight a warp, CTAs an SM, and the shared
// memory for a slab of x, which holds kDepth chunks of every column for each of 4
// warps at least.
template <int NT> struct Budget {
    static constexpr int kDepth = NT == 1 ? 4 : 2;
    static constexpr int kCtas = NT == 1 ? 5 : 4;
    static constexpr int kStageBytes = NT == 1 ? 34 * 1024 : NT == 2 ? 36 * 1024 : 56 * 1024;
    static_assert((kStageBytes / (8 * NT) - 64) / 256 >= kWarps * kDepth, "a slab holds kDepth chunks a warp");
};

template <Kind K> struct XType;
template <> struct XType<kHalf> { using type = __half; };
template <> struct XType<kBfloat> { using type = __nv_bfloat16; };
template <> struct XType<kFloat> { using type = float; };

__device__ __forceinline__ uint32_t mask_or(uint32_t w, uint32_t mask, uint32_t bits) { return (w & mask) | bits; }

__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t *>(&h); }

// The four pairs (q[i] - z, q[i + 4] - z), i < 4, of a word's eight codes, as
// 16-bit floats.  f16: 0x6400 | c is 1024 + c, and 0x6400 | 16 c is 1024 + 16 c,
// whose sixteenth part is 64 + c.
template <bool ZEROS>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t z, uint32_t (&out)[4]) {
    const __half2 low = __half2half2(__ushort_as_half(static_cast<unsigned short>(0xe400u + (ZEROS ? z : 8u))));
    // 64 + z, negative: exact for every z <= 255
    const __half2 high = ZEROS ? __half2half2(__uint2half_rn(64u + z)) : __half2half2(__ushort_as_half(0x5480));
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2c00));
    const uint32_t h = w >> 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t v = i ? h : w;
        const uint32_t even = mask_or(v, 0x000f000fu, 0x64006400u), odd = mask_or(v, 0x00f000f0u, 0x64006400u);
        out[2 * i] = bits_of(__hadd2(*reinterpret_cast<const __half2 *>(&even), low));
        out[2 * i + 1] = bits_of(__hfma2(*reinterpret_cast<const __half2 *>(&odd), sixteenth, __hneg2(high)));
    }
}

// bf16: 0x4300 | c is 128 + c.  128 + z is exact for z = 8; other zero points
// are subtracted after 128 (both steps exact).
template <bool ZEROS>
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t z, uint32_t (&out)[4]) {
    const __nv_bfloat162 base = __bfloat162bfloat162(__ushort_as_bfloat16(ZEROS ? 0xc300 : 0xc308));
    const __nv_bfloat162 zero = __bfloat162bfloat162(__float2bfloat16_rn(-static_cast<float>(z)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = mask_or(w >> (4 * i), 0x000f000fu, 0x43004300u);
        __nv_bfloat162 c = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&v), base);
        if (ZEROS) c = __hadd2(c, zero);
        out[i] = bits_of(c);
    }
}

// d = A * B + (first ? 0 : d)
template <Kind K>
__device__ __forceinline__ void mma(float (&d)[4], bool first, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    const float c0 = first ? 0.f : d[0], c1 = first ? 0.f : d[1], c2 = first ? 0.f : d[2], c3 = first ? 0.f : d[3];
    if (K == kHalf)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The last bytes of a row, zeros past them.
static __device__ __noinline__ uint4 load_tail(const uint8_t *p, int64_t len) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (int i = 0; i < 16; ++i)
        if (i < len) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes at p, inside a row.  Without VEC they are put together from the aligned
// words that cover them (which may reach 3 bytes before p and 4 past them).
template <bool VEC>
__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
    if (VEC) return ld_stream16(p);
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
    const uint32_t *q = reinterpret_cast<const uint32_t *>(p - off);
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = __ldg(q + i);
    const uint32_t s = 8 * off;
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}

// A chunk of a warp: rows g and g + 8 of its 16, 128 columns; scale and zero
// point of the group that this lane loads for its quad, as loaded.
struct Chunk {
    uint4 q[2];
    uint32_t s[2], z[2];
};

__device__ __forceinline__ float scale_value(uint32_t raw, int dtype) {
    const float h = __half2float(__ushort_as_half(static_cast<unsigned short>(raw)));
    return dtype == kF16 ? h : __uint_as_float(raw << (dtype == kBF16 ? 16 : 0));
}

// lane c of a quad holds words v.x .. v.w of columns 32 c .. 32 c + 31; after
// this, word i of every lane lies in group i * NG / 4 of the chunk
template <int NG>
__device__ __forceinline__ void exchange(uint4 &q, int c, uint32_t (&v)[4]) {
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    if (NG == 2) {
        const bool up = c & 2;
        const uint32_t r0 = __shfl_xor_sync(kFull, up ? v[0] : v[2], 2);
        const uint32_t r1 = __shfl_xor_sync(kFull, up ? v[1] : v[3], 2);
        if (up) {
            v[0] = r0, v[1] = r1;
        } else {
            v[2] = r0, v[3] = r1;
        }
    } else if (NG == 4) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t r = __shfl_xor_sync(kFull, (c & 1) ? v[i] : v[i + 1], 1);
            if (c & 1) v[i] = r;
            else v[i + 1] = r;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t r = __shfl_xor_sync(kFull, (c & 2) ? v[i] : v[i + 2], 2);
            if (c & 2) v[i] = r;
            else v[i + 2] = r;
        }
    }
}

// Byte offset, within its chunk's 256 bytes, of the eight columns 8 w .. 8 w + 7
// of x (lane c reads word i at 64 i + 16 c): the inverse of exchange().
template <int NG>
__device__ __forceinline__ uint32_t word_offset(uint32_t w) {
    uint32_t c, i;
    if (NG == 1) {
        c = w >> 2, i = w & 3;
    } else if (NG == 2) {
        c = ((w >> 2) & 1) + (w & 2), i = ((w >> 3) << 1) + (w & 1);
    } else {
        c = w & 3, i = w >> 2;
    }
    return 64 * i + 16 * c;
}

struct Launch {
    int wk;           // warps that split the columns: 1, 2 or 4
    int x_vec;        // rows of x start 16-byte aligned
    int stage_bytes;  // shared memory for x
};

template <typename T>
__device__ __forceinline__ void load8(const T *row, int64_t k0, int64_t k, bool vec, T (&v)[8]) {
    if (vec && k0 + 8 <= k) {
        constexpr int N = 8 * static_cast<int>(sizeof(T)) / 16;
        uint4 raw[N];
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = __ldg(reinterpret_cast<const uint4 *>(row + k0) + i);
        const T *e = reinterpret_cast<const T *>(raw);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = e[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = k0 + j < k ? row[k0 + j] : Elem<T>::from_f(0.f);
    }
}

__device__ __forceinline__ uint32_t pair_bits(uint32_t lo, uint32_t hi) { return lo | (hi << 16); }

// the 16-bit patterns of v in the order in which codes come out of a word
__device__ __forceinline__ uint4 interleave(const uint32_t (&b)[8]) {
    return make_uint4(pair_bits(b[0], b[4]), pair_bits(b[1], b[5]), pair_bits(b[2], b[6]), pair_bits(b[3], b[7]));
}

// hi + mid + lo == v exactly, each with the 8 significant bits of a bf16 (cut off,
// not rounded, so nothing overflows); an infinity or NaN is all in hi
__device__ __forceinline__ void split3(float v, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    const uint32_t u = __float_as_uint(v);
    hi = u >> 16;
    mid = lo = 0u;
    if ((u & 0x7f800000u) == 0x7f800000u) {
        if (u & 0x007fffffu) hi |= 0x40u;
        return;
    }
    const float r = v - __uint_as_float(u & 0xffff0000u);
    const uint32_t ur = __float_as_uint(r);
    mid = ur >> 16;
    lo = __float_as_uint(r - __uint_as_float(ur & 0xffff0000u)) >> 16;
}

// The routed rows of the window that starts at base_row and the expert that this
// CTA serves: the d-th distinct one.  Returns false if there are fewer.  Leaves the
// window's ids in s_ids; also zeroes the CTA's outputs of rows without an expert.
template <typename T>
__device__ __forceinline__ bool find_expert(const Q4Params &p, uint32_t base_row, uint32_t d, int64_t j0, int tile_rows,
                                            uint32_t *s_ids, uint32_t *s_bits, uint32_t &expert) {
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rows = min(p.rows - base_row, static_cast<uint32_t>(kWindow));
    if (tid < 32) s_bits[tid] = 0u;
    __syncthreads();
    bool none = false;
    for (uint32_t i = tid; i < rows; i += kThreads) {
        const uint32_t id = __ldg(p.ids + base_row + i);
        s_ids[i] = id;
        if (id < p.n_experts) atomicOr(&s_bits[id >> 5], 1u << (id & 31));
        else none = true;
    }
    none = __syncthreads_or(none);
    if (none && d == 0) {
        for (uint32_t i = 0; i < rows; ++i)
            if (s_ids[i] >= p.n_experts && tid < tile_rows && j0 + tid < p.n)
                static_cast<T *>(p.out)[static_cast<int64_t>(base_row + i) * p.ldo + j0 + tid] = Elem<T>::from_f(0.f);
    }
    uint32_t word = s_bits[lane];
    const uint32_t bits = __popc(word);
    uint32_t inc = bits;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += v;
    }
    const unsigned owner = __ballot_sync(kFull, d >= inc - bits && d < inc);
    if (owner == 0u) return false;
    const int src = __ffs(owner) - 1;
    word = __shfl_sync(kFull, word, src);
    for (uint32_t skip = d - __shfl_sync(kFull, inc - bits, src); skip > 0; --skip) word &= word - 1;
    expert = src * 32 + __ffs(word) - 1;
    return true;
}

// s_ids becomes the list of the window's routed rows that name `expert`, in
// order; returns their number.  Called by the whole CTA.
__device__ __forceinline__ uint32_t list_rows(const Q4Params &p, uint32_t base_row, uint32_t expert, uint32_t *s_ids,
                                              uint32_t *s_count) {
    const int lane = threadIdx.x & 31;
    const uint32_t rows = min(p.rows - base_row, static_cast<uint32_t>(kWindow));
    __syncthreads();
    if (threadIdx.x < 32) {
        uint32_t n = 0;
        for (uint32_t i = 0; i < rows; i += 32) {  // writes stay at or behind what has been read
            const bool hit = i + lane < rows && s_ids[i + lane] == expert;
            const unsigned hits = __ballot_sync(kFull, hit);
            if (hit) s_ids[n + __popc(hits & ((1u << lane) - 1u))] = base_row + i + lane;
            n += __popc(hits);
            __syncwarp();
        }
        if (lane == 0) *s_count = n;
    }
    __syncthreads();
    return *s_count;
}

// x of `tokens` rows (routed rows list[t0 ..], or rows t0 .. without a list),
// columns k0 .. k0 + 8 words - 1, into shared memory
template <Kind K, int NG>
__device__ __forceinline__ void stage_x(const Q4Params &p, const Launch &cfg, const uint32_t *list, uint32_t t0,
                                        uint32_t tokens, int32_t k0, uint32_t words, uint32_t pitch, uint8_t *stage) {
    using T = typename XType<K>::type;
    constexpr int kTerms = K == kFloat ? 3 : 1;
#pragma unroll 1
    for (uint32_t tok = 0; tok < tokens; ++tok) {
        const uint32_t r = list != nullptr ? list[t0 + tok] : t0 + tok;
        const T *x = static_cast<const T *>(p.x) + static_cast<int64_t>(r / p.top_k) * p.ldx +
                     static_cast<int64_t>(r % p.top_k) * p.x_slot_stride;
        uint8_t *col = stage + tok * kTerms * pitch;
#pragma unroll 1
        for (uint32_t w = threadIdx.x; w < words; w += kThreads) {
            T v[8];
            load8<T>(x, k0 + 8 * w, p.k, cfg.x_vec != 0, v);
            uint8_t *dst = col + (w >> 4) * 256 + word_offset<NG>(w & 15);
            if constexpr (K == kFloat) {
                uint32_t b[3][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) split3(v[j], b[0][j], b[1][j], b[2][j]);
#pragma unroll
                for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4 *>(dst + q * pitch) = interleave(b[q]);
            } else {
                uint32_t b[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] = *reinterpret_cast<const uint16_t *>(&v[j]);
                *reinterpret_cast<uint4 *>(dst) = interleave(b);
            }
        }
    }
}

// NG: groups in a chunk of 128 columns.  NT: mma column tiles, 8 NT / terms rows
// of x a pass.
template <Kind K, int NG, bool ZEROS, bool VEC, int NT>
__global__ void __launch_bounds__(kThreads, Budget<NT>::kCtas)
    q4_kernel(const __grid_constant__ Q4Params p, const __grid_constant__ Launch cfg) {
    using T = typename XType<K>::type;
    constexpr int kTerms = K == kFloat ? 3 : 1;
    constexpr int kDepth = Budget<NT>::kDepth;
    constexpr uint32_t kPass = 8 * NT / kTerms;  // rows of x a pass
    constexpr int kRedPitch = 8 * NT + 1;
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ float red[kWarps][16][kRedPitch];
    __shared__ uint32_t s_ids[kWindow];
    __shared__ uint32_t s_bits[32];
    __shared__ uint32_t s_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int wk = warp & (cfg.wk - 1), wr = warp / cfg.wk, tile_rows = 16 * (kWarps / cfg.wk);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * tile_rows;  // the CTA's first row
    const bool by_id = p.ids != nullptr;

    uint32_t expert = 0;
    const uint32_t base_row = blockIdx.z * kWindow;
    if (by_id && !find_expert<T>(p, base_row, blockIdx.y, j0, tile_rows, s_ids, s_bits, expert)) return;

    // This thread's two rows (rows past the end repeat the last one and are not
    // stored), at this lane's 16 bytes of the warp's next chunk, and the cells of its
    // group's scales and zero points.
    const int32_t row_len = static_cast<int32_t>((p.k + 1) / 2);
    const int32_t chunks = static_cast<int32_t>((p.k + 127) / 128), groups = static_cast<int32_t>(p.groups);
    // chunks that can be read without a look at the row's end: whole ones, and without
    // VEC neither the row's first nor its last words
    const int32_t lo = VEC ? 0 : 1, hi = static_cast<int32_t>(VEC ? p.k / 128 : (p.k - 8) / 128);
    const int lane_group = NG == 4 ? c : NG == 2 ? c >> 1 : 0;  // of the chunk's, whose scale this lane loads
    const int ssize = p.scale_dtype == kF32 ? 4 : 2;
    const uint8_t *qat[2], *zat[2];
    const char *sat[2];
    auto rewind = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int64_t j = j0 + wr * 16 + g + 8 * h;
            if (j >= p.n) j = p.n - 1;
            qat[h] = p.q + static_cast<int64_t>(expert) * p.expert_stride + j * p.ldq + wk * 64 + 16 * c;
            const int64_t cell = (static_cast<int64_t>(expert) * p.n + j) * p.groups + wk * NG + lane_group;
            sat[h] = static_cast<const char *>(p.scales) + cell * ssize;
            zat[h] = ZEROS ? p.zeros + cell : nullptr;
        }
    };
    // the warp's next chunk
    auto fetch = [&](int32_t chunk, Chunk &b) {
        if (chunk < hi && chunk >= lo) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                b.q[h] = load_codes<VEC>(qat[h]);
                b.s[h] = ssize == 4 ? __ldg(reinterpret_cast<const uint32_t *>(sat[h]))
                                    : __ldg(reinterpret_cast<const uint16_t *>(sat[h]));
                b.z[h] = ZEROS ? __ldg(zat[h]) : 0u;
            }
        } else if (chunk < chunks) {
            const bool inside = chunk * NG + lane_group < groups;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                b.q[h] = load_tail(qat[h], row_len - (chunk * 64 + 16 * c));
                b.s[h] = b.z[h] = 0u;
                if (inside) {
                    b.s[h] = ssize == 4 ? __ldg(reinterpret_cast<const uint32_t *>(sat[h]))
                                        : __ldg(reinterpret_cast<const uint16_t *>(sat[h]));
                    if (ZEROS) b.z[h] = __ldg(zat[h]);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            qat[h] += cfg.wk * 64;
            sat[h] += cfg.wk * NG * ssize;
            if (ZEROS) zat[h] += cfg.wk * NG;
        }
    };
    Chunk buf[kDepth];
    rewind();
#pragma unroll
    for (int d = 0; d < kDepth; ++d) fetch(wk + d * cfg.wk, buf[d]);

    const uint32_t first = by_id ? 0u : blockIdx.y * kPass;
    const uint32_t stride = by_id ? kPass : gridDim.y * kPass;
    const uint32_t count = by_id ? list_rows(p, base_row, expert, s_ids, &s_count) : p.rows;

#pragma unroll 1
    for (uint32_t t0 = first; t0 < count; t0 += stride) {
        const uint32_t tokens = min(count - t0, kPass);
        const uint32_t cols = tokens * kTerms;
        const int tiles = static_cast<int>((cols + 7) / 8);
        const int32_t total = (chunks + cfg.wk - 1) / cfg.wk;  // chunks a warp
        // chunks a warp of x that fit, a multiple of kDepth or all of them
        int32_t slab = static_cast<int32_t>((cfg.stage_bytes / cols - 64) / 256) / cfg.wk;
        slab = slab >= total ? total : slab / kDepth * kDepth;
        const uint32_t pitch = static_cast<uint32_t>(slab * cfg.wk) * 256 + 64;
        if (t0 != first) {
            rewind();
#pragma unroll
            for (int d = 0; d < kDepth; ++d) fetch(wk + d * cfg.wk, buf[d]);
        }
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;

#pragma unroll 1
        for (int32_t s0 = 0; s0 < total; s0 += slab) {
            __syncthreads();  // the slab before, or the pass before, is done with
            stage_x<K, NG>(p, cfg, by_id ? s_ids : nullptr, t0, tokens, s0 * cfg.wk * 128,
                           static_cast<uint32_t>(slab * cfg.wk) * 16, pitch, stage);
            __syncthreads();
            const int32_t s1 = s0 + slab < total ? s0 + slab : total;
            // this lane's first word of its column in each tile; lanes past the last column
            // repeat it, and what they compute is not stored
            const uint8_t *xat[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t col = 8 * t + g;
                xat[t] = stage + (col < cols ? col : cols - 1) * pitch + wk * 256 + 16 * c;
            }
            int32_t chunk = wk + s0 * cfg.wk;
            const int32_t end = s1 * cfg.wk < chunks ? s1 * cfg.wk : chunks;
#pragma unroll 1
            while (chunk < end) {
#pragma unroll
                for (int d = 0; d < kDepth; ++d) {
                    if (chunk < end) {
                        uint32_t codes[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) exchange<NG>(buf[d].q[h], c, codes[h]);
                        float part[NT][4];
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int from = (lane & 28) + (NG == 2 ? w & 2 : w);
                            uint32_t a[2][4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t z = 0u;
                                if (ZEROS) z = NG == 1 ? buf[d].z[h] : __shfl_sync(kFull, buf[d].z[h], from);
                                if (K == kHalf) codes_f16<ZEROS>(codes[h][w], z, a[h]);
                                else codes_bf16<ZEROS>(codes[h][w], z, a[h]);
                            }
                            const bool opens = w % (4 / NG) == 0, closes = w % (4 / NG) == 4 / NG - 1;
                            float s[2];
                            if (closes) {
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    s[h] = scale_value(
                                        NG == 1 ? buf[d].s[h] : __shfl_sync(kFull, buf[d].s[h], from), p.scale_dtype);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                if (t < tiles) {
                                    const uint4 b = *reinterpret_cast<const uint4 *>(xat[t] + 64 * w);
                                    mma<K>(part[t], opens, a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                                    mma<K>(part[t], false, a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
                                    if (closes) {
#pragma unroll
                                        for (int q = 0; q < 4; ++q)
                                            acc[t][q] = fmaf(s[q >> 1], part[t][q], acc[t][q]);
                                    }
                                }
                            }
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) xat[t] += cfg.wk * 256;
                        fetch(chunk + kDepth * cfg.wk, buf[d]);
                        chunk += cfg.wk;
                    }
                }
            }
        }

        // the warps that split the columns, and the terms of an f32 row, add up in order
        if (t0 != first) __syncthreads();  // the pass before has read red
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int q = 0; q < 4; ++q) red[warp][g + 8 * (q >> 1)][8 * t + 2 * c + (q & 1)] = acc[t][q];
        }
        __syncthreads();
        for (uint32_t u = tid; u < tile_rows * tokens; u += kThreads) {
            const uint32_t jj = u & (tile_rows - 1), tok = u / tile_rows;
            if (j0 + jj >= p.n) continue;
            float sum = 0.f;
            for (int w = 0; w < cfg.wk; ++w) {
#pragma unroll
                for (int q = 0; q < kTerms; ++q) sum += red[(jj >> 4) * cfg.wk + w][jj & 15][tok * kTerms + q];
            }
            const uint32_t r = by_id ? s_ids[t0 + tok] : t0 + tok;
            static_cast<T *>(p.out)[static_cast<int64_t>(r) * p.ldo + j0 + jj] = Elem<T>::from_f(sum);
        }
    }
}

template <Kind K, int NG, bool ZEROS, bool VEC, int NT>
cudaError_t launch_one(const Q4Params &p, const Launch &cfg, dim3 grid, cudaStream_t s) {
    static unsigned long long done = 0;  // devices on which the kernel may use its shared memory
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(q4_kernel<K, NG, ZEROS, VEC, NT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   Budget<NT>::kStageBytes);
        if (e != cudaSuccess) return e;
        done |= bit;
    }
    q4_kernel<K, NG, ZEROS, VEC, NT><<<grid, kThreads, cfg.stage_bytes, s>>>(p, cfg);
    return cudaGetLastError();
}

template <Kind K, int NG, bool ZEROS>
cudaError_t launch_vec(const Q4Params &p, const Launch &cfg, bool vec, bool wide, dim3 grid, cudaStream_t s) {
    constexpr int kWide = K == kFloat ? 3 : 2;
    if (!vec) return launch_one<K, NG, ZEROS, false, kWide>(p, cfg, grid, s);
    return wide ? launch_one<K, NG, ZEROS, true, kWide>(p, cfg, grid, s)
                : launch_one<K, NG, ZEROS, true, 1>(p, cfg, grid, s);
}

template <Kind K>
cudaError_t launch(const Q4Params &p, int num_sms, cudaStream_t s) {
    using T = typename XType<K>::type;
    constexpr int kTerms = K == kFloat ? 3 : 1;
    const bool vec = reinterpret_cast<uintptr_t>(p.q) % 16 == 0 && p.ldq % 16 == 0 && p.expert_stride % 16 == 0;
    // rows of x that one matrix can meet; past those of one column tile, the wide kernel
    const uint32_t most = p.ids != nullptr && p.rows > static_cast<uint32_t>(kWindow) ? kWindow : p.rows;
    // Per expert id the rows spread over the experts: on average there are `share` rows
    // for each one that occurs, and a second pass over the few with more finds the
    // weights in L2.
    const uint32_t distinct = most < p.n_experts ? most : p.n_experts;
    const uint32_t share = p.ids != nullptr ? (most + distinct - 1) / distinct : most;
    const bool wide = !vec || share * kTerms > 8;
    const uint32_t pass = 8u * (wide ? (K == kFloat ? 3 : 2) : 1) / kTerms;
    const int64_t tiles = (p.n + 15) / 16;
    const int64_t chunks = (p.k + 127) / 128;
    uint32_t gy, gz = 1;
    if (p.ids != nullptr) {
        gz = (p.rows + kWindow - 1) / kWindow;
        gy = most < p.n_experts ? most : p.n_experts;
    } else {
        gy = (p.rows + pass - 1) / pass;
        if (gy > 65535u) gy = 65535u;
    }
    if (gz > 65535u) return cudaErrorInvalidConfiguration;
    Launch cfg{};
    cfg.wk = 1;
    while (cfg.wk < kWarps && cfg.wk < chunks && tiles * gy * cfg.wk < 16LL * num_sms) cfg.wk *= 2;
    cfg.x_vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx * sizeof(T) % 16 == 0 &&
                p.x_slot_stride * sizeof(T) % 16 == 0;
    const int64_t cols = static_cast<int64_t>(most < pass ? most : pass) * kTerms;
    const int64_t want = cols * ((chunks + cfg.wk - 1) / cfg.wk * cfg.wk * 256 + 64);
    const int64_t cap = wide ? Budget<K == kFloat ? 3 : 2>::kStageBytes : Budget<1>::kStageBytes;
    cfg.stage_bytes = static_cast<int>(want < cap ? want : cap);
    const int64_t wr = kWarps / cfg.wk;
    const dim3 grid(static_cast<unsigned>((tiles + wr - 1) / wr), gy, gz);
    const int ng = 128 / p.group;
    if (p.zeros != nullptr) {
        if (ng == 1) return launch_vec<K, 1, true>(p, cfg, vec, wide, grid, s);
        if (ng == 2) return launch_vec<K, 2, true>(p, cfg, vec, wide, grid, s);
        return launch_vec<K, 4, true>(p, cfg, vec, wide, grid, s);
    }
    if (ng == 1) return launch_vec<K, 1, false>(p, cfg, vec, wide, grid, s);
    if (ng == 2) return launch_vec<K, 2, false>(p, cfg, vec, wide, grid, s);
    return launch_vec<K, 4, false>(p, cfg, vec, wide, grid, s);
}

}  // namespace q4
}  // namespace gbmm
