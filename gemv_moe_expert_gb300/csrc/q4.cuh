// q4.cuh -- matrix-vector products with 4-bit weights and group scales, dense or
// per expert id: the kernel, instantiated for one type of x in each q4_*.cu.
//
//   y[i, j] = sum over groups g of s[j,g] * sum over x in g of (q[j,x] - z[j,g]) x[i,x]
//
// The weights are read once from HBM and have to become multiplier operands: the
// kernel is bound by that stream, and next to it by the instructions that unpack
// the codes.  So the products run on the tensor cores straight from registers (mma
// m16n8k16: 16 weight rows x 16 columns against 8 columns of x), and a pair of
// codes becomes half an operand register, less its zero point, with two instructions: a code
// c put under the exponent of 1024 is the f16 number 1024 + c in the lowest four mantissa bits and
// 1024 + 16 c in the next four, from where one subtraction, or one multiply-add with 1/16,
// makes q - z, exactly.  (An f32 product would have to widen every code and multiply it
// once for each row of x.)  A group's sum then takes its scale.
//
// The zero point goes before the product and not after the sum (sum of q x less z times
// sum of x, which needs one instruction for a pair of codes and 4 to 8 % less time where there
// are many weights): the difference of two sums of which each is rounded is off by parts of z sum
// |x|, however small the weights are, and weights of 0 would not give 0.
//
// x is staged in shared memory as f16, after each group of columns of a row has been scaled
// by a power of two that puts its largest magnitude into [2^14, 2^15).  A value keeps all its
// bits unless it lies 2^28 (f16) or 2^31 (bf16) below the largest of its group; then it is off by
// 2^-39 of that at most.  f32 values become the sum of three f16 terms, in three of the mma's eight
// columns, each with what the terms before have left, scaled up by 2^11: 2^37, and 2^-61.  A
// group that holds an infinity, a NaN or a value from 2^112 up is left out and its row computed in
// plain f32 at the end.
//
// The order of a contraction is free, so a thread keeps the 32 bytes it loads (64
// neighbouring codes of a row; the quad of lanes of a row covers a block of 256
// columns, eight rows of whole 128-byte lines an access) and x is stored in the order
// in which those codes come out of the words.  The mma must not add up different
// groups: each row of x (each term of it) takes kParts of the mma's columns, and the
// lanes of a quad that hold another group's codes read zeros there.  With groups of 128
// lanes 0, 1 and 2, 3 hold one group each, with 64 every lane one, with 32 two, which
// are closed one after the other.  The tensor pipe has the room, and nothing is
// exchanged between lanes.
//
// A warp takes 32 rows, so that what it reads of x serves two mma row tiles.  A CTA
// has kWarps warps: wk of them split the columns (blocks, one after the other) of the
// same rows, and kWarps / wk take different rows.  A warp's first block is loaded before x
// is staged, each next one as soon as the one before has been used: twelve to twenty-four
// warps an SM hide the latency.  Loads are predicated, not branched around, and the
// alignment they need is settled at the launch (Access).
//
// Measured (us, and GB/s of codes, scales, zeros, x and y; inputs rotate past L2):
//   dense 11008 x 4096, groups of 128, 1 row     f16 10.2 (2270)   f32 11.3 (2060)
//   the same, 4 f16 rows 13.1, 16 f16 rows 27.9, 8 f32 rows 28.9
//   4 tokens x 8 of 64 experts, 1408 x 2048      bf16 14.5 (2880)   f32 19.0 (2200)
//   16 tokens x 8 of 128 experts, 1536 x 4096: bf16, groups of 32 with zeros 82.7 (3710);
//   bf16, groups of 128 66.0 (4140); f32, groups of 128 104 (2630)
// No pipe is full in the large ones (an SM that has work issues in 53 % of its cycles, the ALU is
// busy in 45 % of them, the tensor pipe in 24 %): a warp's next block is on its way only while the
// warps beside it compute, and the last wave is short.  The last case but one takes 60.1 when x is
// not staged and 61.0 when no zero points are subtracted.  The small ones are over before HBM is at
// its rate.  Tried on the way (the case with groups of 32, which took 77 to 84 then): 16
// rows a warp and 16-byte loads of half lines 151, bound by the L1 data path; a ring of
// shared-memory slots filled by bulk copies of 256-byte row pieces 206; the next block held
// in a second set of registers 91, as it leaves room for fewer instructions in flight; CTAs that
// walk over several row tiles 172; lines fetched to L2 three blocks ahead 88 for 84; a cluster of
// four CTAs that stage a quarter of x each and copy the rest from each other 89 for 79.
#pragma once

#include <algorithm>

#include "device_common.cuh"

namespace gbmm {
namespace q4 {

constexpr uint32_t kWindow = kQ4Window;
constexpr uint32_t kFull = 0xffffffffu;

// mma columns that a row of x takes; how often a block's sums are closed
template <int G> struct Group {
    static constexpr int kParts = G == 128 ? 2 : 4;
    static constexpr int kCloses = G == 32 ? 2 : 1;
    static constexpr int kInBlock = 256 / G;
    static constexpr int kCells = G == 32 ? 4 : 2;  // neighbouring groups whose scales a lane needs
};

enum Kind { kHalf, kBfloat, kFloat };  // type of x

// NT column tiles of 8, MT row tiles of 16 a warp: warps a CTA, CTAs an SM, and the shared
// memory for a slab of x, which holds two blocks for each warp at least.
// Eight warps share the staging of x: 4 f16 rows x 11008 x 4096 13.2 us for 23.3 with four,
// 1 row x 4096 x 11008 12.3 for 15.5, 16 bf16 tokens x 8 of 128 experts 66.1 for 71.8 (groups of
// 32 with zeros 82.9 for 82.3).  f32, which needs the registers, and three and more column
// tiles take four (8 f32 rows 28.9 for 38.9 with eight, 8 bf16 rows with groups of 64 27.8 for
// 30.4).
template <Kind K, int NT, int MT> struct Budget {
    static constexpr int kWarps = K != kFloat && NT <= 2 ? 8 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kCtas = kWarps == 8 ? (MT == 1 && NT == 1 ? 3 : 2) : NT == 1 ? 4 : 3;
    static constexpr int kStageBytes =
        kWarps == 8 ? (NT == 1 ? 48 * 1024 : 80 * 1024) : NT == 1 ? 32 * 1024 : NT == 2 ? 44 * 1024 : 60 * 1024;
};

template <Kind K> struct XType;
template <> struct XType<kHalf> { using type = __half; };
template <> struct XType<kBfloat> { using type = __nv_bfloat16; };
template <> struct XType<kFloat> { using type = float; };

constexpr int kPitchPad = 64;    // spreads the lines of x over the banks
constexpr int kZeroBytes = 512;  // a block: what lanes of another group read
// shared memory of one block of x: `lines` rows (terms of rows), and what undoes each column's scaling
constexpr int block_bytes(int lines, int NT, int closes) { return lines * 512 + 32 * NT * closes; }

// Exponent field of 2^112: 128 values below it times a code less a zero point (255 at most) add
// up to less than 2^127.
constexpr uint32_t kPlainFrom = 239;
// An f16 keeps 11 bits: what the first term of an f32 value leaves is scaled up by 2^11 before it
// becomes the next.
constexpr uint32_t kTermBits = 11;

// d = A * B + (first ? 0 : d)
__device__ __forceinline__ void mma(float (&d)[4], bool first, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    const float c0 = first ? 0.f : d[0], c1 = first ? 0.f : d[1], c2 = first ? 0.f : d[2], c3 = first ? 0.f : d[3];
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Two codes less their row's zero point z, exactly, as f16: the codes in the lowest four bits of w's
// halves, made 1024 + c by the exponent's bits, less 1024 + z; and those in the next four, made 1024 +
// 16 c, a sixteenth of that less 64 + z.
__device__ __forceinline__ uint32_t half2_word(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 word_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
// `exponents` is 0x64006400, in a register that the compiler does not see through: of two constants it
// makes two instructions.
template <uint32_t MASK> __device__ __forceinline__ __half2 pick(uint32_t w, uint32_t exponents) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "n"(MASK), "r"(exponents));  // (w & MASK) | exponents
    return word_half2(r);
}
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t exponents, __half2 z) {
    return half2_word(__hsub2(pick<0x000f000fu>(w, exponents), z));
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w, uint32_t exponents, __half2 minus_z) {
    return half2_word(__hfma2(pick<0x00f000f0u>(w, exponents), word_half2(0x2c002c00u), minus_z));
}

struct Launch {
    int wk_log;   // log2 of the warps that split the columns
    int x_vec;    // rows of x start 16-byte aligned
    int slab;     // blocks of x a warp in shared memory
    int info_at;  // byte offset in shared memory
};

__device__ __forceinline__ float scale_value(uint32_t raw, int dtype) {
    const float h = __half2float(__ushort_as_half(static_cast<unsigned short>(raw)));
    return dtype == kF16 ? h : __uint_as_float(raw << (dtype == kBF16 ? 16 : 0));
}

// Eight neighbouring values of x as loaded, zeros past the row's k columns.
template <typename T> struct Eight {
    static constexpr int N = 8 * static_cast<int>(sizeof(T)) / 16;
    uint4 raw[N];
    __device__ __forceinline__ void load(const T *row, int64_t k0, int64_t k, bool vec) {
        if (vec && k0 + 8 <= k) {
#pragma unroll
            for (int i = 0; i < N; ++i) raw[i] = __ldg(reinterpret_cast<const uint4 *>(row + k0) + i);
        } else {
            T v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = k0 + j < k ? row[k0 + j] : Elem<T>::from_f(0.f);
#pragma unroll
            for (int i = 0; i < N; ++i) raw[i] = reinterpret_cast<const uint4 *>(v)[i];
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) unpack16<T>(raw[i], f + i * (8 / N));
    }
};

__device__ __forceinline__ float power_of_two(uint32_t exponent_field) { return __uint_as_float(exponent_field << 23); }

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Byte offset, within its block's 512 bytes, of columns 8 w .. 8 w + 7 of x: word i =
// w % 4 of half v = w / 4 % 2 of lane c = w / 8, which reads it at 256 v + 64 i + 16 c.
__device__ __forceinline__ uint32_t word_offset(uint32_t w) {
    return 256 * (w >> 2 & 1) + 64 * (w & 3) + 16 * (w >> 3);
}

// The window's expert that this CTA serves: the d-th distinct one of its ids.
// Returns false if there are fewer.  Leaves the window's ids in s_ids; zeroes the CTA's
// outputs of rows without an expert.
template <typename T, int kThreads>
__device__ __forceinline__ bool find_expert(const Q4Params &p, uint32_t base_row, uint32_t d, int64_t j0, int tile_rows,
                                            uint32_t *s_ids, uint32_t *s_bits, uint32_t &expert) {
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rows = min(p.rows - base_row, kWindow);
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
    const uint32_t rows = min(p.rows - base_row, kWindow);
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

// Both for a window of at most 32 rows, which every warp sees at once: the distinct
// experts in the order of their first rows, without a barrier (8 of 64 experts: 1 f32 token
// 7.2 us for 7.5, 4 bf16 tokens 14.6 for 14.8).  `list` is valid after the next barrier.
template <typename T>
__device__ __forceinline__ bool find_in_warp(const Q4Params &p, uint32_t base_row, uint32_t d, int64_t j0,
                                             int tile_rows, uint32_t *list, uint32_t &expert, uint32_t &count) {
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rows = p.rows - base_row;
    const uint32_t id = lane < rows ? __ldg(p.ids + base_row + lane) : p.n_experts;
    const bool has = id < p.n_experts;
    const uint32_t same = __match_any_sync(kFull, id);
    uint32_t firsts = __ballot_sync(kFull, has && (same & ((1u << lane) - 1u)) == 0u);
    if (d == 0) {
        for (uint32_t none = __ballot_sync(kFull, lane < rows && !has); none != 0u; none &= none - 1)
            if (tid < tile_rows && j0 + tid < p.n)
                static_cast<T *>(p.out)[static_cast<int64_t>(base_row + __ffs(none) - 1) * p.ldo + j0 + tid] =
                    Elem<T>::from_f(0.f);
    }
    if (d >= __popc(firsts)) return false;
    for (uint32_t skip = d; skip > 0; --skip) firsts &= firsts - 1;
    const int src = __ffs(firsts) - 1;
    expert = __shfl_sync(kFull, id, src);
    const uint32_t mine = __shfl_sync(kFull, same, src);
    count = __popc(mine);
    if (tid < 32 && mine >> lane & 1u) list[__popc(mine & ((1u << lane) - 1u))] = base_row + lane;
    return true;
}

// x of `tokens` rows, which start at offsets[] (in elements), columns k0 .. k0 + 8 words
// - 1, into shared memory: f16 terms at stage + line * pitch, and for each block (half a
// block with groups of 32) and mma column what undoes the scaling.  Rows with a group that
// cannot be scaled are marked in *bad.
template <Kind K, int G, int NT, int kThreads>
__device__ __forceinline__ void stage_x(const Q4Params &p, const Launch &cfg, const int64_t *offsets, uint32_t tokens,
                                        int32_t k0, uint32_t words, uint32_t pitch, uint8_t *stage, float *info,
                                        uint32_t *bad) {
    using T = typename XType<K>::type;
    constexpr int kTerms = K == kFloat ? 3 : 1;
    constexpr int kLanes = G / 8;  // that share a group
    // Loads in flight a thread (1: 8 bf16 rows 33.8 us for 27.8, 1 f32 row x 4096 x 11008 21.4 for 20.1,
    // but 4 f32 tokens x 8 of 64 experts 18.4 for 19.2).
    constexpr int kAhead = 3;
    const int lane = threadIdx.x & 31;
    // a warp takes 32 words, of one row (words is a multiple of 32), and goes on kThreads further
    uint32_t tok = 0, w = threadIdx.x;
    while (tok < tokens) {
        Eight<T> x8[kAhead];
        uint32_t toks[kAhead], ws[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            while (w >= words && tok < tokens) {
                w -= words;
                ++tok;
            }
            toks[a] = tok;
            ws[a] = w;
            if (tok < tokens)
                x8[a].load(static_cast<const T *>(p.x) + offsets[tok], k0 + 8 * static_cast<int64_t>(w), p.k,
                           cfg.x_vec != 0);
            w += kThreads;
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            if (toks[a] >= tokens) break;
            float f[8];
            x8[a].get(f);
            uint32_t most = 0u;  // of the magnitudes' bits: infinities and NaN are the largest
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) most = max(most, __shfl_xor_sync(kFull, most, o));
            if (most >= kPlainFrom << 23) {
                atomicOr(bad, 1u << toks[a]);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = 0.f;
                most = 0u;
            }
            const uint32_t e = max(most >> 23, 15u + kTermBits * (kTerms - 1));
            const float up = power_of_two(268u - e);  // 2^14 over the largest value's power of two
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= up;
            const uint32_t block = ws[a] >> 5, group = lane / kLanes;
            // column of the row's (term's) first, and the close it belongs to
            const uint32_t part = G == 32 ? group >> 1 : group, close = G == 32 ? group & 1 : 0;
            uint8_t *line = stage + toks[a] * kTerms * pitch + block * 512 + word_offset(lane);
            float *column = info + (block * Group<G>::kCloses + close) * (8 * NT) +
                            toks[a] * kTerms * Group<G>::kParts + part;
#pragma unroll
            for (int q = 0; q < kTerms; ++q) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = half2_bits(f[i], f[i + 4]);
                    if (q + 1 < kTerms) {
                        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                        f[i] = (f[i] - v.x) * static_cast<float>(1 << kTermBits);
                        f[i + 4] = (f[i + 4] - v.y) * static_cast<float>(1 << kTermBits);
                    }
                }
                *reinterpret_cast<uint4 *>(line + q * pitch) = make_uint4(h[0], h[1], h[2], h[3]);
                if (lane % kLanes == 0) column[q * Group<G>::kParts] = power_of_two(e - 14u - kTermBits * q);
            }
        }
    }
}

// One output in plain f32, for a row of x that cannot be scaled: each weight first, as a group's
// sum of codes times x could pass the range of f32 where the result does not.
template <typename T>
__device__ __noinline__ float plain_output(const Q4Params &p, uint32_t expert, int64_t j, uint32_t r) {
    const uint8_t *q = p.q + static_cast<int64_t>(expert) * p.expert_stride + j * p.ldq;
    const int64_t cell = (static_cast<int64_t>(expert) * p.n + j) * p.groups;
    const T *x = static_cast<const T *>(p.x) + static_cast<int64_t>(r / p.top_k) * p.ldx +
                 static_cast<int64_t>(r % p.top_k) * p.x_slot_stride;
    float acc = 0.f;
    for (int64_t g = 0; g < p.groups; ++g) {
        const float s = scale_value(p.scale_dtype == kF32 ? static_cast<const uint32_t *>(p.scales)[cell + g]
                                                          : static_cast<const uint16_t *>(p.scales)[cell + g],
                                    p.scale_dtype);
        const float z = p.zeros != nullptr ? static_cast<float>(p.zeros[cell + g]) : 8.f;
        const int64_t end = (g + 1) * p.group < p.k ? (g + 1) * p.group : p.k;
        float part = 0.f;
        for (int64_t i = g * p.group; i < end; ++i)
            part = fmaf((static_cast<float>((q[i >> 1] >> (4 * (i & 1))) & 15) - z) * s, Elem<T>::to_f(x[i]), part);
        acc += part;
    }
    return acc;
}

// The first n of 16 bytes at p, one by one.
static __device__ __noinline__ uint4 load_bytes(const uint8_t *p, int n) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) w[i / 4] |= static_cast<uint32_t>(__ldg(p + i)) << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Loads under a predicate, without a branch: a branch around each would end a basic
// block, and nothing would be scheduled across it.
__device__ __forceinline__ void load_stream32(bool pred, const void *p, uint4 (&v)[2]) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %9, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t}"
        : "+r"(v[0].x), "+r"(v[0].y), "+r"(v[0].z), "+r"(v[0].w), "+r"(v[1].x), "+r"(v[1].y), "+r"(v[1].z),
          "+r"(v[1].w)
        : "l"(p), "r"(static_cast<uint32_t>(pred)));
}
__device__ __forceinline__ void load_stream16(bool pred, const void *p, uint4 &v) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"(static_cast<uint32_t>(pred)));
}
// zero where the predicate is false
__device__ __forceinline__ uint2 load_cells64(bool pred, const void *p) {
    uint2 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.nc.v2.b32 {%0, %1}, [%2];\n\t}"
        : "=&r"(v.x), "=&r"(v.y)
        : "l"(p), "r"(static_cast<uint32_t>(pred)));
    return v;
}
__device__ __forceinline__ uint32_t load_cells32(bool pred, const void *p) {
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}"
                 : "=&r"(v)
                 : "l"(p), "r"(static_cast<uint32_t>(pred)));
    return v;
}
__device__ __forceinline__ uint32_t load_cells16(bool pred, const void *p) {
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
                 : "=&r"(v)
                 : "l"(p), "r"(static_cast<uint32_t>(pred)));
    return v;
}
__device__ __forceinline__ uint32_t load_cells8(bool pred, const void *p) {
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.u8 %0, [%1];\n\t}"
                 : "=&r"(v)
                 : "l"(p), "r"(static_cast<uint32_t>(pred)));
    return v;
}

// 16 bytes at any p, put together from the five aligned words that cover them.
__device__ __forceinline__ uint4 load_unaligned(bool pred, const uint8_t *p) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u), s = 8 * off;
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = load_cells32(pred, p - off + 4 * i);
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}

// How a kernel reads codes, scales and zero points.  What lies between a row's end and
// the end of an access meets zeros of x; only where the memory ends there, after the last
// row, single bytes are read.
//   kAnyhow  any alignment, scale type and number of rows
//   kLoose   packed rows start on multiples of 16 bytes, 16-bit scales, enough rows for a warp
//   kApart   they start and end on multiples of 32 bytes; the scales of a lane one by one
//            (groups of 32: two by two)
//   kAtOnce  and the scales of a lane, and its zero points, can be read at once
// Measured, 16 bf16 tokens x 8 of 128 experts, groups of 128 (of 32, with zeros): 1536 x 4096,
// kAtOnce, 66 us (83); 1537 x 4090 with rows 2048 bytes apart, kLoose, 82 (134); with rows
// 2045 bytes apart, kAnyhow, 183 (226).  Dense 1 f16 row, groups of 128: 11008 x 4224 (33 groups),
// kApart, 11.2; 11009 x 4098 kLoose 12.6, kAnyhow 19.4.
enum Access { kAnyhow, kLoose, kApart, kAtOnce };

// G: columns of a group.  NT: mma column tiles, 8 NT / (terms kParts) rows of x a pass.
// MT: mma row tiles of a warp.
template <Kind K, int G, Access A, int NT, int MT>
__global__ void __launch_bounds__(Budget<K, NT, MT>::kThreads, Budget<K, NT, MT>::kCtas)
    q4_kernel(const __grid_constant__ Q4Params p, const __grid_constant__ Launch cfg) {
    constexpr int kWarps = Budget<K, NT, MT>::kWarps, kThreads = Budget<K, NT, MT>::kThreads;
    using T = typename XType<K>::type;
    constexpr int kTerms = K == kFloat ? 3 : 1;
    constexpr int kParts = Group<G>::kParts, kCloses = Group<G>::kCloses, kCells = Group<G>::kCells;
    constexpr uint32_t kPass = 8 * NT / (kTerms * kParts);
    static_assert(kPass > 0, "a row of x takes kTerms * kParts columns");
    constexpr int kRedPitch = 8 * NT + 1;
    constexpr int kTile = 16 * MT, kRows = 2 * MT;  // rows of a warp, of a lane
    extern __shared__ __align__(16) uint8_t smem[];  // zeros, x, info
    __shared__ float red[kWarps][kTile][kRedPitch];
    __shared__ uint32_t s_ids[kWindow];
    __shared__ uint32_t s_bits[32];
    __shared__ uint32_t s_count, s_bad;
    __shared__ int64_t s_x[kPass];  // where the rows of x of a pass start
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int wk_count = 1 << cfg.wk_log, wk = warp & (wk_count - 1), wr = warp >> cfg.wk_log;
    const int tile_rows_log = (MT == 2 ? 5 : 4) + (kWarps == 8 ? 3 : 2) - cfg.wk_log;
    const int tile_rows = 1 << tile_rows_log;  // kTile kWarps / wk
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) << tile_rows_log;      // the CTA's first row
    const bool by_id = p.ids != nullptr;

    uint32_t expert = 0;
    const uint32_t base_row = p.first_row + blockIdx.z * kWindow;
    const bool small = by_id && p.rows <= 32;
    uint32_t listed = 0;
    if (small) {
        if (!find_in_warp<T>(p, base_row, blockIdx.y, j0, tile_rows, s_ids, expert, listed)) return;
    } else if (by_id && !find_expert<T, kThreads>(p, base_row, blockIdx.y, j0, tile_rows, s_ids, s_bits, expert)) {
        return;
    }

    const int32_t row_len = static_cast<int32_t>((p.k + 1) / 2);
    const int32_t blocks = static_cast<int32_t>((p.k + 255) / 256);
    const int32_t groups = static_cast<int32_t>(p.groups);
    // The lane's rows are row + 8 h, h < kRows.  A tile that would pass the end starts earlier
    // and computes some rows of the one before again; kAnyhow: the last row is read in place
    // of those past the end, which are not stored.
    const int64_t start = j0 + wr * kTile, row = (A == kAnyhow ? start : min(start, p.n - kTile)) + g;
    const uint8_t *const matrix = p.q + static_cast<int64_t>(expert) * p.expert_stride;
    const uint8_t *const codes = matrix + row * p.ldq + 32 * c;
    const int64_t cells = static_cast<int64_t>(expert) * p.n * p.groups, cell = cells + row * p.groups;
    auto row_of = [&](int h) { return min(row + 8 * h, p.n - 1); };
    const int lane_cell = G == 128 ? 0 : kCells * (c & 1);  // the lane's first group of a block

    uint32_t exponents;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(exponents));
    auto z_of = [&](uint32_t raw, int byte, __half2 &z, __half2 &minus_z) {
        z = word_half2(__byte_perm(raw, exponents, byte == 0 ? 0x5050 : 0x5151));
        minus_z = __hsub2(word_half2(0x63806380u), z);
    };
    __half2 z[kRows], minus_z[kRows];  // 1024 + z and -(64 + z)
#pragma unroll
    for (int h = 0; h < kRows; ++h) z_of(0x0808u, 0, z[h], minus_z[h]);
    int32_t b1 = 0;  // end of the slab: what lies past it is not fetched
    auto fetch_codes = [&](int32_t block, uint4 (&q)[kRows][2]) {
        const int32_t at = block * 128 + 32 * c;  // in the row
        const bool in = block < b1 && at < row_len;
        if (A >= kApart) {
#pragma unroll
            for (int h = 0; h < kRows; ++h) load_stream32(in, codes + block * 128 + h * (8 * p.ldq), q[h]);
        } else if (A == kLoose) {
            const bool in2 = block < b1 && at + 16 < row_len;
            const bool ends = in && at + 32 > row_len;  // the row's end lies in these bytes
#pragma unroll
            for (int h = 0; h < kRows; ++h) {
                const bool last = ends && row + 8 * h == p.n - 1;
                const uint8_t *from = codes + block * 128 + h * (8 * p.ldq);
                load_stream16(in && !last, from, q[h][0]);
                load_stream16(in2 && !last, from + 16, q[h][1]);
            }
            if (ends && row <= p.n - 1 && row + 8 * kRows > p.n - 1) {
#pragma unroll
                for (int h = 0; h < kRows; ++h) {
                    if (row + 8 * h != p.n - 1) continue;
                    const uint8_t *from = codes + block * 128 + h * (8 * p.ldq);
                    q[h][0] = load_bytes(from, row_len - at);
                    q[h][1] = load_bytes(from + 16, row_len - at - 16);
                }
            }
        } else {
            const uint8_t *const first_byte = p.q, *const end = matrix + (p.n - 1) * p.ldq + row_len;
#pragma unroll
            for (int h = 0; h < kRows; ++h) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const uint8_t *from = matrix + row_of(h) * p.ldq + at + 16 * v;
                    const bool some = in && at + 16 * v < row_len;
                    const bool whole = from - 3 >= first_byte && from + 20 <= end;  // the words that cover them
                    q[h][v] = load_unaligned(some && whole, from);
                    if (some && !whole) q[h][v] = load_bytes(from, row_len - at - 16 * v);
                }
            }
        }
    };
    // Zero points of the lane's rows for its own codes of a block: one byte, with groups of 32 two.
    uint32_t z_raw[kRows];
#pragma unroll
    for (int h = 0; h < kRows; ++h) z_raw[h] = 0x0808u;
    auto fetch_zeros = [&](int32_t block) {
        const int32_t group = block * Group<G>::kInBlock + (G == 128 ? c >> 1 : G == 64 ? c : 2 * c);
        const bool have = group < groups;
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
            const uint8_t *z =
                p.zeros + (A == kAnyhow ? cells + row_of(h) * p.groups : cell + h * (8 * p.groups)) + group;
            if (G == 32 && A >= kApart)
                z_raw[h] = load_cells16(have, z);
            else
                z_raw[h] = load_cells8(have, z);
            if (G == 32 && A < kApart) z_raw[h] |= load_cells8(group + 1 < groups, z + 1) << 8;
        }
    };
    // Raw scales of the lane's kCells groups of a block.  kAtOnce: s.x, s.y pairs of scales.
    // Else: s.x, s.y one scale each; with groups of 32, pairs.  (32-bit scales are read where they
    // are used.)
    uint2 s_raw[kRows];
    auto fetch_scales = [&](int32_t block) {
        if (A == kAnyhow && p.scale_dtype == kF32) return;
        const int32_t group = block * Group<G>::kInBlock + lane_cell;
        const bool have = group < groups, more = group + kCells / 2 < groups;
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
            const int64_t at = (A == kAnyhow ? cells + row_of(h) * p.groups : cell + h * (8 * p.groups)) + group;
            const uint16_t *s = static_cast<const uint16_t *>(p.scales) + at;
            if (A == kAtOnce && kCells == 4) {
                s_raw[h] = load_cells64(have, s);
            } else if (A == kAtOnce) {
                s_raw[h].x = load_cells32(have, s);
            } else if (A == kApart && kCells == 4) {
                s_raw[h] = make_uint2(load_cells32(have, s), load_cells32(more, s + 2));
            } else if (kCells == 4) {
                const bool second = group + 1 < groups, fourth = group + 3 < groups;
                s_raw[h].x = load_cells16(have, s) | load_cells16(second, s + 1) << 16;
                s_raw[h].y = load_cells16(more, s + 2) | load_cells16(fourth, s + 3) << 16;
            } else {
                s_raw[h] = make_uint2(load_cells16(have, s), load_cells16(more, s + 1));
            }
        }
    };
    // scales of row h's groups `close` and `close` + kCloses among the lane's of a block
    auto scales_of = [&](int32_t block, int h, int close, float (&s)[2]) {
        if (A != kAnyhow || p.scale_dtype != kF32) {
            uint32_t a, b;
            if (kCells == 4) {  // close 0 takes groups 0 and 2, close 1 takes 1 and 3
                a = s_raw[h].x >> (16 * close) & 0xffffu;
                b = s_raw[h].y >> (16 * close) & 0xffffu;
            } else {
                a = A == kAtOnce ? s_raw[h].x & 0xffffu : s_raw[h].x;
                b = A == kAtOnce ? s_raw[h].x >> 16 : s_raw[h].y;
            }
            s[0] = scale_value(a, p.scale_dtype);
            s[1] = scale_value(b, p.scale_dtype);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t group = block * Group<G>::kInBlock + lane_cell + close + kCloses * i;
                s[i] = group < groups ? __ldg(static_cast<const float *>(p.scales) + cells + row_of(h) * p.groups + group)
                                      : 0.f;
            }
        }
    };
    uint4 q[kRows][2];
    b1 = min(cfg.slab << cfg.wk_log, blocks);
    fetch_codes(wk, q);
    if (p.zeros != nullptr) fetch_zeros(wk);
    fetch_scales(wk);
    // the zeros that lanes of another group read
    if (tid < kZeroBytes / 16) reinterpret_cast<uint4 *>(smem)[tid] = make_uint4(0u, 0u, 0u, 0u);
    uint8_t *stage = smem + kZeroBytes;
    float *info = reinterpret_cast<float *>(smem + cfg.info_at);
    const int32_t slab_blocks = cfg.slab << cfg.wk_log;
    const uint32_t pitch = (static_cast<uint32_t>(slab_blocks) << 9) + kPitchPad;

    const uint32_t first = by_id ? 0u : blockIdx.y * kPass;
    const uint32_t stride = by_id ? kPass : gridDim.y * kPass;
    const uint32_t count = !by_id ? p.rows : small ? listed : list_rows(p, base_row, expert, s_ids, &s_count);

#pragma unroll 1
    for (uint32_t t0 = first; t0 < count; t0 += stride) {
        const uint32_t tokens = min(count - t0, kPass);
        const uint32_t cols = tokens * kTerms * kParts;
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.f;

#pragma unroll 1
        for (int32_t b0 = 0; b0 < blocks; b0 += slab_blocks) {
            __syncthreads();  // the slab before, or the pass before, is done with
            if (b0 == 0) {
                if (tid == 0) s_bad = 0u;
                if (tid < tokens) {
                    const uint32_t r = by_id ? s_ids[t0 + tid] : t0 + tid, t = r / p.top_k;
                    s_x[tid] = t * p.ldx + (r - t * p.top_k) * p.x_slot_stride;
                }
                __syncthreads();
            }
            b1 = min(b0 + slab_blocks, blocks);
            stage_x<K, G, NT, kThreads>(p, cfg, s_x, tokens, b0 * 256,
                              static_cast<uint32_t>(b1 - b0) * 32, pitch, stage, info, &s_bad);
            __syncthreads();
            if (b0 != 0 || t0 != first) {
                fetch_codes(wk + b0, q);
                if (p.zeros != nullptr) fetch_zeros(wk + b0);
                fetch_scales(wk + b0);
            }
            // This lane's first word of the line of mma column 8 t + g, if its codes are of
            // that column's group.  Lanes past the last column repeat it; what they compute
            // is not stored.
            const uint8_t *xat[NT];
            uint32_t xstep[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t col = 8 * t + g < cols ? 8 * t + g : cols - 1;
                const bool own = (kParts == 2 ? c >> 1 : c) == static_cast<int>(col % kParts);
                xat[t] = own ? stage + (col / kParts) * pitch + wk * 512 + 16 * c : smem;
                xstep[t] = own ? 512 << cfg.wk_log : 0;
            }
            // what undoes the scalings of columns 2 c and 2 c + 1
            const float2 *iat = reinterpret_cast<const float2 *>(info + wk * (kCloses * 8 * NT)) + c;
#pragma unroll 1
            for (int32_t block = wk + b0; block < b1; block += wk_count) {
                float part[MT][NT][4];
                uint32_t z_now[kRows];
#pragma unroll
                for (int h = 0; h < kRows; ++h) z_now[h] = z_raw[h];
                if (p.zeros != nullptr) {
                    if (G != 32) {
#pragma unroll
                        for (int h = 0; h < kRows; ++h) z_of(z_now[h], 0, z[h], minus_z[h]);
                    }
                    fetch_zeros(block + wk_count);
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (G == 32) {
#pragma unroll
                        for (int h = 0; h < kRows; ++h) z_of(z_now[h], v, z[h], minus_z[h]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a[kRows][4];  // columns 0 and 4, 1 and 5, 2 and 6, 3 and 7 of a word
#pragma unroll
                        for (int h = 0; h < kRows; ++h) {
                            const uint32_t u = i == 0   ? q[h][v].x
                                               : i == 1 ? q[h][v].y
                                               : i == 2 ? q[h][v].z
                                                        : q[h][v].w;
                            a[h][0] = low_codes(u, exponents, z[h]);
                            a[h][1] = high_codes(u, exponents, minus_z[h]);
                            a[h][2] = low_codes(u >> 8, exponents, z[h]);
                            a[h][3] = high_codes(u >> 8, exponents, minus_z[h]);
                        }
                        const bool opens = i == 0 && (v == 0 || kCloses == 2);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint4 b = *reinterpret_cast<const uint4 *>(xat[t] + 256 * v + 64 * i);
#pragma unroll
                            for (int m = 0; m < MT; ++m) {
                                const uint32_t(&a0)[4] = a[2 * m], (&a1)[4] = a[2 * m + 1];
                                mma(part[m][t], opens, a0[0], a1[0], a0[1], a1[1], b.x, b.y);
                                mma(part[m][t], false, a0[2], a1[2], a0[3], a1[3], b.z, b.w);
                            }
                        }
                    }
                    if (v == 1) {
                        fetch_codes(block + wk_count, q);
                    }
                    if (v == 1 || kCloses == 2) {
                        const int close = kCloses == 2 ? v : 0;
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            float s[2][2];  // [row][column's group]
                            scales_of(block, 2 * m, close, s[0]);
                            scales_of(block, 2 * m + 1, close, s[1]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const float2 f = iat[close * (4 * NT) + 4 * t];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    // (the scale times the factor could pass the range of f32)
                                    float &sum = acc[m][t][i];
                                    sum = fmaf(s[i >> 1][i & 1], (i & 1 ? f.y : f.x) * part[m][t][i], sum);
                                }
                            }
                        }
                    }
                }
                fetch_scales(block + wk_count);
#pragma unroll
                for (int t = 0; t < NT; ++t) xat[t] += xstep[t];
                iat += (kCloses * 4 * NT) << cfg.wk_log;
            }
        }

        // the warps that split the columns, and the terms and groups of a row, add up in order
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    red[warp][16 * m + g + 8 * (i >> 1)][8 * t + 2 * c + (i & 1)] = acc[m][t][i];
        __syncthreads();
        const uint32_t bad = s_bad;
        for (uint32_t u = tid; u < tokens << tile_rows_log; u += kThreads) {
            const uint32_t jj = u & (tile_rows - 1), tok = u >> tile_rows_log;
            int64_t j = j0 + jj;
            if (A != kAnyhow)
                j = min(j0 + jj / kTile * kTile, p.n - kTile) + jj % kTile;
            else if (j >= p.n)
                continue;
            const uint32_t r = by_id ? s_ids[t0 + tok] : t0 + tok;
            float sum = 0.f;
            if (bad >> tok & 1u) {
                sum = plain_output<T>(p, expert, j, r);
            } else {
                for (int w = 0; w < wk_count; ++w) {
#pragma unroll
                    for (int i = 0; i < kTerms * kParts; ++i)
                        sum += red[((jj / kTile) << cfg.wk_log) + w][jj % kTile][tok * (kTerms * kParts) + i];
                }
            }
            static_cast<T *>(p.out)[static_cast<int64_t>(r) * p.ldo + j] = Elem<T>::from_f(sum);
        }
    }
}

template <Kind K, int G, Access A, int NT, int MT>
cudaError_t launch_nt(const Q4Params &p, int num_sms, cudaStream_t s) {
    using T = typename XType<K>::type;
    constexpr int kTerms = K == kFloat ? 3 : 1;
    constexpr uint32_t kPass = 8 * NT / (kTerms * Group<G>::kParts);
    using B = Budget<K, NT, MT>;
    constexpr int kTile = 16 * MT, kWarps = B::kWarps;
    const int64_t tiles = (p.n + kTile - 1) / kTile;
    const int64_t blocks = (p.k + 255) / 256;
    uint32_t gy, gz = 1;
    if (p.ids != nullptr) {
        gz = (std::min(p.rows - p.first_row, kQ4LaunchRows) + kWindow - 1) / kWindow;
        gy = p.rows < kWindow ? p.rows : kWindow;  // distinct experts of a window at most
        if (gy > p.n_experts) gy = p.n_experts;
    } else {
        gy = (p.rows + kPass - 1) / kPass;
        if (gy > 65535u) gy = 65535u;
    }
    Launch cfg{};
    // Warps that split the columns: enough for 16 warps an SM (8, and 4 with f32, where a pass
    // takes more than one column tile, as the staging of its rows is repeated for each CTA),
    // and no warp with 16 blocks or more, so that the last CTAs are short.  Measured: 8 an SM
    // 11.8 us for 10.0 (dense, 1 f16 row) and 24.2 for 19.3 (4 f32 tokens x 8 of 64 experts); 16
    // an SM with more column tiles 35.0 for 28.9 (8 f32 rows), 8 and 2 with f32 60.2 and 69.2
    // for 48.4 (6 tokens x 8 of 13 experts, 1472 x 3200, groups of 32); without the second rule
    // 118 for 105 (16 f32 tokens x 8 of 128 experts, 16 blocks) and 95.0 for 82.9 (bf16, groups
    // of 32), with at most 7 blocks a warp 116 and 87.5.
    int wk = 1;
    constexpr int64_t kEnough = NT == 1 ? 16 : K == kFloat ? 4 : 8;
    while (wk < kWarps && wk < blocks && (tiles * gy * wk < kEnough * num_sms || blocks >= 16 * wk)) {
        wk *= 2;
        ++cfg.wk_log;
    }
    cfg.x_vec = reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && p.ldx * sizeof(T) % 16 == 0 &&
                p.x_slot_stride * sizeof(T) % 16 == 0;
    const int lines = static_cast<int>(p.rows < kPass ? p.rows : kPass) * kTerms;
    const int64_t all = (blocks + wk - 1) / wk;
    const int per_block = wk * block_bytes(lines, NT, Group<G>::kCloses);
    cfg.slab = (B::kStageBytes - lines * kPitchPad) / per_block;
    if (cfg.slab > all) cfg.slab = static_cast<int>(all);
    cfg.info_at = kZeroBytes + lines * (cfg.slab * wk * 512 + kPitchPad);
    const int64_t wr = kWarps / wk;
    const int bytes = kZeroBytes + lines * kPitchPad + cfg.slab * per_block;

    static DeviceBits done{0};  // devices on which the kernel may use its shared memory
    int dev = 0;
    cudaGetDevice(&dev);
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(done & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(q4_kernel<K, G, A, NT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 B::kStageBytes + kZeroBytes);
        if (e != cudaSuccess) return e;
        done |= bit;
    }
    const dim3 grid(static_cast<unsigned>((tiles + wr - 1) / wr), gy, gz);
    // (Launched early, as the MoE layer's kernels are, this one gains 0.2 us with 1 f16 row and
    // loses 1.4 with 1 f32 row: its blocks, one wave, are spread over the SMs as places come free.)
    q4_kernel<K, G, A, NT, MT><<<grid, B::kThreads, bytes, s>>>(p, cfg);
    return cudaGetLastError();
}

template <Kind K, int G, int NT, int MT>
cudaError_t launch_access(const Q4Params &p, int num_sms, cudaStream_t s) {
    constexpr int kCells = Group<G>::kCells;
    auto multiple = [](const void *ptr, int64_t a) { return reinterpret_cast<uintptr_t>(ptr) % a == 0; };
    if (p.scale_dtype == kF32 || p.n < 16 * MT || !multiple(p.q, 16) || p.ldq % 16 != 0 || p.expert_stride % 16 != 0)
        return launch_nt<K, G, kAnyhow, NT, MT>(p, num_sms, s);
    if (!multiple(p.q, 32) || p.ldq % 32 != 0 || p.expert_stride % 32 != 0 || p.k % 64 != 0 ||
        !multiple(p.scales, kCells) || !multiple(p.zeros, G == 32 ? 2 : 1))
        return launch_nt<K, G, kLoose, NT, MT>(p, num_sms, s);
    if (p.groups % kCells == 0 && multiple(p.scales, 2 * kCells))
        return launch_nt<K, G, kAtOnce, NT, MT>(p, num_sms, s);
    return launch_nt<K, G, kApart, NT, MT>(p, num_sms, s);
}

// Column tiles: as few as hold the rows of x that a matrix meets, up to kWide.  A pass
// takes 8 NT / (terms kParts) rows; more tiles cost registers and shared memory, so that
// fewer warps are there to hide latency.  Per expert id the rows spread over the experts:
// on average there are `share` rows for each one that occurs, and a second pass over the
// few with more finds the weights in L2 (16 tokens x 8 of 128 experts with groups of 32:
// 82.9 us with one tile, 91.2 with two).  A matrix of few rows and 16-bit x is cut into row
// tiles of 16, so that every SM has several warps a scheduler (dense, 1 row, 11008 x 4096
// 10.0 us for 12.0, 4096 x 11008 12.3 for 13.4; with many rows 16 tokens x 8 of 128 experts 71.1
// for 66.1, hence the limit).  f32 has three times the staging for each row tile and always
// takes 32 (11008 x 4096: 10.9 for 14.8; 4096 x 11008, with fewer tiles, 20.1 for 17.4).
template <Kind K, int G>
cudaError_t launch_g(const Q4Params &p, int num_sms, cudaStream_t s) {
    constexpr int kColumns = (K == kFloat ? 3 : 1) * Group<G>::kParts;
    constexpr int kNarrow = (kColumns + 7) / 8;
    constexpr int kWide = K == kFloat ? 3 : G == 128 ? 2 : 4;
    const uint32_t distinct = p.rows < p.n_experts ? p.rows : p.n_experts;
    const uint32_t share = p.ids != nullptr ? (p.rows + distinct - 1) / distinct : p.rows;
    if (share * kColumns <= 8 * kNarrow) {
        if constexpr (K != kFloat) {
            const int64_t tiles = (p.n + 31) / 32 * (p.ids != nullptr ? distinct : 1);
            if (tiles < 4LL * num_sms) return launch_access<K, G, kNarrow, 1>(p, num_sms, s);
        }
        return launch_access<K, G, kNarrow, 2>(p, num_sms, s);
    }
    if (share * kColumns <= 8 * (kNarrow + 1)) return launch_access<K, G, kNarrow + 1, 2>(p, num_sms, s);
    return launch_access<K, G, kWide, 2>(p, num_sms, s);
}

template <Kind K>
cudaError_t launch(const Q4Params &p, int num_sms, cudaStream_t s) {
    constexpr int dt = K == kFloat ? kF32 : K == kHalf ? kF16 : kBF16;
    if (p.k == 0) return launch_fill_zero(dt, p.out, 1, p.rows, p.n, p.ldo, 0, s);
    if (p.group == 128) return launch_g<K, 128>(p, num_sms, s);
    if (p.group == 64) return launch_g<K, 64>(p, num_sms, s);
    return launch_g<K, 32>(p, num_sms, s);
}

}  // namespace q4
}  // namespace gbmm
