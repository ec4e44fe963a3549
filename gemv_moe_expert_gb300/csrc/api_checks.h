// api_checks.h -- the argument checks that the entry points of moe_api.cu and
// ffn_api.cu share.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "api_internal.h"

namespace gbmm {

inline gbmm_status fail(gbmm_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return static_cast<gbmm_status>(record_error(s, buf));
}

// one operand of a call: the bytes it spans, its alignment and whether the call writes it.
// row_bytes and ld_bytes, where they are given, let two matrices of the same pitch lie side
// by side in one buffer.
struct Operand {
    const char *label;
    const void *ptr;
    uint64_t bytes;
    uint32_t align;
    bool output;
    uint64_t row_bytes = 0, ld_bytes = 0;
};

// bytes from the first to the last element of [rows, cols] with rows ld elements apart
inline bool span(uint64_t rows, int64_t cols, int64_t ld, uint64_t size, uint64_t *out) {
    if (rows == 0 || cols == 0) {
        *out = 0;
        return true;
    }
    const unsigned __int128 last =
        static_cast<unsigned __int128>(rows - 1) * static_cast<uint64_t>(ld) + static_cast<uint64_t>(cols);
    if (last > INT64_MAX / size) return false;
    *out = static_cast<uint64_t>(last) * size;
    return true;
}

// whether no row of b meets a row of a: both have the same pitch, and modulo that pitch b's
// rows lie between two of a's
inline bool side_by_side(const Operand &a, const Operand &b) {
    if (a.ld_bytes == 0 || a.ld_bytes != b.ld_bytes) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.ptr), pb = reinterpret_cast<uintptr_t>(b.ptr);
    const uint64_t ld = a.ld_bytes, d = pb >= pa ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;
    return d >= a.row_bytes && d + b.row_bytes <= ld;
}

// Non-null, aligned, and no output on top of another operand.  Operands of 0
// bytes are not looked at.
inline gbmm_status check_operands(const char *fn, const Operand *ops, int count) {
    for (int i = 0; i < count; ++i) {
        if (ops[i].bytes == 0) continue;
        if (ops[i].ptr == nullptr) return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: %s is null", fn, ops[i].label);
        if (reinterpret_cast<uintptr_t>(ops[i].ptr) % ops[i].align != 0)
            return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: %s is not aligned to its element", fn, ops[i].label);
        if (ops[i].bytes > UINTPTR_MAX - reinterpret_cast<uintptr_t>(ops[i].ptr))
            return fail(GBMM_ERR_INVALID_ARGUMENT, "%s: %s runs past the address space", fn, ops[i].label);
    }
    for (int i = 0; i < count; ++i) {
        if (!ops[i].output || ops[i].bytes == 0) continue;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(ops[i].ptr), hi = lo + ops[i].bytes;
        for (int j = 0; j < count; ++j) {
            if (j == i || ops[j].bytes == 0) continue;
            const uintptr_t l = reinterpret_cast<uintptr_t>(ops[j].ptr), h = l + ops[j].bytes;
            if (lo < h && l < hi && !side_by_side(ops[i], ops[j]))
                return fail(GBMM_ERR_OVERLAP, "%s: %s overlaps %s", fn, ops[i].label, ops[j].label);
        }
    }
    return GBMM_OK;
}

inline bool known_dtype(gbmm_dtype dt) { return dt == GBMM_F32 || dt == GBMM_F16 || dt == GBMM_BF16; }

inline cudaStream_t cuda_stream(gbmm_stream s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace gbmm
