// Checks that the ABIs of the row operators, the routing and the int8 products
// with scales share (host only).
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "api_internal.h"

namespace dtg {

inline gemm_status fail(gemm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline gemm_status fail(gemm_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return record_error(st, buf);
}

// Bytes from the first to one past the last of `rows` rows of `cols` elements, or -1 past 2^60.
inline int64_t extent(int64_t rows, int64_t stride, int64_t cols, int64_t size) {
    if (rows <= 0 || cols <= 0) return 0;
    const __int128 e = (static_cast<__int128>(rows - 1) * stride + cols) * size;
    return e > (static_cast<__int128>(1) << 60) ? -1 : static_cast<int64_t>(e);
}

// An operand: where it lies, and how its address must be aligned.
struct Operand {
    const char* name;
    const void* p;
    int64_t bytes;
    int align;
    bool written;
};

// Addresses there and aligned, no output overlapping anything.
inline gemm_status check(const Operand* o, int n) {
    for (int i = 0; i < n; ++i) {
        if (o[i].bytes == 0) continue;
        if (!o[i].p) return fail(GEMM_ERR_INVALID_ARG, "%s is NULL", o[i].name);
        if (reinterpret_cast<uintptr_t>(o[i].p) % o[i].align)
            return fail(GEMM_ERR_UNSUPPORTED, "%s must be aligned to its element size", o[i].name);
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (i == j || !o[i].written || o[i].bytes == 0 || o[j].bytes == 0) continue;
            const uintptr_t a = reinterpret_cast<uintptr_t>(o[i].p), b = reinterpret_cast<uintptr_t>(o[j].p);
            if (a < b + o[j].bytes && b < a + o[i].bytes)
                return fail(GEMM_ERR_INVALID_ARG, "%s overlaps %s", o[i].name, o[j].name);
        }
    return GEMM_OK;
}

inline gemm_status launched(hipError_t err, const char* what) {
    return err == hipSuccess ? GEMM_OK : fail(GEMM_ERR_HIP, "launch of the %s: %s", what, hipGetErrorString(err));
}

}  // namespace dtg
