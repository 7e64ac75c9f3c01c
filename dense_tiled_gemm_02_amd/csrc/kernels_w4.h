// Internal interface between the 4-bit matrix-vector ABI (api_w4.cpp) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dtg {

// Y[m, n] = sum_k X[m, k] (q[e, n, k] - z[e, n, k / G]) s[e, n, k / G], e = the
// row's expert (0 without experts).  W holds two k per byte, even k in the
// low nibble.  X, S, Y strides in elements, W, Z strides in bytes.
struct W4Args {
    const uint16_t* X;
    const uint8_t* W;
    const uint16_t* S;
    const uint8_t* Z;       // nullptr: z = 8
    const void* experts;    // nullptr: one matrix for every row
    uint16_t* Y;
    int32_t M, N, K;
    int32_t num_experts;    // 1 without experts
    int32_t id_bytes;       // 4 or 8
    int32_t by_row;         // workgroups for each row's expert in place of each expert (M <= 64)
    int64_t sx, sy;
    int64_t sw_n, sw_e, ss_n, ss_e, sz_n, sz_e;
};

typedef hipError_t (*w4_launch_fn)(const W4Args& args, int64_t tiles, hipStream_t stream);

// One compiled variant: 16 nb columns and 16 mb rows per workgroup pass.
struct W4Entry {
    int32_t nb, mb, waves, group;
    int32_t dtype;          // 0 fp16, 1 bf16
    int32_t zeros;
    w4_launch_fn launch;
    const char* name;
};

const W4Entry* w4_kernel_table(int* count);

}  // namespace dtg
