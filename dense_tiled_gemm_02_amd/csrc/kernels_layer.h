// Internal interface between the ABI of the row operators (api_rows.cpp) and
// their kernels: RMS norm, rows in 8 bits, routing to experts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dtg {

constexpr int64_t kMaxRow = int64_t(1) << 24;   // K

// One row each: h = x (+ r), y = h w / sqrt(mean h^2 + eps) (w nullptr: y = x),
// as 16-bit values (y) or as int8 with the row's scale (q).  Strides in
// elements; rows of K contiguous elements at any address.
struct RowsArgs {
    const uint16_t* x;
    const uint16_t* r;     // nullptr: no addend
    const void* w;         // 16-bit, or fp32 with w32
    uint16_t* h;           // written with an addend
    uint16_t* y;
    int8_t* q;
    float* scale;
    float* rstd;           // nullptr, or 1 / sqrt(mean h^2 + eps) of every row
    int64_t R, sx, sr, sh, sy;
    int32_t K, w32;
    float eps;
    float by;              // filled in by launch_rows: 1, or what values are scaled by before they are squared
};

// dx = dh + (g - h c) rstd with g = dy w, c = rstd^2 mean(g h); parts: per
// workgroup, the K sums over its rows of dy h rstd (nullptr: not wanted).
struct NormGradArgs {
    const uint16_t* dy;
    const uint16_t* dh;    // nullptr: none
    const uint16_t* h;
    const void* w;
    const float* rstd;
    uint16_t* dx;
    float* parts;
    int64_t R, sy, sr, sh, sx;
    int32_t K, w32;
};

hipError_t launch_rows(const RowsArgs& a, int bf16, hipStream_t stream);
// Workgroups of the gradient over R rows of K, each a row of `parts`.
int64_t norm_grad_parts(int64_t R, int64_t K);
hipError_t launch_norm_grad(const NormGradArgs& a, int bf16, hipStream_t stream);
// dw[k] = sum of the parts' k, in order; dw is fp32 (kind 2), bf16 (1) or fp16 (0).
// The parts may be overwritten.
hipError_t launch_norm_weight_grad(float* parts, int64_t nparts, int64_t K, void* dw, int kind, hipStream_t stream);

}  // namespace dtg
