// From an exact int32 sum to an output of the int8 products with scales: in
// fp32 times the row's scale, times the column's, plus the bias, rounded once.
// The sum itself is rounded to fp32 where it passes 2^24.
#pragma once

#include "device_common.h"
#include "kernels_i8.h"

namespace dtg {
namespace dev {

template <int OUT>
__device__ __forceinline__ float bias_at(const void* b, int64_t n) {
    if constexpr (OUT == kOutF32) return static_cast<const float*>(b)[n];
    else return widen<OUT == kOutBF16>(static_cast<const uint16_t*>(b)[n]);
}

__device__ __forceinline__ float scaled(float bits, float sx, float sw) {
    return static_cast<float>(__builtin_bit_cast(int, bits)) * sx * sw;
}

// Four sums of row m, columns n .. n + 3 (those below N).
template <int OUT>
__device__ __forceinline__ void store_scaled(const I8RowsArgs& a, int m, int n, f32x4 sum) {
    if (n >= a.N) return;
    const float sx = a.s.sx[m];
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int c = n + r < a.N ? n + r : a.N - 1;
        v[r] = scaled(sum[r], sx, a.s.sw[c]);
        if (a.s.bias) v[r] += bias_at<OUT>(a.s.bias, c);
    }
    const int64_t at = static_cast<int64_t>(m) * a.ly + n;
    if constexpr (OUT == kOutF32) {
        float* y = static_cast<float*>(a.Y) + at;
        if (n + 4 <= a.N && reinterpret_cast<uintptr_t>(y) % 16 == 0) {
            *reinterpret_cast<f32x4*>(y) = f32x4{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < a.N) y[r] = v[r];
        }
    } else {
        constexpr bool B = OUT == kOutBF16;
        uint16_t* y = static_cast<uint16_t*>(a.Y) + at;
        if (n + 4 <= a.N && reinterpret_cast<uintptr_t>(y) % 8 == 0) {
            *reinterpret_cast<u32x2*>(y) = u32x2{narrow<B>(v[0]) | static_cast<uint32_t>(narrow<B>(v[1])) << 16,
                                                 narrow<B>(v[2]) | static_cast<uint32_t>(narrow<B>(v[3])) << 16};
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < a.N) y[r] = narrow<B>(v[r]);
        }
    }
}

}  // namespace dev
}  // namespace dtg
