// The last step of a weight gradient whose groups were cut into parts
// (grouped_kernel.h): D[g] (+)= the fp32 sums of the group's parts, added in
// order and rounded once.  One thread per 4 consecutive elements; bound by the
// parts' bytes.
#include "grouped_kernel.h"

namespace dtg {
namespace {

constexpr int kThreads = 256;

template <bool BF16, bool O32>
__global__ __launch_bounds__(kThreads) void sum_parts_kernel(GroupedArgs a) {
    const int lane = threadIdx.x & 63;
    const int g = blockIdx.y;
    // parts of the groups before this one, and its own
    uint32_t first = 0, count = 0;
    for (int base = 0; base <= g; base += 64) {
        uint32_t n = 0;
        if (base + lane <= g) n = group_parts(table_segment(a, base + lane + 1).rows, a.part_rows);
        const uint32_t incl = wave_scan(n);
        const int last = g - base < 63 ? g - base : 63;
        first += __builtin_amdgcn_readlane(incl, last);
        count = __builtin_amdgcn_readlane(n, last);
    }
    first -= count;
    const int64_t size = static_cast<int64_t>(a.P) * a.Q;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4;   // Q is a multiple of 8
    if (at >= size) return;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t stop = first + count < static_cast<uint32_t>(a.max_parts) ? first + count : a.max_parts;
    for (uint32_t n = first; n < stop; n += 8) {
        f32x4 part[8];   // eight parts in flight (past the last one: that one again, not added)
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            part[i] = *reinterpret_cast<const f32x4*>(a.parts + static_cast<int64_t>(n + i < stop ? n + i : stop - 1) * size + at);
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i)
            if (n + i < stop) v += part[i];
    }
    const int64_t d = static_cast<int64_t>(g) * a.sd_g + at / a.Q * a.sd_r + at % a.Q;
    const bool vec = (a.sd_r | a.sd_g) % 4 == 0 && reinterpret_cast<uintptr_t>(a.D) % 16 == 0;
    if constexpr (O32) {
        float* D = static_cast<float*>(a.D) + d;
        if (vec) {
            if (a.accumulate) v += *reinterpret_cast<const f32x4*>(D);
            *reinterpret_cast<f32x4*>(D) = v;
        } else {
            for (int e = 0; e < 4; ++e) D[e] = a.accumulate ? v[e] + D[e] : v[e];
        }
    } else {
        uint16_t* D = static_cast<uint16_t*>(a.D) + d;
        uint16_t h[4];
        if (a.accumulate)
            for (int e = 0; e < 4; ++e) v[e] += widen<BF16>(D[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = narrow<BF16>(v[e]);
        if (vec)
            *reinterpret_cast<u32x2*>(D) = u32x2{h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16};
        else
            for (int e = 0; e < 4; ++e) D[e] = h[e];
    }
}

}  // namespace

hipError_t launch_sum_parts(const GroupedArgs& a, int dtype, int out32, hipStream_t stream) {
    const int64_t size = static_cast<int64_t>(a.P) * a.Q;
    const dim3 grid(static_cast<unsigned>((size + 4 * kThreads - 1) / (4 * kThreads)), static_cast<unsigned>(a.groups));
    if (out32) hipLaunchKernelGGL((sum_parts_kernel<false, true>), grid, dim3(kThreads), 0, stream, a);
    else if (dtype) hipLaunchKernelGGL((sum_parts_kernel<true, false>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((sum_parts_kernel<false, false>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace dtg
