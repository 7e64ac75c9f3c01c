// Reductions over 16, 32 or 64 neighbouring lanes of a wave (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dtg {
namespace dev {

// A data-parallel-primitive move inside 16 lanes: 0xB1 and 0x4E exchange with
// lane ^ 1 and ^ 2, 0x141 and 0x140 mirror the lanes of 8 and of 16 (which hold,
// after the steps before, what ^ 4 and ^ 8 would bring).
template <int CTRL>
__device__ __forceinline__ uint32_t lane_swap(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
}

// op (commutative, associative) over T neighbouring lanes, the result in every
// one.  All T lanes must be active; other groups of T need not be.
template <int T, typename Op>
__device__ __forceinline__ uint32_t lanes(uint32_t v, Op op) {
    static_assert(T == 16 || T == 32 || T == 64, "lanes");
    v = op(v, lane_swap<0xB1>(v));
    v = op(v, lane_swap<0x4E>(v));
    v = op(v, lane_swap<0x141>(v));
    v = op(v, lane_swap<0x140>(v));
    if constexpr (T >= 32) v = op(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16)));
    if constexpr (T == 64) v = op(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 32)));
    return v;
}

}  // namespace dev
}  // namespace dtg
