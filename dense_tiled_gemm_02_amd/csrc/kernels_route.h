// Internal interface between the routing ABI (api_route.cpp) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dtg {

constexpr int kMaxExperts = 1024, kMaxExpertGroups = 64, kMaxTop = 64;

struct RouteArgs {
    const void* logits;    // R x E, fp32, fp16 or bf16
    const float* bias;     // E, or nullptr
    float* weights;        // R x top
    int32_t* ids;          // R x top
    int64_t R, sl;         // row stride of logits, elements
    int32_t E, top;
    int32_t groups, top_groups, group_best;
    int32_t sigmoid, renorm;
    float scale;
    uint32_t per_group_inv;   // floor(e per_group_inv / 2^20) = e / (E / groups) for e < E
    // filled in by launch_route: the launch's first row, doubles of LDS to a row,
    // and where the groups' lanes lie
    int64_t first;
    int32_t spare;
    int32_t per;              // E / groups
    int32_t lane_shift;       // a group has 1 << lane_shift lanes
    int32_t in_lanes;         // 1: whose logits are that group's
};

struct RouteGradArgs {
    const void* logits;
    const int32_t* ids;    // R x top
    const float* dw;       // R x top
    void* dl;              // R x E, of the logits' type
    int64_t R, sl;
    int64_t first;         // the launch's first row (filled in by launch_route_grad)
    int32_t E, top;
    int32_t sigmoid, renorm;
    float scale;
};

// kind: 0 fp16, 1 bf16, 2 fp32 logits
hipError_t launch_route(const RouteArgs& a, int kind, hipStream_t stream);
hipError_t launch_route_grad(const RouteGradArgs& a, int kind, hipStream_t stream);

}  // namespace dtg
