// C ABI of the routing of tokens to experts: validation and launch.
// Declarations and the contract are in include/gemm.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/gemm.h"
#include "api_operands.h"
#include "kernels_route.h"

namespace {

using dtg::check;
using dtg::fail;
using dtg::launched;
using dtg::Operand;

gemm_status validate(const gemm_route_problem* p) {
    if (!p) return fail(GEMM_ERR_INVALID_ARG, "problem is NULL");
    if (p->R < 0 || p->E < 1 || p->top < 1)
        return fail(GEMM_ERR_INVALID_ARG, "R=%lld E=%d top=%d: at least no rows, one expert and one choice", (long long)p->R,
                    (int)p->E, (int)p->top);
    if (p->dtype != GEMM_F16 && p->dtype != GEMM_BF16 && p->dtype != GEMM_F32)
        return fail(GEMM_ERR_INVALID_ARG, "dtype %d: logits are GEMM_F16, GEMM_BF16 or GEMM_F32", (int)p->dtype);
    if (p->score != GEMM_SCORE_SOFTMAX && p->score != GEMM_SCORE_SIGMOID)
        return fail(GEMM_ERR_INVALID_ARG, "score %d is none of GEMM_SCORE_SOFTMAX, GEMM_SCORE_SIGMOID", (int)p->score);
    if ((p->has_bias != 0 && p->has_bias != 1) || (p->renormalize != 0 && p->renormalize != 1))
        return fail(GEMM_ERR_INVALID_ARG, "has_bias and renormalize must be 0 or 1, got %d and %d", (int)p->has_bias,
                    (int)p->renormalize);
    if (!isfinite(p->scale)) return fail(GEMM_ERR_INVALID_ARG, "scale must be finite");
    if (p->groups < 1 || p->E % p->groups || p->top_groups < 1 || p->top_groups > p->groups)
        return fail(GEMM_ERR_INVALID_ARG, "groups=%d top_groups=%d: groups must divide E=%d, top_groups be 1 to groups",
                    (int)p->groups, (int)p->top_groups, (int)p->E);
    if (p->group_best != 1 && p->group_best != 2)
        return fail(GEMM_ERR_INVALID_ARG, "group_best must be 1 or 2, got %d", (int)p->group_best);
    if (p->top > p->E / p->groups * p->top_groups)
        return fail(GEMM_ERR_INVALID_ARG, "top=%d is more than the %d experts of %d groups", (int)p->top,
                    (int)(p->E / p->groups * p->top_groups), (int)p->top_groups);
    if (p->E > dtg::kMaxExperts || p->top > dtg::kMaxTop || p->groups > dtg::kMaxExpertGroups || p->R > dtg::kMaxSize)
        return fail(GEMM_ERR_UNSUPPORTED, "at most %d experts, %d choices, %d groups and 2^31-4096 rows", dtg::kMaxExperts,
                    dtg::kMaxTop, dtg::kMaxExpertGroups);
    if (p->sl < 0) return fail(GEMM_ERR_UNSUPPORTED, "negative stride");
    if (p->sl > (int64_t(1) << 60) / (p->R > 0 ? p->R : 1) - p->E)
        return fail(GEMM_ERR_INVALID_ARG, "the stride of the logits reaches past 2^60 elements");
    return GEMM_OK;
}

int64_t size_of(const gemm_route_problem* p) { return p->dtype == GEMM_F32 ? 4 : 2; }
int64_t logit_bytes(const gemm_route_problem* p) { return p->R > 0 ? ((p->R - 1) * p->sl + p->E) * size_of(p) : 0; }
int kind_of(const gemm_route_problem* p) { return p->dtype == GEMM_F32 ? 2 : p->dtype == GEMM_BF16 ? 1 : 0; }

}  // namespace

extern "C" {

gemm_status gemm_route(const gemm_route_problem* prob, const void* logits, const float* bias, float* weights, int32_t* ids,
                       void* stream) {
    gemm_status st = validate(prob);
    if (st != GEMM_OK) return st;
    const gemm_route_problem& p = *prob;
    if (!p.has_bias && bias) return fail(GEMM_ERR_INVALID_ARG, "bias given but the problem has has_bias = 0");
    const int64_t chosen = p.R * p.top * 4;
    const Operand o[4] = {{"logits", logits, logit_bytes(prob), static_cast<int>(size_of(prob)), false},
                          {"bias", bias, p.has_bias && p.R > 0 ? p.E * 4 : 0, 4, false},
                          {"weights", weights, chosen, 4, true},
                          {"ids", ids, chosen, 4, true}};
    st = check(o, 4);
    if (st != GEMM_OK || p.R == 0) return st;
    dtg::RouteArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.weights = weights;
    a.ids = ids;
    a.R = p.R;
    a.sl = p.sl;
    a.E = p.E;
    a.top = p.top;
    a.groups = p.groups;
    a.top_groups = p.top_groups;
    a.group_best = p.group_best;
    a.sigmoid = p.score == GEMM_SCORE_SIGMOID;
    a.renorm = p.renormalize;
    a.scale = p.scale;
    // ceil(2^20 / n): e times its excess, below 1, stays under 2^20 / n for e < 2^20 / n, n and e up to 1024
    const int n = p.E / p.groups;
    a.per_group_inv = static_cast<uint32_t>(((1 << 20) + n - 1) / n);
    return launched(dtg::launch_route(a, kind_of(prob), static_cast<hipStream_t>(stream)), "routing");
}

gemm_status gemm_route_grad(const gemm_route_problem* prob, const void* logits, const int32_t* ids, const float* dweights,
                            void* dlogits, void* stream) {
    gemm_status st = validate(prob);
    if (st != GEMM_OK) return st;
    const gemm_route_problem& p = *prob;
    const int64_t chosen = p.R * p.top * 4;
    const Operand o[4] = {{"logits", logits, logit_bytes(prob), static_cast<int>(size_of(prob)), false},
                          {"ids", ids, chosen, 4, false},
                          {"dweights", dweights, chosen, 4, false},
                          {"dlogits", dlogits, p.R * p.E * size_of(prob), static_cast<int>(size_of(prob)), true}};
    st = check(o, 4);
    if (st != GEMM_OK || p.R == 0) return st;
    dtg::RouteGradArgs a = {};
    a.logits = logits;
    a.ids = ids;
    a.dw = dweights;
    a.dl = dlogits;
    a.R = p.R;
    a.sl = p.sl;
    a.E = p.E;
    a.top = p.top;
    a.sigmoid = p.score == GEMM_SCORE_SIGMOID;
    a.renorm = p.renormalize;
    a.scale = p.scale;
    return launched(dtg::launch_route_grad(a, kind_of(prob), static_cast<hipStream_t>(stream)), "routing's gradient");
}

}  // extern "C"
