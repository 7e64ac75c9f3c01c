// C ABI of the row operators (RMS norm and its gradients, rows in 8 bits):
// validation and launch.  Declarations and the contract are in include/gemm.h.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/gemm.h"
#include "api_operands.h"
#include "kernels_layer.h"

namespace {

using dtg::check;
using dtg::extent;
using dtg::fail;
using dtg::launched;
using dtg::Operand;

// Sizes and one stride of each operand that the call has.
struct Stride {
    const char* name;
    int64_t stride;
    bool written;
};

gemm_status sizes(int64_t R, int64_t K, gemm_dtype dtype, const Stride* s, int n) {
    if (R < 0 || K < 0) return fail(GEMM_ERR_INVALID_ARG, "negative size R=%lld K=%lld", (long long)R, (long long)K);
    if (dtype != GEMM_F16 && dtype != GEMM_BF16)
        return fail(GEMM_ERR_INVALID_ARG, "dtype %d: rows are GEMM_F16 or GEMM_BF16", (int)dtype);
    if (R > dtg::kMaxSize || K > dtg::kMaxRow)
        return fail(GEMM_ERR_UNSUPPORTED, "more than 2^31-4096 rows or 2^24 values a row are not supported");
    for (int i = 0; i < n; ++i) {
        if (s[i].stride < 0) return fail(GEMM_ERR_UNSUPPORTED, "negative stride of %s", s[i].name);
        if (extent(R, s[i].stride, K, 4) < 0) return fail(GEMM_ERR_INVALID_ARG, "the stride of %s reaches past 2^60 bytes", s[i].name);
        if (s[i].written && R > 1 && s[i].stride < K)
            return fail(GEMM_ERR_INVALID_ARG, "row stride %lld < K=%lld makes rows of %s overlap", (long long)s[i].stride,
                        (long long)K, s[i].name);
    }
    return GEMM_OK;
}

gemm_status norm_problem(const gemm_norm_problem* p, const Stride* s, int n) {
    const gemm_status st = sizes(p->R, p->K, p->dtype, s, n);
    if (st != GEMM_OK) return st;
    if (p->weight != p->dtype && p->weight != GEMM_F32)
        return fail(GEMM_ERR_INVALID_ARG, "weight type %d: the rows' type or GEMM_F32", (int)p->weight);
    if (p->has_residual != 0 && p->has_residual != 1)
        return fail(GEMM_ERR_INVALID_ARG, "has_residual must be 0 or 1, got %d", (int)p->has_residual);
    if (!(p->eps > 0.0f) || !isfinite(p->eps))
        return fail(GEMM_ERR_INVALID_ARG, "eps must be positive and finite, got %g", (double)p->eps);
    return GEMM_OK;
}

// The norm into y (16-bit) or into q and scale.
gemm_status norm(const gemm_norm_problem* p, const void* x, const void* r, const void* w, void* h, void* y, int8_t* q,
                 float* scale, float* rstd, void* stream) {
    if (!p) return fail(GEMM_ERR_INVALID_ARG, "problem is NULL");
    const bool res = p->has_residual != 0;
    const Stride s[4] = {{"x", p->sx, false}, {"y", p->sy, true}, {"r", res ? p->sr : 0, false}, {"h", p->sh, true}};
    gemm_status st = norm_problem(p, s, res ? 4 : 2);
    if (st != GEMM_OK) return st;
    if (!res && (r || h)) return fail(GEMM_ERR_INVALID_ARG, "r or h given but the problem has has_residual = 0");
    const int64_t wide = p->weight == GEMM_F32 ? 4 : 2, some = p->K > 0 ? p->R * 4 : 0;
    const Operand o[7] = {{"x", x, extent(p->R, p->sx, p->K, 2), 2, false},
                          {"r", r, res ? extent(p->R, p->sr, p->K, 2) : 0, 2, false},
                          {"w", w, p->R > 0 ? p->K * wide : 0, static_cast<int>(wide), false},
                          {"h", h, res ? extent(p->R, p->sh, p->K, 2) : 0, 2, true},
                          {q ? "q" : "y", q ? static_cast<void*>(q) : y, extent(p->R, p->sy, p->K, q ? 1 : 2), q ? 1 : 2, true},
                          {"scale", scale, q ? p->R * 4 : 0, 4, true},
                          {"rstd", rstd, rstd ? some : 0, 4, true}};
    st = check(o, 7);
    if (st != GEMM_OK) return st;
    // rows of no values: their scales are zeros
    if (p->R == 0 || (p->K == 0 && !q)) return GEMM_OK;
    dtg::RowsArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.r = static_cast<const uint16_t*>(res ? r : nullptr);
    a.w = w;
    a.h = static_cast<uint16_t*>(h);
    a.y = static_cast<uint16_t*>(y);
    a.q = q;
    a.scale = scale;
    a.rstd = rstd;
    a.R = p->R;
    a.K = static_cast<int32_t>(p->K);
    a.sx = p->sx;
    a.sr = p->sr;
    a.sh = p->sh;
    a.sy = p->sy;
    a.w32 = p->weight == GEMM_F32;
    a.eps = p->eps;
    if (p->K == 0) a.w = nullptr;
    return launched(dtg::launch_rows(a, p->dtype == GEMM_BF16, static_cast<hipStream_t>(stream)), "norm");
}

// Bytes of the gradient's parts, or -1.
int64_t parts_bytes(const gemm_norm_problem* p) {
    return p->R > 0 && p->K > 0 ? extent(dtg::norm_grad_parts(p->R, p->K), p->K, p->K, 4) : 0;
}

}  // namespace

extern "C" {

gemm_status gemm_rms_norm(const gemm_norm_problem* prob, const void* x, const void* r, const void* w, void* h, void* y,
                          float* rstd, void* stream) {
    return norm(prob, x, r, w, h, y, nullptr, nullptr, rstd, stream);
}

gemm_status gemm_rms_norm_i8(const gemm_norm_problem* prob, const void* x, const void* r, const void* w, void* h, int8_t* q,
                             float* scale, void* stream) {
    if (prob && prob->R > 0 && !q) {
        if (prob->K > 0 || !scale) return fail(GEMM_ERR_INVALID_ARG, "q or scale is NULL");
        q = reinterpret_cast<int8_t*>(scale);   // of no bytes
    }
    return norm(prob, x, r, w, h, nullptr, q, scale, nullptr, stream);
}

gemm_status gemm_rms_norm_grad_workspace(const gemm_norm_problem* prob, size_t* bytes) {
    if (!prob || !bytes) return fail(GEMM_ERR_INVALID_ARG, "problem or bytes is NULL");
    *bytes = 0;
    const gemm_status st = norm_problem(prob, nullptr, 0);
    if (st != GEMM_OK) return st;
    *bytes = static_cast<size_t>(parts_bytes(prob));
    return GEMM_OK;
}

gemm_status gemm_rms_norm_grad(const gemm_norm_problem* prob, const void* dy, const void* dh, const void* h, const void* w,
                               const float* rstd, void* dx, void* dw, void* workspace, size_t workspace_bytes, void* stream) {
    if (!prob) return fail(GEMM_ERR_INVALID_ARG, "problem is NULL");
    const gemm_norm_problem* p = prob;
    const bool res = p->has_residual != 0;
    const Stride s[4] = {{"dy", p->sy, false}, {"h", p->sh, false}, {"dx", p->sx, true}, {"dh", p->sr, false}};
    gemm_status st = norm_problem(p, s, res ? 4 : 3);
    if (st != GEMM_OK) return st;
    if (!res && dh) return fail(GEMM_ERR_INVALID_ARG, "dh given but the problem has has_residual = 0");
    const int64_t wide = p->weight == GEMM_F32 ? 4 : 2, need = dw ? parts_bytes(p) : 0;
    if (need > 0 && (!workspace || workspace_bytes < static_cast<size_t>(need)))
        return fail(GEMM_ERR_WORKSPACE, "workspace of %lld bytes needed, got %lld", (long long)need,
                    (long long)(workspace ? workspace_bytes : 0));
    const Operand o[8] = {{"dy", dy, extent(p->R, p->sy, p->K, 2), 2, false},
                          {"dh", dh, res ? extent(p->R, p->sr, p->K, 2) : 0, 2, false},
                          {"h", h, extent(p->R, p->sh, p->K, 2), 2, false},
                          {"w", w, p->R > 0 ? p->K * wide : 0, static_cast<int>(wide), false},
                          {"rstd", rstd, p->K > 0 ? p->R * 4 : 0, 4, false},
                          {"dx", dx, extent(p->R, p->sx, p->K, 2), 2, true},
                          {"dw", dw, dw ? p->K * wide : 0, static_cast<int>(wide), true},
                          {"workspace", workspace, need, 16, true}};
    st = check(o, 8);
    if (st != GEMM_OK || p->K == 0) return st;
    const hipStream_t on = static_cast<hipStream_t>(stream);
    if (p->R > 0) {
        dtg::NormGradArgs a = {};
        a.dy = static_cast<const uint16_t*>(dy);
        a.dh = static_cast<const uint16_t*>(res ? dh : nullptr);
        a.h = static_cast<const uint16_t*>(h);
        a.w = w;
        a.rstd = rstd;
        a.dx = static_cast<uint16_t*>(dx);
        a.parts = static_cast<float*>(dw ? workspace : nullptr);
        a.R = p->R;
        a.K = static_cast<int32_t>(p->K);
        a.sy = p->sy;
        a.sr = p->sr;
        a.sh = p->sh;
        a.sx = p->sx;
        a.w32 = p->weight == GEMM_F32;
        st = launched(dtg::launch_norm_grad(a, p->dtype == GEMM_BF16, on), "norm's gradient");
        if (st != GEMM_OK) return st;
    }
    if (!dw) return GEMM_OK;   // without rows: zeros
    return launched(dtg::launch_norm_weight_grad(static_cast<float*>(workspace),
                                                 p->R > 0 ? dtg::norm_grad_parts(p->R, p->K) : 0, p->K, dw,
                                                 p->weight == GEMM_F32 ? 2 : p->weight == GEMM_BF16 ? 1 : 0, on),
                    "norm's weight gradient");
}

gemm_status gemm_i8_quantize(const void* x, gemm_dtype dtype, int64_t R, int64_t K, int64_t sx, int8_t* q, int64_t sq,
                             float* scale, void* stream) {
    const Stride s[2] = {{"x", sx, false}, {"q", sq, true}};
    gemm_status st = sizes(R, K, dtype, s, 2);
    if (st != GEMM_OK) return st;
    const Operand o[3] = {{"x", x, extent(R, sx, K, 2), 2, false},
                          {"q", q, extent(R, sq, K, 1), 1, true},
                          {"scale", scale, R * 4, 4, true}};
    st = check(o, 3);
    if (st != GEMM_OK || R == 0) return st;
    dtg::RowsArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.q = q;
    a.scale = scale;
    a.R = R;
    a.K = static_cast<int32_t>(K);
    a.sx = sx;
    a.sy = sq;
    return launched(dtg::launch_rows(a, dtype == GEMM_BF16, static_cast<hipStream_t>(stream)), "quantization");
}

}  // extern "C"
