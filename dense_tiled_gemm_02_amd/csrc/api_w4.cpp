// C ABI of the matrix-vector product with 4-bit weights: validation, variant
// choice and launch.  Declarations and the contract are in include/gemm.h.
#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/gemm.h"
#include "api_internal.h"
#include "kernels_w4.h"

struct gemm_w4_plan {
    gemm_w4_problem prob;
    const dtg::W4Entry* entry;
    int64_t tiles;
};

namespace {

gemm_status fail(gemm_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gemm_status fail(gemm_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return dtg::record_error(st, buf);
}

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Units from the first to one past the last of `experts` matrices of `rows`
// rows of `cols`, or -1 past 2^60.
int64_t extent(int64_t experts, int64_t se, int64_t rows, int64_t sr, int64_t cols) {
    if (experts <= 0 || rows <= 0 || cols <= 0) return 0;
    const __int128 e = static_cast<__int128>(experts - 1) * se + static_cast<__int128>(rows - 1) * sr + cols;
    return e > (static_cast<__int128>(1) << 60) ? -1 : static_cast<int64_t>(e);
}

int64_t matrices(const gemm_w4_problem* p) { return p->experts > 0 ? p->experts : 1; }
int64_t w_bytes(const gemm_w4_problem* p) { return extent(matrices(p), p->sw_e, p->N, p->sw_n, p->K / 2); }
int64_t s_elems(const gemm_w4_problem* p) {
    return extent(matrices(p), p->ss_e, p->N, p->ss_n, cdiv(p->K, p->group));
}
int64_t z_bytes(const gemm_w4_problem* p) {
    return p->has_zeros ? extent(matrices(p), p->sz_e, p->N, p->sz_n, cdiv(p->K, p->group)) : 0;
}
int64_t x_elems(const gemm_w4_problem* p) { return extent(1, 0, p->M, p->sx, p->K); }
int64_t y_elems(const gemm_w4_problem* p) { return extent(1, 0, p->M, p->sy, p->N); }

// Workgroups for each row's expert in place of each expert (one row over 41
// experts of 288 x 8797: 29 us with workgroups for every expert).
bool by_row(const gemm_w4_problem* p) { return p->experts > p->M && p->M <= 64; }

gemm_status validate(const gemm_w4_problem* p) {
    if (!p) return fail(GEMM_ERR_INVALID_ARG, "problem is NULL");
    if (p->M < 0 || p->N < 0 || p->K < 0 || p->experts < 0)
        return fail(GEMM_ERR_INVALID_ARG, "negative size M=%lld N=%lld K=%lld experts=%lld", (long long)p->M,
                    (long long)p->N, (long long)p->K, (long long)p->experts);
    if (p->dtype != GEMM_F16 && p->dtype != GEMM_BF16)
        return fail(p->dtype == GEMM_I8 ? GEMM_ERR_UNSUPPORTED : GEMM_ERR_INVALID_ARG,
                    "dtype %d: 4-bit weights take GEMM_F16 or GEMM_BF16 rows", (int)p->dtype);
    if (p->has_zeros != 0 && p->has_zeros != 1)
        return fail(GEMM_ERR_INVALID_ARG, "has_zeros must be 0 or 1, got %d", (int)p->has_zeros);
    if (p->experts > 0 && p->id_bytes != 4 && p->id_bytes != 8)
        return fail(GEMM_ERR_INVALID_ARG, "id_bytes must be 4 or 8, got %d", (int)p->id_bytes);
    if (p->group != 32 && p->group != 64 && p->group != 128)
        return fail(GEMM_ERR_UNSUPPORTED, "group=%lld: scales are per 32, 64 or 128 k", (long long)p->group);
    if (p->M > dtg::kMaxSize || p->N > dtg::kMaxSize || p->K > dtg::kMaxSize)
        return fail(GEMM_ERR_UNSUPPORTED, "dimensions above 2^31-4096 are not supported");
    if (p->experts > 65535)
        return fail(GEMM_ERR_UNSUPPORTED, "%lld experts, at most 65535", (long long)p->experts);
    if (p->K % 32) return fail(GEMM_ERR_UNSUPPORTED, "K=%lld must be a multiple of 32", (long long)p->K);
    if (p->sx < 0 || p->sy < 0 || p->sw_n < 0 || p->sw_e < 0 || p->ss_n < 0 || p->ss_e < 0 ||
        (p->has_zeros && (p->sz_n < 0 || p->sz_e < 0)))
        return fail(GEMM_ERR_UNSUPPORTED, "negative stride");
    if (p->sx % 8 || p->sw_n % 16 || p->sw_e % 16)
        return fail(GEMM_ERR_UNSUPPORTED, "rows of X must be multiples of 8 elements apart, rows of W and experts "
                    "multiples of 16 bytes (sx=%lld sw_n=%lld sw_e=%lld)", (long long)p->sx, (long long)p->sw_n,
                    (long long)p->sw_e);
    if (w_bytes(p) < 0 || s_elems(p) < 0 || z_bytes(p) < 0 || x_elems(p) < 0 || y_elems(p) < 0)
        return fail(GEMM_ERR_INVALID_ARG, "strides reach past 2^60 elements");
    if (p->sx > kMaxDim || p->ss_n > kMaxDim || (p->has_zeros && p->sz_n > kMaxDim) || p->sw_n > kMaxDim / 32)
        return fail(GEMM_ERR_UNSUPPORTED, "rows too far apart: X, S and Z at most 2^31-1 elements, W 2^26 bytes");
    if (p->M > 1 && p->N > 0 && p->sy < p->N)
        return fail(GEMM_ERR_INVALID_ARG, "Y row stride %lld < N=%lld makes output rows overlap", (long long)p->sy,
                    (long long)p->N);
    return GEMM_OK;
}

gemm_status plan_impl(const gemm_w4_problem* prob, const gemm_device_info* dev, gemm_w4_plan** out) {
    if (!out) return fail(GEMM_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    const gemm_status st = validate(prob);
    if (st != GEMM_OK) return st;
    if (!dev || dev->cu_count <= 0) return fail(GEMM_ERR_INVALID_ARG, "device info missing, or without CUs");
    // rows per pass: two blocks of 16 where a dense batch fills them; a
    // workgroup of an expert sees that expert's rows only
    const int mb = prob->experts == 0 && prob->M > 16 ? 2 : 1;
    // Columns per workgroup, in blocks of 16, and the waves that share out K.
    //  one block, eight waves, while that gives no CU two workgroups (16 x 4096
    //    x 4096: 7.4 us, two blocks 8.5);
    //  two blocks, one or two waves, where there are four of them to a CU and
    //    more (30 rows over 60 experts, 1024 x 2786: 20 us, 44 with four waves;
    //    32 over 16, 4096 x 2048: 25 and 27) or K is short;
    //  four blocks, eight waves, where they still reach four CUs in five (16 x
    //    8192 x 14336: 22 us, two blocks 25; 8 x 8192 x 8192, 128 workgroups: 18
    //    us, two blocks 14);
    //  two blocks, eight waves, where one workgroup to a CU is all there is and K
    //    is short (16 x 608 x 7000: 7.3 us with four, 6.0; 16 x 2048: 6.7 and 7.6);
    //  else two blocks, four waves, two workgroups to a CU.
    int64_t used = matrices(prob);
    if (used > prob->M) used = prob->M > 0 ? prob->M : 1;
    const int64_t cus = dev->cu_count, pairs = used * cdiv(prob->N, 32);
    int nb = 2, waves = 4;
    if (used * cdiv(prob->N, 16) <= cus) {
        nb = 1;
        waves = mb == 1 ? 8 : 4;
    } else if (mb == 2) {
        // four waves fill a CU's LDS: past one workgroup each, two (32 x 608 x 14336: 11.5 us, 17)
        waves = pairs > cus && prob->K <= 4096 ? 2 : 4;
    } else {
        if (pairs >= 4 * cus) {
            waves = prob->K <= 1024 ? 1 : 2;
        } else if (prob->K <= 1024 && 2 * pairs >= 3 * cus) {
            waves = 2;
        } else if (prob->group > 32 && 5 * used * cdiv(prob->N, 64) >= 4 * cus) {
            nb = 4;
            waves = 8;
        } else if (pairs <= cus && prob->K < 2048) {
            waves = 8;
        }
    }
    int n = 0;
    const dtg::W4Entry* t = dtg::w4_kernel_table(&n);
    const dtg::W4Entry* e = nullptr;
    for (int i = 0; i < n && !e; ++i)
        if (t[i].nb == nb && t[i].waves == waves && t[i].mb == mb && t[i].group == prob->group && t[i].zeros == prob->has_zeros &&
            t[i].dtype == (prob->dtype == GEMM_BF16 ? 1 : 0))
            e = &t[i];
    if (!e) return fail(GEMM_ERR_UNSUPPORTED, "no 4-bit kernel for group %lld", (long long)prob->group);
    gemm_w4_plan* pl = new (std::nothrow) gemm_w4_plan;
    if (!pl) return fail(GEMM_ERR_INVALID_ARG, "out of host memory");
    pl->prob = *prob;
    pl->entry = e;
    pl->tiles = cdiv(prob->N, 16 * e->nb);
    *out = pl;
    return GEMM_OK;
}

struct Span {
    uintptr_t lo, hi;
    Span(const void* p, int64_t bytes)
        : lo(reinterpret_cast<uintptr_t>(p)), hi(reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(bytes)) {}
    bool meets(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};

}  // namespace

extern "C" {

gemm_status gemm_w4_plan_create_for(const gemm_w4_problem* prob, const gemm_device_info* info, gemm_w4_plan** out) {
    return plan_impl(prob, info, out);
}

gemm_status gemm_w4_plan_create(const gemm_w4_problem* prob, int device, gemm_w4_plan** out) {
    if (out) *out = nullptr;
    gemm_status st = validate(prob);
    if (st != GEMM_OK) return st;
    gemm_device_info info;
    st = dtg::cached_device_info(device, &info);
    if (st != GEMM_OK) return st;
    return plan_impl(prob, &info, out);
}

void gemm_w4_plan_destroy(gemm_w4_plan* plan) { delete plan; }

gemm_status gemm_w4_plan_describe(const gemm_w4_plan* plan, char* buf, size_t len) {
    if (!plan || !buf || len == 0) return fail(GEMM_ERR_INVALID_ARG, "plan or buf is NULL");
    snprintf(buf, len, "kernel=%s columns=%d rows=%d waves=%d group=%d grid=%lldx%lld", plan->entry->name,
             16 * plan->entry->nb, 16 * plan->entry->mb, plan->entry->waves, plan->entry->group,
             (long long)plan->tiles, (long long)(by_row(&plan->prob) ? plan->prob.M : matrices(&plan->prob)));
    return GEMM_OK;
}

gemm_status gemm_w4_run(const gemm_w4_plan* plan, const void* X, const void* W, const void* S, const void* Z,
                        const void* expert_ids, void* Y, void* stream) {
    if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
    const gemm_w4_problem& p = plan->prob;
    if (!p.has_zeros && Z) return fail(GEMM_ERR_INVALID_ARG, "Z given but the problem has has_zeros = 0");
    if (p.experts == 0 && expert_ids) return fail(GEMM_ERR_INVALID_ARG, "expert_ids given but experts = 0");
    if (p.M == 0 || p.N == 0) return GEMM_OK;
    if (!Y) return fail(GEMM_ERR_INVALID_ARG, "Y is NULL");
    if (p.K > 0 && (!X || !W || !S || (p.has_zeros && !Z))) return fail(GEMM_ERR_INVALID_ARG, "X, W, S or Z is NULL");
    if (p.experts > 0 && !expert_ids) return fail(GEMM_ERR_INVALID_ARG, "expert_ids is NULL");
    if (reinterpret_cast<uintptr_t>(X) % 16 || reinterpret_cast<uintptr_t>(W) % 16)
        return fail(GEMM_ERR_UNSUPPORTED, "X and W must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(S) % 2 || reinterpret_cast<uintptr_t>(Y) % 2 ||
        (p.experts > 0 && reinterpret_cast<uintptr_t>(expert_ids) % p.id_bytes))
        return fail(GEMM_ERR_UNSUPPORTED, "S, Y and expert_ids must be aligned to their element size");
    const Span y(Y, y_elems(&p) * 2);
    const struct { Span s; const char* name; } in[5] = {
        {Span(X, x_elems(&p) * 2), "X"}, {Span(W, w_bytes(&p)), "W"}, {Span(S, s_elems(&p) * 2), "S"},
        {Span(Z, z_bytes(&p)), "Z"}, {Span(expert_ids, p.experts > 0 ? p.M * p.id_bytes : 0), "expert_ids"}};
    for (const auto& i : in)
        if (y.meets(i.s)) return fail(GEMM_ERR_INVALID_ARG, "Y overlaps %s", i.name);
    dtg::W4Args a;
    a.X = static_cast<const uint16_t*>(X);
    a.W = static_cast<const uint8_t*>(W);
    a.S = static_cast<const uint16_t*>(S);
    a.Z = static_cast<const uint8_t*>(Z);
    a.experts = p.experts > 0 ? expert_ids : nullptr;
    a.Y = static_cast<uint16_t*>(Y);
    a.M = static_cast<int32_t>(p.M);
    a.N = static_cast<int32_t>(p.N);
    a.K = static_cast<int32_t>(p.K);
    a.num_experts = static_cast<int32_t>(matrices(&p));
    a.id_bytes = p.id_bytes;
    a.by_row = by_row(&p);
    a.sx = p.sx;
    a.sy = p.sy;
    a.sw_n = p.sw_n;
    a.sw_e = p.sw_e;
    a.ss_n = p.ss_n;
    a.ss_e = p.ss_e;
    a.sz_n = p.sz_n;
    a.sz_e = p.sz_e;
    const hipError_t err = plan->entry->launch(a, plan->tiles, static_cast<hipStream_t>(stream));
    if (err != hipSuccess)
        return fail(GEMM_ERR_HIP, "launch of %s: %s", plan->entry->name, hipGetErrorString(err));
    return GEMM_OK;
}

}  // extern "C"
