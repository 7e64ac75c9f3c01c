// C ABI of the int8 products with scales: validation, variant choice and
// launch.  Declarations and the contract are in include/gemm.h.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <new>

#include "../../include/gemm.h"
#include "api_operands.h"
#include "kernels_i8.h"

struct gemm_i8_plan {
    gemm_i8_problem prob;
    int out;                          // kOutF16, kOutBF16, kOutF32
    const dtg::I8TileEntry* tile;     // one of these two, or neither: the kernel for any address
    const dtg::I8FewEntry* few;
    int64_t tiles_m, tiles_n;
    int group_m, xcds, cus;
};

namespace {

using dtg::extent;
using dtg::fail;
using dtg::Operand;

constexpr int64_t kMaxRows = int64_t(1) << 27;        // of X and W: the grids of the smallest tiles
constexpr int64_t kMaxOutputs = int64_t(1) << 35;
constexpr int64_t kMaxK = int64_t(1) << 17;           // 2^17 products of 2^14 make 2^31
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int out_bytes(const gemm_i8_problem* p) { return p->out == GEMM_F32 ? 4 : 2; }

gemm_status validate(const gemm_i8_problem* p) {
    if (!p) return fail(GEMM_ERR_INVALID_ARG, "problem is NULL");
    if (p->M < 0 || p->N < 0 || p->K < 0)
        return fail(GEMM_ERR_INVALID_ARG, "negative size M=%lld N=%lld K=%lld", (long long)p->M, (long long)p->N,
                    (long long)p->K);
    if (p->out != GEMM_F16 && p->out != GEMM_BF16 && p->out != GEMM_F32)
        return fail(GEMM_ERR_INVALID_ARG, "output type %d is none of GEMM_F16, GEMM_BF16, GEMM_F32", (int)p->out);
    if (p->has_bias != 0 && p->has_bias != 1)
        return fail(GEMM_ERR_INVALID_ARG, "has_bias must be 0 or 1, got %d", (int)p->has_bias);
    if (p->M > kMaxRows || p->N > kMaxRows || p->M * p->N > kMaxOutputs)
        return fail(GEMM_ERR_UNSUPPORTED, "M and N above 2^27 or more than 2^35 outputs are not supported");
    if (p->K >= kMaxK)
        return fail(GEMM_ERR_UNSUPPORTED, "K=%lld: sums of 2^17 products and more can pass int32", (long long)p->K);
    if (p->sx < 0 || p->sw < 0 || p->sy < 0) return fail(GEMM_ERR_UNSUPPORTED, "negative stride");
    if (extent(p->M, p->sx, p->K, 1) < 0 || extent(p->N, p->sw, p->K, 1) < 0 || extent(p->M, p->sy, p->N, 4) < 0)
        return fail(GEMM_ERR_INVALID_ARG, "strides reach past 2^60 bytes");
    if (p->M > 1 && p->sy < p->N)
        return fail(GEMM_ERR_INVALID_ARG, "Y row stride %lld < N=%lld makes output rows overlap", (long long)p->sy,
                    (long long)p->N);
    return GEMM_OK;
}

// Rows 16 bytes apart and whole chunks of 16 k: the direct-to-LDS kernels.
bool chunked(const gemm_i8_problem* p) {
    return p->K > 0 && p->K % 16 == 0 && p->sx % 16 == 0 && p->sw % 16 == 0;
}

// 32-bit offsets of `rows` rows from a rebased descriptor.
bool near(int64_t rows, int64_t stride, int64_t K) {
    return stride < (int64_t(1) << 31) && rows * stride + K < (int64_t(1) << 31) - 4096;
}

// The smallest tile of at most 64 x 32 whose workgroups the CUs hold at once: K is
// long beside the tile, and its waves share it out, so that a second round or a
// larger tile costs more than reading X or W again (us, W from memory):
//   64 x 1024 x 1024   16 x 16 tiles 3.4, 32 x 32 4.1, 64 x 64 5.2
//   32 x 4096 x 4096   16 x 32 7.1, 32 x 32 8.0; 16 x 16, two rounds 10.6
//   128 x 4096 x 4096  64 x 32 10.2, 32 x 32, two rounds 12.4, 64 x 64 12.8
//   64 x 14336 x 4096  64 x 64 16.2, 64 x 32, two rounds 20.7
// Up to 32 rows the widest tile stays on where no tile fits: 32 x 28672 x 8192 42.9
// us, 64 x 64 46.3.
const dtg::I8FewEntry* pick_few(const gemm_i8_problem* p, const gemm_device_info* dev) {
    static const struct { int mb, nb, rows; } order[] = {{1, 1, 0}, {1, 2, 0}, {1, 4, 16}, {2, 2, 0}, {2, 4, 32}, {4, 2, 0}};
    int n = 0;
    const dtg::I8FewEntry* t = dtg::i8_few_table(&n);
    for (const auto& o : order) {
        // past a tile's rows the next one; tiles of many columns are for few rows
        if (o.rows ? p->M > o.rows : o.mb > 1 && p->M <= 16 * o.mb / 2) continue;
        const bool fits = cdiv(p->M, 16 * o.mb) * cdiv(p->N, 16 * o.nb) <= dev->cu_count;
        if (!fits && !(o.nb == 4 && p->M > 16 * (o.mb - 1))) continue;
        if (!near(16 * o.nb, p->sw, p->K) || !near(16 * o.mb, p->sx, p->K)) continue;
        for (int i = 0; i < n; ++i)
            if (t[i].mb == o.mb && t[i].nb == o.nb) return &t[i];
    }
    return nullptr;
}

const dtg::I8TileEntry* pick_tile(const gemm_i8_problem* p, const gemm_device_info* dev, int out) {
    // Rounds of workgroups times a tile's cost relative to 256 x 256, fitted to K =
    // 4096 (us a round): 256 x 256 53, 256 x 128 29.4, 128 x 256 31, 128 x 128 21.2, 64
    // x 64 12.7, and 19.4 with two to a CU.  A last round of at most half the CUs goes
    // in halves (gemm_i8s_mixed_kernel).  192 x 256 is for what these leave between
    // them (K = 4096, us of it, 256 x 256, the halves and 128 x 256: 1500 x 6000 48.9,
    // 54.0, none, 58.3; 6000 x 6000 150, 160, 147, 158; 2500 x 8192 95.4, 113, 88.4, 92.9).
    // Short K keeps the order: K = 512, 1500 x 6000 13.6, 14.8, none, 17.9; 6000 x 6000
    // 42.5, 47.7, 43.1, 46.2; 4096 x 4096 23.4, 16.9, none, 20.3.
    const int64_t cus = dev->cu_count;
    auto cost = [&](const dtg::I8TileEntry& e) {
        const int64_t tiles = cdiv(p->M, e.bm) * cdiv(p->N, e.bn), left = tiles % cus;
        if (e.mixed) return tiles > cus && left > 0 && 2 * left <= cus ? static_cast<double>(tiles / cus) + 0.56 : 1e18;
        if (e.bm == 64) {
            const int64_t two = tiles % (2 * cus);
            return static_cast<double>(tiles / (2 * cus)) * 0.366 + (two == 0 ? 0.0 : two <= cus ? 0.24 : 0.366);
        }
        return static_cast<double>(cdiv(tiles, cus)) * (e.bm + e.bn == 512 ? 1.0 : e.bm == 192 ? 0.8 : e.bm == 256 ? 0.56 : e.bn == 256 ? 0.59 : 0.4);
    };
    int n = 0, best = -1;
    double best_t = 0.0;
    const dtg::I8TileEntry* t = dtg::i8_scaled_table(&n);
    for (int i = 0; i < n; ++i) {
        if (t[i].out != out || !near(t[i].bm, p->sx, p->K) || !near(t[i].bn, p->sw, p->K)) continue;
        const double c = cost(t[i]);
        if (best < 0 || c < best_t) best = i, best_t = c;
    }
    return best < 0 ? nullptr : &t[best];
}

gemm_status plan_impl(const gemm_i8_problem* given, const gemm_device_info* dev, gemm_i8_plan** out) {
    if (!out) return fail(GEMM_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    const gemm_status st = validate(given);
    if (st != GEMM_OK) return st;
    gemm_i8_problem seen = *given;   // without the strides that no access uses
    if (seen.M <= 1) seen.sx = 0;
    if (seen.N <= 1) seen.sw = 0;
    const gemm_i8_problem* const p = &seen;
    if (!dev || dev->cu_count <= 0) return fail(GEMM_ERR_INVALID_ARG, "device info missing, or without CUs");
    gemm_i8_plan* pl = new (std::nothrow) gemm_i8_plan();
    if (!pl) return fail(GEMM_ERR_INVALID_ARG, "out of host memory");
    pl->prob = *p;
    pl->out = p->out == GEMM_F32 ? dtg::kOutF32 : p->out == GEMM_BF16 ? dtg::kOutBF16 : dtg::kOutF16;
    pl->cus = dev->cu_count;
    pl->xcds = dev->xcd_count > 0 ? dev->xcd_count : 1;
    if (chunked(p)) {
        pl->few = pick_few(p, dev);
        if (!pl->few) pl->tile = pick_tile(p, dev, pl->out);
    }
    if (pl->tile) {
        pl->tiles_m = cdiv(p->M, pl->tile->bm);
        pl->tiles_n = cdiv(p->N, pl->tile->bn);
        pl->group_m = 8;
    } else {
        const int side = dtg::i8_any_tile(p->M, p->N, pl->cus);
        pl->tiles_m = cdiv(p->M, pl->few ? 16 * pl->few->mb : side);
        pl->tiles_n = cdiv(p->N, pl->few ? 16 * pl->few->nb : side);
    }
    *out = pl;
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status gemm_i8_plan_create_for(const gemm_i8_problem* prob, const gemm_device_info* info, gemm_i8_plan** out) {
    return plan_impl(prob, info, out);
}

gemm_status gemm_i8_plan_create(const gemm_i8_problem* prob, int device, gemm_i8_plan** out) {
    if (out) *out = nullptr;
    gemm_status st = validate(prob);
    if (st != GEMM_OK) return st;
    gemm_device_info info;
    st = dtg::cached_device_info(device, &info);
    if (st != GEMM_OK) return st;
    return plan_impl(prob, &info, out);
}

void gemm_i8_plan_destroy(gemm_i8_plan* plan) { delete plan; }

gemm_status gemm_i8_plan_describe(const gemm_i8_plan* plan, char* buf, size_t len) {
    if (!plan || !buf || len == 0) return fail(GEMM_ERR_INVALID_ARG, "plan or buf is NULL");
    snprintf(buf, len, "kernel=%s grid=%lldx%lld", plan->tile ? plan->tile->name : plan->few ? plan->few->name : "i8_any_kernel",
             (long long)plan->tiles_m, (long long)plan->tiles_n);
    return GEMM_OK;
}

gemm_status gemm_i8_run(const gemm_i8_plan* plan, const int8_t* X, const float* x_scale, const int8_t* W, const float* w_scale,
                        const void* bias, void* Y, void* stream) {
    if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
    const gemm_i8_problem& p = plan->prob;
    if (!p.has_bias && bias) return fail(GEMM_ERR_INVALID_ARG, "bias given but the problem has has_bias = 0");
    if (p.M == 0 || p.N == 0) return GEMM_OK;
    const int size = out_bytes(&p);
    const Operand o[6] = {{"X", X, extent(p.M, p.sx, p.K, 1), 1, false},
                          {"W", W, extent(p.N, p.sw, p.K, 1), 1, false},
                          {"x_scale", x_scale, p.M * 4, 4, false},
                          {"w_scale", w_scale, p.N * 4, 4, false},
                          {"bias", bias, p.has_bias ? p.N * size : 0, size, false},
                          {"Y", Y, extent(p.M, p.sy, p.N, size), size, true}};
    const gemm_status st = dtg::check(o, 6);
    if (st != GEMM_OK) return st;
    const dtg::ScaledI8 scales = {x_scale, w_scale, p.has_bias ? bias : nullptr};
    const hipStream_t on = static_cast<hipStream_t>(stream);
    const bool aligned = reinterpret_cast<uintptr_t>(X) % 16 == 0 && reinterpret_cast<uintptr_t>(W) % 16 == 0;
    hipError_t err;
    if (plan->tile && aligned) {
        dtg::ScaledArgs a = {};
        a.A = reinterpret_cast<const uint16_t*>(X);
        a.B = reinterpret_cast<const uint16_t*>(W);
        a.D = static_cast<uint16_t*>(Y);
        a.M = static_cast<int32_t>(p.M);
        a.N = static_cast<int32_t>(p.N);
        a.K = static_cast<int32_t>(p.K / 2);
        a.num_pid_m = static_cast<int32_t>(plan->tiles_m);
        a.num_pid_n = static_cast<int32_t>(plan->tiles_n);
        a.group_m = plan->group_m;
        a.xcds = plan->xcds;
        a.splits = 1;
        a.lda = p.M > 1 ? p.sx / 2 : a.K;   // of one row: none is taken
        a.sbn = p.N > 1 ? p.sw / 2 : a.K;
        a.sak = a.ldb = 1;
        a.ldd = p.sy;
        a.s = scales;
        a.cus = plan->cus;
        err = plan->tile->launch(a, plan->tiles_m * plan->tiles_n, on);
    } else {
        dtg::I8RowsArgs a = {};
        a.X = X;
        a.W = W;
        a.Y = Y;
        a.s = scales;
        a.M = static_cast<int32_t>(p.M);
        a.N = static_cast<int32_t>(p.N);
        a.K = static_cast<int32_t>(p.K);
        a.lx = p.sx;
        a.lw = p.sw;
        a.ly = p.sy;
        err = plan->few && aligned ? plan->few->launch[plan->out](a, on) : dtg::launch_i8_any(a, plan->out, plan->cus, plan->xcds, on);
    }
    return dtg::launched(err, "int8 product");
}

}  // extern "C"
