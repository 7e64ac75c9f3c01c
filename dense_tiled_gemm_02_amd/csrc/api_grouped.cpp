// C ABI of the products grouped by an offset table and of the row grouping:
// validation, tile choice and launch.  Declarations and the contract of every
// entry point are in include/gemm.h.
#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <new>

#include "../../include/gemm.h"
#include "api_internal.h"
#include "kernels_grouped.h"

struct gemm_grouped_plan {
    gemm_grouped_problem prob;
    gemm_device_info dev;
    gemm_config cfg;
    const dtg::GroupedEntry* entry;
    const dtg::GroupedEntry* fallback;   // for bases that are not 16-byte aligned
    int64_t grid;
    // with a workspace: groups cut into parts of part_rows (0: never)
    const dtg::GroupedEntry* part_entry;
    int32_t part_rows;
    int64_t max_parts;
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
constexpr int64_t kMaxGroups = 65535;
constexpr int32_t kFewRows = 16, kFewK = 32;   // the smaller tile for few rows per group; the k chunk of both
constexpr double kMostPartBytes = 256e6;   // of workspace for a gradient's parts
// mean rows of a group from which the weight gradient takes the longest first
constexpr int64_t kSortRows = 256;
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Elements from the first to one past the last of a strided box (0 when it is
// empty), or -1 past 2^60.
int64_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1, int64_t s2 = 0) {
    if (n0 <= 0 || n1 <= 0 || n2 <= 0) return 0;
    const __int128 e = static_cast<__int128>(n0 - 1) * s0 + static_cast<__int128>(n1 - 1) * s1 +
                       static_cast<__int128>(n2 - 1) * s2 + 1;
    return e > (static_cast<__int128>(1) << 60) ? -1 : static_cast<int64_t>(e);
}

bool reduce_kind(const gemm_grouped_problem* p) { return p->kind == GEMM_GROUPED_REDUCE; }
int64_t a_extent(const gemm_grouped_problem* p) { return extent(p->R, p->sa_r, p->P, p->sa_p); }
int64_t b_extent(const gemm_grouped_problem* p) {
    return reduce_kind(p) ? extent(p->R, p->sb_r, p->Q, p->sb_q)
                          : extent(p->groups, p->sb_g, p->P, p->sb_r, p->Q, p->sb_q);
}
int64_t d_extent(const gemm_grouped_problem* p) {
    return reduce_kind(p) ? extent(p->groups, p->sd_g, p->P, p->sd_r, p->Q, 1)
                          : extent(p->R, p->sd_r, p->Q, 1);
}

gemm_status validate(const gemm_grouped_problem* p) {
    if (!p) return fail(GEMM_ERR_INVALID_ARG, "problem is NULL");
    if (p->groups < 0 || p->R < 0 || p->P < 0 || p->Q < 0)
        return fail(GEMM_ERR_INVALID_ARG, "negative size groups=%lld R=%lld P=%lld Q=%lld", (long long)p->groups,
                    (long long)p->R, (long long)p->P, (long long)p->Q);
    if (p->kind != GEMM_GROUPED_ROWS && p->kind != GEMM_GROUPED_REDUCE)
        return fail(GEMM_ERR_INVALID_ARG, "kind %d is not a gemm_grouped_kind", (int)p->kind);
    if (p->dtype != GEMM_F16 && p->dtype != GEMM_BF16)
        return fail(p->dtype == GEMM_I8 ? GEMM_ERR_UNSUPPORTED : GEMM_ERR_INVALID_ARG,
                    "dtype %d: grouped products take GEMM_F16 or GEMM_BF16", (int)p->dtype);
    if (p->out != GEMM_GROUPED_OUT_SAME && p->out != GEMM_GROUPED_OUT_F32)
        return fail(GEMM_ERR_INVALID_ARG, "out %d is not a gemm_grouped_out", (int)p->out);
    if (p->accumulate != 0 && p->accumulate != 1)
        return fail(GEMM_ERR_INVALID_ARG, "accumulate must be 0 or 1, got %d", (int)p->accumulate);
    if (!reduce_kind(p) && (p->out != GEMM_GROUPED_OUT_SAME || p->accumulate))
        return fail(GEMM_ERR_UNSUPPORTED, "fp32 output and accumulate are of GEMM_GROUPED_REDUCE only");
    if (p->R > dtg::kMaxSize || p->P > dtg::kMaxSize || p->Q > dtg::kMaxSize)
        return fail(GEMM_ERR_UNSUPPORTED, "dimensions above 2^31-4096 are not supported");
    if (p->groups > kMaxGroups)
        return fail(GEMM_ERR_UNSUPPORTED, "%lld groups, at most %lld", (long long)p->groups, (long long)kMaxGroups);
    if (p->sa_r < 0 || p->sa_p < 0 || p->sb_g < 0 || p->sb_r < 0 || p->sb_q < 0 || p->sd_g < 0 || p->sd_r < 0)
        return fail(GEMM_ERR_UNSUPPORTED, "negative stride");
    if (a_extent(p) < 0 || b_extent(p) < 0 || d_extent(p) < 0)
        return fail(GEMM_ERR_INVALID_ARG, "strides reach past 2^60 elements");
    const int64_t drows = reduce_kind(p) ? p->P : p->R;
    if (drows > 1 && p->Q > 0 && p->sd_r < p->Q)
        return fail(GEMM_ERR_INVALID_ARG, "D row stride %lld < Q=%lld makes output rows overlap", (long long)p->sd_r,
                    (long long)p->Q);
    if (reduce_kind(p) && p->groups > 1 && p->P > 0 && p->Q > 0 && p->sd_g < (p->P - 1) * p->sd_r + p->Q)
        return fail(GEMM_ERR_INVALID_ARG, "D group stride %lld makes the groups' outputs overlap",
                    (long long)p->sd_g);
    return GEMM_OK;
}

// Whether B's inner matrices are stored Q x P (rows kind).  A single column
// counts as row-major.
bool b_transposed(const gemm_grouped_problem* p) {
    return !reduce_kind(p) && p->Q > 1 && p->sb_q != 1 && (p->P <= 1 || p->sb_r == 1);
}

// Operands the direct-to-LDS tiles can take (bases aside): 16-byte chunks
// along each contiguous index, rows that do not overlap (the tiles rely on the
// buffer range to zero what lies past an operand), and 32-bit byte offsets
// within a tile's panel.
bool vec_ok(const gemm_grouped_problem* p) {
    const int64_t lim = ((int64_t(1) << 31) - 4096) / (2 * 256);
    if (p->P == 0 || p->Q == 0 || p->R == 0) return false;
    if (p->sa_p != 1 || p->P % 8 || p->sa_r % 8 || p->sa_r < p->P || p->sa_r + p->P >= lim) return false;
    if (reduce_kind(p))
        return p->sb_q == 1 && p->Q % 8 == 0 && p->sb_r % 8 == 0 && p->sb_r >= p->Q && p->sb_r + p->Q < lim;
    if (p->sb_g % 8) return false;
    if (b_transposed(p)) return p->sb_q % 8 == 0 && p->sb_q >= p->P && p->sb_q + p->P < lim;
    return p->sb_q == 1 && p->Q % 8 == 0 && p->sb_r % 8 == 0 && p->sb_r >= p->Q && p->sb_r + p->Q < lim;
}

// Operands of the chunked tiles: an index contiguous over 8 elements or more,
// at any address.
bool odd_ok(const gemm_grouped_problem* p) {
    if (p->sa_p != 1 || p->P < 8) return false;
    if (!reduce_kind(p) && b_transposed(p)) return p->sb_r == 1;
    return p->sb_q == 1 && p->Q >= 8;
}

bool mixed(const dtg::GroupedEntry* e) {
    int n = 0;
    const dtg::GroupedEntry* t = dtg::grouped_mixed_table(&n);
    return e >= t && e < t + n;
}

// Workgroups of a launch: every tile any table can need (see grouped_kernel.h).
int64_t grid_of(const gemm_grouped_problem* p, const dtg::GroupedEntry* e, int64_t cus) {
    if (reduce_kind(p)) return p->groups * cdiv(p->P, e->bm) * cdiv(p->Q, e->bn);
    const int64_t tiles = (p->R / e->bm + p->groups + 2) * cdiv(p->Q, e->bn);
    // the mixed tiles: two small ones in place of a group's last row of tiles, at most a round in place of others
    return mixed(e) ? tiles + (p->groups + 2) * cdiv(p->Q, e->bn) + cus : tiles;
}

const dtg::GroupedEntry* find_entry(const gemm_grouped_problem* p, const gemm_device_info& dev,
                                    dtg::GroupedLoads loads, const gemm_config& w) {
    int n = 0;
    const dtg::GroupedEntry* t = loads == dtg::kGroupedAny   ? dtg::grouped_any_table(&n)
                                 : loads == dtg::kGroupedOdd ? dtg::grouped_odd_table(&n)
                                 : reduce_kind(p)            ? dtg::grouped_reduce_table(&n)
                                 : w.bm == kFewRows || w.bk == kFewK ? dtg::grouped_few_table(&n)
                                                             : dtg::grouped_rows_table(&n);
    const int dtype = p->dtype == GEMM_BF16 ? 1 : 0, out32 = p->out == GEMM_GROUPED_OUT_F32 ? 1 : 0;
    for (int i = 0; i < n; ++i) {
        const dtg::GroupedEntry* e = &t[i];
        if (e->kind != (reduce_kind(p) ? dtg::kGroupedReduce : dtg::kGroupedRows) || e->dtype != dtype ||
            e->out32 != out32 || (loads != dtg::kGroupedAny && e->tb != (b_transposed(p) ? 1 : 0)) || e->lds_bytes > dev.lds_per_wg)
            continue;
        if ((w.bm && w.bm != e->bm) || (w.bn && w.bn != e->bn) || (w.bk && w.bk != e->bk) ||
            (w.stages && w.stages != e->stages) || (w.mfma && w.mfma != e->mfma) ||
            (w.waves_m && w.waves_m != e->waves_m) || (w.waves_n && w.waves_n != e->waves_n))
            continue;
        return e;
    }
    return nullptr;
}

// What a compiled tile costs, measured on gfx950: microseconds per 64 k of one
// workgroup with the card to itself and with `resident` on every CU, and the
// part of its output's time that other workgroups do not hide.
struct TileCost {
    int bm, bn, bk, st, resident;
    double alone, loaded, shown;
};
constexpr TileCost kRowTiles[] = {{256, 256, 64, 2, 1, 1.2, 1.6, 1.0}, {128, 256, 64, 3, 1, 0.69, 1.05, 1.0},
                                  {128, 128, 64, 4, 1, 0.6, 0.7, 1.0}, {128, 128, 64, 2, 2, 0.74, 1.1, 0.5},
                                  {64, 64, 64, 4, 2, 0.3, 0.5, 0.5}};
constexpr TileCost kReduceTiles[] = {{256, 256, 64, 2, 1, 1.2, 1.6, 1.0}, {128, 256, 64, 3, 1, 0.69, 1.05, 1.0},
                                     {128, 128, 64, 2, 2, 0.74, 1.1, 0.5}, {128, 128, 32, 2, 4, 1.05, 2.2, 0.25},
                                     {64, 64, 64, 4, 2, 0.3, 0.5, 0.5}};
constexpr double kStart = 4.0;          // us before a workgroup's first product and after its last
constexpr double kBytesPerUs = 4.7e6;   // what large copies reach

gemm_config tile_config(const TileCost& t) {
    gemm_config c;
    memset(&c, 0, sizeof c);
    c.bm = t.bm;
    c.bn = t.bn;
    c.bk = t.bk;
    c.stages = t.st;
    return c;
}

// Time of `items` workgroups of `steps` 64-k steps each, the longest of
// `longest` steps.
double workgroups_us(const TileCost& t, double items, double steps, double longest, int cus) {
    const double slots = static_cast<double>(cus) * t.resident;
    if (items <= cus) return kStart + longest * t.alone;
    const double one = kStart + longest * t.loaded;
    const double all = items / slots * (kStart + steps * t.loaded);
    return all > one ? all : one;
}

// Rows kind: the host knows only the mean group length; a group of r rows
// counts r / bm tiles and half a tile for its ragged end, at least one.  B is
// read once from memory, whatever the tile.
void choose_rows_tile(const gemm_grouped_problem* p, const gemm_device_info& dev, gemm_config* want) {
    const double groups = static_cast<double>(p->groups < p->R ? p->groups : p->R);
    const double steps = static_cast<double>(cdiv(p->P, 64));
    const double bytes = 2.0 * (static_cast<double>(p->R) * p->P + groups * p->P * p->Q + static_cast<double>(p->R) * p->Q);
    double best = 0.0;
    for (const TileCost& t : kRowTiles) {
        const gemm_config c = tile_config(t);
        if (!find_entry(p, dev, dtg::kGroupedDirect, c)) continue;
        const double per = groups > 0 ? static_cast<double>(p->R) / groups / t.bm + 0.5 : 1.0;
        const double items = (groups > 0 ? groups : 1) * (per > 1 ? per : 1) * cdiv(p->Q, t.bn);
        double est = workgroups_us(t, items, steps, steps, dev.cu_count);
        // the last round of many is half empty on average
        if (items > dev.cu_count * t.resident) est += 0.5 * (kStart + steps * t.loaded);
        const double memory = bytes / kBytesPerUs;
        est = (est > memory ? est : memory) + 0.1 * est;
        if (best == 0.0 || est < best) {
            best = est;
            *want = c;
        }
    }
}

// Few rows per group: the waves of a workgroup share out K, 0.35 us per 32 k of
// each; 16-row tiles to a mean of 16 rows a group, 64-row ones to 48 (a longer
// group's second tile reads B[g] again).  Worth it while no CU gets two tiles (16
// x 1024 x 512 over 8 groups: 5.2 us, 64 x 64 tiles 7.0; 46 x 2184 x 736 over 2:
// 7.9 and 11.3; 64 x 4096 x 4096 over 8, two tiles to a CU: 70 and 59).  nullptr
// where it is not.
const dtg::GroupedEntry* few_rows(const gemm_grouped_problem* p, const gemm_device_info& dev, const gemm_config& tile) {
    const double groups = static_cast<double>(p->groups < p->R ? p->groups : p->R);
    if (groups < 1) return nullptr;
    const double mean = static_cast<double>(p->R) / groups;
    double alone = 0.0;   // stays 0, and nothing is chosen, where no whole tile fits the device
    for (const TileCost& t : kRowTiles)
        if (t.bm == tile.bm && t.bn == tile.bn && t.st == tile.stages) alone = t.alone;
    int n = 0;
    const dtg::GroupedEntry* few = dtg::grouped_few_table(&n);
    for (int i = 0; i < n; ++i) {
        const dtg::GroupedEntry& e = few[i];
        if (e.dtype != (p->dtype == GEMM_BF16 ? 1 : 0) || e.tb != (b_transposed(p) ? 1 : 0) ||
            e.lds_bytes > dev.lds_per_wg || mean > (e.bm == kFewRows ? kFewRows : 48))
            continue;
        const double per = mean / e.bm + 0.5;
        if (groups * (per > 1 ? per : 1) * cdiv(p->Q, e.bn) > dev.cu_count) continue;
        if (0.35 * cdiv(p->P, kFewK * e.waves_n) < alone * cdiv(p->P, 64)) return &e;
    }
    return nullptr;
}

// Reduce kind: the tile, and whether to cut the groups' rows into parts (few
// output tiles, many rows: 12000 rows of one 264 x 520 gradient 58 us whole,
// 25 us in parts of 704).  Lengths vary: the longest group counts 1.5 means.
void choose_reduce_tile(const gemm_grouped_problem* p, const gemm_device_info& dev, gemm_config* want,
                        int32_t* part_rows) {
    const double groups = static_cast<double>(p->groups > 0 ? p->groups : 1);
    const double rows = static_cast<double>(p->R) / groups;
    const double longest = groups > 1 && 1.5 * rows < p->R ? 1.5 * rows : static_cast<double>(p->R);
    const double sums = static_cast<double>(p->P) * p->Q * 4;
    const double out = groups * sums / (p->out == GEMM_GROUPED_OUT_F32 ? 1 : 2) / kBytesPerUs;
    auto steps = [](double r) { return r > 64 ? r / 64 : 1.0; };
    double best = 0.0;
    for (const TileCost& t : kReduceTiles) {
        const gemm_config c = tile_config(t);
        if (!find_entry(p, dev, dtg::kGroupedDirect, c)) continue;
        const double tiles = static_cast<double>(cdiv(p->P, t.bm) * cdiv(p->Q, t.bn));
        const double work = workgroups_us(t, groups * tiles, steps(rows), steps(longest), dev.cu_count);
        const double est = work > out ? work + t.shown * out : out + t.shown * work;
        if (best == 0.0 || est < best) {
            best = est;
            *want = c;
            *part_rows = 0;
        }
        for (int32_t q : {512, 768, 1024, 1536, 2048, 4096}) {
            const double parts = static_cast<double>(p->R / q + p->groups);
            if (p->groups == 0 || q >= longest || parts * sums > kMostPartBytes) continue;
            // their sums are written, read again, and a second launch adds them
            const double cut = workgroups_us(t, parts * tiles, q / 64, q / 64, dev.cu_count) +
                               2 * parts * sums / kBytesPerUs + out + 8.0;
            if (cut < best) {
                best = cut;
                *want = c;
                *part_rows = q;
            }
        }
    }
}

gemm_status plan_impl(const gemm_grouped_problem* prob, const gemm_device_info* dev, const gemm_config* force,
                      gemm_grouped_plan** out) {
    if (!out) return fail(GEMM_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    const gemm_status st = validate(prob);
    if (st != GEMM_OK) return st;
    if (!dev || dev->cu_count <= 0 || dev->lds_per_wg <= 0)
        return fail(GEMM_ERR_INVALID_ARG, "device info missing, or without CUs or LDS");
    gemm_config want;
    memset(&want, 0, sizeof want);
    const gemm_config none = want;
    int32_t group_m = 8;
    bool xcd = true, forced = false;
    if (force) {
        if (force->splitk < 0 || force->splitk > 1 || force->kernel)
            return fail(GEMM_ERR_UNSUPPORTED, "grouped products take no kernel family and no K slices");
        if (force->group_m < 0 || force->xcd_remap < 0 || force->xcd_remap > 2)
            return fail(GEMM_ERR_INVALID_ARG, "group_m must be >= 0 and xcd_remap one of 0, 1, 2");
        forced = force->bm || force->bn || force->bk || force->stages || force->mfma || force->waves_m || force->waves_n;
        if (forced) want = *force;
        if (force->group_m) group_m = force->group_m;
        if (force->xcd_remap) xcd = force->xcd_remap == GEMM_XCD_ON;
    }
    // chunked loads where an index is contiguous (777 x 1003 x 517 over 5 groups: 10.8 us, 200 us element by element)
    const dtg::GroupedLoads loose = odd_ok(prob) ? dtg::kGroupedOdd : dtg::kGroupedAny;
    const dtg::GroupedLoads loads = vec_ok(prob) ? dtg::kGroupedDirect : loose;
    int32_t part_rows = 0;
    const dtg::GroupedEntry* few = nullptr;
    if (loads == dtg::kGroupedDirect && !forced) {
        if (reduce_kind(prob)) choose_reduce_tile(prob, *dev, &want, &part_rows);
        else choose_rows_tile(prob, *dev, &want);
        if (!reduce_kind(prob)) few = few_rows(prob, *dev, want);
    }
    const dtg::GroupedEntry* e = few ? few : find_entry(prob, *dev, loads, want);
    const dtg::GroupedEntry* any = find_entry(prob, *dev, loose, none);
    if (!e || !any)
        return fail(GEMM_ERR_UNSUPPORTED, "no grouped kernel for bm=%d bn=%d bk=%d stages=%d waves=%dx%d mfma=%d on "
                    "these operands within %lld bytes of LDS", want.bm, want.bn, want.bk, want.stages, want.waves_m,
                    want.waves_n, want.mfma, (long long)dev->lds_per_wg);
    // both tile sizes in one launch, where the lanes of a wave hold all segments
    if (loads == dtg::kGroupedDirect && !reduce_kind(prob) && !forced && e->bm == 256 && prob->groups + 2 <= 64) {
        int n = 0;
        const dtg::GroupedEntry* t = dtg::grouped_mixed_table(&n);
        for (int i = 0; i < n; ++i)
            if (t[i].dtype == e->dtype && t[i].tb == e->tb) e = &t[i];
    }
    if (grid_of(prob, e, dev->cu_count) > kMaxDim || grid_of(prob, any, dev->cu_count) > kMaxDim)
        return fail(GEMM_ERR_UNSUPPORTED, "output too large for one launch");
    gemm_grouped_plan* pl = new (std::nothrow) gemm_grouped_plan;
    if (!pl) return fail(GEMM_ERR_INVALID_ARG, "out of host memory");
    pl->prob = *prob;
    pl->dev = *dev;
    pl->entry = e;
    pl->fallback = any;
    pl->grid = grid_of(prob, e, dev->cu_count);
    pl->part_entry = nullptr;
    pl->part_rows = 0;
    pl->max_parts = 0;
    if (part_rows > 0) {
        gemm_grouped_problem sums = *prob;
        sums.out = GEMM_GROUPED_OUT_F32;
        pl->part_entry = find_entry(&sums, *dev, loads, want);
        if (pl->part_entry) {
            pl->part_rows = part_rows;
            pl->max_parts = prob->R / part_rows + prob->groups;
        }
    }
    gemm_config& c = pl->cfg;
    c = none;
    c.bm = e->bm;
    c.bn = e->bn;
    c.bk = e->bk;
    c.stages = e->stages;
    c.mfma = e->mfma;
    c.waves_m = e->waves_m;
    c.waves_n = e->waves_n;
    c.splitk = 1;
    // the kernels clamp the band to a group's rows of tiles; this keeps its arithmetic in 32 bits
    c.group_m = group_m > 1024 ? 1024 : group_m;
    c.xcd_remap = (xcd && dev->xcd_count > 1) ? GEMM_XCD_ON : GEMM_XCD_OFF;
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

gemm_status gemm_grouped_plan_create_for(const gemm_grouped_problem* prob, const gemm_device_info* info,
                                         const gemm_config* force, gemm_grouped_plan** out) {
    return plan_impl(prob, info, force, out);
}

gemm_status gemm_grouped_plan_create(const gemm_grouped_problem* prob, int device, const gemm_config* force,
                                     gemm_grouped_plan** out) {
    if (out) *out = nullptr;
    gemm_status st = validate(prob);
    if (st != GEMM_OK) return st;
    gemm_device_info info;
    st = dtg::cached_device_info(device, &info);
    if (st != GEMM_OK) return st;
    return plan_impl(prob, &info, force, out);
}

void gemm_grouped_plan_destroy(gemm_grouped_plan* plan) { delete plan; }

gemm_status gemm_grouped_plan_config(const gemm_grouped_plan* plan, gemm_config* out) {
    if (!plan || !out) return fail(GEMM_ERR_INVALID_ARG, "plan or out is NULL");
    *out = plan->cfg;
    return GEMM_OK;
}

gemm_status gemm_grouped_plan_launch(const gemm_grouped_plan* plan, int64_t* grid, int32_t* threads, int64_t* lds) {
    if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
    if (grid) *grid = plan->grid;
    if (threads) *threads = plan->entry->threads;
    if (lds) *lds = plan->entry->lds_bytes;
    return GEMM_OK;
}

gemm_status gemm_grouped_plan_describe(const gemm_grouped_plan* plan, char* buf, size_t len) {
    if (!plan || !buf || len == 0) return fail(GEMM_ERR_INVALID_ARG, "plan or buf is NULL");
    const gemm_config& c = plan->cfg;
    snprintf(buf, len,
             "kernel=%s bm=%d bn=%d bk=%d stages=%d mfma=%d waves=%dx%d group_m=%d xcd_remap=%d grid=%lld threads=%d "
             "lds=%lld part_rows=%d",
             plan->entry->name, c.bm, c.bn, c.bk, c.stages, c.mfma, c.waves_m, c.waves_n, c.group_m, c.xcd_remap,
             (long long)plan->grid, plan->entry->threads, (long long)plan->entry->lds_bytes, plan->part_rows);
    return GEMM_OK;
}

gemm_status gemm_grouped_workspace(const gemm_grouped_plan* plan, size_t* bytes) {
    if (!plan || !bytes) return fail(GEMM_ERR_INVALID_ARG, "plan or bytes is NULL");
    *bytes = static_cast<size_t>(plan->max_parts * plan->prob.P * plan->prob.Q) * 4;
    return GEMM_OK;
}

gemm_status gemm_grouped_run(const gemm_grouped_plan* plan, const void* A, const void* B, const int32_t* offsets,
                             void* D, void* stream) {
    return gemm_grouped_run_parts(plan, A, B, offsets, D, nullptr, 0, stream);
}

gemm_status gemm_grouped_run_parts(const gemm_grouped_plan* plan, const void* A, const void* B,
                                   const int32_t* offsets, void* D, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
    const gemm_grouped_problem& p = plan->prob;
    const int64_t dn = d_extent(&p), an = a_extent(&p), bn = b_extent(&p);
    if (dn == 0) return GEMM_OK;
    if (!D) return fail(GEMM_ERR_INVALID_ARG, "D is NULL");
    if (!offsets) return fail(GEMM_ERR_INVALID_ARG, "offsets is NULL");
    if ((an > 0 && !A) || (bn > 0 && !B)) return fail(GEMM_ERR_INVALID_ARG, "A or B is NULL");
    const int esz = p.out == GEMM_GROUPED_OUT_F32 ? 4 : 2;
    const uintptr_t ia = reinterpret_cast<uintptr_t>(A), ib = reinterpret_cast<uintptr_t>(B);
    if (reinterpret_cast<uintptr_t>(D) % esz || ia % 2 || ib % 2 || reinterpret_cast<uintptr_t>(offsets) % 4)
        return fail(GEMM_ERR_UNSUPPORTED, "A, B, D and offsets must be aligned to their element size");
    const Span d(D, dn * esz);
    if (d.meets(Span(A, an * 2))) return fail(GEMM_ERR_INVALID_ARG, "D overlaps A");
    if (d.meets(Span(B, bn * 2))) return fail(GEMM_ERR_INVALID_ARG, "D overlaps B");
    if (d.meets(Span(offsets, (p.groups + 1) * 4))) return fail(GEMM_ERR_INVALID_ARG, "D overlaps offsets");
    const bool aligned = ia % 16 == 0 && ib % 16 == 0;
    const bool parts = plan->part_rows > 0 && workspace && aligned;
    if (workspace) {
        const size_t need = static_cast<size_t>(plan->max_parts * p.P * p.Q) * 4;
        if (workspace_bytes < need)
            return fail(GEMM_ERR_WORKSPACE, "%zu bytes of workspace needed (%zu given)", need, workspace_bytes);
        if (reinterpret_cast<uintptr_t>(workspace) % 16)
            return fail(GEMM_ERR_WORKSPACE, "workspace must be 16-byte aligned");
        const Span w(workspace, static_cast<int64_t>(need));
        if (w.meets(d) || w.meets(Span(A, an * 2)) || w.meets(Span(B, bn * 2)) ||
            w.meets(Span(offsets, (p.groups + 1) * 4)))
            return fail(GEMM_ERR_INVALID_ARG, "the workspace overlaps an operand");
    }
    const dtg::GroupedEntry* e = parts ? plan->part_entry : plan->entry;
    if (e->loads == dtg::kGroupedDirect && !aligned) e = plan->fallback;
    dtg::GroupedArgs a;
    a.A = static_cast<const uint16_t*>(A);
    a.B = static_cast<const uint16_t*>(B);
    a.D = D;
    a.offsets = offsets;
    a.groups = static_cast<int32_t>(p.groups);
    a.R = static_cast<int32_t>(p.R);
    a.P = static_cast<int32_t>(p.P);
    a.Q = static_cast<int32_t>(p.Q);
    a.num_pid_p = static_cast<int32_t>(cdiv(p.P, e->bm));
    a.num_pid_q = static_cast<int32_t>(cdiv(p.Q, e->bn));
    a.group_m = plan->cfg.group_m;
    a.xcds = plan->cfg.xcd_remap == GEMM_XCD_ON ? plan->dev.xcd_count : 1;
    a.accumulate = p.accumulate;
    a.sa_r = p.sa_r;
    a.sa_p = p.sa_p;
    a.sb_g = p.sb_g;
    a.sb_r = p.sb_r;
    a.sb_q = p.sb_q;
    a.sd_g = p.sd_g;
    a.sd_r = p.sd_r;
    a.cus = plan->dev.cu_count;
    a.longest_first = p.groups <= 64 && p.R / kSortRows >= p.groups;
    a.part_rows = parts ? plan->part_rows : 0;
    a.max_parts = static_cast<int32_t>(plan->max_parts);
    a.parts = static_cast<float*>(workspace);
    const int64_t grid = parts ? plan->max_parts * a.num_pid_p * a.num_pid_q
                               : e == plan->entry ? plan->grid : grid_of(&p, e, plan->dev.cu_count);
    hipError_t err = e->launch(a, grid, static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return fail(GEMM_ERR_HIP, "launch of %s: %s", e->name, hipGetErrorString(err));
    if (parts) {
        err = dtg::launch_sum_parts(a, p.dtype == GEMM_BF16 ? 1 : 0, esz == 4 ? 1 : 0, static_cast<hipStream_t>(stream));
        if (err != hipSuccess) return fail(GEMM_ERR_HIP, "launch of the parts' sum: %s", hipGetErrorString(err));
    }
    return GEMM_OK;
}

gemm_status gemm_group_rows_workspace(int64_t R, int64_t groups, size_t* bytes) {
    if (!bytes) return fail(GEMM_ERR_INVALID_ARG, "bytes is NULL");
    if (R < 0 || groups < 0) return fail(GEMM_ERR_INVALID_ARG, "negative size");
    if (R > kMaxDim || groups >= dtg::kMaxRowGroups)
        return fail(GEMM_ERR_UNSUPPORTED, "R=%lld, groups=%lld: at most 2^31-1 rows and %d groups", (long long)R,
                    (long long)groups, dtg::kMaxRowGroups - 1);
    *bytes = static_cast<size_t>(dtg::group_rows_workspace_bytes(R, groups));
    return GEMM_OK;
}

gemm_status gemm_group_rows(const void* ids, int32_t id_bytes, int64_t R, int64_t groups, int32_t* offsets,
                            int32_t* order, void* workspace, size_t workspace_bytes, void* stream) {
    size_t need = 0;
    const gemm_status st = gemm_group_rows_workspace(R, groups, &need);
    if (st != GEMM_OK) return st;
    if (id_bytes != 4 && id_bytes != 8)
        return fail(GEMM_ERR_INVALID_ARG, "id_bytes must be 4 or 8, got %d", (int)id_bytes);
    if (!offsets || (R > 0 && (!ids || !order))) return fail(GEMM_ERR_INVALID_ARG, "ids, offsets or order is NULL");
    if (reinterpret_cast<uintptr_t>(ids) % id_bytes || reinterpret_cast<uintptr_t>(offsets) % 4 ||
        reinterpret_cast<uintptr_t>(order) % 4)
        return fail(GEMM_ERR_UNSUPPORTED, "ids, offsets and order must be aligned to their element size");
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(GEMM_ERR_WORKSPACE, "%zu bytes of workspace needed (%zu given)", need,
                    workspace ? workspace_bytes : static_cast<size_t>(0));
    if (need > 0 && reinterpret_cast<uintptr_t>(workspace) % 4)
        return fail(GEMM_ERR_WORKSPACE, "workspace must be 4-byte aligned");
    const Span s[4] = {Span(ids, R * id_bytes), Span(offsets, (groups + 1) * 4), Span(order, R * 4),
                       Span(workspace, static_cast<int64_t>(need))};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (s[i].meets(s[j])) return fail(GEMM_ERR_INVALID_ARG, "ids, offsets, order and workspace overlap");
    const hipError_t err = dtg::launch_group_rows(ids, id_bytes, R, static_cast<int32_t>(groups), offsets, order,
                                                  workspace, static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return fail(GEMM_ERR_HIP, "launch of the row grouping: %s", hipGetErrorString(err));
    return GEMM_OK;
}

}  // extern "C"
