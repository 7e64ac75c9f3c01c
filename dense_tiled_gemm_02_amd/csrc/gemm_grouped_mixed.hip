// The grouped product over ragged rows with two tile sizes in one launch: 256 x
// 256 tiles, and 128 x 128 ones where a whole tile would leave the card half
// empty.
//
//  * A group's last rows, if 128 or fewer, take tiles of 128 rows.
//  * The whole tiles that do not fill a last round of the CUs are cut in four, if
//    they and the small tiles fit one round.
// Small tiles come last; a round of them takes 0.45 of a round of whole ones.
// 16384 x 4096 x 4096 over 8 groups 472 us (1.16 PFLOP/s; 506 us with whole tiles
// only), 8000 x 2048 x 2048 over 16 groups 83 us (110); where the small tiles
// save no round they cost 2 %.  Bound by the matrix units.  The groups and the
// two segments of no group share one wave's lanes: up to 62 groups.
#include "grouped_kernel.h"

namespace dtg {
namespace {

struct MixedTile {
    int seg, lo, rows;      // the segment and its rows
    int pid_m, pid_n;       // the tile, in its own size
    bool whole;
};

// Rows of whole tiles of a segment, and whether a half one follows them.
__device__ __forceinline__ int whole_rows(int rows) {
    return static_cast<int>((static_cast<uint32_t>(rows) + 127) / 256);
}
__device__ __forceinline__ bool half_row(int rows) { return rows % 256 >= 1 && rows % 256 <= 128; }

__device__ __forceinline__ bool find_mixed(const GroupedArgs& a, MixedTile* out) {
    const int lane = threadIdx.x & 63, nseg = a.groups + 2;
    Segment s = {0, 0};
    if (lane < nseg) s = table_segment(a, lane);
    const uint32_t full = whole_rows(s.rows), half = half_row(s.rows) ? 1 : 0;
    const uint32_t full_incl = wave_scan(full), half_incl = wave_scan(half);
    const uint32_t fulls = __builtin_amdgcn_readlane(full_incl, 63), halves = __builtin_amdgcn_readlane(half_incl, 63);
    // no increasing table has more rows of tiles (the grid's count, so the products fit 32 bits)
    if (fulls > static_cast<uint32_t>(a.R / 256 + nseg)) return false;
    const int nq = a.num_pid_q;                         // 256-column tiles
    const int nh = (a.Q + 127) / 128;                   // 128-column ones
    const int slots = a.cus;
    int wholes = static_cast<int>(fulls) * nq, cut = wholes % slots;
    const int smalls = static_cast<int>(halves) * nh;
    if (4 * cut + smalls > slots) cut = 0;
    wholes -= cut;
    const int wg = blockIdx.x;
    uint32_t row;                                       // row of tiles over all segments
    if (wg < wholes + 4 * cut) {                        // a whole tile, or a quarter of one
        int t, q = 0;
        if (wg < wholes) {
            t = xcd_permute<int>(wg, wholes, a.xcds);
        } else {
            t = wholes + (wg - wholes) / 4;
            q = (wg - wholes) % 4;
        }
        row = t / nq;
        const int l = __builtin_ctzll(__ballot(full_incl > row));
        const int before = static_cast<int>(__builtin_amdgcn_readlane(full_incl - full, l));
        const int tiles = __builtin_amdgcn_readlane(full, l);
        out->seg = l;
        out->lo = __builtin_amdgcn_readlane(s.lo, l);
        out->rows = __builtin_amdgcn_readlane(s.rows, l);
        out->whole = wg < wholes;
        grouped_tile<int>(t - before * nq, tiles, nq, a.group_m < tiles ? a.group_m : tiles, &out->pid_m, &out->pid_n);
        if (!out->whole) {
            out->pid_m = 2 * out->pid_m + (q >> 1);
            out->pid_n = 2 * out->pid_n + (q & 1);
            return out->pid_m * 128 < out->rows && out->pid_n < nh;   // a quarter can lie outside
        }
        return true;
    }
    const int t = wg - wholes - 4 * cut;
    if (t >= smalls) return false;
    row = t / nh;
    const int l = __builtin_ctzll(__ballot(half_incl > row));
    out->seg = l;
    out->lo = __builtin_amdgcn_readlane(s.lo, l);
    out->rows = __builtin_amdgcn_readlane(s.rows, l);
    out->whole = false;
    out->pid_m = 2 * static_cast<int>(__builtin_amdgcn_readlane(full, l));
    out->pid_n = t % nh;
    return true;
}

template <bool BF16, bool TB>
__global__ __launch_bounds__(512) void gemm_grouped_rows_mixed_kernel(GroupedArgs a) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[65536];   // either tile's ring
    MixedTile m;
    if (!find_mixed(a, &m)) return;
    RowTile t;
    t.seg = m.seg;
    t.lo = m.lo;
    t.rows = m.rows;
    t.tiles = m.pid_m + 1;
    t.tile = 0;
    KArgs p = row_args(a, t);
    // the tile is known: row-major order finds it again
    p.group_m = 1;
    constexpr int EL = BF16 ? kElBF16 : kElF16;
    const int steps = (p.K + 63) / 64;
    if (m.whole) {
        dma_tile_in<256, 256, 64, 2, 4, 16, 2, EL, false, TB>(smem, p, whole_tile(m.pid_m * p.num_pid_n + m.pid_n, steps));
    } else {
        p.num_pid_n = (a.Q + 127) / 128;
        dma_tile_in<128, 128, 64, 2, 4, 16, 4, EL, false, TB>(smem, p, whole_tile(m.pid_m * p.num_pid_n + m.pid_n, steps));
    }
}

template <bool BF16, bool TB>
hipError_t launch_mixed(const GroupedArgs& a, int64_t grid, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_grouped_rows_mixed_kernel<BF16, TB>), dim3(static_cast<unsigned>(grid)), dim3(512), 0,
                       stream, a);
    return hipGetLastError();
}

#define MIXED_ENTRY(BF, TB)                                                                       \
    {kGroupedRows, 256, 256, 64, 2, 16, 2, 4, BF, kGroupedDirect, TB, 0, 512, 131072,             \
     &launch_mixed<(BF != 0), (TB != 0)>, "gemm_grouped_rows_mixed_kernel<" DTG_STR(BF) "," DTG_STR(TB) ">"}

const GroupedEntry kTable[] = {MIXED_ENTRY(0, 0), MIXED_ENTRY(1, 0), MIXED_ENTRY(0, 1), MIXED_ENTRY(1, 1)};

}  // namespace

const GroupedEntry* grouped_mixed_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
