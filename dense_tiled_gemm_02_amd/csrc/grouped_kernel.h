// Products grouped by an offset table, on the tile bodies of the dense kernels.
//
//  rows kind:    D[i, :] = A[i, :] x B[g]   for offsets[g] <= i < offsets[g + 1]
//  reduce kind:  D[g] = sum over those i of A[i, :]^T x B[i, :]
//
// The table is on the device, so the host knows neither a group's length nor
// the number of tiles: the rows kind launches the most tiles that any table
// over R rows can need (floor(R / BM) + groups + 2 rows of tiles; every segment
// but the last tile of each is full), each workgroup counts the tiles of the
// segments from the table itself, and workgroups past the count leave.  A
// workgroup then is one tile of one ordinary product whose A, B and D start
// at its segment.
//
// The R rows are cut into groups + 2 segments: the rows before offsets[0], the
// groups, and the rows from offsets[groups] on.  The first and last belong to
// no group and run with no K steps, which writes zeros.  Bounds are clamped
// to [0, R], so no table can lead an access outside the operands; a table that
// decreases can leave rows unwritten, nothing worse.
#pragma once

#include "gemm_dma_kernel.h"
#include "kernels_grouped.h"

namespace dtg {
namespace {

struct Segment {
    int lo, rows;
};

// Segment i (0 .. groups + 1) of the table; no rows when the table decreases.
__device__ __forceinline__ Segment table_segment(const GroupedArgs& a, int i) {
    auto bound = [&](int j) {
        const int b = a.offsets[j];
        return b < 0 ? 0 : b > a.R ? a.R : b;
    };
    const int lo = i == 0 ? 0 : bound(i - 1);
    const int hi = i == a.groups + 1 ? a.R : bound(i);
    return {lo, hi > lo ? hi - lo : 0};
}

struct RowTile {
    int seg, lo, rows;     // the segment and its rows
    int tile, tiles;       // position among the segment's tiles, its rows of tiles
};

// Tile number `wg` (a workgroup's own, by default), the same in every wave (no
// LDS, no barrier): lane l counts the tiles of segment base + l, an inclusive
// scan over the wave places them.  False past the last tile.
template <int BM>
__device__ __forceinline__ bool find_row_tile(const GroupedArgs& a, RowTile* out, int wg = blockIdx.x) {
    const int lane = threadIdx.x & 63;
    const int nseg = a.groups + 2;
    auto count = [&](int i, Segment* s) {
        if (i >= nseg) {
            *s = {0, 0};
            return 0u;
        }
        *s = table_segment(a, i);
        return (static_cast<uint32_t>(s->rows) + BM - 1) / BM;
    };
    auto scan = [&](uint32_t v) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t u = __shfl_up(v, d, 64);
            if (lane >= d) v += u;
        }
        return v;
    };
    // Rows of tiles of all segments.  No increasing table has more than `most`
    // (the launch's own count, so total * num_pid_q fits 32 bits).
    const uint32_t most = static_cast<uint32_t>(a.R / BM) + static_cast<uint32_t>(nseg);
    Segment s;
    uint32_t incl = scan(count(lane, &s));
    uint32_t total = __builtin_amdgcn_readlane(incl, 63);
    for (int base = 64; base < nseg && total <= most; base += 64) {
        Segment t;
        total += __builtin_amdgcn_readlane(scan(count(base + lane, &t)), 63);
    }
    if (total > most) return false;
    const int positions = static_cast<int>(total) * a.num_pid_q;
    if (wg >= positions) return false;
    const int pos = xcd_permute<int>(wg, positions, a.xcds);
    const uint32_t want = pos / a.num_pid_q;   // row of tiles over all segments
    uint32_t before = 0;                        // rows of tiles before this chunk of segments
    for (int base = 0; base < nseg; base += 64) {
        if (base > 0) incl = scan(count(base + lane, &s));
        const uint64_t past = __ballot(before + incl > want);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int upto = static_cast<int>(before + __builtin_amdgcn_readlane(incl, l));
            out->seg = base + l;
            out->lo = __builtin_amdgcn_readlane(s.lo, l);
            out->rows = __builtin_amdgcn_readlane(s.rows, l);
            out->tiles = static_cast<int>((static_cast<uint32_t>(out->rows) + BM - 1) / BM);
            out->tile = pos - (upto - out->tiles) * a.num_pid_q;
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

// The workgroup's segment as an ordinary product's arguments (rows kind).
__device__ __forceinline__ KArgs row_args(const GroupedArgs& a, const RowTile& t) {
    const bool grouped = t.seg >= 1 && t.seg <= a.groups;
    KArgs p;
    p.A = a.A + static_cast<int64_t>(t.lo) * a.sa_r;
    p.B = a.B + (grouped ? static_cast<int64_t>(t.seg - 1) * a.sb_g : 0);
    p.C = nullptr;
    p.D = static_cast<uint16_t*>(a.D) + static_cast<int64_t>(t.lo) * a.sd_r;
    p.M = t.rows;
    p.N = a.Q;
    p.K = grouped ? a.P : 0;
    p.num_pid_m = t.tiles;
    p.num_pid_n = a.num_pid_q;
    p.group_m = a.group_m < t.tiles ? a.group_m : t.tiles;
    p.xcds = 1;
    p.has_c = 0;
    p.splits = 1;
    p.lda = a.sa_r;
    p.sak = a.sa_p;
    p.ldb = a.sb_r;
    p.sbn = a.sb_q;
    p.ldc = 0;
    p.ldd = a.sd_r;
    p.ws = nullptr;
    return p;
}

// Parts of a group of `rows` rows; a group without rows is one part (of zeros).
__device__ __forceinline__ uint32_t group_parts(int rows, int part_rows) {
    const uint32_t n = (static_cast<uint32_t>(rows) + part_rows - 1) / static_cast<uint32_t>(part_rows);
    return n > 0 ? n : 1;
}

// Inclusive scan over the wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

// Part number `want` of all groups' parts in order: its group and rows.  False
// past the last one.
__device__ __forceinline__ bool find_part(const GroupedArgs& a, uint32_t want, int* group, Segment* rows) {
    const int lane = threadIdx.x & 63;
    uint32_t before = 0;
    for (int base = 0; base < a.groups; base += 64) {
        Segment s = {0, 0};
        uint32_t n = 0;
        if (base + lane < a.groups) {
            s = table_segment(a, base + lane + 1);
            n = group_parts(s.rows, a.part_rows);
        }
        const uint32_t incl = wave_scan(n);
        const uint64_t past = __ballot(before + incl > want);
        if (past) {
            const int l = __builtin_ctzll(past);
            const uint32_t first = before + __builtin_amdgcn_readlane(incl - n, l);
            const int lo = __builtin_amdgcn_readlane(s.lo, l), len = __builtin_amdgcn_readlane(s.rows, l);
            const int skip = static_cast<int>(want - first) * a.part_rows;
            *group = base + l;
            rows->lo = lo + skip;
            rows->rows = len - skip < a.part_rows ? len - skip : a.part_rows;
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

// The group that is number `rank` in order of length (up to 64 groups).
__device__ __forceinline__ int group_of_rank(const GroupedArgs& a, int rank) {
    const int lane = threadIdx.x & 63;
    const int rows = lane < a.groups ? table_segment(a, lane + 1).rows : -1;
    int ahead = 0;
    for (int j = 0; j < a.groups; ++j) {
        const int other = __builtin_amdgcn_readlane(rows, j);
        ahead += other > rows || (other == rows && j < lane);
    }
    return __builtin_ctzll(__ballot(lane < a.groups && ahead == rank));
}

// Workgroup -> (group or part, tile of it).  Where the tiles divide by the
// dies, each die takes the same share of every group, neighbouring tiles
// together; in one contiguous range each, the die with the longest group
// finished last (16384 rows over 8 groups: 415 us).
__device__ __forceinline__ void reduce_position(const GroupedArgs& a, int* item, int* tile) {
    const int tiles = a.num_pid_p * a.num_pid_q;
    const int wg = blockIdx.x;
    if (a.xcds > 1 && tiles % a.xcds == 0) {
        const int per = tiles / a.xcds, local = wg / a.xcds;
        *item = local / per;
        *tile = wg % a.xcds * per + local % per;
    } else {
        *item = wg / tiles;
        *tile = wg % tiles;
    }
}

// A group's product as an ordinary one's arguments (reduce kind): the
// contraction runs over `rows` rows from `lo` on, D is the group's or the part's.
template <bool O32>
__device__ __forceinline__ KArgs reduce_args(const GroupedArgs& a, int g, int lo, int rows) {
    const int64_t at = static_cast<int64_t>(g) * a.sd_g;
    KArgs p;
    p.A = a.A + static_cast<int64_t>(lo) * a.sa_r;
    p.B = a.B + static_cast<int64_t>(lo) * a.sb_r;
    p.D = O32 ? reinterpret_cast<uint16_t*>(static_cast<float*>(a.D) + at) : static_cast<uint16_t*>(a.D) + at;
    p.C = a.accumulate ? p.D : nullptr;
    p.M = a.P;
    p.N = a.Q;
    p.K = rows;
    p.num_pid_m = a.num_pid_p;
    p.num_pid_n = a.num_pid_q;
    p.group_m = a.group_m < a.num_pid_p ? a.group_m : a.num_pid_p;
    p.xcds = 1;
    p.has_c = a.accumulate;
    p.splits = 1;
    p.lda = a.sa_p;
    p.sak = a.sa_r;
    p.ldb = a.sb_r;
    p.sbn = a.sb_q;
    p.ldc = a.sd_r;
    p.ldd = a.sd_r;
    p.ws = nullptr;
    return p;
}

__device__ __forceinline__ Work whole_tile(int tile, int ksteps) {
    Work w;
    w.tile = tile;
    w.kt0 = 0;
    w.kt1 = ksteps;
    w.part = 0;
    w.nparts = 1;
    w.base = w.slot0 = w.slot1 = 0;
    w.nslots = 1;
    return w;
}

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, bool TB>
__global__ __launch_bounds__(64 * WM * WN) void gemm_grouped_rows_kernel(GroupedArgs a) {
    RowTile t;
    if (!find_row_tile<BM>(a, &t)) return;
    const KArgs p = row_args(a, t);
    dma_tile<BM, BN, BK, WM, WN, MF, ST, BF16 ? kElBF16 : kElF16, false, TB>(
        p, whole_tile(t.tile, (p.K + BK - 1) / BK));
}

// The workgroup's product and tile; false for a workgroup past the last part.
template <bool O32>
__device__ __forceinline__ bool reduce_work(const GroupedArgs& a, KArgs* p, int* tile) {
    int item, g;
    Segment s;
    reduce_position(a, &item, tile);
    if (a.part_rows > 0) {
        if (!find_part(a, item, &g, &s)) return false;
        *p = reduce_args<O32>(a, g, s.lo, s.rows);
        p->D = reinterpret_cast<uint16_t*>(a.parts + static_cast<int64_t>(item) * a.P * a.Q);
        p->ldd = a.Q;
        p->C = nullptr;
        p->has_c = 0;
    } else {
        g = a.longest_first ? group_of_rank(a, item) : item;
        s = table_segment(a, g + 1);
        *p = reduce_args<O32>(a, g, __builtin_amdgcn_readfirstlane(s.lo), __builtin_amdgcn_readfirstlane(s.rows));
    }
    return true;
}

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, bool O32>
__global__ __launch_bounds__(64 * WM * WN) void gemm_grouped_reduce_kernel(GroupedArgs a) {
    KArgs p;
    int tile;
    if (!reduce_work<O32>(a, &p, &tile)) return;
    dma_tile<BM, BN, BK, WM, WN, MF, ST, BF16 ? kElBF16 : kElF16, true, false, false, false, O32>(
        p, whole_tile(tile, (p.K + BK - 1) / BK));
}

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, bool TB>
hipError_t launch_grouped_rows(const GroupedArgs& a, int64_t grid, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_grouped_rows_kernel<BM, BN, BK, WM, WN, MF, ST, BF16, TB>),
                       dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, stream, a);
    return hipGetLastError();
}

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, bool O32>
hipError_t launch_grouped_reduce(const GroupedArgs& a, int64_t grid, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_grouped_reduce_kernel<BM, BN, BK, WM, WN, MF, ST, BF16, O32>),
                       dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, stream, a);
    return hipGetLastError();
}

#define GROUPED_LDS(BM, BN, BK, ST) static_cast<int64_t>(ST) * (BM + BN) * BK * 2
#define GROUPED_ROWS_ENTRY(BM, BN, BK, WM, WN, MF, ST, BF, TB)                                       \
    {kGroupedRows, BM, BN, BK, ST, MF, WM, WN, BF, kGroupedDirect, TB, 0, 64 * WM * WN, GROUPED_LDS(BM, BN, BK, ST), \
     &launch_grouped_rows<BM, BN, BK, WM, WN, MF, ST, (BF != 0), (TB != 0)>,                         \
     "gemm_grouped_rows_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) ","      \
     DTG_STR(WN) "," DTG_STR(MF) "," DTG_STR(ST) "," DTG_STR(BF) "," DTG_STR(TB) ">"}
#define GROUPED_ROWS(BM, BN, BK, WM, WN, MF, ST)             \
    GROUPED_ROWS_ENTRY(BM, BN, BK, WM, WN, MF, ST, 0, 0),    \
    GROUPED_ROWS_ENTRY(BM, BN, BK, WM, WN, MF, ST, 1, 0),    \
    GROUPED_ROWS_ENTRY(BM, BN, BK, WM, WN, MF, ST, 0, 1),    \
    GROUPED_ROWS_ENTRY(BM, BN, BK, WM, WN, MF, ST, 1, 1)
#define GROUPED_REDUCE_ENTRY(BM, BN, BK, WM, WN, MF, ST, BF, O32)                                      \
    {kGroupedReduce, BM, BN, BK, ST, MF, WM, WN, BF, kGroupedDirect, 0, O32, 64 * WM * WN, GROUPED_LDS(BM, BN, BK, ST), \
     &launch_grouped_reduce<BM, BN, BK, WM, WN, MF, ST, (BF != 0), (O32 != 0)>,                        \
     "gemm_grouped_reduce_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) ","      \
     DTG_STR(WN) "," DTG_STR(MF) "," DTG_STR(ST) "," DTG_STR(BF) "," DTG_STR(O32) ">"}
#define GROUPED_REDUCE(BM, BN, BK, WM, WN, MF, ST)           \
    GROUPED_REDUCE_ENTRY(BM, BN, BK, WM, WN, MF, ST, 0, 0),  \
    GROUPED_REDUCE_ENTRY(BM, BN, BK, WM, WN, MF, ST, 1, 0),  \
    GROUPED_REDUCE_ENTRY(BM, BN, BK, WM, WN, MF, ST, 0, 1),  \
    GROUPED_REDUCE_ENTRY(BM, BN, BK, WM, WN, MF, ST, 1, 1)

}  // namespace
}  // namespace dtg
