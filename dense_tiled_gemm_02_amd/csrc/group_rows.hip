// Row grouping: the counting sort that turns the router's ids into the offset
// table and the row order of the grouped products.
//
//     offsets[g] = number of rows with id < g        (ids outside [0, groups) count as `groups`)
//     order[offsets[id] + rank] = row,  rank = earlier rows of the same id
//
// Stable, so the result does not depend on the launch.  The rows are dealt to
// the waves in contiguous runs; a first pass counts the ids of each run in LDS
// (integer atomics: the counts do not depend on their order), an exclusive
// scan over (id, run) places each run's first row of each id, and a second
// pass walks the runs 64 rows at a time: rows of one id within the 64 find
// one another by one ballot per id bit, and the first of them draws the
// places for all.
//
// Up to kRowsOneBlock rows one workgroup does everything; above, two launches:
// per-block counts, then the placement, where every block adds up the counts
// of the blocks before it for itself.  Past kSelfScan blocks that sum would
// outgrow the placement, and a launch between them scans the counts.
// Bound by latency, not bytes: 131072 ids over 128 groups, 1 MB, take 9 us
// (with the scan launch and one placing workgroup per count 14.7).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels_grouped.h"

namespace dtg {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kClasses = kMaxRowGroups;   // LDS counters per wave: groups + 1 classes at most
constexpr int kSelfScan = 64;             // blocks up to which the placement sums the counts itself

template <typename ID>
__device__ __forceinline__ int class_of(const ID* ids, int64_t row, int groups) {
    const ID id = ids[row];
    return (id >= 0 && id < groups) ? static_cast<int>(id) : groups;
}

// Exclusive scan of one value per thread over the workgroup.
__device__ __forceinline__ int block_exclusive(int v, int* waves) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int u = __shfl_up(incl, d, 64);
        if (lane >= d) incl += u;
    }
    if (lane == 63) waves[wave] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w) before += waves[w];
    return before + incl - v;
}

// Rows [first, last) of a block, `run` (a multiple of 64, at most 64 KEEP) to
// each wave; their classes stay in registers between the passes.  prepare()
// runs before the first barrier, gather() after it, and place(tid, total) then
// gives thread tid < groups + 1 the place of the block's first row of that
// class, of which the block has `total`; every thread calls all three.
template <int KEEP, typename ID, typename Prepare, typename Gather, typename Place>
__device__ __forceinline__ void place_rows(const ID* ids, int64_t first, int64_t last, int64_t run, int groups,
                                           int32_t* order, Prepare&& prepare, Gather&& gather, Place&& place) {
    __shared__ int count[kWaves * kClasses];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int classes = groups + 1;
    const int64_t r0 = first + wave * run;
    const int64_t r1 = r0 + run < last ? r0 + run : last;
    int cls[KEEP];
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        const int64_t r = r0 + 64 * k + lane;
        cls[k] = r < r1 ? class_of(ids, r, groups) : -1;
    }
    prepare();
    for (int i = tid; i < kWaves * classes; i += kThreads) count[i] = 0;
    __syncthreads();
    int* const mine = count + wave * classes;
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
        if (cls[k] >= 0) atomicAdd(&mine[cls[k]], 1);
    gather();
    __syncthreads();
    int total = 0, held[kWaves];
    if (tid < classes) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) held[w] = count[w * classes + tid];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int c = held[w];
            held[w] = total;
            total += c;
        }
    }
    const int base = place(tid, total);
    if (tid < classes) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) count[w * classes + tid] = held[w] + base;
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < classes) ++bits;
#pragma unroll
    for (int k = 0; k < KEEP; ++k) {
        const int64_t r = r0 + 64 * k + lane;
        if (r0 + 64 * k >= r1) break;
        const bool live = cls[k] >= 0;
        const int c = live ? cls[k] : 0;
        uint64_t same = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((c >> b) & 1);
            same &= ((c >> b) & 1) ? set : ~set;
        }
        const int leader = live ? __builtin_ctzll(same) : 0;
        int at = 0;
        if (live && lane == leader) at = atomicAdd(&mine[c], __popcll(same));
        at = __shfl(at, leader, 64);
        if (live) order[at + __popcll(same & ((uint64_t(1) << lane) - 1))] = static_cast<int32_t>(r);
    }
}

// Up to 1024 KEEP rows in one workgroup.
template <int KEEP, typename ID>
__global__ __launch_bounds__(kThreads) void group_rows_kernel(const ID* ids, int64_t R, int64_t run, int groups,
                                                              int32_t* offsets, int32_t* order) {
    __shared__ int waves[kWaves];
    place_rows<KEEP>(ids, 0, R, run, groups, order, [] {}, [] {}, [&](int tid, int total) {
        const int base = block_exclusive(total, waves);
        if (tid <= groups) offsets[tid] = base;
        return base;
    });
}

template <typename ID>
__global__ __launch_bounds__(kThreads) void group_count_kernel(const ID* ids, int64_t R, int groups, int32_t* counts) {
    __shared__ int count[kClasses];
    const int classes = groups + 1;
    for (int i = threadIdx.x; i < classes; i += kThreads) count[i] = 0;
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock;
#pragma unroll
    for (int i = 0; i < kRowsPerBlock / kThreads; ++i) {
        const int64_t r = first + i * kThreads + threadIdx.x;
        if (r < R) atomicAdd(&count[class_of(ids, r, groups)], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < classes; i += kThreads)
        counts[static_cast<int64_t>(blockIdx.x) * classes + i] = count[i];
}

// One workgroup, a thread per class: counts[block][class] becomes the class's
// rows in earlier blocks, offsets the classes' first places.
__global__ __launch_bounds__(kThreads) void group_scan_kernel(int32_t* counts, int blocks, int groups,
                                                              int32_t* offsets) {
    __shared__ int waves[kWaves];
    const int c = threadIdx.x, classes = groups + 1;
    int total = 0;
    if (c < classes) {
        for (int b0 = 0; b0 < blocks; b0 += 16) {
            int v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = b0 + i < blocks ? counts[static_cast<int64_t>(b0 + i) * classes + c] : 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (b0 + i < blocks) counts[static_cast<int64_t>(b0 + i) * classes + c] = total;
                total += v[i];
            }
        }
    }
    const int base = block_exclusive(total, waves);
    if (c < classes) offsets[c] = base;
}

// kSubs workgroups place the rows of one counting block, each its share of
// kThreads rows: it counts the shares before its own itself, and its own in one
// step of 64 rows per wave (with one workgroup per block 7.5 us, so 6.4).
// SCANNED: the counts are already sums over earlier blocks, and offsets written.
constexpr int kSubs = kRowsPerBlock / kThreads;

template <typename ID, bool SCANNED>
__global__ __launch_bounds__(kThreads) void group_place_kernel(const ID* ids, int64_t R, int groups,
                                                               const int32_t* counts, int blocks, int32_t* offsets,
                                                               int32_t* order) {
    __shared__ int before[kClasses], all[kClasses], waves[kWaves];
    const int classes = groups + 1, here = blockIdx.x / kSubs, sub = blockIdx.x % kSubs;
    const int64_t block0 = static_cast<int64_t>(here) * kRowsPerBlock, first = block0 + sub * kThreads;
    if (first >= R) return;
    // the counts of all blocks, HELD of them in flight per thread while the rows are counted
    constexpr int HELD = 8;
    const int cells = blocks * classes;
    int v[HELD], earlier[kSubs - 1];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < HELD; ++u) {
            const int i = i0 + u * kThreads;
            v[u] = i < cells ? counts[i] : 0;
        }
    };
    auto prepare = [&] {
        if constexpr (!SCANNED) fetch(threadIdx.x);
#pragma unroll
        for (int u = 0; u < kSubs - 1; ++u)   // whole shares: this one starts before R
            earlier[u] = u < sub ? class_of(ids, block0 + u * kThreads + threadIdx.x, groups) : -1;
        for (int i = threadIdx.x; i < classes; i += kThreads) before[i] = all[i] = 0;
    };
    auto gather = [&] {   // integer sums, in any order
#pragma unroll
        for (int u = 0; u < kSubs - 1; ++u)
            if (earlier[u] >= 0) atomicAdd(&before[earlier[u]], 1);
        if constexpr (SCANNED) return;
        for (int i0 = threadIdx.x; i0 < cells; i0 += HELD * kThreads) {
            if (i0 >= kThreads) fetch(i0);
#pragma unroll
            for (int u = 0; u < HELD; ++u) {
                const int i = i0 + u * kThreads, b = i / classes, c = i - b * classes;
                if (v[u]) {
                    atomicAdd(&all[c], v[u]);
                    if (b < here) atomicAdd(&before[c], v[u]);
                }
            }
        }
    };
    auto place = [&](int tid, int) {
        if constexpr (SCANNED)
            return tid < classes ? counts[static_cast<int64_t>(here) * classes + tid] + offsets[tid] + before[tid] : 0;
        const int base = block_exclusive(tid < classes ? all[tid] : 0, waves);
        if (blockIdx.x == 0 && tid < classes) offsets[tid] = base;
        return base + (tid < classes ? before[tid] : 0);
    };
    place_rows<1>(ids, first, first + kThreads < R ? first + kThreads : R, 64, groups, order, prepare, gather, place);
}

template <typename ID>
hipError_t launch_ids(const ID* ids, int64_t R, int32_t groups, int32_t* offsets, int32_t* order, int32_t* counts,
                      hipStream_t stream) {
    if (R <= kRowsOneBlock) {
        const int64_t run = ((R + kWaves - 1) / kWaves + 63) / 64 * 64;
        if (run <= 64 * 4)
            hipLaunchKernelGGL((group_rows_kernel<4, ID>), dim3(1), dim3(kThreads), 0, stream, ids, R, run, groups,
                               offsets, order);
        else
            hipLaunchKernelGGL((group_rows_kernel<kRowsOneBlock / kThreads, ID>), dim3(1), dim3(kThreads), 0, stream,
                               ids, R, run, groups, offsets, order);
        return hipGetLastError();
    }
    const unsigned blocks = static_cast<unsigned>((R + kRowsPerBlock - 1) / kRowsPerBlock);
    hipLaunchKernelGGL(group_count_kernel<ID>, dim3(blocks), dim3(kThreads), 0, stream, ids, R, groups, counts);
    if (blocks <= kSelfScan) {
        hipLaunchKernelGGL((group_place_kernel<ID, false>), dim3(blocks * kSubs), dim3(kThreads), 0, stream, ids, R, groups,
                           counts, static_cast<int>(blocks), offsets, order);
    } else {
        hipLaunchKernelGGL(group_scan_kernel, dim3(1), dim3(kThreads), 0, stream, counts, static_cast<int>(blocks),
                           groups, offsets);
        hipLaunchKernelGGL((group_place_kernel<ID, true>), dim3(blocks * kSubs), dim3(kThreads), 0, stream, ids, R, groups,
                           counts, static_cast<int>(blocks), offsets, order);
    }
    return hipGetLastError();
}

}  // namespace

int64_t group_rows_workspace_bytes(int64_t R, int64_t groups) {
    if (R <= kRowsOneBlock) return 0;
    return (R + kRowsPerBlock - 1) / kRowsPerBlock * (groups + 1) * 4;
}

hipError_t launch_group_rows(const void* ids, int id_bytes, int64_t R, int32_t groups, int32_t* offsets,
                             int32_t* order, void* workspace, hipStream_t stream) {
    int32_t* counts = static_cast<int32_t*>(workspace);
    if (id_bytes == 8) return launch_ids(static_cast<const int64_t*>(ids), R, groups, offsets, order, counts, stream);
    return launch_ids(static_cast<const int32_t*>(ids), R, groups, offsets, order, counts, stream);
}

}  // namespace dtg
