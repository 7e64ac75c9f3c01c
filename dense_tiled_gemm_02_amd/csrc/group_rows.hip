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
// Up to kRowsOneBlock rows one workgroup does everything; above, three
// launches: per-block counts, their scan over the blocks, the placement.
// Bound by latency, not bytes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels_grouped.h"

namespace dtg {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kClasses = kMaxRowGroups;   // LDS counters per wave: groups + 1 classes at most

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

// Rows [first, last) of a block, `run` (a multiple of 64) to each wave.
// `start`: nullptr for a block that holds every row (it also writes offsets);
// else the rows of each class in the blocks before this one, with offsets
// already written.
template <typename ID>
__device__ __forceinline__ void place_rows(const ID* ids, int64_t first, int64_t last, int64_t run, int groups,
                                           const int32_t* start, int32_t* offsets, int32_t* order) {
    __shared__ int count[kWaves * kClasses];
    __shared__ int waves[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int classes = groups + 1;
    for (int i = tid; i < kWaves * classes; i += kThreads) count[i] = 0;
    __syncthreads();
    const int64_t r0 = first + wave * run;
    const int64_t r1 = r0 + run < last ? r0 + run : last;
    int* const mine = count + wave * classes;
    for (int64_t r = r0 + lane; r < r1; r += 64) atomicAdd(&mine[class_of(ids, r, groups)], 1);
    __syncthreads();
    int total = 0;
    if (tid < classes) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int c = count[w * classes + tid];
            count[w * classes + tid] = total;
            total += c;
        }
    }
    int base;
    if (start) {
        base = tid < classes ? start[tid] + offsets[tid] : 0;
    } else {
        base = block_exclusive(total, waves);
        if (tid < classes) offsets[tid] = base;
    }
    if (tid < classes) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) count[w * classes + tid] += base;
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < classes) ++bits;
    for (int64_t r = r0; r < r1; r += 64) {
        const bool live = r + lane < r1;
        const int c = live ? class_of(ids, r + lane, groups) : 0;
        uint64_t same = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((c >> b) & 1);
            same &= ((c >> b) & 1) ? set : ~set;
        }
        const int leader = live ? __builtin_ctzll(same) : 0;
        int place = 0;
        if (live && lane == leader) place = atomicAdd(&mine[c], __popcll(same));
        place = __shfl(place, leader, 64);
        if (live) order[place + __popcll(same & ((uint64_t(1) << lane) - 1))] = static_cast<int32_t>(r + lane);
    }
}

template <typename ID>
__global__ __launch_bounds__(kThreads) void group_rows_kernel(const ID* ids, int64_t R, int64_t run, int groups,
                                                              int32_t* offsets, int32_t* order) {
    place_rows(ids, 0, R, run, groups, nullptr, offsets, order);
}

template <typename ID>
__global__ __launch_bounds__(kThreads) void group_count_kernel(const ID* ids, int64_t R, int groups, int32_t* counts) {
    __shared__ int count[kClasses];
    const int classes = groups + 1;
    for (int i = threadIdx.x; i < classes; i += kThreads) count[i] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * kRowsPerBlock;
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

template <typename ID>
__global__ __launch_bounds__(kThreads) void group_place_kernel(const ID* ids, int64_t R, int groups,
                                                               const int32_t* counts, int32_t* offsets,
                                                               int32_t* order) {
    const int64_t first = blockIdx.x * kRowsPerBlock;
    place_rows(ids, first, first + kRowsPerBlock < R ? first + kRowsPerBlock : R, kRowsPerBlock / kWaves, groups,
               counts + static_cast<int64_t>(blockIdx.x) * (groups + 1), offsets, order);
}

template <typename ID>
hipError_t launch_ids(const ID* ids, int64_t R, int32_t groups, int32_t* offsets, int32_t* order, int32_t* counts,
                      hipStream_t stream) {
    if (R <= kRowsOneBlock) {
        const int64_t run = ((R + kWaves - 1) / kWaves + 63) / 64 * 64;
        hipLaunchKernelGGL(group_rows_kernel<ID>, dim3(1), dim3(kThreads), 0, stream, ids, R, run, groups, offsets,
                           order);
        return hipGetLastError();
    }
    const unsigned blocks = static_cast<unsigned>((R + kRowsPerBlock - 1) / kRowsPerBlock);
    hipLaunchKernelGGL(group_count_kernel<ID>, dim3(blocks), dim3(kThreads), 0, stream, ids, R, groups, counts);
    hipLaunchKernelGGL(group_scan_kernel, dim3(1), dim3(kThreads), 0, stream, counts, static_cast<int>(blocks),
                       groups, offsets);
    hipLaunchKernelGGL(group_place_kernel<ID>, dim3(blocks), dim3(kThreads), 0, stream, ids, R, groups, counts,
                       offsets, order);
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
