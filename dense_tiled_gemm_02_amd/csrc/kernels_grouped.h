// Internal interface between the grouped-product ABI (api_grouped.cpp) and its kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dtg {

// Arguments of a product grouped by an offset table.  offsets[0 .. groups]
// lives on the device: group g owns the rows [offsets[g], offsets[g + 1]) of
// the R rows, each bound clamped to [0, R] where it is read.
//  rows kind:   D (R x Q) = A (R x P) x B[g] (P x Q); rows in no group give zeros
//  reduce kind: D[g] (P x Q) (+)= A_g^T x B_g, A (R x P), B (R x Q)
// Strides in elements; D's column stride is 1.
struct GroupedArgs {
    const uint16_t* A;
    const uint16_t* B;
    void* D;
    const int32_t* offsets;
    int32_t groups, R, P, Q;
    int32_t num_pid_p;      // tiles over P (reduce kind)
    int32_t num_pid_q;      // tiles over Q
    int32_t group_m, xcds;
    int32_t accumulate;     // reduce kind: add to D instead of overwriting it
    int64_t sa_r, sa_p;     // A element (row, p)
    int64_t sb_g, sb_r, sb_q;  // B element (g, p, q) of the rows kind, (row, q) of the reduce kind
    int64_t sd_g, sd_r;
    int32_t cus;            // of the device
    int32_t longest_first;  // reduce kind: groups in order of length
    int32_t part_rows;      // reduce kind: rows of one part of a group (0: whole groups), part n's
    int32_t max_parts;      // fp32 P x Q sum at parts + n * P * Q; no increasing
    float* parts;           // table has more than max_parts
};

typedef hipError_t (*grouped_launch_fn)(const GroupedArgs& args, int64_t grid, hipStream_t stream);

enum GroupedKind { kGroupedRows = 0, kGroupedReduce = 1 };

// How a variant reads its operands: element by element (any strides), in
// chunks of 8 of the contiguous index at any address, or straight into LDS in
// aligned 16-byte chunks.
enum GroupedLoads { kGroupedAny = 0, kGroupedDirect = 1, kGroupedOdd = 2 };

// One compiled variant (bm = 16: few rows per group, waves_n waves over K).  tb: B[g] is stored Q x P (rows kind).
struct GroupedEntry {
    int32_t kind;
    int32_t bm, bn, bk, stages, mfma, waves_m, waves_n;
    int32_t dtype;          // 0 fp16, 1 bf16
    int32_t loads, tb, out32;   // loads: GroupedLoads
    int32_t threads;
    int64_t lds_bytes;
    grouped_launch_fn launch;
    const char* name;
};

// D[g] (+)= the sum of the parts of group g in order, for each of the groups.
hipError_t launch_sum_parts(const GroupedArgs& a, int dtype, int out32, hipStream_t stream);

const GroupedEntry* grouped_rows_table(int* count);
const GroupedEntry* grouped_reduce_table(int* count);
const GroupedEntry* grouped_mixed_table(int* count);
const GroupedEntry* grouped_few_table(int* count);
const GroupedEntry* grouped_odd_table(int* count);
const GroupedEntry* grouped_any_table(int* count);

// Row grouping: offsets (groups + 1) and the stable order of the R rows by
// id (32- or 64-bit); ids outside [0, groups) come last.  Up to kRowsOneBlock
// rows take one workgroup and no workspace.
constexpr int64_t kRowsOneBlock = 16384;
constexpr int64_t kRowsPerBlock = 4096;
constexpr int32_t kMaxRowGroups = 1024;   // classes: groups + 1, one LDS counter per wave each
int64_t group_rows_workspace_bytes(int64_t R, int64_t groups);
hipError_t launch_group_rows(const void* ids, int id_bytes, int64_t R, int32_t groups, int32_t* offsets,
                             int32_t* order, void* workspace, hipStream_t stream);

}  // namespace dtg
