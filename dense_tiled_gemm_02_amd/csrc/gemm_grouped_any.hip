// The grouped products for operands without a contiguous index (broadcast or
// twice-strided views): the register-staged tile body with element loads.
#include "gemm_tile_kernel.h"
#include "grouped_kernel.h"

namespace dtg {
namespace {

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16>
__global__ __launch_bounds__(64 * WM * WN) void gemm_grouped_rows_any_kernel(GroupedArgs a) {
    RowTile t;
    if (!find_row_tile<BM>(a, &t)) return;
    const KArgs p = row_args(a, t);
    int pid_m, pid_n;
    grouped_tile<int>(t.tile, p.num_pid_m, p.num_pid_n, p.group_m, &pid_m, &pid_n);
    reg_tile<BM, BN, BK, WM, WN, MF, ST, BF16, false>(p, pid_m, pid_n);
}

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, bool O32>
__global__ __launch_bounds__(64 * WM * WN) void gemm_grouped_reduce_any_kernel(GroupedArgs a) {
    KArgs p;
    int tile, pid_m, pid_n;
    if (!reduce_work<O32>(a, &p, &tile)) return;
    grouped_tile<int>(tile, p.num_pid_m, p.num_pid_n, p.group_m, &pid_m, &pid_n);
    reg_tile<BM, BN, BK, WM, WN, MF, ST, BF16, false, O32>(p, pid_m, pid_n);
}

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, int KIND, bool O32>
hipError_t launch_grouped_any(const GroupedArgs& a, int64_t grid, hipStream_t stream) {
    const dim3 g(static_cast<unsigned>(grid)), b(64 * WM * WN);
    if constexpr (KIND == kGroupedRows)
        hipLaunchKernelGGL((gemm_grouped_rows_any_kernel<BM, BN, BK, WM, WN, MF, ST, BF16>), g, b, 0, stream, a);
    else
        hipLaunchKernelGGL((gemm_grouped_reduce_any_kernel<BM, BN, BK, WM, WN, MF, ST, BF16, O32>), g, b, 0, stream,
                           a);
    return hipGetLastError();
}

#define GROUPED_ANY(BM, BN, BK, WM, WN, MF, ST, BF, KIND, O32, NAME)                                          \
    {KIND, BM, BN, BK, ST, MF, WM, WN, BF, kGroupedAny, 0, O32, 64 * WM * WN, GROUPED_LDS(BM, BN, BK, ST),               \
     &launch_grouped_any<BM, BN, BK, WM, WN, MF, ST, (BF != 0), KIND, (O32 != 0)>,                            \
     NAME "<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) "," DTG_STR(WN) "," DTG_STR(MF) "," \
     DTG_STR(ST) "," DTG_STR(BF) ">"}

const GroupedEntry kTable[] = {
    GROUPED_ANY(64, 64, 32, 2, 2, 16, 2, 0, kGroupedRows, 0, "gemm_grouped_rows_any_kernel"),
    GROUPED_ANY(64, 64, 32, 2, 2, 16, 2, 1, kGroupedRows, 0, "gemm_grouped_rows_any_kernel"),
    GROUPED_ANY(64, 64, 32, 2, 2, 16, 2, 0, kGroupedReduce, 0, "gemm_grouped_reduce_any_kernel"),
    GROUPED_ANY(64, 64, 32, 2, 2, 16, 2, 1, kGroupedReduce, 0, "gemm_grouped_reduce_any_kernel"),
    GROUPED_ANY(64, 64, 32, 2, 2, 16, 2, 0, kGroupedReduce, 1, "gemm_grouped_reduce_any_kernel"),
    GROUPED_ANY(64, 64, 32, 2, 2, 16, 2, 1, kGroupedReduce, 1, "gemm_grouped_reduce_any_kernel"),
};

}  // namespace

const GroupedEntry* grouped_any_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
