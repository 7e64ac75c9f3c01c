// Register-staged tiled GEMM kernels (the tile body is gemm_tile_kernel.h):  D = A x B (+ C).
//
// Output tiles are visited in the grouped order of tile_order.h.

#include "gemm_tile_kernel.h"

namespace dtg {
namespace {

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, bool VEC>
__global__ __launch_bounds__(64 * WM * WN) void gemm_tile_kernel(KArgs p) {
    int pid_m, pid_n;
    tile_of_workgroup<int>(blockIdx.x, p.num_pid_m, p.num_pid_n, p.group_m, p.xcds, &pid_m, &pid_n);
    reg_tile<BM, BN, BK, WM, WN, MF, ST, BF16, VEC>(p, pid_m, pid_n);
}

template <int BM, int BN, int BK, int WM, int WN, int MF, int ST, bool BF16, bool VEC>
hipError_t launch_tile(const KArgs& a, int64_t grid, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_tile_kernel<BM, BN, BK, WM, WN, MF, ST, BF16, VEC>),
                       dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, stream, a);
    return hipGetLastError();
}

#define DTG_STR2(x) #x
#define DTG_STR(x) DTG_STR2(x)
#define TILE_ENTRY(BM, BN, BK, WM, WN, MF, ST, BF, VEC)                                      \
    {KF_TILE, BM, BN, BK, ST, MF, WM, WN, 1, BF, VEC, 64 * WM * WN,                           \
     static_cast<int64_t>(ST) * (BM + BN) * BK * 2,                                          \
     &launch_tile<BM, BN, BK, WM, WN, MF, ST, (BF != 0), (VEC != 0)>,                        \
     "gemm_tile_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) ","     \
     DTG_STR(WN) "," DTG_STR(MF) "," DTG_STR(ST) "," DTG_STR(BF) "," DTG_STR(VEC) ">", (VEC) ? 0 : -1}

#define TILE_BOTH(BM, BN, BK, WM, WN, MF, ST, VEC) \
    TILE_ENTRY(BM, BN, BK, WM, WN, MF, ST, 0, VEC), TILE_ENTRY(BM, BN, BK, WM, WN, MF, ST, 1, VEC)

const KernelEntry kTileTable[] = {
    TILE_BOTH(256, 256, 64, 2, 4, 32, 2, 1),
    TILE_BOTH(256, 128, 64, 2, 2, 16, 2, 1),
    TILE_BOTH(256, 128, 64, 2, 2, 32, 2, 1),
    TILE_BOTH(128, 256, 64, 2, 2, 16, 2, 1),
    TILE_BOTH(128, 128, 64, 2, 2, 16, 2, 1),
    TILE_BOTH(128, 128, 64, 2, 2, 32, 2, 1),
    TILE_BOTH(128, 128, 64, 2, 2, 16, 1, 1),
    TILE_BOTH(128, 128, 32, 2, 2, 16, 2, 1),
    TILE_BOTH(64, 64, 64, 2, 2, 16, 2, 1),
    TILE_BOTH(64, 64, 32, 2, 2, 16, 2, 1),
    TILE_BOTH(64, 64, 32, 2, 2, 16, 1, 1),
    TILE_BOTH(32, 32, 32, 2, 2, 16, 2, 1),
    TILE_BOTH(16, 64, 64, 1, 4, 16, 2, 1),
    TILE_BOTH(64, 64, 32, 2, 2, 16, 2, 0),
};

}  // namespace

const KernelEntry* tile_kernel_table(int* count) {
    *count = static_cast<int>(sizeof(kTileTable) / sizeof(kTileTable[0]));
    return kTileTable;
}

}  // namespace dtg
