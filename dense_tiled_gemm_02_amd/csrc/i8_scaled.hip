// The int8 tile kernel (gemm_dma_kernel.h) with a scale for each row of X and
// row of W: the same ring and contraction as GEMM_I8's, the sums scaled and
// rounded in registers and stored as 16-byte chunks of rows.  Bound by the matrix
// units and the clock that they leave: 4096 x 14336 x 4096 190 to 200 us of a layer's
// values (2.4 to 2.5 POP/s), 213 to 247 of uniform ones; 8192^3 464 us of those (2.4).
#include "gemm_dma_kernel.h"

namespace dtg {
namespace {

#define I8S(BM, BN, BK, WM, WN, MF, ST, KIND, OUT_NAME)                                                    \
    {BM, BN, ST, MF, WM, WN, KIND, 0, &launch_i8s<BM, BN, BK, WM, WN, MF, ST, KIND>,                       \
     "gemm_i8s_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) "," DTG_STR(WN) "," DTG_STR(MF) \
     "," DTG_STR(ST) "," OUT_NAME ">"}
#define I8S_ALL(BM, BN, BK, WM, WN, MF, ST)                    \
    I8S(BM, BN, BK, WM, WN, MF, ST, kOutF16, "f16"),           \
    I8S(BM, BN, BK, WM, WN, MF, ST, kOutBF16, "bf16"),         \
    I8S(BM, BN, BK, WM, WN, MF, ST, kOutF32, "f32")

// Whole 256 x 256 tiles for full rounds of the card's CUs, and the tiles that are
// left, at most half a round, as halves of 256 x 128, which fit a round of their own:
// 4096 x 14336 x 4096, 3.5 rounds, takes 3.56 in place of 4.
template <int KIND>
__global__ __launch_bounds__(512) void gemm_i8s_mixed_kernel(ScaledArgs p, int whole) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[3 * (256 + 128) * 64];   // either tile's ring
    constexpr int EL = kElI8ToF16 + KIND;
    const int wg = static_cast<int>(blockIdx.x), steps = (p.K + 63) / 64;
    const int halves = 2 * (p.num_pid_m * p.num_pid_n - whole);
    const int half = wg < whole ? -1 : xcd_permute<int>(wg - whole, halves, p.xcds);
    const int pos = half < 0 ? xcd_permute<int>(wg, whole, p.xcds) : whole + half / 2;
    int pm, pn;
    grouped_tile<int>(pos, p.num_pid_m, p.num_pid_n, p.group_m, &pm, &pn);
    p.group_m = 1;   // the tile is known: row-major order finds it again
    Work w = {0, 0, steps, 0, 1, 0, 0, 0, 1};
    if (half < 0) {
        w.tile = pm * p.num_pid_n + pn;
        dma_tile_in<256, 256, 64, 2, 4, 16, 2, EL, false, true>(smem, p, w);
    } else {
        pn = 2 * pn + half % 2;
        p.num_pid_n = (p.N + 127) / 128;
        if (pn >= p.num_pid_n) return;   // a half can lie outside
        w.tile = pm * p.num_pid_n + pn;
        dma_tile_in<256, 128, 64, 4, 2, 16, 3, EL, false, true>(smem, p, w);
    }
}

// grid: the tiles; at least one round of whole ones.
template <int KIND>
hipError_t launch_mixed(const ScaledArgs& a, int64_t grid, hipStream_t stream) {
    const int64_t whole = grid - grid % a.cus;
    hipLaunchKernelGGL((gemm_i8s_mixed_kernel<KIND>), dim3(static_cast<unsigned>(whole + 2 * (grid - whole))), dim3(512), 0, stream, a,
                       static_cast<int>(whole));
    return hipGetLastError();
}
#define I8S_MIXED(KIND, OUT_NAME) {256, 256, 2, 16, 2, 4, KIND, 1, &launch_mixed<KIND>, "gemm_i8s_mixed_kernel<" OUT_NAME ">"}

const I8TileEntry kTable[] = {
    I8S_ALL(256, 256, 64, 2, 4, 16, 2),
    I8S_MIXED(kOutF16, "f16"), I8S_MIXED(kOutBF16, "bf16"), I8S_MIXED(kOutF32, "f32"),
    I8S_ALL(192, 256, 64, 2, 4, 16, 2),
    I8S_ALL(256, 128, 64, 4, 2, 16, 3),
    I8S_ALL(128, 256, 64, 2, 4, 16, 3),
    I8S_ALL(128, 128, 64, 2, 4, 16, 4),
    I8S_ALL(64, 64, 64, 2, 2, 16, 4),
};

}  // namespace

const I8TileEntry* i8_scaled_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
