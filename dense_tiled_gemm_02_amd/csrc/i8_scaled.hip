// The int8 tile kernel (gemm_dma_kernel.h) with a scale for each row of X and
// row of W: the same ring and contraction as GEMM_I8's, the sums scaled and
// rounded in registers and stored as 16-byte chunks of rows.
#include "gemm_dma_kernel.h"

namespace dtg {
namespace {

#define I8S(BM, BN, BK, WM, WN, MF, ST, KIND, OUT_NAME)                                                    \
    {BM, BN, ST, MF, WM, WN, KIND, &launch_i8s<BM, BN, BK, WM, WN, MF, ST, KIND>,                          \
     "gemm_i8s_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) "," DTG_STR(WN) "," DTG_STR(MF) \
     "," DTG_STR(ST) "," OUT_NAME ">"}
#define I8S_ALL(BM, BN, BK, WM, WN, MF, ST)                    \
    I8S(BM, BN, BK, WM, WN, MF, ST, kOutF16, "f16"),           \
    I8S(BM, BN, BK, WM, WN, MF, ST, kOutBF16, "bf16"),         \
    I8S(BM, BN, BK, WM, WN, MF, ST, kOutF32, "f32")

const I8TileEntry kTable[] = {
    I8S_ALL(256, 256, 64, 2, 4, 16, 2),
    I8S_ALL(256, 128, 64, 4, 2, 16, 3),
    I8S_ALL(128, 256, 64, 2, 4, 16, 3),
    I8S_ALL(128, 128, 64, 2, 4, 16, 4),
    I8S_ALL(128, 128, 64, 2, 4, 16, 2),
    I8S_ALL(64, 64, 64, 2, 2, 16, 4),
};

}  // namespace

const I8TileEntry* i8_scaled_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
