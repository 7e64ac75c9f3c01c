// Internal interface between the ABI of the int8 products with scales
// (api_i8.cpp) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace dtg {

// Y[m, n] = (sum_k X[m, k] W[n, k]) sx[m] sw[n] + bias[n], Y and bias of one type.
struct ScaledI8 {
    const float* sx;
    const float* sw;
    const void* bias;   // nullptr: none
};

// The tile kernels' view: A = X, B = W in pairs of k (see gemm_dma_kernel.h).
struct ScaledArgs : KArgs {
    ScaledI8 s;
    int32_t cus;        // of the device: a round of tiles
};

// The other kernels': strides in bytes (X, W) and elements (Y).
struct I8RowsArgs {
    const int8_t* X;
    const int8_t* W;
    void* Y;
    ScaledI8 s;
    int32_t M, N, K;
    int64_t lx, lw, ly;
};

enum { kOutF16 = 0, kOutBF16 = 1, kOutF32 = 2 };

typedef hipError_t (*i8_tile_fn)(const ScaledArgs& args, int64_t grid, hipStream_t stream);
struct I8TileEntry {
    int32_t bm, bn, stages, mfma, waves_m, waves_n, out;
    int32_t mixed;      // 1: the last, partial round in halves
    i8_tile_fn launch;
    const char* name;
};
const I8TileEntry* i8_scaled_table(int* count);

// Tiles of 16 mb rows and 16 nb columns whose waves share out K.  K and row
// strides multiples of 16, X and W 16-byte aligned.
typedef hipError_t (*i8_few_fn)(const I8RowsArgs& args, hipStream_t stream);
struct I8FewEntry {
    int32_t mb, nb;
    i8_few_fn launch[3];   // by output type
    const char* name;
};
const I8FewEntry* i8_few_table(int* count);

// Sizes, strides and addresses of any kind, in square tiles of i8_any_tile.
int i8_any_tile(int64_t M, int64_t N, int cus);
hipError_t launch_i8_any(const I8RowsArgs& a, int out, int cus, int xcds, hipStream_t stream);

}  // namespace dtg
