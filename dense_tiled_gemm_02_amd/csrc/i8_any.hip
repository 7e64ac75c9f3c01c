// int8 products with scales, Y = (X W^T) sx sw + b, for operands that the
// direct-to-LDS kernels do not take: K, row strides or bases that are no
// multiples of 16 bytes.
//
// 64 x 64 outputs to a workgroup of four waves, 128 k a step.  Every chunk of
// 16 k is one load at its own address, whatever that is, through registers one
// step ahead into one of two LDS stages; the chunk that K cuts is loaded byte by
// byte.  Rows past the operands read the last row, and what they make is not
// stored.  The sums are exact (int32), so nothing depends on their order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "i8_epilogue.h"
#include "kernels_i8.h"

namespace dtg {
namespace {

using namespace dev;

struct __attribute__((packed, aligned(1))) Loose16 {
    u32x4 v;
};

constexpr int kTile = 64, kStep = 128, kThreads = 256;
constexpr int kChunks = kStep / 16;                                // to a row
constexpr int kLoads = kTile * kChunks / kThreads;                 // of an operand, to a thread
constexpr int kStage = kTile * kStep;                              // bytes of an operand

template <int OUT>
__global__ __launch_bounds__(kThreads) void i8_any_kernel(I8RowsArgs a, int tiles_n) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * 2 * kStage];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int64_t tile = blockIdx.x;
    const int m0 = static_cast<int>(tile / tiles_n) * kTile, n0 = static_cast<int>(tile % tiles_n) * kTile;
    const int K = a.K;

    const int8_t* src[2][kLoads];
    int at[kLoads], lds[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int q = tid + i * kThreads, row = q / kChunks, c = q % kChunks;
        const int m = m0 + row < a.M ? m0 + row : a.M - 1, n = n0 + row < a.N ? n0 + row : a.N - 1;
        src[0][i] = a.X + static_cast<int64_t>(m) * a.lx;
        src[1][i] = a.W + static_cast<int64_t>(n) * a.lw;
        at[i] = 16 * c;
        lds[i] = row * kStep + 16 * (c ^ swz<kChunks>(row));
    }
    u32x4 reg[2][kLoads];
    auto load = [&](int k0) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int k = k0 + at[i];
                u32x4 v = {0u, 0u, 0u, 0u};
                if (k + 16 <= K) {
                    v = reinterpret_cast<const Loose16*>(src[o][i] + k)->v;
                } else if (k < K) {
#pragma unroll
                    for (int e = 0; e < 15; ++e)
                        if (k + e < K) v[e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(src[o][i][k + e])) << (8 * (e % 4));
                }
                reg[o][i] = v;
            }
    };
    auto store = [&](int s) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(smem + (2 * s + o) * kStage + lds[i]) = reg[o][i];
    };

    f32x4 acc[2][2];   // int32 bits; [m block][n block], a lane: one m, four n
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int steps = (K + kStep - 1) / kStep;
    if (steps > 0) load(0);
    for (int s = 0; s < steps; ++s) {
        store(s & 1);
        if (s + 1 < steps) load((s + 1) * kStep);
        __syncthreads();   // the readers of this stage two steps ago passed the previous barrier
        const uint8_t *x = smem + 2 * (s & 1) * kStage, *w = x + kStage;
#pragma unroll
        for (int ks = 0; ks < kStep / 64; ++ks) {
            u32x4 fx[2], fw[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 4 * ks + (lane >> 4), rx = wm * 32 + i * 16 + (lane & 15), rw = wn * 32 + i * 16 + (lane & 15);
                fx[i] = *reinterpret_cast<const u32x4*>(x + rx * kStep + 16 * (c ^ swz<kChunks>(rx)));
                fw[i] = *reinterpret_cast<const u32x4*>(w + rw * kStep + 16 * (c ^ swz<kChunks>(rw)));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma_i8<16>(fw[j], fx[i], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = m0 + wm * 32 + i * 16 + (lane & 15);
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            store_scaled<OUT>(a, m, n0 + wn * 32 + j * 16 + 4 * (lane >> 4), acc[i][j]);
    }
}

}  // namespace

hipError_t launch_i8_any(const I8RowsArgs& a, int out, hipStream_t stream) {
    const int64_t tm = (static_cast<int64_t>(a.M) + kTile - 1) / kTile, tn = (static_cast<int64_t>(a.N) + kTile - 1) / kTile;
    const dim3 grid(static_cast<unsigned>(tm * tn)), block(kThreads);
    const int n = static_cast<int>(tn);
    if (out == kOutF32) hipLaunchKernelGGL((i8_any_kernel<kOutF32>), grid, block, 0, stream, a, n);
    else if (out == kOutBF16) hipLaunchKernelGGL((i8_any_kernel<kOutBF16>), grid, block, 0, stream, a, n);
    else hipLaunchKernelGGL((i8_any_kernel<kOutF16>), grid, block, 0, stream, a, n);
    return hipGetLastError();
}

}  // namespace dtg
