// int8 products with scales, Y = (X W^T) sx sw + b, for operands that the
// direct-to-LDS kernels do not take: K, row strides or bases that are no
// multiples of 16 bytes.
//
// 64 x 64 or 128 x 128 outputs to a workgroup, 128 k a step.  Every chunk of 16 k is one load
// at its own address, whatever that is, through registers one step ahead into one
// of two LDS stages.  Rows past the operands read the last row, and what they make
// is not stored.  Where the tiles are at most one to a CU KG groups of four waves
// take the steps in turn, each with its own stages, and their sums meet in LDS.
// The sums are exact (int32), so nothing depends on their order.
//
// Bound by the loads of single bytes' alignment, which take a CU 49 cycles each
// where aligned ones take 26 (512 k of a tile 1.5 and 0.8 us): 777 x 1003 x 2005 12.7
// us, with rows of whole words (K = 2004) 11.2.  Whole words around each chunk, shifted
// in registers, cost as much (1.02 times the time, and 1.2 times for whole words).  Two
// or three steps ahead: 1.03 and 1.13 times the time of one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "i8_epilogue.h"
#include "kernels_i8.h"
#include "tile_order.h"

namespace dtg {
namespace {

using namespace dev;

struct __attribute__((packed, aligned(1))) Loose16 {
    u32x4 v;
};

constexpr int kStep = 128, kThreads = 256;
constexpr int kChunks = kStep / 16;   // to a row

// Where a workgroup's tile lies (tile_order.h): a die's tiles next to one another,
// in bands of kBand rows of tiles (4096 x 4097 x 4095 of equal values, 64 x 64 tiles:
// 183 us in plain order, bands of 1, 4, 8, 16 rows 171, 136, 131, 139).
constexpr int kBand = 8;
struct Order {
    int tiles_m, tiles_n, group_m, xcds;
};

// Tiles of 32 TB rows and columns; a wave has TB x TB blocks of 16 x 16.
template <int TB, int KG, int OUT>
__global__ __launch_bounds__(KG * kThreads) void i8_any_kernel(I8RowsArgs a, Order order) {
    constexpr int kTile = 32 * TB;
    constexpr int kLoads = kTile * kChunks / kThreads;   // of an operand, to a thread
    constexpr int kStage = kTile * kStep;                // bytes of an operand
    static_assert(KG == 1 || TB == 2, "the groups' sums are four blocks a wave");
    __shared__ __attribute__((aligned(16))) uint8_t all[KG * 2 * 2 * kStage];
    const int group = threadIdx.x / kThreads;   // whole waves
    const int tid = threadIdx.x % kThreads, lane = tid & 63, wave = tid >> 6;
    uint8_t* const smem = all + group * 2 * 2 * kStage;
    const int wm = wave >> 1, wn = wave & 1;
    int pm, pn;
    grouped_tile<int>(xcd_permute<int>(blockIdx.x, gridDim.x, order.xcds), order.tiles_m, order.tiles_n, order.group_m, &pm, &pn);
    const int m0 = pm * kTile, n0 = pn * kTile;
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
    // A chunk that K cuts is the row's last 16 bytes, moved down when it is staged;
    // one past K is those, moved out.  (Loads under a condition would wait for one
    // another: 1.2 times the time at 777 x 1003 x 2005.)
    u32x4 reg[2][kLoads];
    auto load = [&](int k0) {
        if (K >= 16) {
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int k = k0 + at[i];
                    reg[o][i] = reinterpret_cast<const Loose16*>(src[o][i] + (k + 16 <= K ? k : K - 16))->v;
                }
        } else {   // one step of one chunk
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    uint64_t lo = 0, hi = 0;
#pragma unroll 1
                    for (int e = 0; e < K; ++e) {
                        const uint64_t c = k0 + at[i] == 0 ? static_cast<uint8_t>(src[o][i][e]) : 0;
                        (e < 8 ? lo : hi) |= c << (8 * (e & 7));
                    }
                    const u32x4 v = {static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                                     static_cast<uint32_t>(hi >> 32)};
                    reg[o][i] = v;
                }
        }
    };
    auto store = [&](int s, int k0) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                u32x4 v = reg[o][i];
                if (k0 + kStep > K && K >= 16) {
                    const int over = k0 + at[i] + 16 - K, sh = 8 * over;   // bits to move down
                    const uint64_t lo = v[0] | static_cast<uint64_t>(v[1]) << 32, hi = v[2] | static_cast<uint64_t>(v[3]) << 32;
                    const uint64_t up = over >= 16 ? 0 : hi >> (sh & 63);
                    const uint64_t down = over >= 8 ? up : (lo >> (sh & 63)) | (hi << 1 << (63 - (sh & 63)));
                    const uint64_t l = over <= 0 ? lo : down, h = over <= 0 ? hi : over >= 8 ? 0 : up;
                    v = u32x4{static_cast<uint32_t>(l), static_cast<uint32_t>(l >> 32), static_cast<uint32_t>(h),
                              static_cast<uint32_t>(h >> 32)};
                }
                *reinterpret_cast<u32x4*>(smem + (2 * s + o) * kStage + lds[i]) = v;
            }
    };

    f32x4 acc[TB][TB];   // int32 bits; [m block][n block], a lane: one m, four n
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // of every group as many: steps past K are zeros
    const int steps = ((K + kStep - 1) / kStep + KG - 1) / KG;
    if (steps > 0) load(group * kStep);
    for (int s = 0; s < steps; ++s) {
        store(s & 1, (s * KG + group) * kStep);
        if (s + 1 < steps) load(((s + 1) * KG + group) * kStep);
        __syncthreads();   // the readers of this stage two steps ago passed the previous barrier
        const uint8_t *x = smem + 2 * (s & 1) * kStage, *w = x + kStage;
#pragma unroll
        for (int ks = 0; ks < kStep / 64; ++ks) {
            u32x4 fx[TB], fw[TB];
#pragma unroll
            for (int i = 0; i < TB; ++i) {
                const int c = 4 * ks + (lane >> 4), rx = (wm * TB + i) * 16 + (lane & 15), rw = (wn * TB + i) * 16 + (lane & 15);
                fx[i] = *reinterpret_cast<const u32x4*>(x + rx * kStep + 16 * (c ^ swz<kChunks>(rx)));
                fw[i] = *reinterpret_cast<const u32x4*>(w + rw * kStep + 16 * (c ^ swz<kChunks>(rw)));
            }
#pragma unroll
            for (int i = 0; i < TB; ++i)
#pragma unroll
                for (int j = 0; j < TB; ++j) acc[i][j] = mfma_i8<16>(fw[j], fx[i], acc[i][j]);
        }
    }
    if constexpr (KG > 1) {
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        i32x4* const sums = reinterpret_cast<i32x4*>(all);
        __syncthreads();   // every group is past its last operand reads
        if (group > 0) {
#pragma unroll
            for (int b = 0; b < 4; ++b) sums[((group - 1) * 4 + b) * kThreads + tid] = __builtin_bit_cast(i32x4, acc[b / 2][b % 2]);
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            i32x4 v = __builtin_bit_cast(i32x4, acc[b / 2][b % 2]);
#pragma unroll
            for (int g = 0; g < KG - 1; ++g) v += sums[(g * 4 + b) * kThreads + tid];
            acc[b / 2][b % 2] = __builtin_bit_cast(f32x4, v);
        }
    }
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        const int m = m0 + (wm * TB + i) * 16 + (lane & 15);
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < TB; ++j)
            store_scaled<OUT>(a, m, n0 + (wn * TB + j) * 16 + 4 * (lane >> 4), acc[i][j]);
    }
}

template <int TB, int KG>
hipError_t launch(const I8RowsArgs& a, int out, int xcds, hipStream_t stream) {
    const Order order = {static_cast<int>((static_cast<int64_t>(a.M) + 32 * TB - 1) / (32 * TB)),
                         static_cast<int>((static_cast<int64_t>(a.N) + 32 * TB - 1) / (32 * TB)), kBand, xcds};
    const dim3 grid(static_cast<unsigned>(order.tiles_m) * order.tiles_n), block(KG * kThreads);
    if (out == kOutF32) hipLaunchKernelGGL((i8_any_kernel<TB, KG, kOutF32>), grid, block, 0, stream, a, order);
    else if (out == kOutBF16) hipLaunchKernelGGL((i8_any_kernel<TB, KG, kOutBF16>), grid, block, 0, stream, a, order);
    else hipLaunchKernelGGL((i8_any_kernel<TB, KG, kOutF16>), grid, block, 0, stream, a, order);
    return hipGetLastError();
}

}  // namespace

// us of 64 x 64 tiles with four groups and with one, and of 128 x 128, rows at any byte:
//   1000 x 1000 x 1000   7.9, 7.8, 17.0   (256 of the small tiles, 64 of the large)
//   777 x 1003 x 2005    12.7, 14.0, 30   (208, 56)
//   300 x 4097 x 4095    36, 30, 47       (325, 99)
//   20000 x 100 x 4095   53, 45, 45       (626, 157)
//   128 x 28001 x 4095   90, 79, 55       (876, 219)
//   4096 x 4097 x 4095   282, 222, 176    (4160, 1056)
//   5000 x 5000 x 300    123, 44, 53      (6241, 1600)
int i8_any_tile(int64_t M, int64_t N, int cus) {
    return 4 * ((M + 127) / 128) * ((N + 127) / 128) < 3 * static_cast<int64_t>(cus) ? 64 : 128;
}

hipError_t launch_i8_any(const I8RowsArgs& a, int out, int cus, int xcds, hipStream_t stream) {
    if (i8_any_tile(a.M, a.N, cus) == 128) return launch<4, 1>(a, out, xcds, stream);
    const int64_t tiles = (static_cast<int64_t>(a.M) + 63) / 64 * ((static_cast<int64_t>(a.N) + 63) / 64);
    return tiles <= cus ? launch<2, 4>(a, out, xcds, stream) : launch<2, 1>(a, out, xcds, stream);
}

}  // namespace dtg
