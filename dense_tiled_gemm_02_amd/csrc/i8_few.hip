// int8 products with scales where 64 x 64 tiles would leave most of the card
// empty: few rows (a token to a decode batch), or little of everything.
// Y = (X W^T) sx sw + b, bound by streaming W: 16 x 8192 x 8192 12.6 us, 5.3 TB/s.
//
// A workgroup owns 16 NB columns of 16 MB rows; its WV waves take the units of
// KB k in turn.  Each wave brings its units of W (16 NB rows) and of X through a
// ring of ST stages in LDS that no other wave touches: direct loads, waited for
// by count, no barrier in the loop.  A load instruction fills 1 KB of LDS with
// runs of KB bytes of each row, its 16-byte chunks placed so that the operand
// reads have no bank conflicts.  W is the instruction's first operand, so a lane
// ends with four consecutive columns of one row.  The waves' exact int32 sums
// meet in LDS at the end.
//
// Rows past M and N and chunks past K load as zeros (an offset past any range).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "i8_epilogue.h"
#include "kernels_i8.h"

namespace dtg {
namespace {

using namespace dev;

template <int MB, int NB, int KB, int ST, int XI, int WV, int OUT>
__device__ __forceinline__ void few_tile(const I8RowsArgs& a) {
    constexpr int CH = KB / 16, R = 64 / CH;          // chunks of a row, rows of a load
    constexpr int WI = 16 * NB / R, L = WI + XI;      // loads of a unit
    constexpr int KS = KB / 64;                       // instructions along a unit
    static_assert(XI * R == 16 * MB, "rows of X");
    constexpr int STAGE = 16 * (NB + MB) * KB;         // bytes; X behind W
    static_assert(L * (ST - 1) < 64, "loads in flight");
    static_assert(WV * MB * NB * 1024 <= WV * ST * STAGE, "the sums fit in the ring");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[WV * ST * STAGE];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = static_cast<int>(blockIdx.x) * 16 * NB, m0 = static_cast<int>(blockIdx.y) * 16 * MB, K = a.K;
    const int rows_x = a.M - m0 < 16 * MB ? a.M - m0 : 16 * MB;
    uint8_t* const mine = ring + wave * ST * STAGE;

    const int64_t w_first = static_cast<int64_t>(n0) * a.lw;
    const int rows_w = a.N - n0 < 16 * NB ? a.N - n0 : 16 * NB;
    __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(a.W + w_first), 0, clamp_records(static_cast<int64_t>(rows_w - 1) * a.lw + K), kRsrcWord3);
    __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(a.X + static_cast<int64_t>(m0) * a.lx), 0,
        clamp_records(static_cast<int64_t>(rows_x - 1) * a.lx + K), kRsrcWord3);
    uint32_t off[L];
    int k_of[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int row = (i < WI ? i : i - WI) * R + lane / CH;
        const int c = (lane % CH) ^ swz<CH>(row);
        k_of[i] = 16 * c;
        const bool in = row < (i < WI ? rows_w : rows_x);
        off[i] = in ? static_cast<uint32_t>(row * (i < WI ? a.lw : a.lx) + 16 * c) : kOOB;
    }
    const int units = (K + KB - 1) / KB;
    const int mine_units = units > wave ? (units - wave + WV - 1) / WV : 0;
    // Each workgroup starts elsewhere along k: rows a power of two apart would
    // otherwise all be read at one offset, from a few of the memory's channels.
    const int turn = mine_units > 0 ? static_cast<int>(blockIdx.x) % mine_units : 0;
    auto issue = [&](int i) {   // this wave's unit i (past the last one: zeros)
        const int u = i + turn < mine_units ? i + turn : i + turn - mine_units;
        const int k0 = i < mine_units ? (wave + u * WV) * KB : K;
        const int so = k0 < K ? k0 : 0;
        uint8_t* const stage = mine + (i % ST) * STAGE;
        __amdgpu_buffer_rsrc_t w = rw, x = rx;
#pragma unroll
        for (int l = 0; l < WI; ++l)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(w, (lds_void_t*)(stage + l * 1024), 16,
                                                     off[l] | (k0 + k_of[l] < K ? 0u : kOOB), so, 0, kNonTemporal);
#pragma unroll
        for (int l = WI; l < L; ++l)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x, (lds_void_t*)(stage + l * 1024), 16,
                                                     off[l] | (k0 + k_of[l] < K ? 0u : kOOB), so, 0, 0);
    };

    f32x4 acc[MB][NB];   // int32 bits
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // operand reads: row l % 16 of a block, chunk 4 ks + l / 16
    const uint32_t base = lds_addr(reinterpret_cast<const uint16_t*>(mine));
    uint32_t chunk[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) chunk[ks] = (lane & 15) * KB + 16 * ((4 * ks + (lane >> 4)) ^ swz<CH>(lane & 15));

    if (mine_units > 0) {
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) issue(i);
        for (int i = 0; i < mine_units; ++i) {
            // the stage that this fills was read, and waited for, in the round before
            issue(i + ST - 1);
            asm volatile("" ::: "memory");
            wait_vm<(ST - 1) * L>();
            asm volatile("" ::: "memory");
            const uint32_t at = base + (i % ST) * STAGE;
            u32x4 fw[KS][NB], fx[KS][MB];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                static_for<NB>([&](auto j) { fw[ks][j] = lds_read16<decltype(j)::value * 16 * KB>(at + chunk[ks]); });
                static_for<MB>([&](auto j) { fx[ks][j] = lds_read16<(NB + decltype(j)::value) * 16 * KB>(at + chunk[ks]); });
            }
            lds_wait_all();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                for (int j = 0; j < NB; ++j) tie(fw[ks][j]);
#pragma unroll
                for (int j = 0; j < MB; ++j) tie(fx[ks][j]);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int n = 0; n < NB; ++n) acc[m][n] = mfma_i8<16>(fw[ks][n], fx[ks][m], acc[m][n]);
        }
        wait_vm<0>();   // nothing may still be written to LDS
    }
    __syncthreads();
    f32x4* const sums = reinterpret_cast<f32x4*>(ring);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n) sums[((m * NB + n) * WV + wave) * 64 + lane] = acc[m][n];
    __syncthreads();
    for (int b = wave; b < MB * NB; b += WV) {
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        i32x4 s = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WV; ++w) s += __builtin_bit_cast(i32x4, sums[(b * WV + w) * 64 + lane]);
        const int m = m0 + b / NB * 16 + (lane & 15);
        if (m < a.M) store_scaled<OUT>(a, m, n0 + b % NB * 16 + 4 * (lane >> 4), __builtin_bit_cast(f32x4, s));
    }
}

template <int MB, int NB, int KB, int ST, int XI, int WV, int OUT>
__global__ __launch_bounds__(64 * WV) void i8_few_kernel(I8RowsArgs a) {
    few_tile<MB, NB, KB, ST, XI, WV, OUT>(a);
}

template <int MB, int NB, int KB, int ST, int XI, int WV, int OUT>
hipError_t launch(const I8RowsArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((i8_few_kernel<MB, NB, KB, ST, XI, WV, OUT>), dim3(static_cast<unsigned>((a.N + 16 * NB - 1) / (16 * NB)),
                       static_cast<unsigned>((a.M + 16 * MB - 1) / (16 * MB))), dim3(64 * WV), 0, stream, a);
    return hipGetLastError();
}

#define DTG_STR2(x) #x
#define DTG_STR(x) DTG_STR2(x)
#define FEW(MB, NB, KB, ST, XI, WV)                                                                                     \
    {MB, NB,                                                                                                             \
     {&launch<MB, NB, KB, ST, XI, WV, kOutF16>, &launch<MB, NB, KB, ST, XI, WV, kOutBF16>,                               \
      &launch<MB, NB, KB, ST, XI, WV, kOutF32>},                                                                         \
     "i8_few_kernel<" DTG_STR(MB) "," DTG_STR(NB) "," DTG_STR(KB) "," DTG_STR(ST) "," DTG_STR(XI) "," DTG_STR(WV) ">"}

// Waves, stages and runs by measurement over 12 shapes, W from memory (us):
//   16 x 16   16 waves, 2 stages  1 x 4096 x 4096 5.7 (4 waves, 6 stages of 128: 6.2)
//   16 x 32   4 waves, 3 stages   16 x 8192 x 8192 12.6 (8 waves, 2 stages: 15.9)
//   16 x 64   4 waves, 3 stages   16 x 11008 x 4096 10.8 (8 waves, 2 stages: 11.0)
//   32 x 32   4 waves, 2 stages   32 x 8192 x 8192 14.1 (8 waves, 2 stages: 17.1)
//   32 x 64, 64 x 32  the same    32 x 14336 x 4096 13.3, 64 x 8192 x 8192 18.0
const I8FewEntry kTable[] = {
    FEW(1, 1, 128, 2, 2, 16),
    FEW(1, 2, 128, 3, 2, 4),
    FEW(1, 4, 128, 3, 2, 4),
    FEW(2, 2, 128, 2, 4, 4),
    FEW(2, 4, 128, 2, 4, 4),
    FEW(4, 2, 128, 2, 8, 4),
};

}  // namespace

const I8FewEntry* i8_few_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
