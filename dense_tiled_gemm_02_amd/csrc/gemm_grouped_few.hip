// The grouped product for few rows per group (a decode batch through unquantized
// experts): B[g] is streamed once and K is what there is to spread.
//
// A workgroup computes BM (16 or 64) rows x BN columns of one group; its NWV waves take
// the 32-k chunks of K in turn, each through a private ST-stage LDS ring filled
// by direct loads (the layouts of the direct tiles, OpShape), so no barrier is
// needed until the waves' sums meet in LDS, added in wave order.  Bound by
// latency, about 0.35 us per chunk of a wave and 3 us around them: 16 x 1024 x
// 512 over 8 groups 5.2 us (64 x 64 tiles with one K loop 7.0), 4 x 3880 x 136
// over 19 groups 8.8 us (16.9), 1 x 4096 x 4096 10.5 us (17.7); with 64 rows 46 x
// 2184 x 736 over 2 groups 7.9 us (11.3), 375 x 3384 x 400 over 8 16.9 us (18.8;
// 16-row tiles read B[g] three times).  64 rows and 64 columns leave LDS for four
// waves with four stages.  A deeper ring (6
// stages) starts later and gains nothing; non-temporal loads of B, which the
// next step's call reads again, cost 1 x 4096 x 4096 6 us.
#include "grouped_kernel.h"

namespace dtg {
namespace {

template <int BM, int BN, int NWV, int ST, bool BF16, bool TB>
__device__ __forceinline__ void few_tile(const KArgs& p, int pid_m, int pid_n) {
    constexpr int CK = 32, FM = BM / 16, FN = BN / 16;
    typedef OpShape<true, BM, CK, 1> OA;
    typedef OpShape<TB, BN, CK, 1> OB;
    constexpr int STG = OA::SZ + OB::SZ, OPS = OA::IW + OB::IW;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[NWV * ST * STG];
    static_assert(NWV * BM * BN * 4 <= NWV * ST * STG * 2, "the waves' sums go over the ring");

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = pid_m * BM, n0 = pid_n * BN;
    const int M = p.M, N = p.N, K = p.K;
    const int64_t lda = p.lda, ldb = TB ? p.sbn : p.ldb;

    // Per-lane load offsets, as the direct tiles have them: rows past an operand
    // lie past its descriptor, chunks past K or N get an offset past any range.
    uint32_t a_voff[OA::IW], b_voff[OB::IW];
    int a_k[OA::IW], b_k[OB::IW];
#pragma unroll
    for (int i = 0; i < OA::IW; ++i) {
        const int row = i * OA::R + lane / OA::CH, c = (lane % OA::CH) ^ OA::sw(row);
        a_voff[i] = static_cast<uint32_t>(row * lda * 2 + c * 16);
        a_k[i] = 8 * c;
    }
#pragma unroll
    for (int i = 0; i < OB::IW; ++i) {
        const int row = i * OB::R + lane / OB::CH, c = (lane % OB::CH) ^ OB::sw(row);
        b_voff[i] = static_cast<uint32_t>(row * ldb * 2 + c * 16);
        if (!TB && n0 + 8 * c >= N) b_voff[i] = kOOB;
        b_k[i] = TB ? 8 * c : 0;
    }
    const uint64_t a_full = 2u * static_cast<uint64_t>(static_cast<int64_t>(M - 1 - m0) * lda + K);
    const uint64_t b_full = 2u * static_cast<uint64_t>(TB ? static_cast<int64_t>(N - 1 - n0) * ldb + K
                                                          : static_cast<int64_t>(K - 1) * ldb + (N - n0));
    const uint16_t* const a_tile = p.A + static_cast<int64_t>(m0) * lda;
    const uint16_t* const b_tile = TB ? p.B + static_cast<int64_t>(n0) * ldb : p.B + n0;
    uint16_t* const ring = smem + wave * ST * STG;
    const int chunks = (K + CK - 1) / CK;
    auto issue = [&](int c, int slot) {
        const bool live = c < chunks;   // past the last one: empty ranges, so that the waits stay uniform
        const int k0 = live ? c * CK : 0;
        const int64_t boff = TB ? k0 : static_cast<int64_t>(k0) * ldb;
        __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(a_tile + k0), 0, live ? capped_records(a_full, 2u * static_cast<uint64_t>(k0)) : 0u,
            kRsrcWord3);
        __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(b_tile + boff), 0,
            live ? capped_records(b_full, 2u * static_cast<uint64_t>(boff)) : 0u, kRsrcWord3);
        uint16_t* const sa = ring + slot * STG;
#pragma unroll
        for (int i = 0; i < OB::IW; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t*)(sa + OA::SZ + i * 512), 16,
                                                     b_voff[i] | (k0 + b_k[i] < K ? 0u : kOOB), 0, 0, 0);
#pragma unroll
        for (int i = 0; i < OA::IW; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(sa + i * 512), 16,
                                                     a_voff[i] | (k0 + a_k[i] < K ? 0u : kOOB), 0, 0, 0);
    };

    // operand addresses within a stage: 8 k of one row or column per lane
    const int r16 = lane & 15, g = lane >> 4;
    const uint32_t a_off = (r16 * CK + ((g ^ OA::sw(r16)) * 8)) * 2;   // + 16 rows per fragment: the swizzle repeats
    uint32_t b_off[FN][TB ? 1 : 2];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
        if constexpr (TB) {
            const int row = f * 16 + r16;
            b_off[f][0] = (OA::SZ + row * CK + ((g ^ OB::sw(row)) * 8)) * 2;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 8 * g + 4 * h + (r16 >> 2);
                b_off[f][h] = (OA::SZ + row * BN + (((2 * f) ^ OB::sw(row)) * 8) + 4 * (r16 & 3)) * 2;
            }
        }
    }

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < FN; ++f) acc[i][f] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t ring0 = lds_addr(ring);
    if (wave < chunks) {
#pragma unroll
        for (int s = 0; s < ST - 1; ++s) issue(wave + s * NWV, s);
        int slot = 0;
        for (int c = wave; c < chunks; c += NWV) {
            wait_vm<(ST - 2) * OPS>();
            issue(c + (ST - 1) * NWV, slot == 0 ? ST - 1 : slot - 1);
            const uint32_t at = ring0 + slot * (STG * 2);
            u32x4 fa[FM], fb[FN];
            static_for<FM>([&](auto i_tag) {
                constexpr int I = decltype(i_tag)::value;
                fa[I] = lds_read16<I * 16 * CK * 2>(at + a_off);
            });
            i16x4 h[FN][2];
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                if constexpr (TB) {
                    fb[f] = lds_read16<0>(at + b_off[f][0]);
                } else {
                    h[f][0] = lds_read_tr<0>(at + b_off[f][0]);
                    h[f][1] = lds_read_tr<0>(at + b_off[f][1]);
                }
            }
            lds_wait_all();
#pragma unroll
            for (int i = 0; i < FM; ++i) tie(fa[i]);
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                if constexpr (!TB) {
                    tie(h[f][0]);
                    tie(h[f][1]);
                    fb[f] = __builtin_bit_cast(u32x4, __builtin_shufflevector(h[f][0], h[f][1], 0, 1, 2, 3, 4, 5, 6, 7));
                }
                tie(fb[f]);
#pragma unroll
                for (int i = 0; i < FM; ++i) acc[i][f] = mfma<16, BF16>(fa[i], fb[f], acc[i][f]);
            }
            slot = slot + 1 == ST ? 0 : slot + 1;
        }
        wait_vm<0>();   // no load may still be writing the ring
    }

    // ---- the waves' sums in wave order, rounded once
    __syncthreads();
    float* const red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[(wave * BM + 16 * i + 4 * g + r) * BN + f * 16 + r16] = acc[i][f][r];
    __syncthreads();
    for (int t = tid; t < BM * BN; t += 64 * NWV) {
        const int row = t / BN, col = t % BN;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < NWV; ++w) v += red[w * BM * BN + t];
        if (m0 + row < M && n0 + col < N) p.D[static_cast<int64_t>(m0 + row) * p.ldd + n0 + col] = narrow<BF16>(v);
    }
}

template <int BM, int BN, int NWV, int ST, bool BF16, bool TB>
__global__ __launch_bounds__(64 * NWV) void gemm_grouped_rows_few_kernel(GroupedArgs a, int most) {
    // at most one workgroup per CU, taking tiles in turn: most of the tiles that
    // a table could need are not there (8 x 2048 x 1024 over 64 groups: 256 of
    // 2112, 17 us with a workgroup for each, 11 us so)
    for (int wg = blockIdx.x;; wg += gridDim.x) {
        RowTile t;
        if (!find_row_tile<BM>(a, &t, wg)) return;
        const KArgs p = row_args(a, t);
        int pid_m, pid_n;
        grouped_tile<int>(t.tile, p.num_pid_m, p.num_pid_n, p.group_m, &pid_m, &pid_n);
        few_tile<BM, BN, NWV, ST, BF16, TB>(p, pid_m, pid_n);
        if (wg + static_cast<int>(gridDim.x) >= most) return;   // the table need not be asked
        __syncthreads();   // the sums are read; the ring is free
    }
}

template <int BM, int BN, int NWV, int ST, bool BF16, bool TB>
hipError_t launch_few(const GroupedArgs& a, int64_t grid, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_grouped_rows_few_kernel<BM, BN, NWV, ST, BF16, TB>), dim3(static_cast<unsigned>(grid < a.cus ? grid : a.cus)),
                       dim3(64 * NWV), 0, stream, a, static_cast<int>(grid));
    return hipGetLastError();
}

#define FEW_ENTRY(BM, BN, NWV, ST, BF, TB)                                                                    \
    {kGroupedRows, BM, BN, 32, ST, 16, 1, NWV, BF, kGroupedDirect, TB, 0, 64 * NWV,                           \
     static_cast<int64_t>(NWV) * ST * (BM + BN) * 32 * 2, &launch_few<BM, BN, NWV, ST, (BF != 0), (TB != 0)>,  \
     "gemm_grouped_rows_few_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(NWV) "," DTG_STR(ST) "," DTG_STR(BF) "," \
     DTG_STR(TB) ">"}

// k-contiguous B: 32 columns, twice the workgroups; row-major B: 64 (the
// transposing reads' layout needs 128-byte rows)
const GroupedEntry kTable[] = {
    FEW_ENTRY(16, 32, 8, 4, 0, 1), FEW_ENTRY(16, 32, 8, 4, 1, 1),
    FEW_ENTRY(16, 64, 8, 3, 0, 0), FEW_ENTRY(16, 64, 8, 3, 1, 0),
    FEW_ENTRY(64, 32, 8, 3, 0, 1), FEW_ENTRY(64, 32, 8, 3, 1, 1),
    FEW_ENTRY(64, 64, 4, 4, 0, 0), FEW_ENTRY(64, 64, 4, 4, 1, 0),
};

}  // namespace

const GroupedEntry* grouped_few_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
