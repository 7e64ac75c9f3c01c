// Matrix-vector product with 4-bit weights and group scales for gfx950:
//
//     Y[m, n] = sum over groups j of s[n, j] * sum over k in j of X[m, k] (q[n, k] - z[n, j])
//
// for a few rows m (one token to a small decode batch), or for rows that each
// pick one of several experts' matrices.  Bound by streaming W.
//
// The weights never become floating-point values of their own.  A nibble q
// OR'd into the mantissa of 16.0 is the exact value 16 + q in both storage
// types (bf16 0x4180 | q << 3, fp16 0x4C00 | q << 6), one shift and one
// and-or for two weights, so the matrix instruction takes X and 16 + q, and
//
//     sum X (q - z) = sum X (16 + q) - (16 + z) sum X,
//
// the second sum from the same instruction against ones (its result lands in
// the same lanes and registers).  Both sums are fp32 and the group's scale is
// applied to their difference in fp32; the offset of 16 costs at most
// 31/|q - z| times the rounding of an fp32 sum, 2^-24 of sum |X| per step.  An
// output that comes out infinite or NaN (an infinity in X makes both sums
// infinite) is summed again term by term.
//
// A wave takes 128 k at a time of 16 NB rows of W: each lane one 16-byte load
// per 16 rows (row l mod 16, k 32 (l / 16) .. + 31), non-temporal, U chunks
// ahead in registers.  The order of k inside the instruction is free as long
// as X follows it, so with groups of 128 a lane's four dwords are simply four
// instructions; for groups of 64 or 32 the dwords are first exchanged between
// the wave's halves (and quarters) so that every instruction stays inside one
// group.  The waves of a workgroup take the chunks in turn and their sums are
// added through LDS in wave order, so a call's result does not depend on timing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "kernels_w4.h"

namespace dtg {
namespace {

using namespace dev;

constexpr int kListRows = 1024;   // rows gathered per pass over the expert ids

// Nibbles r and r + 4 of w as the pair (16 + q_r, 16 + q_{r + 4}).
template <bool BF16, int R>
__device__ __forceinline__ uint32_t offset_pair(uint32_t w) {
    constexpr int to = BF16 ? 3 : 6;                    // lowest mantissa bit of the units place
    constexpr int sh = 4 * R - to;
    const uint32_t v = sh > 0 ? w >> (sh > 0 ? sh : 0) : w << (sh < 0 ? -sh : 0);
    return (v & (0x000F000Fu << to)) | (BF16 ? 0x41804180u : 0x4C004C00u);
}

// X's 8 consecutive k in the nibbles' pair order: (k, k + 4) for k = 0..3.
__device__ __forceinline__ u32x4 pair_order(u32x4 x) {
    return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100), __builtin_amdgcn_perm(x[2], x[0], 0x07060302),
                 __builtin_amdgcn_perm(x[3], x[1], 0x05040100), __builtin_amdgcn_perm(x[3], x[1], 0x07060302)};
}

__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap_quarters(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// First k (within a chunk of 128) of the 8 that lane quarter g feeds to
// instruction t.
template <int G>
__device__ __forceinline__ int step_k(int t, int g) {
    if constexpr (G == 128) return 32 * g + 8 * t;
    else if constexpr (G == 64) return 64 * (t >> 1) + 8 * (t & 1) + 32 * (g & 1) + 16 * (g >> 1);
    else return 32 * t + 8 * g;
}

// The sum of one output by the formula, term by term in fp32: for outputs
// that the offset form leaves infinite or NaN.
template <int G, bool BF16, bool ZP>
__device__ __noinline__ float plain_sum(const uint16_t* x, const uint8_t* w, const uint16_t* s, const uint8_t* z,
                                        int K) {
    float y = 0.0f;
    for (int k0 = 0; k0 < K; k0 += G) {
        const float zero = ZP ? static_cast<float>(z[k0 / G]) : 8.0f;
        float t = 0.0f;
        for (int k = k0; k < k0 + G && k < K; ++k) {
            const int q = (w[k >> 1] >> (4 * (k & 1))) & 15;
            t += widen<BF16>(x[k]) * (static_cast<float>(q) - zero);
        }
        y += widen<BF16>(s[k0 / G]) * t;
    }
    return y;
}

template <int NB, int MB, int NWV, int G, bool BF16, bool ZP>
__global__ __launch_bounds__(64 * NWV) void gemm_w4_kernel(W4Args a) {
    constexpr int NG = 128 / G;                          // groups per chunk
    constexpr int U = NB * MB == 1 ? 4 : 2;               // chunks in flight
    constexpr int ROWS = 16 * MB;
    __shared__ float red[NWV * NB * MB * 256];
    __shared__ int list[kListRows];
    __shared__ int listed;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4;
    const int e = blockIdx.y;
    const int n0 = blockIdx.x * (16 * NB);
    const int M = a.M, N = a.N, K = a.K;
    const uint8_t* const W = a.W + static_cast<int64_t>(e) * a.sw_e;
    const uint16_t* const S = a.S + static_cast<int64_t>(e) * a.ss_e;
    const uint8_t* const Z = ZP ? a.Z + static_cast<int64_t>(e) * a.sz_e : nullptr;

    // this lane's columns (those past N repeat the last one and are not stored)
    const uint8_t* wrow[NB];
    const uint16_t* srow[NB];
    const uint8_t* zrow[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int n = n0 + 16 * j + (lane & 15);
        const int64_t nc = n < N ? n : N - 1;
        wrow[j] = W + nc * a.sw_n + 16 * g;
        srow[j] = S + nc * a.ss_n;
        zrow[j] = ZP ? Z + nc * a.sz_n : nullptr;
    }
    const int full = K / 128;

    u32x4 ones;
#pragma unroll
    for (int r = 0; r < 4; ++r) ones[r] = BF16 ? 0x3F803F80u : 0x3C003C00u;

    for (int first = 0; first < M; first += kListRows) {
        // ---- the rows of this pass
        int rows;
        if (a.experts) {
            if (first > 0) __syncthreads();
            if (wave == 0) {
                int n = 0;
                const int end = first + kListRows < M ? first + kListRows : M;
                for (int r = first; r < end; r += 64) {
                    const int row = r + lane;
                    int64_t id = -1;
                    if (row < end)
                        id = a.id_bytes == 8 ? static_cast<const int64_t*>(a.experts)[row]
                                             : static_cast<const int32_t*>(a.experts)[row];
                    const bool mine = row < end && id == e;
                    const uint64_t hits = __ballot(mine);
                    if (mine) list[n + __popcll(hits & ((uint64_t(1) << lane) - 1))] = row;
                    n += __popcll(hits);
                    // rows of no expert are zeros, written by the first expert's workgroups
                    if (e == 0 && row < end && (id < 0 || id >= a.num_experts))
                        for (int c = n0; c < n0 + 16 * NB && c < N; ++c)
                            a.Y[static_cast<int64_t>(row) * a.sy + c] = 0;
                }
                if (lane == 0) listed = n;
            }
            __syncthreads();
            rows = listed;
        } else {
            rows = M - first < kListRows ? M - first : kListRows;
        }
        auto row_of = [&](int i) { return a.experts ? list[i] : first + i; };

        for (int m0 = 0; m0 < rows; m0 += ROWS) {
            const uint16_t* xrow[MB];
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const int i = m0 + 16 * b + (lane & 15);
                xrow[b] = a.X + static_cast<int64_t>(row_of(i < rows ? i : rows - 1)) * a.sx;
            }

            f32x4 tot[MB][NB];
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int j = 0; j < NB; ++j) tot[b][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

            struct Chunk {
                u32x4 w[NB];
                u32x4 x[MB][4];
                uint16_t s[NB][NG];
                uint8_t z[NB][NG];
            };
            auto load = [&](Chunk& c, int chunk) {
                const int k0 = chunk * 128;
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    c.w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow[j] + k0 / 2));
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        c.x[b][t] = *reinterpret_cast<const u32x4*>(xrow[b] + k0 + step_k<G>(t, g));
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        c.s[j][i] = srow[j][chunk * NG + i];
                        if constexpr (ZP) c.z[j][i] = zrow[j][chunk * NG + i];
                    }
            };
            auto contract = [&](Chunk& c) {
                if constexpr (G < 128) {
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        uint32_t d0 = c.w[j][0], d1 = c.w[j][1], d2 = c.w[j][2], d3 = c.w[j][3];
                        swap_halves(d0, d2);
                        swap_halves(d1, d3);
                        if constexpr (G == 32) {
                            swap_quarters(d0, d1);
                            swap_quarters(d2, d3);
                        }
                        c.w[j] = u32x4{d0, d1, d2, d3};
                    }
                }
                f32x4 acc[MB][NB], sum[MB];
                static_for<4>([&](auto t_tag) {
                    constexpr int T = decltype(t_tag)::value;
                    constexpr int STEPS = G / 32;              // instructions per group
                    if constexpr (T % STEPS == 0) {
#pragma unroll
                        for (int b = 0; b < MB; ++b) {
                            sum[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int j = 0; j < NB; ++j) acc[b][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                        }
                    }
                    u32x4 wf[NB];
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const uint32_t w = c.w[j][T];
                        wf[j] = u32x4{offset_pair<BF16, 0>(w), offset_pair<BF16, 1>(w), offset_pair<BF16, 2>(w),
                                      offset_pair<BF16, 3>(w)};
                    }
#pragma unroll
                    for (int b = 0; b < MB; ++b) {
                        const u32x4 xf = pair_order(c.x[b][T]);
                        sum[b] = mfma<16, BF16>(xf, ones, sum[b]);
#pragma unroll
                        for (int j = 0; j < NB; ++j) acc[b][j] = mfma<16, BF16>(xf, wf[j], acc[b][j]);
                    }
                    if constexpr (T % STEPS == STEPS - 1) {
                        constexpr int I = T / STEPS;
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            const float sc = widen<BF16>(c.s[j][I]);
                            const float off = ZP ? 16.0f + static_cast<float>(c.z[j][I]) : 24.0f;
#pragma unroll
                            for (int b = 0; b < MB; ++b)
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    tot[b][j][r] += sc * (acc[b][j][r] - off * sum[b][r]);
                        }
                    }
                });
            };

            // whole chunks wave, wave + NWV, ...
            const int mine = full > wave ? (full - wave + NWV - 1) / NWV : 0;
            if (mine > 0) {
                Chunk c[U];
                auto at = [&](int i) { return wave + (i < mine ? i : mine - 1) * NWV; };
#pragma unroll
                for (int u = 0; u < U; ++u) load(c[u], at(u));
                for (int i = 0; i < mine; i += U) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (i + u < mine) {
                            contract(c[u]);
                            load(c[u], at(i + u + U));
                        }
                    }
                }
            }
            // the last K mod 128: one wave, lanes past K read the chunk's start and X as zeros
            if (K % 128 != 0 && wave == full % NWV) {
                Chunk c;
                const int k0 = full * 128;
                const bool in = k0 + 32 * g < K;
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    c.w[j] = *reinterpret_cast<const u32x4*>(wrow[j] + k0 / 2 - (in ? 0 : 16 * g));
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int k = k0 + step_k<G>(t, g);
                        c.x[b][t] = u32x4{0, 0, 0, 0};
                        if (k < K) c.x[b][t] = *reinterpret_cast<const u32x4*>(xrow[b] + k);
                    }
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        const bool has = k0 + i * G < K;
                        c.s[j][i] = has ? srow[j][full * NG + i] : static_cast<uint16_t>(0);
                        if constexpr (ZP) c.z[j][i] = has ? zrow[j][full * NG + i] : static_cast<uint8_t>(0);
                    }
                contract(c);
            }

            // ---- the waves' sums in wave order, rounded once
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        red[(wave * MB * NB + b * NB + j) * 256 + (4 * g + r) * 16 + (lane & 15)] = tot[b][j][r];
            __syncthreads();
            for (int x = tid; x < NB * MB * 256; x += 64 * NWV) {
                const int col = x % 16, row = (x / 16) % 16, blk = x / 256;
                const int i = m0 + 16 * (blk / NB) + row, n = n0 + 16 * (blk % NB) + col;
                if (i >= rows || n >= N) continue;
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < NWV; ++w) v += red[(w * MB * NB + blk) * 256 + row * 16 + col];
                const int r = row_of(i);
                if (!__builtin_isfinite(v))
                    v = plain_sum<G, BF16, ZP>(a.X + static_cast<int64_t>(r) * a.sx,
                                               W + static_cast<int64_t>(n) * a.sw_n,
                                               S + static_cast<int64_t>(n) * a.ss_n,
                                               ZP ? Z + static_cast<int64_t>(n) * a.sz_n : nullptr, K);
                a.Y[static_cast<int64_t>(r) * a.sy + n] = narrow<BF16>(v);
            }
            __syncthreads();   // red is written again by the next block of rows
        }
    }
}

template <int NB, int MB, int NWV, int G, bool BF16, bool ZP>
hipError_t launch_w4(const W4Args& a, int64_t tiles, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_w4_kernel<NB, MB, NWV, G, BF16, ZP>),
                       dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.num_experts)), dim3(64 * NWV), 0,
                       stream, a);
    return hipGetLastError();
}

#define DTG_STR2(x) #x
#define DTG_STR(x) DTG_STR2(x)
#define W4_ENTRY(NB, MB, NWV, G, BF, ZP)                                                     \
    {NB, MB, NWV, G, BF, ZP, &launch_w4<NB, MB, NWV, G, (BF != 0), (ZP != 0)>,               \
     "gemm_w4_kernel<" DTG_STR(NB) "," DTG_STR(MB) "," DTG_STR(NWV) "," DTG_STR(G) "," DTG_STR(BF) "," DTG_STR(ZP) ">"}
#define W4_GROUPS(NB, MB, NWV)                                                                                   \
    W4_ENTRY(NB, MB, NWV, 128, 0, 0), W4_ENTRY(NB, MB, NWV, 128, 0, 1), W4_ENTRY(NB, MB, NWV, 128, 1, 0),         \
    W4_ENTRY(NB, MB, NWV, 128, 1, 1), W4_ENTRY(NB, MB, NWV, 64, 0, 0), W4_ENTRY(NB, MB, NWV, 64, 0, 1),           \
    W4_ENTRY(NB, MB, NWV, 64, 1, 0), W4_ENTRY(NB, MB, NWV, 64, 1, 1), W4_ENTRY(NB, MB, NWV, 32, 0, 0),            \
    W4_ENTRY(NB, MB, NWV, 32, 0, 1), W4_ENTRY(NB, MB, NWV, 32, 1, 0), W4_ENTRY(NB, MB, NWV, 32, 1, 1)

const W4Entry kTable[] = {
    W4_GROUPS(1, 1, 8), W4_GROUPS(2, 1, 8),
    W4_GROUPS(1, 2, 8),
};

}  // namespace

const W4Entry* w4_kernel_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
