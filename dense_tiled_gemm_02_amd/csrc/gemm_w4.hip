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
// A wave takes chunks of 128 k of 16 NB rows of W: each lane one 16-byte load
// per 16 rows (row l mod 16, k 32 (l / 16) .. + 31), issued UW chunks ahead into
// registers (cached: non-temporal, the two waves that share each 128-byte line
// both fetch it, 24 us in place of 22 when that was tried); X comes through a ring in LDS,
// filled by direct loads; the scales and offsets of the workgroup's columns are
// converted into an LDS table once.  The order of k inside the instruction is
// free as long as X follows it, so with groups of 128 a lane's four dwords are
// simply four instructions; for groups of 64 or 32 the dwords are first
// exchanged between the wave's halves (and quarters) so that every instruction
// stays inside one group.  The waves of a workgroup take the chunks in turn and
// their sums are added through LDS in wave order, so a call's result does not
// depend on timing.
//
// Blocks of up to 4 rows (a token, or the few rows of one of many experts) load
// and keep a quarter of X, issued four chunks ahead like W: 1 x 4096 x 4096 6.1 ->
// 5.6 us, 32 rows over 16 experts, 4096 x 2048, groups of 32 24 -> 21 us (eight
// chunks ahead: 22) when they came in; 5.3 and 19 us now.  Four column blocks (one
// row of 8192 x 14336, groups of 128: 16.9 us) have no such path.
//
// What is issued ahead does not stay in flight for a whole round of UW chunks:
// as compiled, one wait in a round (two where UW is 2) is for every load there
// is, the compiler's own for W's registers while loads to LDS are pending, and
// the loop pays a memory latency there.
//
// Measured: 16 x 8192 x 14336, groups of 64 with zero points, 19.3 us with W from
// memory, against 13.0 us for reading W alone in this order of lanes (10.5 us in
// consecutive 1 KB).  Bound by those waits (half of a wave's cycles) and by 3 us
// before the first product; vector instructions, about 70 per 1 KB of W, issue
// in a third of the cycles.  With many workgroups those 3 us
// count most, and one wave with 32 columns to itself wins (30 rows over 60
// experts, 1024 x 2786: 20 us, 44 with four waves to 32 columns).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "kernels_w4.h"

namespace dtg {
namespace {

using namespace dev;

constexpr int kListRows = 256;    // rows gathered per pass over the expert ids

// Lowest mantissa bit of the units place of 16.0.
template <bool BF16> constexpr int kUnits = BF16 ? 3 : 6;

// Nibbles r and r + 4 of w as the pair (16 + q_r, 16 + q_{r + 4}); `mask` and
// `sixteen` are the nibbles' places and two times 16.0, in registers (as
// literals they would cost an instruction each).
template <bool BF16, int R>
__device__ __forceinline__ uint32_t offset_pair(uint32_t w, uint32_t mask, uint32_t sixteen) {
    constexpr int to = kUnits<BF16>;
    constexpr int sh = 4 * R - to;
    const uint32_t v = sh > 0 ? w >> (sh > 0 ? sh : 0) : w << (sh < 0 ? -sh : 0);
    return (v & mask) | sixteen;
}

// Between X's loads and W's.  A wait for X counts the loads that follow it, so
// X has to go out first; nothing else keeps the scheduler from moving W's.  Only
// memory loads are held (mask: arithmetic, matrix and LDS instructions may pass).
__device__ __forceinline__ void x_before_w() { __builtin_amdgcn_sched_barrier(0x48F); }

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
// instruction t: quarter_k(g) + step_k(t).
template <int G>
__device__ __forceinline__ int quarter_k(int g) {
    if constexpr (G == 128) return 32 * g;
    else if constexpr (G == 64) return 32 * (g & 1) + 16 * (g >> 1);
    else return 8 * g;
}
template <int G>
constexpr int step_k(int t) {
    return G == 128 ? 8 * t : G == 64 ? 64 * (t >> 1) + 8 * (t & 1) : 32 * t;
}

// Of a chunk of X with 4 rows, piece p of row r sits at p ^ few_place(r): the 16
// pieces that one instruction's lanes read meet no LDS bank twice.
template <int G>
__device__ __forceinline__ int few_place(int r) {
    return G == 128 ? r : G == 64 ? (r & 1) | (r & 2) << 2 : 4 * r;
}

// The sum of one output by the formula, term by term in fp32: for outputs
// that the offset form leaves infinite or NaN.
template <int G, bool BF16, bool ZP>
__device__ __forceinline__ float plain_sum(const uint16_t* x, const uint8_t* w, const uint16_t* s, const uint8_t* z,
                                        int K) {
    float y = 0.0f;
#pragma nounroll
    for (int k0 = 0; k0 < K; k0 += G) {
        const float zero = ZP ? static_cast<float>(z[k0 / G]) : 8.0f;
        float t = 0.0f;
#pragma nounroll
        for (int k = k0; k < k0 + G && k < K; ++k) {
            const int q = (w[k >> 1] >> (4 * (k & 1))) & 15;
            t += widen<BF16>(x[k]) * (static_cast<float>(q) - zero);
        }
        y += widen<BF16>(s[k0 / G]) * t;
    }
    return y;
}

// PANEL: groups of k whose scales and zero points are held in LDS at a time.
template <int NB, int MB, int NWV, int PANEL, int G, bool BF16, bool ZP>
__global__ __launch_bounds__(64 * NWV, 2) void gemm_w4_kernel(W4Args a) {
    constexpr int kPanel = !ZP && PANEL < 128 ? 2 * PANEL : PANEL;   // without zero points the table holds scales alone
    constexpr int kPitch = kPanel + 1;   // odd: 16 columns' reads of one group meet no LDS bank twice
    constexpr int LPC = kPanel / 4;      // lanes per column of the table, four groups each
    typedef std::conditional_t<ZP, float2, float> Entry;
    typedef std::conditional_t<ZP, u32x2, uint32_t> Scale;
    constexpr int CPL = 64 / LPC;        // columns per load
    constexpr int NG = 128 / G;          // groups per chunk
    constexpr int UW = NB == 4 || (MB == 2 && NWV == 2) ? 2 : 4;   // chunks of W in flight, in registers
    constexpr int UX = 2;                                         // chunks of X in flight, in LDS (16 MB rows each)
    constexpr int ROWS = 16 * MB;
    constexpr int CW = 16 * NB / NWV;    // columns of the table per wave
    __shared__ Entry tab[16 * NB * kPitch];
    __shared__ __attribute__((aligned(1024))) uint16_t xring[NWV * UX * MB * 2048];
    __shared__ int list[kListRows];
    __shared__ int listed;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4;
    const int n0 = blockIdx.x * (16 * NB);
    const int M = a.M, N = a.N, K = a.K;
    auto id_of = [&](int row) -> int64_t {
        return a.id_bytes == 8 ? static_cast<const int64_t*>(a.experts)[row]
                               : static_cast<const int32_t*>(a.experts)[row];
    };
    int expert = blockIdx.y;
    if (a.by_row) {   // more experts than rows, 64 of those at most: the blockIdx.y-th that a row names
        const int64_t id = lane < M ? id_of(lane) : -1;
        const bool named = id >= 0 && id < a.num_experts;
        uint64_t same = __ballot(named);   // the rows of this lane's id, one bit of the ids at a time
        for (int b = 0; (a.num_experts - 1) >> b; ++b) {
            const bool bit = (id >> b) & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const bool again = (same & ((uint64_t(1) << lane) - 1)) != 0;
        uint64_t first = __ballot(named && !again);
        if (__popcll(first) <= expert && expert > 0) return;
        for (int k = 0; k < expert; ++k) first &= first - 1;
        expert = first ? __builtin_amdgcn_readlane(static_cast<int>(id), __builtin_ctzll(first)) : -1;
    }
    // no row names an expert: nothing but the zeros to write
    const int e = expert < 0 ? 0 : expert;
    const uint8_t* const W = a.W + static_cast<int64_t>(e) * a.sw_e + static_cast<int64_t>(n0) * a.sw_n;
    const uint16_t* const S = a.S + static_cast<int64_t>(e) * a.ss_e + static_cast<int64_t>(n0) * a.ss_n;
    const uint8_t* const Z = ZP ? a.Z + static_cast<int64_t>(e) * a.sz_e + static_cast<int64_t>(n0) * a.sz_n : nullptr;
    const int cols = N - n0 < 16 * NB ? N - n0 : 16 * NB;   // columns past N repeat the last one and are not stored

    // this lane's bytes within the workgroup's columns (the planner keeps 64 row strides below 2^32)
    uint32_t woff[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int n = 16 * j + (lane & 15);
        woff[j] = static_cast<uint32_t>(n < cols ? n : cols - 1) * static_cast<uint32_t>(a.sw_n) + 16 * g;
    }
    const int full = K / 128;
    const int groups = (K + G - 1) / G;

    // {scale, offset} of groups [p0, p0 + held) of every column, zeros up to a multiple of 4.
    // In two steps, all loads before the first store: loaded and stored one by
    // one, the table took half of a wave's time.
    struct __attribute__((packed, aligned(2))) Loose8 {
        uint32_t v[2];
    };
    struct __attribute__((packed, aligned(1))) Loose4 {
        uint32_t v;
    };
    static_assert(CW % CPL == 0, "whole loads of table columns");
    const int tcol = wave * CW + lane / LPC, tgroup = 4 * (lane % LPC);   // columns tcol + CPL c, groups tgroup + 0..3
    uint32_t ts[CW / CPL][2], tz[CW / CPL];
    auto load_table = [&](int p0, int held) {
#pragma unroll
        for (int c = 0; c < CW / CPL; ++c) {
            const uint32_t n = tcol + CPL * c < cols ? tcol + CPL * c : cols - 1;
            const uint16_t* s = S + static_cast<uint64_t>(n) * static_cast<uint32_t>(a.ss_n) + p0;
            const uint8_t* z = ZP ? Z + static_cast<uint64_t>(n) * static_cast<uint32_t>(a.sz_n) + p0 : nullptr;
            ts[c][0] = ts[c][1] = 0;
            tz[c] = 0x08080808u;
            if (held % 4 == 0) {
                if (tgroup < held) {
                    const Loose8 v = *reinterpret_cast<const Loose8*>(s + tgroup);
                    ts[c][0] = v.v[0];
                    ts[c][1] = v.v[1];
                    if constexpr (ZP) tz[c] = reinterpret_cast<const Loose4*>(z + tgroup)->v;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (tgroup + i < held) {
                        ts[c][i / 2] |= static_cast<uint32_t>(s[tgroup + i]) << (16 * (i % 2));
                        if constexpr (ZP) tz[c] = (tz[c] & ~(255u << (8 * i))) | static_cast<uint32_t>(z[tgroup + i]) << (8 * i);
                    }
            }
        }
    };
    auto store_table = [&](int held) {
#pragma unroll
        for (int c = 0; c < CW / CPL; ++c) {
            Entry* row = tab + (tcol + CPL * c) * kPitch;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (tgroup < held) {
                    const float scale = widen<BF16>(static_cast<uint16_t>(ts[c][i / 2] >> (16 * (i % 2))));
                    if constexpr (ZP) row[tgroup + i] = float2{scale, 16.0f + static_cast<float>((tz[c] >> (8 * i)) & 255u)};
                    else row[tgroup + i] = scale;
                }
        }
    };
    int in_table = -1;   // first group of the table's panel
    float* const red = reinterpret_cast<float*>(xring);
    uint16_t* const xwave = xring + wave * UX * MB * 2048;
    const uint32_t tab_addr = lds_addr(reinterpret_cast<const uint16_t*>(tab)) + (lane & 15) * (kPitch * sizeof(Entry));

    uint32_t mask = 0x000F000Fu << kUnits<BF16>, sixteen = BF16 ? 0x41804180u : 0x4C004C00u;
    asm volatile("" : "+s"(mask), "+v"(sixteen));
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
                    if (row < end) id = id_of(row);
                    const bool mine = row < end && id == expert && expert >= 0;
                    const uint64_t hits = __ballot(mine);
                    if (mine) list[n + __popcll(hits & ((uint64_t(1) << lane) - 1))] = row;
                    n += __popcll(hits);
                    // rows of no expert are zeros, written by the first workgroups
                    if (blockIdx.y == 0 && row < end && (id < 0 || id >= a.num_experts))
                        for (int c = 0; c < cols; ++c) a.Y[static_cast<int64_t>(row) * a.sy + n0 + c] = 0;
                }
                if (lane == 0) listed = n;
            }
            __syncthreads();
            rows = __builtin_amdgcn_readfirstlane(listed);
        } else {
            rows = M - first < kListRows ? M - first : kListRows;
        }
        auto row_of = [&](int i) { return a.experts ? list[i] : first + i; };

        // One block of rows.  FEW (4 rows or less of a block of 16): X's chunk is 1 KB,
        // a row from each quarter of a wave's load, in place of 4 KB of which 3 repeat
        // the last row, and the ring holds as many chunks of it as of W.
        auto block = [&](auto few_tag, int m0) {
            constexpr bool FEW = decltype(few_tag)::value;
            constexpr int U = FEW ? 4 : UW, XS = FEW ? U : UX, XL = FEW ? 1 : 4 * MB;   // X: slots, loads per chunk
            static_assert(!FEW || (MB == 1 && U * 512 <= UX * 2048), "the ring holds a row of each quarter");
            u32x4 w[U][NB];
            auto load_w = [&](u32x4 (&d)[NB], int chunk) {
                const uint8_t* wk = W + static_cast<int64_t>(chunk) * 64;
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    d[j] = *reinterpret_cast<const u32x4*>(wk + woff[j]);
            };
            // The wave's whole chunks of the panel from group p0 on: c0 + wave,
            // c0 + wave + NWV, ... (`mine` of them).
            int c0, mine;
            auto at = [&](int i) { return wave + (i < mine ? i : mine - 1) * NWV; };
            auto chunks = [&](int p0) {
                c0 = p0 / NG;
                mine = ((full < c0 + kPanel / NG ? full : c0 + kPanel / NG) - c0 - wave + NWV - 1) / NWV;
            };
            // W of the first chunks is on its way before anything else is computed
            auto start = [&] {
                if (!FEW && mine > 0)
#pragma unroll
                    for (int u = 0; u < U - 1; ++u) load_w(w[u], c0 + at(u));
            };
            chunks(0);
            start();
            // Row i of a block of 16 sits in instruction row 4 (i % 4) + i / 4, so
            // that register r of the result holds rows 4 r .. 4 r + 3: blocks of up
            // to 4 rows scale one register in place of four.
            // X goes to LDS a chunk at a time, each wave its own: load t brings
            // instruction rows 4 t .. 4 t + 3, 256 bytes of each in one piece (read
            // straight into the operand's lanes, consecutive lanes lie in different
            // rows, and the 16-row product took 32 us in place of 27).  Piece p of
            // row r sits at p ^ r.
            const uint16_t* xsrc[FEW ? 1 : MB][FEW ? 1 : 4];
#pragma unroll
            for (int b = 0; b < (FEW ? 1 : MB); ++b)
#pragma unroll
                for (int t = 0; t < (FEW ? 1 : 4); ++t) {
                    const int i = m0 + (FEW ? g : 16 * b + t + 4 * g);
                    xsrc[b][t] = a.X + static_cast<uint64_t>(static_cast<uint32_t>(row_of(i < rows ? i : rows - 1))) *
                                           static_cast<uint32_t>(a.sx) +
                                 8 * ((lane & 15) ^ (FEW ? few_place<G>(g) : 4 * t + g));
                }
            const bool few = FEW || ((MB > 1 || NB == 4) && rows - m0 <= 4);
            uint32_t xaddr[4];   // this lane's pieces of X: instruction row lane % 16, FEW: row lane / 4 % 4
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int piece = (quarter_k<G>(g) + step_k<G>(t)) / 8, ir = lane & 15;
                xaddr[t] = lds_addr(xwave) + (FEW ? (ir >> 2) * 256 + (piece ^ few_place<G>(ir >> 2)) * 16
                                                  : ir * 256 + (piece ^ ir) * 16);
            }

            f32x4 tot[MB][NB];
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int j = 0; j < NB; ++j) tot[b][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

            auto load_x = [&](int slot, int chunk) {
                if constexpr (FEW)
                    __builtin_amdgcn_global_load_lds(
                        (const __attribute__((address_space(1))) void*)(xsrc[0][0] + static_cast<int64_t>(chunk) * 128),
                        (lds_void_t*)(xwave + slot * 512), 16, 0, 0);
                else
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        __builtin_amdgcn_global_load_lds(
                            (const __attribute__((address_space(1))) void*)(xsrc[b][t] + static_cast<int64_t>(chunk) * 128),
                            (lds_void_t*)(xwave + (slot * MB + b) * 2048 + t * 512), 16, 0, 0);
            };
            // A chunk's operands out of LDS: X of `slot`, its groups from number `g0`
            // of the table on.  The reads are explicit: the compiler would hold each
            // until every load in flight to LDS has landed.
            struct Frag {
                u32x4 x[MB][4];
                Scale q[NG][NB];
            };
            auto fetch = [&](auto slot_tag, Frag& f, int g0) {
                static_for<4>([&](auto t_tag) {
                    static_for<MB>([&](auto b_tag) {
                        constexpr int T = decltype(t_tag)::value, B = decltype(b_tag)::value;
                        f.x[B][T] = lds_read16<FEW ? decltype(slot_tag)::value * 1024 : (decltype(slot_tag)::value * MB + B) * 4096>(xaddr[T]);
                    });
                });
                const uint32_t taddr = tab_addr + sizeof(Entry) * g0;
                static_for<NG>([&](auto i_tag) {
                    static_for<NB>([&](auto j_tag) {
                        constexpr int I = decltype(i_tag)::value, J = decltype(j_tag)::value;
                        if constexpr (ZP) f.q[I][J] = lds_read8<(16 * J * kPitch + I) * 8>(taddr);
                        else f.q[I][J] = lds_read4<(16 * J * kPitch + I) * 4>(taddr);
                    });
                });
            };
            auto landed = [&](Frag& f) {
                lds_wait_all();
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int t = 0; t < 4; ++t) tie(f.x[b][t]);
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j) tie(f.q[i][j]);
            };
            auto contract = [&](const Frag& f, u32x4 (&w)[NB]) {
                if constexpr (G < 128) {
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        uint32_t d0 = w[j][0], d1 = w[j][1], d2 = w[j][2], d3 = w[j][3];
                        swap_halves(d0, d2);
                        swap_halves(d1, d3);
                        if constexpr (G == 32) {
                            swap_quarters(d0, d1);
                            swap_quarters(d2, d3);
                        }
                        w[j] = u32x4{d0, d1, d2, d3};
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
                        const uint32_t d = w[j][T];
                        wf[j] = u32x4{offset_pair<BF16, 0>(d, mask, sixteen), offset_pair<BF16, 1>(d, mask, sixteen),
                                      offset_pair<BF16, 2>(d, mask, sixteen), offset_pair<BF16, 3>(d, mask, sixteen)};
                    }
#pragma unroll
                    for (int b = 0; b < MB; ++b) {
                        const u32x4 xf = pair_order(f.x[b][T]);
                        sum[b] = mfma<16, BF16>(xf, ones, sum[b]);
#pragma unroll
                        for (int j = 0; j < NB; ++j) acc[b][j] = mfma<16, BF16>(xf, wf[j], acc[b][j]);
                    }
                    if constexpr (T % STEPS == STEPS - 1) {
                        constexpr int I = T / STEPS;
                        auto scale = [&](int r) {
#pragma unroll
                            for (int b = 0; b < MB; ++b)
#pragma unroll
                                for (int j = 0; j < NB; ++j)
                                    if constexpr (ZP)
                                        tot[b][j][r] += __uint_as_float(f.q[I][j][0]) *
                                                        (acc[b][j][r] - __uint_as_float(f.q[I][j][1]) * sum[b][r]);
                                    else
                                        tot[b][j][r] += __uint_as_float(f.q[I][j]) * (acc[b][j][r] - 24.0f * sum[b][r]);
                        };
                        scale(0);
                        if (!few) {
                            scale(1);
                            scale(2);
                            scale(3);
                        }
                    }
                });
            };

            for (int p0 = 0; p0 < groups; p0 += kPanel) {
                const int held = groups - p0 < kPanel ? groups - p0 : kPanel;
                const bool fresh = in_table != p0;
                if constexpr (FEW) {   // in the order in which they are waited for
                    if (fresh) load_table(p0, held);
                    if (mine > 0) {
                        static_for<U>([&](auto u_tag) { load_x(decltype(u_tag)::value, c0 + at(decltype(u_tag)::value)); });
                        x_before_w();
#pragma unroll
                        for (int u = 0; u < U; ++u) load_w(w[u], c0 + at(u));
                    }
                } else {
                    if (mine > 0) {
                        load_x(0, c0 + at(0));
                        load_x(1, c0 + at(1));
                    }
                    if (fresh) load_table(p0, held);
                }
                if (fresh) {
                    if (in_table >= 0) __syncthreads();   // the last panel's readers are done
                    store_table(held);
                    in_table = p0;
                    __syncthreads();
                }
                // Step i contracts chunk i while the next one's operands come out of
                // LDS, then refills their slot of the ring and W's registers.  X goes
                // out before W: waiting for the next X leaves a later step of X and two
                // of W in flight.  FEW: the first step's W is followed by U - 1 chunks of
                // W and one of X, the later ones' by more.
                Frag f[2];
                auto step = [&](auto u_tag, int i) {
                    constexpr int V = decltype(u_tag)::value, S1 = (V + 1) % XS, F1 = (V + 1) % 2;
                    wait_vm<FEW ? NB * (U - 1) + 1 : 2 * NB + XL>();
                    fetch(std::integral_constant<int, S1>{}, f[F1], at(i + 1) * NG);
                    contract(f[V % 2], w[V]);
                    landed(f[F1]);
                    load_x(S1, c0 + at(i + 1 + XS));
                    x_before_w();
                    load_w(w[V], c0 + at(i + U));
                };
                if (mine > 0) {
                    // both chunks of X: fewer loads follow the second one here than the count in step() allows for
                    wait_vm<FEW ? NB * U + U - 1 : 0>();
                    fetch(std::integral_constant<int, 0>{}, f[0], at(0) * NG);
                    landed(f[0]);
                    load_x(0, c0 + at(XS));
                    x_before_w();
                    if constexpr (!FEW) load_w(w[U - 1], c0 + at(U - 1));
                    for (int i = 0;; i += U) {
                        step(std::integral_constant<int, 0>{}, i);
                        if (i + 1 >= mine) break;
                        step(std::integral_constant<int, 1>{}, i + 1);
                        if (i + 2 >= mine) break;
                        if constexpr (U == 4) {
                            step(std::integral_constant<int, 2>{}, i + 2);
                            if (i + 3 >= mine) break;
                            step(std::integral_constant<int, 3>{}, i + 3);
                            if (i + 4 >= mine) break;
                        }
                    }
                    wait_vm<0>();   // no load may still be writing the ring
                }
                // the last K mod 128: one wave, lanes past K read the chunk's start and X as zeros
                if (K % 128 != 0 && p0 + kPanel >= groups && wave == full % NWV) {
                    const int k0 = full * 128;
                    const uint8_t* wk = W + static_cast<int64_t>(full) * 64;
                    const uint32_t back = k0 + 32 * g < K ? 0 : 16 * g;
#pragma unroll
                    for (int j = 0; j < NB; ++j) w[0][j] = *reinterpret_cast<const u32x4*>(wk + (woff[j] - back));
#pragma unroll
                    for (int b = 0; b < (FEW ? 1 : MB); ++b)
#pragma unroll
                        for (int t = 0; t < (FEW ? 1 : 4); ++t) {
                            u32x4 v = {0, 0, 0, 0};
                            if (k0 + 8 * ((lane & 15) ^ (FEW ? few_place<G>(g) : 4 * t + g)) < K)
                                v = *reinterpret_cast<const u32x4*>(xsrc[b][t] + k0);
                            *reinterpret_cast<u32x4*>(xwave + b * 2048 + t * 512 + 8 * lane) = v;
                        }
                    lds_wait_all();
                    fetch(std::integral_constant<int, 0>{}, f[0], (full - c0) * NG);
                    landed(f[0]);
                    contract(f[0], w[0]);
                }
                if (p0 + kPanel < groups) {
                    chunks(p0 + kPanel);
                    start();
                }
            }

            // ---- the waves' sums in wave order, rounded once (over the ring)
            __syncthreads();
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int j = 0; j < NB; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        red[(wave * MB * NB + b * NB + j) * 256 + (g + 4 * r) * 16 + (lane & 15)] = tot[b][j][r];
            __syncthreads();
            for (int x = tid; x < NB * MB * 256; x += 64 * NWV) {
                const int col = x % 16, row = (x / 16) % 16, blk = x / 256;
                const int i = m0 + 16 * (blk / NB) + row, n = 16 * (blk % NB) + col;
                if (i >= rows || n >= cols) continue;
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < NWV; ++w) v += red[(w * MB * NB + blk) * 256 + row * 16 + col];
                const int64_t r = row_of(i);
                if (!__builtin_isfinite(v))
                    v = plain_sum<G, BF16, ZP>(a.X + r * a.sx, W + n * a.sw_n, S + n * a.ss_n,
                                               ZP ? Z + n * a.sz_n : nullptr, K);
                a.Y[r * a.sy + n0 + n] = narrow<BF16>(v);
            }
            __syncthreads();   // red is written again by the next block of rows
        };
        for (int m0 = 0; m0 < rows; m0 += ROWS) {
            if constexpr (MB == 1 && NB < 4) {
                if (rows - m0 <= 4) {
                    block(std::true_type{}, m0);
                    continue;
                }
            }
            block(std::false_type{}, m0);
        }
    }
}

template <int NB, int MB, int NWV, int PANEL, int G, bool BF16, bool ZP>
hipError_t launch_w4(const W4Args& a, int64_t tiles, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_w4_kernel<NB, MB, NWV, PANEL, G, BF16, ZP>),
                       dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.by_row ? a.M : a.num_experts)), dim3(64 * NWV), 0,
                       stream, a);
    return hipGetLastError();
}

#define DTG_STR2(x) #x
#define DTG_STR(x) DTG_STR2(x)
#define W4_ENTRY(NB, MB, NWV, PN, G, BF, ZP)                                                 \
    {NB, MB, NWV, G, BF, ZP, &launch_w4<NB, MB, NWV, PN, G, (BF != 0), (ZP != 0)>,           \
     "gemm_w4_kernel<" DTG_STR(NB) "," DTG_STR(MB) "," DTG_STR(NWV) "," DTG_STR(PN) "," DTG_STR(G) "," DTG_STR(BF) "," \
     DTG_STR(ZP) ">"}
// (groups of 32 keep twice the scales in registers: four column blocks would spill)
#define W4_WIDE(NB, MB, NWV, PN)                                                                                 \
    W4_ENTRY(NB, MB, NWV, PN, 128, 0, 0), W4_ENTRY(NB, MB, NWV, PN, 128, 0, 1),                                   \
    W4_ENTRY(NB, MB, NWV, PN, 128, 1, 0), W4_ENTRY(NB, MB, NWV, PN, 128, 1, 1),                                   \
    W4_ENTRY(NB, MB, NWV, PN, 64, 0, 0), W4_ENTRY(NB, MB, NWV, PN, 64, 0, 1),                                     \
    W4_ENTRY(NB, MB, NWV, PN, 64, 1, 0), W4_ENTRY(NB, MB, NWV, PN, 64, 1, 1)
#define W4_GROUPS(NB, MB, NWV, PN)                                                                               \
    W4_WIDE(NB, MB, NWV, PN), W4_ENTRY(NB, MB, NWV, PN, 32, 0, 0), W4_ENTRY(NB, MB, NWV, PN, 32, 0, 1),           \
    W4_ENTRY(NB, MB, NWV, PN, 32, 1, 0), W4_ENTRY(NB, MB, NWV, PN, 32, 1, 1)

const W4Entry kTable[] = {
    W4_GROUPS(1, 1, 8, 128), W4_GROUPS(2, 1, 4, 128), W4_WIDE(4, 1, 8, 128),
    W4_GROUPS(1, 2, 4, 128), W4_GROUPS(2, 2, 4, 128), W4_GROUPS(2, 2, 2, 64), W4_GROUPS(2, 1, 1, 32), W4_GROUPS(2, 1, 2, 64), W4_GROUPS(2, 1, 8, 128),
};

}  // namespace

const W4Entry* w4_kernel_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
