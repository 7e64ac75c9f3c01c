// The grouped products for operands with a contiguous index but sizes, strides
// or bases that are no multiple of 16 bytes (an odd feature size, a view that
// starts anywhere): the direct-to-LDS loads need aligned 16-byte chunks, plain
// global loads do not.  Every chunk of 8 elements is one 16-byte load at its
// own 2-byte-aligned address.  A chunk that the row's end cuts is loaded from
// where its last element ends the 16 bytes and shifted down when it is staged,
// so nothing outside a row is touched (the planner admits rows of 8 elements
// and more).
//
// Staging is through registers, two K steps ahead, into an LDS tile laid out as
// the direct kernels lay theirs (OpShape): an operand with contiguous k as rows
// of k, the other kind as rows of its outer index, read with the transposing
// LDS read.  Two LDS stages, one barrier per step.  Bound by the latency of a K
// step, not by bytes: 777 x 1003 x 517 over 5 groups has 135 tiles for 256 CUs
// and takes 10.8 us (200 us with element loads).
#include "grouped_kernel.h"

namespace dtg {
namespace {

// 16 bytes from any 2-byte-aligned address (one load instruction: gfx9 runs
// HSA code with unaligned access enabled).
struct __attribute__((packed, aligned(2))) Loose16 {
    u32x4 v;
};

template <int BM, int BN, int BK, int WM, int WN, bool BF16, bool AKC, bool BKC, bool O32>
__device__ __forceinline__ void odd_tile(const KArgs& p, int pid_m, int pid_n) {
    constexpr int NW = WM * WN, NT = 64 * NW;
    constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    typedef OpShape<AKC, BM, BK, NW> OA;
    typedef OpShape<BKC, BN, BK, NW> OB;
    constexpr int DEPTH = 2;   // K steps in flight (4: 11.6 us instead of 10.8 at 777 x 1003 x 517, and fewer resident)
    constexpr int PA = BM * BK / 8 / NT, PB = BN * BK / 8 / NT;   // chunks per thread per stage
    __shared__ __attribute__((aligned(16))) uint16_t smem[2 * (OA::SZ + OB::SZ)];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // The last tile along an outer-contiguous index moves back to end with the
    // operand, where that is wider than a tile: whole chunks only, 11.6 us instead
    // of 14.5 at 777 x 1003 x 517.  What the tile before it holds is not stored
    // again.
    const int m_first = pid_m * BM, n_first = pid_n * BN;
    const int m0 = !AKC && m_first + BM > p.M && p.M > BM ? p.M - BM : m_first;
    const int n0 = !BKC && n_first + BN > p.N && p.N > BN ? p.N - BN : n_first;
    const int K = p.K;
    const int64_t lda = AKC ? p.lda : p.sak, ldb = BKC ? p.sbn : p.ldb;

    // One operand's chunk i of this thread (LDS row q / CH, chunk q % CH): where
    // it loads from in the next whole K step and how far a step moves that, its
    // k within a step, its place in LDS, and how many of its 8 elements the
    // outer index leaves (k contiguous: all or none).  A chunk with none left
    // reads the operand's start and stays there: what it holds only reaches
    // outputs that are not stored.
    struct Lane {
        const uint16_t* src;
        int64_t inc;
        int at, avail, lds;
    };
    auto place = [&](auto kc_tag, auto shape_tag, int i, const uint16_t* op, int64_t ld, int e0, int count) {
        constexpr bool KC = decltype(kc_tag)::value;
        typedef decltype(shape_tag) OS;
        const int q = tid + i * NT, row = q / OS::CH, c = q % OS::CH;
        Lane l;
        l.lds = (row * OS::CH + (c ^ OS::sw(row))) * 8;
        if constexpr (KC) {
            l.src = op + static_cast<int64_t>(e0 + row) * ld + 8 * c;
            l.inc = BK;
            l.at = 8 * c;
            l.avail = e0 + row < count ? 8 : 0;
        } else {
            const int left = count - (e0 + 8 * c);
            l.src = op + static_cast<int64_t>(row) * ld + e0 + 8 * c;
            l.inc = BK * ld;
            l.at = row;
            l.avail = left < 8 ? left : 8;
            if (left > 0) l.src -= 8 - l.avail;
        }
        if (l.avail <= 0) {
            l.src = op;
            l.inc = 0;
        }
        return l;
    };
    Lane la[PA], lb[PB];
#pragma unroll
    for (int i = 0; i < PA; ++i) la[i] = place(std::integral_constant<bool, AKC>{}, OA{}, i, p.A, lda, m0, p.M);
#pragma unroll
    for (int i = 0; i < PB; ++i) lb[i] = place(std::integral_constant<bool, BKC>{}, OB{}, i, p.B, ldb, n0, p.N);

    // Every lane loads at every step, so that the compiler counts the loads in
    // flight (the branches left are a whole wave's, around the last steps'
    // addresses).  Past the whole steps, lanes with no k left read the operand's
    // start.
    const int whole = K / BK;
    auto fetch = [&](auto kc_tag, Lane& l, const uint16_t* op, int kt) {
        const uint16_t* src = l.src;
        if (kt >= whole) {
            const int left = K - kt * BK - l.at;
            if (left <= 0) src = op;
            else if (decltype(kc_tag)::value && left < 8 && l.avail > 0) src -= 8 - left;
        }
        l.src += l.inc;
        return reinterpret_cast<const Loose16*>(src)->v;
    };
    // The n elements at the end of v moved to its start, zeros after them (none
    // left: all zeros).  Selects, not branches: in divergent branches this cost
    // 0.25 us per step in a tile that the row's end cuts.
    auto shift_down = [&](u32x4 v, int n) {
        const int cut = n < 8 ? 8 - n : 0;
        const bool four = (cut & 4) != 0, two = (cut & 2) != 0;
        const uint32_t a0 = four ? v[2] : v[0], a1 = four ? v[3] : v[1], a2 = four ? 0u : v[2], a3 = four ? 0u : v[3];
        const uint32_t b0 = two ? a1 : a0, b1 = two ? a2 : a1, b2 = two ? a3 : a2, b3 = two ? 0u : a3;
        const uint32_t s = 16u * (cut & 1);
        const uint32_t keep = n > 0 ? ~0u : 0u;
        return u32x4{__builtin_amdgcn_alignbit(b1, b0, s) & keep, __builtin_amdgcn_alignbit(b2, b1, s) & keep,
                     __builtin_amdgcn_alignbit(b3, b2, s) & keep, __builtin_amdgcn_alignbit(0u, b3, s) & keep};
    };
    // The chunk as it goes to LDS; k past K must be zeros in both operands.
    const bool a_edge = !AKC && m0 + BM > p.M, b_edge = !BKC && n0 + BN > p.N;
    auto settle = [&](auto kc_tag, u32x4 v, const Lane& l, int kt, bool edge) {
        constexpr bool KC = decltype(kc_tag)::value;
        if (edge || kt >= whole) {
            const int left = K - kt * BK - l.at;
            v = shift_down(v, KC ? left : (left > 0 ? l.avail : 0));
        }
        return v;
    };

    u32x4 ra[DEPTH][PA], rb[DEPTH][PB];
    auto gload = [&](auto s_tag, int kt) {
        constexpr int S = decltype(s_tag)::value;
#pragma unroll
        for (int i = 0; i < PA; ++i) ra[S][i] = fetch(std::integral_constant<bool, AKC>{}, la[i], p.A, kt);
#pragma unroll
        for (int i = 0; i < PB; ++i) rb[S][i] = fetch(std::integral_constant<bool, BKC>{}, lb[i], p.B, kt);
    };
    auto stage = [&](auto s_tag, int kt) {
        constexpr int R = decltype(s_tag)::value, S = R % 2;
#pragma unroll
        for (int i = 0; i < PA; ++i)
            *reinterpret_cast<u32x4*>(smem + S * OA::SZ + la[i].lds) =
                settle(std::integral_constant<bool, AKC>{}, ra[R][i], la[i], kt, a_edge);
#pragma unroll
        for (int i = 0; i < PB; ++i)
            *reinterpret_cast<u32x4*>(smem + 2 * OA::SZ + S * OB::SZ + lb[i].lds) =
                settle(std::integral_constant<bool, BKC>{}, rb[R][i], lb[i], kt, b_edge);
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // 8 consecutive k of outer index e0 + lane % 16, k = ks * 32 + 8 (lane / 16) + 0..7
    auto frag = [&](auto kc_tag, auto shape_tag, const uint16_t* t, int e0, int ks) {
        constexpr bool KC = decltype(kc_tag)::value;
        typedef decltype(shape_tag) OS;
        if constexpr (KC) {
            const int row = e0 + (lane & 15);
            return *reinterpret_cast<const u32x4*>(t + (row * OS::CH + ((ks * 4 + (lane >> 4)) ^ OS::sw(row))) * 8);
        } else {
            i16x4 h[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = ks * 32 + 8 * (lane >> 4) + 4 * x + ((lane & 15) >> 2);
                // the swizzle is even, so the two chunks of 16 indices stay neighbours
                const uint16_t* at = t + (row * OS::CH + ((e0 >> 3) ^ OS::sw(row))) * 8 + 4 * (lane & 3);
                h[x] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)at);
            }
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
        }
    };
    auto contract = [&](auto s_tag) {
        constexpr int S = decltype(s_tag)::value % 2;
        const uint16_t* ta = smem + S * OA::SZ;
        const uint16_t* tb = smem + 2 * OA::SZ + S * OB::SZ;
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks) {
            u32x4 fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[i] = frag(std::integral_constant<bool, AKC>{}, OA{}, ta, wm * TM + i * 16, ks);
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[j] = frag(std::integral_constant<bool, BKC>{}, OB{}, tb, wn * TN + j * 16, ks);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma<16, BF16>(fa[i], fb[j], acc[i][j]);
        }
    };

    const int nkt = (K + BK - 1) / BK;
    if (nkt > 0) static_for<DEPTH>([&](auto r_tag) { gload(r_tag, decltype(r_tag)::value); });
    // DEPTH steps at a time, so that the loop has no branch either: steps past K contract zeros
    for (int k0 = 0; k0 < nkt; k0 += DEPTH)
        static_for<DEPTH>([&](auto r_tag) {
            const int kt = k0 + decltype(r_tag)::value;
            stage(r_tag, kt);
            gload(r_tag, kt + DEPTH);
            __syncthreads();   // the last readers of this LDS stage passed the previous step's barrier
            contract(r_tag);
        });

#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int col = n0 + wn * TN + j * 16 + (lane & 15);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = m0 + wm * TM + i * 16 + 4 * (lane >> 4) + r;
                if (row < m_first || row >= p.M || col < n_first || col >= p.N) continue;
                float v = acc[i][j][r];
                if constexpr (O32) {
                    if (p.has_c) v += reinterpret_cast<const float*>(p.C)[static_cast<int64_t>(row) * p.ldc + col];
                    reinterpret_cast<float*>(p.D)[static_cast<int64_t>(row) * p.ldd + col] = v;
                } else {
                    if (p.has_c) v += widen<BF16>(p.C[static_cast<int64_t>(row) * p.ldc + col]);
                    p.D[static_cast<int64_t>(row) * p.ldd + col] = narrow<BF16>(v);
                }
            }
        }
}

template <int BM, int BN, int BK, int WM, int WN, bool BF16, bool TB>
__global__ __launch_bounds__(64 * WM * WN) void gemm_grouped_rows_odd_any_kernel(GroupedArgs a) {
    RowTile t;
    if (!find_row_tile<BM>(a, &t)) return;
    const KArgs p = row_args(a, t);
    int pid_m, pid_n;
    grouped_tile<int>(t.tile, p.num_pid_m, p.num_pid_n, p.group_m, &pid_m, &pid_n);
    odd_tile<BM, BN, BK, WM, WN, BF16, true, TB, false>(p, pid_m, pid_n);
}

template <int BM, int BN, int BK, int WM, int WN, bool BF16, bool O32>
__global__ __launch_bounds__(64 * WM * WN) void gemm_grouped_reduce_odd_any_kernel(GroupedArgs a) {
    KArgs p;
    int tile, pid_m, pid_n;
    if (!reduce_work<O32>(a, &p, &tile)) return;
    grouped_tile<int>(tile, p.num_pid_m, p.num_pid_n, p.group_m, &pid_m, &pid_n);
    odd_tile<BM, BN, BK, WM, WN, BF16, false, false, O32>(p, pid_m, pid_n);
}

template <int BM, int BN, int BK, int WM, int WN, bool BF16, bool TB>
hipError_t launch_rows_odd(const GroupedArgs& a, int64_t grid, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_grouped_rows_odd_any_kernel<BM, BN, BK, WM, WN, BF16, TB>),
                       dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, stream, a);
    return hipGetLastError();
}

template <int BM, int BN, int BK, int WM, int WN, bool BF16, bool O32>
hipError_t launch_reduce_odd(const GroupedArgs& a, int64_t grid, hipStream_t stream) {
    hipLaunchKernelGGL((gemm_grouped_reduce_odd_any_kernel<BM, BN, BK, WM, WN, BF16, O32>),
                       dim3(static_cast<unsigned>(grid)), dim3(64 * WM * WN), 0, stream, a);
    return hipGetLastError();
}

#define ODD_ROWS(BM, BN, BK, WM, WN, BF, TB)                                                             \
    {kGroupedRows, BM, BN, BK, 2, 16, WM, WN, BF, kGroupedOdd, TB, 0, 64 * WM * WN, GROUPED_LDS(BM, BN, BK, 2), \
     &launch_rows_odd<BM, BN, BK, WM, WN, (BF != 0), (TB != 0)>,                                         \
     "gemm_grouped_rows_odd_any_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) ","  \
     DTG_STR(WN) "," DTG_STR(BF) "," DTG_STR(TB) ">"}
#define ODD_REDUCE(BM, BN, BK, WM, WN, BF, O32)                                                           \
    {kGroupedReduce, BM, BN, BK, 2, 16, WM, WN, BF, kGroupedOdd, 0, O32, 64 * WM * WN, GROUPED_LDS(BM, BN, BK, 2), \
     &launch_reduce_odd<BM, BN, BK, WM, WN, (BF != 0), (O32 != 0)>,                                       \
     "gemm_grouped_reduce_odd_any_kernel<" DTG_STR(BM) "," DTG_STR(BN) "," DTG_STR(BK) "," DTG_STR(WM) "," \
     DTG_STR(WN) "," DTG_STR(BF) "," DTG_STR(O32) ">"}

const GroupedEntry kTable[] = {
    ODD_ROWS(64, 64, 64, 2, 2, 0, 0),   ODD_ROWS(64, 64, 64, 2, 2, 1, 0),
    ODD_ROWS(64, 64, 64, 2, 2, 0, 1),   ODD_ROWS(64, 64, 64, 2, 2, 1, 1),
    ODD_REDUCE(64, 64, 64, 2, 2, 0, 0), ODD_REDUCE(64, 64, 64, 2, 2, 1, 0),
    ODD_REDUCE(64, 64, 64, 2, 2, 0, 1), ODD_REDUCE(64, 64, 64, 2, 2, 1, 1),
};

}  // namespace

const GroupedEntry* grouped_odd_table(int* count) {
    *count = static_cast<int>(sizeof(kTable) / sizeof(kTable[0]));
    return kTable;
}

}  // namespace dtg
