// Routing of tokens to experts, and its gradient, for gfx950.  For a row of E
// logits l:
//
//     p = softmax(l) or sigmoid(l),  c = p + bias (the choice alone)
//     a group's strength = the sum of its best one or two c
//     ids = the `top` largest c within the strongest groups, lowest index first
//     w = scale p, divided by the sum of the chosen p where renormalized
//
// LANES lanes take a row, J logits each (expert j LANES + lane), all of it in
// registers; what is largest comes from a reduction over the lanes, `top` times.
// Bound by these chains of dependent instructions, not by bytes.
//
// Which of two experts comes first must not depend on fp32 rounding.  Without a
// bias the scores have the logits' order, and the logits are compared: exact.
// With one (and for the groups' sums) the fp32 values decide only where they
// differ by more than both can be off; a row with a closer pair among its first
// top + 1, unless the two have the same logit and the same bias, is chosen again
// from 64-bit scores.  That is a row in a hundred or so for 256 experts.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "kernels_route.h"
#include "row_lanes.h"

namespace dtg {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr float kInf = __builtin_huge_valf();
constexpr int kNone = 1 << 30;

template <int KIND>
__device__ __forceinline__ float logit(const void* p, int64_t at) {
    if constexpr (KIND == 2) return static_cast<const float*>(p)[at];
    else return widen<KIND == 1>(static_cast<const uint16_t*>(p)[at]);
}

template <int LANES>
__device__ __forceinline__ float row_max(float v) {
    return __uint_as_float(lanes<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
template <int LANES>
__device__ __forceinline__ double row_max(double v) {
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) v = fmax(v, __shfl_xor(v, m));
    return v;
}
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
    return __uint_as_float(lanes<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int LANES>
__device__ __forceinline__ double row_sum(double v) {
#pragma unroll
    for (int m = 1; m < LANES; m <<= 1) v += __shfl_xor(v, m);
    return v;
}
template <int LANES>
__device__ __forceinline__ int row_min(int v) {
    return static_cast<int>(lanes<LANES>(static_cast<uint32_t>(v), [](uint32_t a, uint32_t b) { return a < b ? a : b; }));
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// 1 / (1 + e^-l), without the overflow of e^-l
template <typename F>
__device__ __forceinline__ F sigmoid(F l) {
    const F e = exp_of(l < 0 ? l : -l);
    return (l < 0 ? e : F(1)) / (1 + e);
}

// LDS written by some lanes of a wave and read by others: the hardware keeps a
// wave's LDS accesses in order, this keeps the compiler's.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The scores of a row from its logits (NaN as -inf: no score), the row's largest
// logit and, for a softmax, the reciprocal of its sum.  Infinite logits share
// the whole.
template <typename F, int LANES, int J>
__device__ __forceinline__ void scores(const float (&l)[J], bool sig, F (&s)[J], float& top, F& inv) {
    if (sig) {
#pragma unroll
        for (int j = 0; j < J; ++j) s[j] = sigmoid<F>(l[j]);
        return;
    }
    top = l[0];
#pragma unroll
    for (int j = 1; j < J; ++j) top = fmaxf(top, l[j]);
    top = row_max<LANES>(top);
    F sum = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        s[j] = l[j] == top ? F(1) : exp_of(F(l[j]) - F(top));
        sum += s[j];
    }
    inv = F(1) / row_sum<LANES>(sum);
#pragma unroll
    for (int j = 0; j < J; ++j) s[j] *= inv;
}

// The ids of a row from its choice values c (-inf: not to be had), by F's
// comparisons; part: what the groups' strengths are summed from.  True where a
// difference that decided is at most tol, of sums four times group_tol (below
// 0: none is).
template <typename F, int LANES, int J, int KIND>
__device__ __forceinline__ bool choose(const RouteArgs& a, int64_t row, int lane, F (&c)[J], const F (&part)[J], F tol,
                                       F group_tol, F* shared, int* ids) {
    constexpr F none = -static_cast<F>(kInf);
    bool close = false;
    if (a.groups > 1) {
        const int G = a.groups, per = a.E / G;
        wave_lds_fence();
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (j * LANES + lane < a.E) shared[j * LANES + lane] = part[j];
        wave_lds_fence();
        // P lanes to a group, each the best two of its share; the groups start
        // at different places, which spreads their reads over the banks
        int P = 1;
        while (2 * P * G <= LANES) P *= 2;
        const int g = lane / P, p = lane % P, n = (per + P - 1) / P;
        F t1 = none, t2 = none;
        if (g < G) {
            int i = g % n;
            for (int k = 0; k < n; ++k) {
                const int m = p + P * i;
                if (m < per) {
                    const F v = shared[g * per + m];
                    t2 = fmax(t2, fmin(t1, v));
                    t1 = fmax(t1, v);
                }
                i = i + 1 == n ? 0 : i + 1;
            }
        }
        for (int x = 1; x < P; x <<= 1) {
            const F o1 = __shfl_xor(t1, x), o2 = __shfl_xor(t2, x);
            t2 = fmax(fmin(t1, o1), fmax(t2, o2));
            t1 = fmax(t1, o1);
        }
        F strength = p == 0 ? (a.group_best == 2 && t2 != none ? t1 + t2 : t1) : none;
        uint64_t kept = 0;
        F last = 0;
        for (int k = 0; k < a.top_groups; ++k) {
            const F m = row_max<LANES>(strength);
            if (m == none) break;
            const int at = row_min<LANES>(strength == m ? lane : kNone);
            kept |= uint64_t(1) << (at / P);
            if (lane == at) strength = none;
            last = m;
        }
        const F next = row_max<LANES>(strength);
        if (next != none && last - next <= 4 * group_tol) close = true;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t e = j * LANES + lane;
            if (!(kept >> ((e * a.per_group_inv >> 20) & 63) & 1)) c[j] = none;
        }
    }
    F before = 0;
    int before_at = 0;
    for (int t = 0; t <= a.top; ++t) {   // the last one only for its distance
        if (t == a.top && tol < 0) break;
        F m = c[0];
#pragma unroll
        for (int j = 1; j < J; ++j) m = fmax(m, c[j]);
        m = row_max<LANES>(m);
        if (m == none) {
            for (int k = t + lane; k < a.top; k += LANES) ids[k] = -1;
            break;
        }
        int at = kNone;
#pragma unroll
        for (int j = J - 1; j >= 0; --j)
            if (c[j] == m) at = j * LANES + lane;
        at = row_min<LANES>(at);
        if (t > 0 && before - m <= tol) {
            // the same logit and bias make the same score in any precision
            const int64_t r = row * a.sl;
            if (__float_as_uint(logit<KIND>(a.logits, r + at)) != __float_as_uint(logit<KIND>(a.logits, r + before_at)) ||
                (a.bias && __float_as_uint(a.bias[at]) != __float_as_uint(a.bias[before_at])))
                close = true;
        }
        if (t < a.top && lane == 0) ids[t] = at;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (j * LANES + lane == at) c[j] = none;
        before = m;
        before_at = at;
    }
    return close;
}

// A chosen expert's share before any normalization: of the chosen ones' largest
// logit where renormalized (nothing underflows that counts), else the score.
__device__ __forceinline__ float share(float l, bool sig, bool renorm, float most, float top, float inv) {
    if (!sig) return renorm ? (l == most ? 1.0f : expf(l - most)) : (l == top ? 1.0f : expf(l - top)) * inv;
    if (!renorm || most >= 0.0f) return sigmoid<float>(l);
    return (l == most ? 1.0f : expf(l - most)) / (1.0f + expf(l));
}

template <int LANES, int J, int KIND>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
    constexpr int ROWS = kThreads / LANES, SLOTS = kMaxTop / LANES;
    __shared__ int id_rows[ROWS][kMaxTop];
    extern __shared__ double part_rows[];   // with groups: E values a row
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    int* const ids = id_rows[slot];
    double* const shared = part_rows + static_cast<int64_t>(slot) * (a.E + 8);
    const bool sig = a.sigmoid != 0, renorm = a.renorm != 0;
    float b[J];
#pragma unroll
    for (int j = 0; j < J; ++j) b[j] = a.bias && j * LANES + lane < a.E ? a.bias[j * LANES + lane] : 0.0f;

    for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + slot; row < a.R; row += static_cast<int64_t>(gridDim.x) * ROWS) {
        float l[J];
        bool nan = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            l[j] = j * LANES + lane < a.E ? logit<KIND>(a.logits, row * a.sl + j * LANES + lane) : -kInf;
            if (l[j] != l[j]) {
                nan = true;
                l[j] = -kInf;
            }
        }
        // this row's lanes of the wave
        const uint64_t mine = LANES == 64 ? ~uint64_t(0) : ((uint64_t(1) << (LANES % 64)) - 1) << ((threadIdx.x & 63) / LANES * LANES);
        nan = (__ballot(nan) & mine) != 0;

        // what is compared: the logits themselves, or scores and group sums that rounding can confuse
        const bool sums = a.groups > 1 && a.group_best == 2;
        float top = 0.0f, inv = 0.0f, s[J];
        if (a.bias || sums || (!sig && !renorm)) scores<float, LANES, J>(l, sig, s, top, inv);
        if (!a.bias && !sums) {
            float c[J];
#pragma unroll
            for (int j = 0; j < J; ++j) c[j] = l[j];
            choose<float, LANES, J, KIND>(a, row, lane, c, l, -1.0f, -1.0f, reinterpret_cast<float*>(shared), ids);
        } else {
            // fills the choice values and the groups' terms from scores of either precision
            auto values = [&](const auto& p, auto& c, auto& part) {
                typedef std::remove_reference_t<decltype(c[0])> F;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const bool had = l[j] > -kInf && b[j] > -kInf;   // false for a NaN, too
                    const F none = -static_cast<F>(kInf);
                    part[j] = had ? p[j] + F(b[j]) : none;
                    c[j] = a.bias ? part[j] : F(l[j]);
                }
            };
            float c[J], part[J], size = 0.0f;
            values(s, c, part);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float v = s[j] + fabsf(b[j]);
                if (part[j] > -kInf && v < kInf) size = fmaxf(size, v);
            }
            // both scores' errors: up to 22 roundings of a sum and 8 of the rest each
            const float tol = row_max<LANES>(size) * 0x1p-17f;
            if (choose<float, LANES, J, KIND>(a, row, lane, c, part, a.bias ? tol : -1.0f, tol, reinterpret_cast<float*>(shared), ids)) {
                double s2[J], c2[J], part2[J], inv2;
                float top2;
                scores<double, LANES, J>(l, sig, s2, top2, inv2);
                values(s2, c2, part2);
                choose<double, LANES, J, KIND>(a, row, lane, c2, part2, -1.0, -1.0, shared, ids);
            }
        }
        wave_lds_fence();

        int id[SLOTS];
        float cl[SLOTS], u[SLOTS], most = -kInf, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int t = i * LANES + lane;
            id[i] = t < a.top ? ids[t] : -1;
            cl[i] = id[i] >= 0 ? logit<KIND>(a.logits, row * a.sl + id[i]) : -kInf;
            most = fmaxf(most, cl[i]);
        }
        if (renorm) most = row_max<LANES>(most);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            u[i] = id[i] >= 0 ? share(cl[i], sig, renorm, most, top, inv) : 0.0f;
            sum += u[i];
        }
        if (renorm) sum = row_sum<LANES>(sum);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int t = i * LANES + lane;
            if (t >= a.top) continue;
            float w = renorm && id[i] >= 0 ? u[i] / sum * a.scale : u[i] * a.scale;
            if (nan && id[i] >= 0) w = __builtin_nanf("");
            a.weights[row * a.top + t] = w;
            a.ids[row * a.top + t] = id[i];
        }
    }
}

// dl from dw: with g = scale dw on the chosen, u their normalized shares,
//     renormalized   softmax u (g - sum u g),  sigmoid u (1 - p) (g - sum u g)
//     as they are    softmax p (g - sum p g) over all experts,  sigmoid p (1 - p) g
// Ids outside [0, E) have no part in it; an id given twice counts twice.
template <int LANES, int J, int KIND>
__global__ __launch_bounds__(kThreads) void route_grad_kernel(RouteGradArgs a) {
    constexpr int ROWS = kThreads / LANES, SLOTS = kMaxTop / LANES;
    __shared__ int id_rows[ROWS][kMaxTop];
    __shared__ float d_rows[ROWS][kMaxTop];
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    int* const ids = id_rows[slot];
    float* const ds = d_rows[slot];
    const bool sig = a.sigmoid != 0, renorm = a.renorm != 0, all = !sig && !renorm;

    for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + slot; row < a.R; row += static_cast<int64_t>(gridDim.x) * ROWS) {
        float s[J], top = 0.0f, inv = 0.0f;
        if (all) {
            float l[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                l[j] = j * LANES + lane < a.E ? logit<KIND>(a.logits, row * a.sl + j * LANES + lane) : -kInf;
                if (l[j] != l[j]) l[j] = -kInf;
            }
            scores<float, LANES, J>(l, false, s, top, inv);
        }
        int id[SLOTS];
        float cl[SLOTS], g[SLOTS], u[SLOTS], most = -kInf, sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int t = i * LANES + lane;
            id[i] = t < a.top ? a.ids[row * a.top + t] : -1;
            if (id[i] >= a.E) id[i] = -1;
            cl[i] = id[i] >= 0 ? logit<KIND>(a.logits, row * a.sl + id[i]) : -kInf;
            g[i] = id[i] >= 0 ? a.dw[row * a.sg + t] * a.scale : 0.0f;
            most = fmaxf(most, cl[i]);
        }
        if (renorm) most = row_max<LANES>(most);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            u[i] = id[i] >= 0 ? share(cl[i], sig, renorm, most, top, inv) : 0.0f;
            sum += u[i];
        }
        if (renorm) {
            sum = row_sum<LANES>(sum);
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) u[i] = id[i] >= 0 ? u[i] / sum : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) dot = fmaf(u[i], g[i], dot);
        dot = sig && !renorm ? 0.0f : row_sum<LANES>(dot);
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int t = i * LANES + lane;
            if (t >= a.top) continue;
            float d = u[i] * (all ? g[i] : g[i] - dot);
            if (sig) d *= sigmoid<float>(-cl[i]);   // 1 - p
            ids[t] = id[i];
            ds[t] = id[i] >= 0 ? d : 0.0f;
        }
        wave_lds_fence();
        float out[J];
#pragma unroll
        for (int j = 0; j < J; ++j) out[j] = all ? -s[j] * dot : 0.0f;
        for (int t = 0; t < a.top; ++t) {
            const int e = ids[t];
            const float d = ds[t];
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j * LANES + lane == e) out[j] += d;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = j * LANES + lane;
            if (e >= a.E) continue;
            if constexpr (KIND == 2) static_cast<float*>(a.dl)[row * a.sd + e] = out[j];
            else static_cast<uint16_t*>(a.dl)[row * a.sd + e] = narrow<KIND == 1>(out[j]);
        }
    }
}

constexpr int64_t kMostGroups = int64_t(1) << 20;   // workgroups of a launch; each then takes several rows

// fn(lanes, logits a lane, kind) for E experts.
template <typename Fn>
hipError_t with_shape(int E, int groups, int kind, Fn&& fn) {
    const int L = E > 256 || groups > 16 ? 64 : 16;
    const int need = (E + L - 1) / L;
#define DTG_ROUTE(L_, J_)                                                                                      \
    if (L == L_ && need <= J_) {                                                                               \
        const std::integral_constant<int, L_> l;                                                               \
        const std::integral_constant<int, J_> j;                                                               \
        return kind == 2   ? fn(l, j, std::integral_constant<int, 2>{})                                        \
               : kind == 1 ? fn(l, j, std::integral_constant<int, 1>{})                                        \
                           : fn(l, j, std::integral_constant<int, 0>{});                                       \
    }
    DTG_ROUTE(16, 1)
    DTG_ROUTE(16, 2)
    DTG_ROUTE(16, 4)
    DTG_ROUTE(16, 8)
    DTG_ROUTE(16, 16)
    DTG_ROUTE(64, 1)
    DTG_ROUTE(64, 4)
    DTG_ROUTE(64, 8)
    DTG_ROUTE(64, 16)
#undef DTG_ROUTE
    return hipErrorInvalidValue;
}

unsigned grid_of(int64_t R, int rows) {
    const int64_t need = (R + rows - 1) / rows;
    return static_cast<unsigned>(need < kMostGroups ? need : kMostGroups);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int kind, hipStream_t stream) {
    return with_shape(a.E, a.groups, kind, [&](auto l, auto j, auto k) {
        constexpr int ROWS = kThreads / decltype(l)::value;
        const size_t lds = a.groups > 1 ? sizeof(double) * ROWS * (a.E + 8) : 0;
        hipLaunchKernelGGL((route_kernel<decltype(l)::value, decltype(j)::value, decltype(k)::value>), dim3(grid_of(a.R, ROWS)),
                           dim3(kThreads), lds, stream, a);
        return hipGetLastError();
    });
}

hipError_t launch_route_grad(const RouteGradArgs& a, int kind, hipStream_t stream) {
    return with_shape(a.E, 1, kind, [&](auto l, auto j, auto k) {
        constexpr int ROWS = kThreads / decltype(l)::value;
        hipLaunchKernelGGL((route_grad_kernel<decltype(l)::value, decltype(j)::value, decltype(k)::value>),
                           dim3(grid_of(a.R, ROWS)), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    });
}

}  // namespace dtg
