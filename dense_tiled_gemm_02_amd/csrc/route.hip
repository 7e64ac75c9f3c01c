// Routing of tokens to experts, and its gradient, for gfx950.  For a row of E
// logits l:
//
//     p = softmax(l) or sigmoid(l),  c = p + bias (the choice alone)
//     a group's strength = the sum of its best one or two c
//     ids = the `top` largest c within the strongest groups, lowest index first
//     w = scale p, divided by the sum of the chosen p where renormalized
//
// LANES lanes take a row, J consecutive logits each, all of it in registers.
// Every expert becomes one 32-bit key, 22 bits of its value above 10 of 1023 -
// index, so that one integer maximum over the lanes gives both, and equal values
// go to the lower index; a lane sorts its J keys by maxima and minima, and `top`
// rounds of (maximum of the lanes' first keys, that lane moves its list up) give
// the ids in order.  16 lanes where 16 logits each are enough: a round's maximum is
// then four moves inside a quarter wave, and a wave has four rows under way.
//
// Bound by instructions, not by bytes: 16384 x 256 in bf16, top 8, 8.9 us (softmax),
// 18.5 us (sigmoid with a bias), 21 us (and the best 4 of 8 groups by their best two);
// its bytes take 2.  512 experts 13, 30 and 34 us, 64 experts 5 to 11.  The gradient
// of 16384 x 256 8.8 to 9.4 us, of which its bytes are 3.5: each of a lane's J outputs
// is compared with every one of the `top` chosen.
//
// Which of two experts comes first must not depend on rounding.  fp16 and bf16
// logits without a bias are compared whole: the scores have the logits' order,
// and 16 bits fit a key.  Else a key's value is a fixed-point one of the logit (a
// window of 32 below the row's largest) or of the score with its bias, and two
// experts count as told apart only where their values differ by more than both
// can be off; a row with a closer pair among its first top + 1 (unless the two have
// the same logit and the same bias) or at the groups' border is chosen again from
// 64-bit scores in LDS.  That is a row in a hundred or so for 256 experts.
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
constexpr int kIndexBits = 10;                       // kMaxExperts
constexpr int kValues = 1 << (32 - kIndexBits);      // a key's values: 1 .. kValues - 1; 0: no such expert

template <int KIND>
__device__ __forceinline__ float logit(const void* p, int64_t at) {
    if constexpr (KIND == 2) return static_cast<const float*>(p)[at];
    else return widen<KIND == 1>(static_cast<const uint16_t*>(p)[at]);
}

struct MaxU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct MinU {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a < b ? a : b; }
};
struct MaxF {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
};
struct AddF {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }
};
template <int LANES>
__device__ __forceinline__ float row_max(float v) { return __uint_as_float(lanes<LANES>(__float_as_uint(v), MaxF())); }
template <int LANES>
__device__ __forceinline__ float row_sum(float v) { return __uint_as_float(lanes<LANES>(__float_as_uint(v), AddF())); }
template <int LANES>
__device__ __forceinline__ int row_min(int v) { return static_cast<int>(lanes<LANES>(static_cast<uint32_t>(v), MinU())); }
template <int LANES>
__device__ __forceinline__ double row_max(double v) {
    for (int m = 1; m < LANES; m <<= 1) v = fmax(v, __shfl_xor(v, m));
    return v;
}
template <int LANES>
__device__ __forceinline__ double row_sum(double v) {
    for (int m = 1; m < LANES; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// e^v by the hardware's 2^t, with t's rounding made up for: for v up to 88 three
// steps of 2^-24 off at most (the bare 2^t: |v| steps), and 0 where e^v is below
// 2^-126.  Past 88 it stays at e^88: an infinite 2^t times a rest that is zero or
// negative would be a NaN.  Only the scores of a sigmoid ask for such a v, and
// their 1 / (1 + e^88) is zero to every key.
__device__ __forceinline__ float quick_exp(float v) {
    constexpr float hi = 1.44269502f, lo = 1.92596299e-8f, ln2 = 0.693147181f;   // hi + lo = log2 e
    v = fminf(fmaxf(v, -200.0f), 88.0f);
    const float t = v * hi, rest = fmaf(v, lo, fmaf(v, hi, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, rest * ln2, e);
}

// 1 / (1 + e^-l), without the overflow of e^-l
__device__ __forceinline__ float sigmoid(float l) {
    const float e = quick_exp(l < 0 ? l : -l);
    return (l < 0 ? e : 1.0f) / (1.0f + e);
}

// LDS written by some lanes of a wave and read by others: the hardware keeps a
// wave's LDS accesses in order, this keeps the compiler's.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// J consecutive logits of a row from e on, those below E; the others are -inf,
// NaN ones too (and `nan` is set).
template <int J, int KIND>
__device__ __forceinline__ void load_logits(const void* logits, int64_t row_at, int e, int E, float (&l)[J], bool& nan) {
    constexpr int SIZE = KIND == 2 ? 4 : 2;
    struct __attribute__((packed, aligned(SIZE))) Block {
        uint16_t h[J * SIZE / 2];
    };
    const char* const row = static_cast<const char*>(logits) + row_at * SIZE;
    if (e + J <= E) {
        const Block b = *reinterpret_cast<const Block*>(row + e * SIZE);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if constexpr (KIND == 2) l[j] = __uint_as_float(b.h[2 * j] | static_cast<uint32_t>(b.h[2 * j + 1]) << 16);
            else l[j] = widen<KIND == 1>(b.h[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j) {   // all of them, some the last one again: loads that wait for one another cost more
            const float v = logit<KIND>(row, e + j < E ? e + j : E - 1);
            l[j] = e + j < E ? v : -kInf;
        }
    }
    nan = false;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const bool bad = l[j] != l[j];
        nan = nan | bad;
        l[j] = bad ? -kInf : l[j];
    }
}

template <int LANES, int J>
__device__ __forceinline__ float largest(const float (&l)[J]) {
    float top = l[0];
#pragma unroll
    for (int j = 1; j < J; ++j) top = fmaxf(top, l[j]);
    return row_max<LANES>(top);
}

// The scores of a row by quick_exp and the hardware's reciprocal (a few steps of
// 2^-24 of each score off, which is what the keys allow for) and, for a softmax,
// the reciprocal of the sum.  top: the row's largest logit; infinite logits
// share the whole.
template <int LANES, int J>
__device__ __forceinline__ void scores(const float (&l)[J], bool sig, float top, float (&s)[J], float& inv) {
    if (sig) {
#pragma unroll
        for (int j = 0; j < J; ++j) s[j] = __builtin_amdgcn_rcpf(1.0f + quick_exp(-l[j]));
        return;
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        s[j] = l[j] == top ? 1.0f : quick_exp(l[j] - top);
        sum += s[j];
    }
    inv = 1.0f / row_sum<LANES>(sum);
#pragma unroll
    for (int j = 0; j < J; ++j) s[j] *= inv;
}

__device__ __forceinline__ uint32_t key_of(uint32_t value, int e) { return value << kIndexBits | (kMaxExperts - 1 - e); }
__device__ __forceinline__ int expert_of(uint32_t key) { return kMaxExperts - 1 - static_cast<int>(key & (kMaxExperts - 1)); }
__device__ __forceinline__ int value_of(uint32_t key) { return static_cast<int>(key >> kIndexBits); }

// 16-bit logits in their order, from the fp32 that they were widened to: its
// upper bits hold all of them.  Both zeros are one value.
template <bool BF16>
__device__ __forceinline__ uint32_t whole_value(float l) {
    const uint32_t x = __float_as_uint(l + 0.0f);
    return (x ^ (static_cast<uint32_t>(static_cast<int>(x) >> 31) | 0x80000000u)) >> (BF16 ? 16 : 13);
}

// A logit in a window of 32 below the row's largest: steps of 2^-17.  Equal
// logits have equal values; values two steps apart are in the logits' order (the
// difference and its scaling are each off by a quarter of a step, and the rest is
// cut off).  What lies below the window is one value.
constexpr int kWindowClose = 1;
__device__ __forceinline__ uint32_t window_value(float l, float top) {
    const float v = l == top ? 0.0f : l - top;
    return 1 + static_cast<uint32_t>(fmaxf(fmaf(v, (kValues - 4) / 32.0f, kValues - 4.0f), 0.0f));
}

// A score with its bias, in -size .. size: steps of 2^-21 size.  Each such fp32
// value is off by at most 8 roundings of 2^-24 size, one step, and by a quarter
// of one here; two of them and the cut-off make less than 4.  A softmax's sum
// (up to 22 roundings) is off for all alike, which moves two scores by at most
// 2.75 steps against each other.
constexpr int kSigmoidClose = 4, kSoftmaxClose = 7;
constexpr float kScoreHalf = kValues / 2 - 2.0f;
__device__ __forceinline__ uint32_t score_value(float c, float by_size) {
    return 1 + static_cast<uint32_t>(fminf(fmaxf(fmaf(c * by_size, kScoreHalf, kScoreHalf), 0.0f), 2 * kScoreHalf));
}

// Descending, by Batcher's merge-exchange network on J (a power of two) keys.
template <int J>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[J]) {
#pragma unroll
    for (int p = 1; p < J; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < J; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (j + i + q < J && (j + i) / (2 * p) == (j + i + q) / (2 * p)) {
                        const uint32_t a = k[j + i], b = k[j + i + q];
                        k[j + i] = a > b ? a : b;
                        k[j + i + q] = a > b ? b : a;
                    }
}

// The groups that take part, as bits.  part: every expert's key, best: how many of
// a group's keys make its strength.  close is set where two strengths at the
// border differ by at most `far` values.
template <int LANES, int J>
__device__ __forceinline__ uint64_t strongest(const RouteArgs& a, int lane, const uint32_t (&part)[J], int far, uint32_t* shared,
                                              bool& close) {
    const int G = a.groups, per = a.per, P = 1 << a.lane_shift;   // lane g P holds group g in the end
    const bool two = a.group_best == 2;
    const int g = lane >> a.lane_shift, p = lane & (P - 1);
    uint32_t t1 = 0, t2 = 0;
    if (a.in_lanes) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t v = part[j];
            t2 = MaxU()(t2, MinU()(t1, v));
            t1 = MaxU()(t1, v);
        }
    } else {
        // through LDS, each lane the best two of its share of a group; the groups
        // start at different places, which spreads their reads over the banks
        wave_lds_fence();
#pragma unroll
        for (int j = 0; j < J; ++j) shared[lane * J + j] = part[j];
        wave_lds_fence();
        const int n = (per + P - 1) >> a.lane_shift;
        int i = g < n ? g : 0;
        if (g < G)
#pragma unroll 2
            for (int k = 0; k < n; ++k) {
                const int m = p + P * i;
                const uint32_t v = shared[g * per + (m < per ? m : p)];
                const uint32_t w = m < per ? v : 0;
                t2 = MaxU()(t2, MinU()(t1, w));
                t1 = MaxU()(t1, w);
                i = i + 1 == n ? 0 : i + 1;
            }
    }
    for (int x = 1; x < P; x <<= 1) {
        const uint32_t o1 = __shfl_xor(static_cast<int>(t1), x), o2 = __shfl_xor(static_cast<int>(t2), x);
        t2 = MaxU()(MinU()(t1, o1), MaxU()(t2, o2));
        t1 = MaxU()(t1, o1);
    }
    // a strength as a key again: a sum's values over the group's place from behind (a group
    // with one expert left has a sum with zero, which the scores' middle value is)
    uint32_t strength = t1;
    if (two && t1 != 0) strength = (value_of(t1) + (t2 != 0 ? value_of(t2) : 1 + static_cast<int>(kScoreHalf))) << 7 | (63 - g);
    if (p != 0 || g >= G) strength = 0;
    uint64_t kept = 0;
    uint32_t last = 0;
    for (int k = 0; k < a.top_groups; ++k) {
        const uint32_t m = lanes<LANES>(strength, MaxU());
        if (m == 0) break;
        kept |= uint64_t(1) << (two ? 63 - (m & 63) : static_cast<uint32_t>(expert_of(m)) * a.per_group_inv >> 20);
        if (strength == m) strength = 0;
        last = m;
    }
    const uint32_t next = lanes<LANES>(strength, MaxU());
    const int shift = two ? 7 : kIndexBits;
    if (next != 0 && static_cast<int>(last >> shift) - static_cast<int>(next >> shift) <= far) close = true;
    return kept;
}

// 64-bit values of a row: loops without unrolling, since few rows come here and
// instructions that are not in the cache yet cost more than they do.
template <int LANES, int KIND>
struct Exact {
    const RouteArgs& a;
    int64_t at;         // the row's first logit
    int lane;
    float top;          // the largest logit
    double inv = 0.0;   // the reciprocal of the softmax's sum, once it is asked for

    __device__ float value(int e) const {
        const float l = logit<KIND>(a.logits, at + e);
        return l == l ? l : -kInf;
    }
    __device__ void sum() {
        if (a.sigmoid || inv != 0.0) return;
        double s = 0.0;
#pragma unroll 1
        for (int e = lane; e < a.E; e += LANES) {
            const float l = value(e);
            s += l == top ? 1.0 : exp(static_cast<double>(l) - static_cast<double>(top));
        }
        inv = 1.0 / row_sum<LANES>(s);
    }
    // an expert's score with its bias, or its logit; -inf where it is not to be had
    __device__ double of(int e, bool by_score) const {
        const float l = value(e), b = a.bias ? a.bias[e] : 0.0f;
        double v = l;
        if (by_score) {
            const double x = a.sigmoid ? -fabs(v) : v - static_cast<double>(top);
            const double ex = !a.sigmoid && l == top ? 1.0 : exp(x);
            v = (a.sigmoid ? (l < 0 ? ex : 1.0) / (1.0 + ex) : ex * inv) + static_cast<double>(b);
        }
        return l > -kInf && b > -kInf ? v : -static_cast<double>(kInf);
    }
    __device__ void fill(double* shared, bool by_score, uint64_t kept) {
        if (by_score) sum();
        wave_lds_fence();
#pragma unroll 1
        for (int e = lane; e < a.E; e += LANES)
            shared[e] = kept >> ((e * a.per_group_inv >> 20) & 63) & 1 ? of(e, by_score) : -static_cast<double>(kInf);
        wave_lds_fence();
    }
    __device__ uint64_t strongest(double* shared, bool by_score) {
        const double none = -static_cast<double>(kInf);
        const int G = a.groups, per = a.per;
        fill(shared, by_score, ~uint64_t(0));
        double t1 = none, t2 = none;
        if (lane < G)
#pragma unroll 4
            for (int m = 0; m < per; ++m) {
                const double v = shared[lane * per + m];
                t2 = fmax(t2, fmin(t1, v));
                t1 = fmax(t1, v);
            }
        double strength = a.group_best == 2 && t2 != none ? t1 + t2 : t1;
        uint64_t kept = 0;
#pragma unroll 1
        for (int k = 0; k < a.top_groups; ++k) {
            const double m = row_max<LANES>(strength);
            if (m == none) break;
            const int g = row_min<LANES>(strength == m ? lane : kNone);
            kept |= uint64_t(1) << g;
            if (lane == g) strength = none;
        }
        return kept;
    }
    // the best of n candidates in ids, in order
    __device__ void rank(double* shared, int* ids, int n, bool by_score) {
        if (by_score) sum();
        wave_lds_fence();
#pragma unroll 1
        for (int i = lane; i < n; i += LANES) shared[i] = of(ids[i], by_score);
        wave_lds_fence();
        int id[kMaxTop / LANES], place[kMaxTop / LANES];
#pragma unroll
        for (int s = 0; s < kMaxTop / LANES; ++s) {
            const int i = s * LANES + lane;
            id[s] = i < n ? ids[i] : 0;
            place[s] = n;
            if (i >= n) continue;
            const double v = shared[i];
            int before = 0;
#pragma unroll 1
            for (int k = 0; k < n; ++k) {
                const double o = shared[k];
                before += o > v || (o == v && ids[k] < id[s]) ? 1 : 0;
            }
            place[s] = before;
        }
        wave_lds_fence();
#pragma unroll
        for (int s = 0; s < kMaxTop / LANES; ++s)
            if (place[s] < n) ids[place[s]] = id[s];
    }
    // all ids anew
    __device__ void choose(double* shared, int* ids, bool by_score, uint64_t kept) {
        const double none = -static_cast<double>(kInf);
        fill(shared, by_score, kept);
#pragma unroll 1
        for (int t = 0; t < a.top; ++t) {
            double m = none;
            int mine = kNone;
#pragma unroll 1
            for (int e = lane; e < a.E; e += LANES) {
                const double v = shared[e];
                if (v > m) {
                    m = v;
                    mine = e;
                }
            }
            const double most = row_max<LANES>(m);
            const int id = row_min<LANES>(m == most && most != none ? mine : kNone);
            if (lane == 0) ids[t] = id == kNone ? -1 : id;
            if (mine == id && id != kNone) shared[id] = none;
            wave_lds_fence();
        }
    }
};

// A chosen expert's share before any normalization: of the chosen ones' largest
// logit where renormalized (nothing underflows that counts), else the score.
__device__ __forceinline__ float share(float l, bool sig, bool renorm, float most, float top, float inv) {
    const bool plain = sig && (!renorm || most >= 0.0f);
    const float from = renorm ? most : top;
    const float e = l == from && !plain ? 1.0f : quick_exp(plain ? -fabsf(l) : l - from);
    if (!sig) return renorm ? e : e * inv;
    const float under = 1.0f + (plain ? e : quick_exp(l));
    return (plain && l >= 0.0f ? 1.0f : e) / under;
}

// SCORED: scores are compared (a bias, or the sums of groups), else logits alone.
template <int LANES, int J, int KIND, bool SCORED>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
    constexpr int ROWS = kThreads / LANES;
    constexpr bool WHOLE = KIND != 2;   // logits fit a key
    __shared__ int id_rows[ROWS][kMaxTop];
    extern __shared__ double spare[];   // E values a row, or LANES x J keys
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES, e0 = lane * J;
    int* const ids = id_rows[slot];
    double* const shared = spare + slot * a.spare;
    const bool sig = a.sigmoid != 0, renorm = a.renorm != 0, biased = SCORED && a.bias != nullptr;
    const bool grouped = a.groups > 1, sums = SCORED && grouped && a.group_best == 2;
    // this row's lanes of the wave
    const uint64_t mine = LANES == 64 ? ~uint64_t(0) : ((uint64_t(1) << (LANES % 64)) - 1) << ((threadIdx.x & 63) / LANES * LANES);

    // one row, without a loop: what a loop's compiler takes out of it costs half the registers
    const int64_t row = a.first + static_cast<int64_t>(blockIdx.x) * ROWS + slot;
    if (row >= a.R) return;
    float l[J], b[SCORED ? J : 1];
    bool nan;
    if constexpr (SCORED) {
#pragma unroll
        for (int j = 0; j < J; ++j) b[j] = biased ? a.bias[e0 + j < a.E ? e0 + j : a.E - 1] : 0.0f;
    }
    load_logits<J, KIND>(a.logits, row * a.sl, e0, a.E, l, nan);
    nan = (__ballot(nan) & mine) != 0;

    float top = 0.0f, inv = 0.0f, s[J];
    const bool shares = !sig && !renorm;   // the weights need the softmax's sum
    if (SCORED || !WHOLE || shares) top = largest<LANES, J>(l);
    if (SCORED || shares) scores<LANES, J>(l, sig, top, s, inv);
    Exact<LANES, KIND> exact{a, row * a.sl, lane, top};
    uint32_t key[J];
    int far = -1;   // values closer than this are not told apart
    bool close = false;
    uint64_t kept = ~uint64_t(0);
    if constexpr (SCORED) {
        float size = 0x1p-100f;
        bool endless = false;   // an infinite bias has no fixed-point value
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool had = (l[j] > -kInf) & (b[j] > -kInf);   // false for a NaN, too
            const float v = s[j] + fabsf(b[j]);
            s[j] = had ? s[j] + b[j] : -kInf;
            size = (had & (v < kInf)) ? fmaxf(size, v) : size;
            endless = endless | (had & (b[j] == kInf));
        }
        close = (__ballot(endless) & mine) != 0;
        const float by_size = 1.0f / row_max<LANES>(size);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t k = key_of(score_value(s[j], by_size), e0 + j);
            key[j] = s[j] > -kInf ? k : 0;
        }
        far = sig ? kSigmoidClose : kSoftmaxClose;
        if (grouped) {
            bool border = close;
            kept = strongest<LANES, J>(a, lane, key, sums ? 2 * far : far, reinterpret_cast<uint32_t*>(shared), border);
            if (__builtin_expect(border, 0)) kept = exact.strongest(shared, true);
        }
    }
    if (!biased) {   // the logits have the scores' order
        far = WHOLE ? -1 : kWindowClose;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            uint32_t v;
            if constexpr (WHOLE) v = whole_value<KIND == 1>(l[j]);
            else v = window_value(l[j], top);
            v = key_of(v, e0 + j);
            key[j] = l[j] > -kInf ? v : 0;
        }
        if (grouped && !sums) {
            bool border = false;
            kept = strongest<LANES, J>(a, lane, key, far, reinterpret_cast<uint32_t*>(shared), border);
            if (!WHOLE && __builtin_expect(border, 0)) kept = exact.strongest(shared, false);
        }
    }
    if (grouped) {
#pragma unroll
        for (int j = 0; j < J; ++j) key[j] = kept >> (((e0 + j) * a.per_group_inv >> 20) & 63) & 1 ? key[j] : 0;
    }
    sort_keys<J>(key);
    uint32_t before = 0;
    int n = 0;   // ids so far: `top` of them, or more where those after the last are close to it
    for (; n < kMaxTop; ++n) {
        const uint32_t m = lanes<LANES>(key[0], MaxU());
        if (m == 0) break;
        const int at = expert_of(m);
        const bool near = n > 0 && value_of(before) - value_of(m) <= far;
        if (n >= a.top && !near) break;
        if (__builtin_expect(near, 0)) {
            // the same logit and bias make the same score in any precision
            const int other = expert_of(before);
            const int64_t r = row * a.sl;
            if (__float_as_uint(logit<KIND>(a.logits, r + at)) != __float_as_uint(logit<KIND>(a.logits, r + other)) ||
                (biased && __float_as_uint(a.bias[at]) != __float_as_uint(a.bias[other])))
                close = true;
        }
        if (lane == 0) ids[n] = at;
        // by masks: selects of neighbours become an index, and that a search
        const uint32_t moved = key[0] == m ? ~0u : 0u;
#pragma unroll
        for (int j = 0; j + 1 < J; ++j) key[j] = (key[j + 1] & moved) | (key[j] & ~moved);
        key[J - 1] &= ~moved;
        before = m;
    }
    bool all = true;   // that are close to one another are in ids
    if constexpr (SCORED || !WHOLE) {
        if (n == kMaxTop) {
            const uint32_t m = lanes<LANES>(key[0], MaxU());
            all = m == 0 || value_of(before) - value_of(m) > far;
        }
    }
    for (int k = n + lane; k < a.top; k += LANES) ids[k] = -1;
    if constexpr (SCORED || !WHOLE) {
        if (__builtin_expect(close | !all, 0)) {
            wave_lds_fence();
            if (all) exact.rank(shared, ids, n, biased);
            else exact.choose(shared, ids, biased, kept);
        }
    }
    wave_lds_fence();

    float most = -kInf, sum = 1.0f;
    const int64_t at = row * a.sl;
    if (renorm) {
#pragma unroll 1
        for (int t = lane; t < a.top; t += LANES)
            if (ids[t] >= 0) most = fmaxf(most, logit<KIND>(a.logits, at + ids[t]));
        most = row_max<LANES>(most);
        sum = 0.0f;
#pragma unroll 1
        for (int t = lane; t < a.top; t += LANES)
            if (ids[t] >= 0) sum += share(logit<KIND>(a.logits, at + ids[t]), sig, true, most, top, inv);
        sum = row_sum<LANES>(sum);
    }
#pragma unroll 1
    for (int t = lane; t < a.top; t += LANES) {
        const int id = ids[t];
        float w = 0.0f;
        if (id >= 0) w = nan ? __builtin_nanf("") : share(logit<KIND>(a.logits, at + id), sig, renorm, most, top, inv) / sum * a.scale;
        a.weights[row * a.top + t] = w;
        a.ids[row * a.top + t] = id;
    }
}

// J consecutive values of a row from e on, those below E, in the logits' type.
template <int J, int KIND>
__device__ __forceinline__ void store_logits(void* dl, int64_t row_at, int e, int E, const float (&v)[J]) {
    if constexpr (KIND == 2) {
        struct __attribute__((packed, aligned(4))) Block {
            float f[J];
        };
        float* const to = static_cast<float*>(dl) + row_at + e;
        if (e + J <= E) {
            Block b;
#pragma unroll
            for (int j = 0; j < J; ++j) b.f[j] = v[j];
            *reinterpret_cast<Block*>(to) = b;
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (e + j < E) to[j] = v[j];
        }
    } else {
        struct __attribute__((packed, aligned(2))) Block {
            uint16_t h[J];
        };
        uint16_t* const to = static_cast<uint16_t*>(dl) + row_at + e;
        Block b;
#pragma unroll
        for (int j = 0; j < J; ++j) b.h[j] = narrow<KIND == 1>(v[j]);
        if (e + J <= E) {
            *reinterpret_cast<Block*>(to) = b;
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (e + j < E) to[j] = b.h[j];
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
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES, e0 = lane * J;
    int* const ids = id_rows[slot];
    float* const ds = d_rows[slot];
    const bool sig = a.sigmoid != 0, renorm = a.renorm != 0, all = !sig && !renorm;

    const int64_t row = a.first + static_cast<int64_t>(blockIdx.x) * ROWS + slot;
    if (row >= a.R) return;
    float s[J], top = 0.0f, inv = 0.0f;
    if (all) {
        float l[J];
        bool nan;
        load_logits<J, KIND>(a.logits, row * a.sl, e0, a.E, l, nan);
        top = largest<LANES, J>(l);
        scores<LANES, J>(l, false, top, s, inv);
    }
    int id[SLOTS];
    float cl[SLOTS], g[SLOTS], u[SLOTS], most = -kInf, sum = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        const int t = i * LANES + lane;
        id[i] = t < a.top ? a.ids[row * a.top + t] : -1;
        if (id[i] >= a.E) id[i] = -1;
        cl[i] = id[i] >= 0 ? logit<KIND>(a.logits, row * a.sl + id[i]) : -kInf;
        g[i] = id[i] >= 0 ? a.dw[row * a.top + t] * a.scale : 0.0f;
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
        if (sig) d *= sigmoid(-cl[i]);   // 1 - p
        ids[t] = id[i];
        ds[t] = id[i] >= 0 ? d : 0.0f;
    }
    wave_lds_fence();
    float out[J];
#pragma unroll
    for (int j = 0; j < J; ++j) out[j] = all ? -s[j] * dot : 0.0f;
    for (int t = 0; t < a.top; ++t) {
        const int e = ids[t] - e0;
        const float d = ds[t];
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (j == e) out[j] += d;
    }
    store_logits<J, KIND>(a.dl, row * a.E, e0, a.E, out);
}

// Rows of a launch: of more, several follow one another.
constexpr int64_t kMostRows = int64_t(1) << 24;

// fn(lanes, logits a lane, kind) for E experts; GROUPED: there can be groups, which
// want a lane each.
template <bool GROUPED, typename Fn>
hipError_t with_shape(int E, int groups, int kind, Fn&& fn) {
    const int L = E > 512 || groups > 32 ? 64 : E > 256 || groups > 16 ? 32 : 16;
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
    if constexpr (GROUPED) {
        DTG_ROUTE(32, 1)
        DTG_ROUTE(32, 4)
        DTG_ROUTE(64, 1)
        DTG_ROUTE(64, 4)
    }
    DTG_ROUTE(32, 16)
    DTG_ROUTE(64, 16)
#undef DTG_ROUTE
    return hipErrorInvalidValue;
}

unsigned grid_of(int64_t rows, int per) { return static_cast<unsigned>(((rows < kMostRows ? rows : kMostRows) + per - 1) / per); }

}  // namespace

hipError_t launch_route(const RouteArgs& a, int kind, hipStream_t stream) {
    return with_shape<true>(a.E, a.groups, kind, [&](auto l, auto j, auto k) {
        constexpr int ROWS = kThreads / decltype(l)::value;
        // rows that are compared whole need no second choice, and no room for groups where they are lanes
        const bool spare = a.bias || a.groups > 1 || decltype(k)::value == 2;
        constexpr int L = decltype(l)::value, J = decltype(j)::value;
        RouteArgs g = a;
        g.spare = a.E > L * J / 2 ? a.E : L * J / 2;
        const size_t lds = spare ? sizeof(double) * ROWS * g.spare : 0;
        g.per = a.E / a.groups;
        const int own = g.per % J == 0 ? g.per / J : 0;   // lanes that hold one group, if they hold nothing else
        g.in_lanes = own > 0 && (own & (own - 1)) == 0 && own * a.groups <= L;
        g.lane_shift = 0;
        while ((g.in_lanes ? 1 << g.lane_shift < own : (2 << g.lane_shift) * a.groups <= L)) ++g.lane_shift;
        const bool scored = a.bias || (a.groups > 1 && a.group_best == 2);
        for (g.first = 0; g.first < a.R; g.first += kMostRows) {
            const dim3 grid(grid_of(a.R - g.first, ROWS)), block(kThreads);
            if (scored) hipLaunchKernelGGL((route_kernel<L, J, decltype(k)::value, true>), grid, block, lds, stream, g);
            else hipLaunchKernelGGL((route_kernel<L, J, decltype(k)::value, false>), grid, block, lds, stream, g);
        }
        return hipGetLastError();
    });
}

hipError_t launch_route_grad(const RouteGradArgs& a, int kind, hipStream_t stream) {
    return with_shape<false>(a.E, 1, kind, [&](auto l, auto j, auto k) {
        constexpr int ROWS = kThreads / decltype(l)::value;
        RouteGradArgs g = a;
        for (g.first = 0; g.first < a.R; g.first += kMostRows)
            hipLaunchKernelGGL((route_grad_kernel<decltype(l)::value, decltype(j)::value, decltype(k)::value>),
                               dim3(grid_of(a.R - g.first, ROWS)), dim3(kThreads), 0, stream, g);
        return hipGetLastError();
    });
}

}  // namespace dtg
