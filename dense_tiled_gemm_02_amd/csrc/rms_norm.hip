// RMS norm with the residual's addition, rows in 8 bits, and the norm's
// gradients, for gfx950.  One row of K values:
//
//     h = x + r (rounded to the stream's type),  n = sqrt(mean h^2 + eps)
//     y = h w / n                                      (16-bit output)
//     s = max |y| / 127,  q = y / s to the nearest     (int8 output)
//
// All of it from one read: T threads hold the row in registers, C chunks of 8
// values each, packed as they are stored (what is summed has been rounded to 16
// bits), with the sums across them through the wave's lanes and, where a row
// takes more than a wave, one LDS word per wave and one barrier.  Bound by memory:
// x, r are read and y or q (and h) are written once (8192 x 4096 with a residual 45
// us, 5.9 TB/s; into int8 46; 4096 x 14336 into int8 alone 33).  Rows longer than the
// registers hold are read again for each pass (C = 0); kMaxRow keeps their sums
// (a chunk's 8, then up to 2048 chunks a thread, in a row) within 2^-13.
//
// The quotient y / s is defined as an IEEE division by the stored scale, rounded
// to the nearest integer; see steps_of for how most of it is done without one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "kernels_layer.h"
#include "row_lanes.h"

namespace dtg {
namespace {

using namespace dev;

// 16 and 8 bytes at any address that their elements' alignment allows.
struct __attribute__((packed, aligned(2))) Loose16 {
    u32x4 v;
};
struct __attribute__((packed, aligned(1))) Loose8 {
    u32x2 v;
};
struct __attribute__((packed, aligned(4))) LooseF4 {
    f32x4 v;
};

constexpr float kInf = __builtin_huge_valf();

struct Add {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }
};
// Magnitudes as bits: their order as integers is their order, and any NaN is above infinity.
struct Max {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// op over the T threads of a row.  Rows of several waves meet in LDS: the two
// halves of `meet` take turns, so one barrier a call is enough (a half is
// written again only after the next call's barrier, which every reader of it
// has reached).
template <int T>
struct Meet {
    uint32_t* at;
    int turn = 0;
    template <typename Op>
    __device__ uint32_t all(uint32_t v, Op op) {
        if constexpr (T <= 64) {
            return lanes<T>(v, op);
        } else {
            v = lanes<64>(v, op);
            uint32_t* m = at + turn * (T / 64);
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) m[threadIdx.x / 64] = v;
            __syncthreads();
            v = m[0];
#pragma unroll
            for (int i = 1; i < T / 64; ++i) v = op(v, m[i]);
            return v;
        }
    }
    __device__ float sum(float v) { return __uint_as_float(all(__float_as_uint(v), Add())); }
    __device__ float most(float v) { return __uint_as_float(all(__float_as_uint(v), Max())); }
};

// Elements k .. k + 7 of a row of K (zeros past its end).
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int k, int K) {
    u32x4 u = {0u, 0u, 0u, 0u};
    if (k + 8 <= K) {
        u = reinterpret_cast<const Loose16*>(row + k)->v;
    } else if (k < K) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (k + e < K) u[e / 2] |= static_cast<uint32_t>(row[k + e]) << (16 * (e % 2));
    }
    return u;
}

__device__ __forceinline__ void store8(uint16_t* row, int k, int K, u32x4 u) {
    if (k + 8 <= K) {
        reinterpret_cast<Loose16*>(row + k)->v = u;
    } else if (k < K) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (k + e < K) row[k + e] = static_cast<uint16_t>(u[e / 2] >> (16 * (e % 2)));
    }
}

template <bool BF16>
__device__ __forceinline__ void widen8(u32x4 u, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = widen<BF16>(static_cast<uint16_t>(u[e / 2] >> (16 * (e % 2))));
}

template <bool BF16>
__device__ __forceinline__ u32x4 narrow8(const float (&v)[8]) {
    u32x4 u;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        u[e] = narrow<BF16>(v[2 * e]) | static_cast<uint32_t>(narrow<BF16>(v[2 * e + 1])) << 16;
    return u;
}

// Elements k .. k + 7 of the weights, all of them there.
template <bool BF16>
__device__ __forceinline__ void whole_weights8(const void* w, int w32, int k, float (&v)[8]) {
    if (w32) {
        const float* p = static_cast<const float*>(w) + k;
        const f32x4 lo = reinterpret_cast<const LooseF4*>(p)->v, hi = reinterpret_cast<const LooseF4*>(p + 4)->v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
    } else {
        widen8<BF16>(reinterpret_cast<const Loose16*>(static_cast<const uint16_t*>(w) + k)->v, v);
    }
}

// Elements k .. k + 7 of the weights (zeros past the end).
template <bool BF16>
__device__ __forceinline__ void weights8(const void* w, int w32, int k, int K, float (&v)[8]) {
    if (w32) {
        const float* p = static_cast<const float*>(w);
        if (k + 8 <= K) {
            const f32x4 lo = reinterpret_cast<const LooseF4*>(p + k)->v, hi = reinterpret_cast<const LooseF4*>(p + k + 4)->v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = k + e < K ? p[k + e] : 0.0f;
        }
    } else {
        widen8<BF16>(load8(static_cast<const uint16_t*>(w), k, K), v);
    }
}

// bf16 values whose squares fp32 cannot hold.  Where the mean plus eps is infinite
// (values past 1e19, or the largest eps), it is taken again, of values scaled by
// kSmaller.  Where eps is below kLeastEps, squares below 2^-126 can count beside it
// and have lost their last bits: such a launch scales all values by kLarger
// (RowsArgs::by; powers of two change no other bit), and eps by its square, which is
// then 2^-117 and more.  Values that overflow with that, 2^36 and more, are not lost
// to kSmaller.  Rows held in registers are not scaled (16384 x 2048 into int8 44.4
// us, 46.1 with the factor), so these launches take shapes that read rows again.
constexpr float kSmaller = 0x1p-80f, kLarger = 0x1p16f, kLeastEps = 0x1p-100f;

// Eight quotients v / s as bytes.  v times the reciprocal of s, added to 1.5 x 2^23,
// leaves the nearest integer in the sum's low bits; it is the division's wherever
// the product is further than 2^-15 from halfway between two integers (both are
// within 2^-23 of the quotient, relative, and that is at most 127 and a bit).
// Chunks that hold a closer one, one in several hundred, are divided.  Scales so
// small that the reciprocal overflows or the quotients pass 127 are, too.
__device__ __forceinline__ u32x2 steps_of(const float (&v)[8], float s, float inv) {
    constexpr float magic = 12582912.0f;
    uint32_t b[8];
    float worst = s < 0x1p-100f ? 1.0f : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = fmaf(v[e], inv, magic);
        worst = fmaxf(worst, fabsf(fmaf(v[e], inv, magic - t)));
        b[e] = __float_as_uint(t);
    }
    if (__builtin_expect(!(worst < 0.5f - 0x1p-15f), 0)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float n = s > 0.0f ? fminf(fmaxf(rintf(v[e] / s), -127.0f), 127.0f) : 0.0f;
            b[e] = static_cast<uint32_t>(static_cast<int>(n));
        }
    }
    u32x2 u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * e + 1], b[4 * e], 0x0c0c0400), hi = __builtin_amdgcn_perm(b[4 * e + 3], b[4 * e + 2], 0x0c0c0400);
        u[e] = lo | hi << 16;
    }
    return u;
}

template <bool BF16, int T, int C, bool NORM, bool QUANT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rows_kernel(RowsArgs a) {
    constexpr int THREADS = T < 256 ? 256 : T, ROWS = THREADS / T;
    __shared__ uint32_t meet_words[T > 64 ? 2 * (T / 64) : 1];
    Meet<T> meet{meet_words};
    const int t = threadIdx.x % T, K = a.K;
    const bool odd = K % 8 != 0;

    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < a.R; first += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t row = first + threadIdx.x / T;
        const bool live = row < a.R;
        const int Kr = live ? K : 0;   // lanes past the last row touch nothing
        const int64_t at = live ? row : 0;
        const uint16_t* x = a.x + at * a.sx;
        const uint16_t* r = a.r ? a.r + at * a.sr : nullptr;
        uint16_t* h = a.r ? a.h + at * a.sh : nullptr;

        // Chunk k .. k + 7 of a row held in registers starts at `from`: the last one
        // moves back to end with the row (whole loads and stores only), and its
        // first k - from values are the chunk's before it, not to be summed again.
        auto from = [&](int k) { return k + 8 <= K ? k : K - 8; };
        auto load = [&](const uint16_t* p, int k) {
            if constexpr (C > 0) return k < Kr ? reinterpret_cast<const Loose16*>(p + from(k))->v : u32x4{0u, 0u, 0u, 0u};
            else return load8(p, k, Kr);
        };
        auto store = [&](uint16_t* p, int k, u32x4 u) {
            if constexpr (C > 0) {
                if (k < Kr) reinterpret_cast<Loose16*>(p + from(k))->v = u;
            } else {
                store8(p, k, Kr, u);
            }
        };
        // the row's values at a chunk, summed and rounded to the stream's type
        auto fetch = [&](int k) {
            u32x4 u = load(x, k);
            if (r) {
                float v[8], v2[8];
                widen8<BF16>(u, v);
                widen8<BF16>(load(r, k), v2);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += v2[e];
                u = narrow8<BF16>(v);
                store(h, k, u);
            }
            return u;
        };
        u32x4 keep[C > 0 ? C : 1];
        // fn(k, chunk) over this thread's chunks; `again`: the row has been summed
        auto chunks = [&](bool again, auto&& fn) {
            if constexpr (C > 0) {
#pragma unroll
                for (int c = 0; c < C; ++c) fn(8 * (t + c * T), keep[c]);
            } else {
                for (int k = 8 * t; k < Kr; k += 8 * T) fn(k, again ? load(r ? h : x, k) : fetch(k));
            }
        };
        if constexpr (C > 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) keep[c] = fetch(8 * (t + c * T));
        }

        float rstd = 1.0f;
        if constexpr (NORM) {
            auto squares = [&](bool again, float by) {
                float ss = 0.0f;
                chunks(again, [&](int k, u32x4 u) {
                    float v[8];
                    widen8<BF16>(u, v);
                    const int skip = C > 0 && odd ? k - from(k) : 0;
                    float part = 0.0f;   // a chunk by itself: a long row's sum is not rounded for every value
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float w = (C > 0 && odd && e < skip ? 0.0f : v[e]) * by;
                        part = fmaf(w, w, part);
                    }
                    ss += part;
                });
                return meet.sum(ss);
            };
            const float by = BF16 && C == 0 ? a.by : 1.0f;
            const float mean = squares(false, by) / static_cast<float>(K) + a.eps;
            // rows of one wave meet by lanes alone; of several, every thread of the workgroup is here
            if (BF16 && __builtin_expect(mean == kInf, 0))
                rstd = kSmaller / sqrtf(squares(true, kSmaller) / static_cast<float>(K) + a.eps * kSmaller * kSmaller);
            else rstd = by / sqrtf(mean);
            if (a.rstd && live && t == 0) a.rstd[row] = rstd;
        }
        auto values = [&](int k, u32x4 u, float (&v)[8]) {
            widen8<BF16>(u, v);
            if constexpr (NORM) {
                float w[8];
                if constexpr (C > 0) whole_weights8<BF16>(a.w, a.w32, k < Kr ? from(k) : 0, w);
                else weights8<BF16>(a.w, a.w32, k, Kr, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * w[e];
            }
        };
        if constexpr (!QUANT) {
            uint16_t* y = a.y + at * a.sy;
            chunks(true, [&](int k, u32x4 u) {
                float v[8];
                values(k, u, v);
                store(y, k, narrow8<BF16>(v));
            });
        } else {
            uint32_t most = 0;   // as bits: see Max
            if constexpr (NORM) {
                chunks(true, [&](int k, u32x4 u) {
                    float v[8];
                    values(k, u, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) most = Max()(most, __float_as_uint(fabsf(v[e])));
                });
            } else {   // 16-bit magnitudes, two to a word
                typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
                u16x2 two = {0, 0};
                chunks(false, [&](int, u32x4 u) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) two = __builtin_elementwise_max(two, __builtin_bit_cast(u16x2, u[e] & 0x7fff7fffu));
                });
                most = __float_as_uint(widen<BF16>(two[0] > two[1] ? two[0] : two[1]));
            }
            const float largest = __uint_as_float(meet.all(most, Max()));
            // a row with an infinity or a NaN has no steps: its scale says so
            const bool fine = __float_as_uint(largest) < __float_as_uint(kInf);
            const float s = fine ? largest / 127.0f : __builtin_nanf("");
            const float by = fine ? s : 0.0f, inv = 1.0f / by;
            if (live && t == 0) a.scale[row] = s;
            int8_t* q = a.q + at * a.sy;
            chunks(true, [&](int k, u32x4 chunk) {
                float v[8];
                values(k, chunk, v);
                const u32x2 u = steps_of(v, by, inv);
                if (C > 0 ? k < Kr : k + 8 <= Kr) {
                    reinterpret_cast<Loose8*>(q + (C > 0 ? from(k) : k))->v = u;
                } else if (C == 0 && k < Kr) {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (k + e < Kr) q[k + e] = static_cast<int8_t>(u[e / 4] >> (8 * (e % 4)));
                }
            });
        }
    }
}

// The gradients.  With g = dy w and u = h rstd,
//     dx = dh + (g - u mean(g u)) rstd,     dw = sum over rows of dy u,
// from one read of dy and h.  A workgroup takes every gridDim-th row (or group
// of rows) and keeps its sums for dw in registers, one fp32 row of `parts` at the
// end; norm_weight_grad_kernel adds these in order, so nothing depends on timing.
template <bool BF16, int T, int C>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_grad_kernel(NormGradArgs a) {
    constexpr int THREADS = T < 256 ? 256 : T, ROWS = THREADS / T;
    __shared__ uint32_t meet_words[T > 64 ? 2 * (T / 64) : 1];
    __shared__ float side[ROWS > 1 ? THREADS * C * 8 : 1];
    Meet<T> meet{meet_words};
    const int t = threadIdx.x % T, K = a.K;
    const float count = static_cast<float>(K);
    float dw[C > 0 ? C : 1][8], w[C > 0 ? C : 1][8];
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            weights8<BF16>(a.w, a.w32, 8 * (t + c * T), K, w[c]);
#pragma unroll
            for (int e = 0; e < 8; ++e) dw[c][e] = 0.0f;
        }
    }
    float* const part = a.parts ? a.parts + static_cast<int64_t>(blockIdx.x) * K : nullptr;
    bool begun = false;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < a.R; first += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t row = first + threadIdx.x / T;
        const bool live = row < a.R;
        const int Kr = live ? K : 0;
        const int64_t at = live ? row : 0;
        const uint16_t *dy = a.dy + at * a.sy, *h = a.h + at * a.sh, *dh = a.dh ? a.dh + at * a.sr : nullptr;
        uint16_t* dx = a.dx + at * a.sx;
        const float rstd = a.rstd[at];
        auto finish = [&](int k, const float (&g)[8], const float (&u)[8], float mean) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (g[e] - u[e] * mean) * rstd;
            if (dh) {
                float d[8];
                widen8<BF16>(load8(dh, k, Kr), d);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += d[e];
            }
            store8(dx, k, Kr, narrow8<BF16>(o));
        };
        if constexpr (C > 0) {
            float g[C][8], u[C][8], dot = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = 8 * (t + c * T);
                widen8<BF16>(load8(dy, k, Kr), g[c]);
                widen8<BF16>(load8(h, k, Kr), u[c]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    u[c][e] *= rstd;
                    dw[c][e] = fmaf(g[c][e], u[c][e], dw[c][e]);
                    g[c][e] *= w[c][e];
                    dot = fmaf(g[c][e], u[c][e], dot);
                }
            }
            const float mean = meet.sum(dot) / count;
#pragma unroll
            for (int c = 0; c < C; ++c) finish(8 * (t + c * T), g[c], u[c], mean);
        } else {
            float dot = 0.0f;
            auto both = [&](int k, float (&g)[8], float (&u)[8], float (&wk)[8]) {
                widen8<BF16>(load8(dy, k, Kr), g);
                widen8<BF16>(load8(h, k, Kr), u);
                weights8<BF16>(a.w, a.w32, k, K, wk);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= rstd;
            };
            for (int k = 8 * t; k < Kr; k += 8 * T) {
                float g[8], u[8], wk[8];
                both(k, g, u, wk);
                float part = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) part = fmaf(g[e] * wk[e], u[e], part);
                dot += part;
            }
            const float mean = meet.sum(dot) / count;
            for (int k = 8 * t; k < Kr; k += 8 * T) {
                float g[8], u[8], wk[8];
                both(k, g, u, wk);
                if (part) {   // this thread's own places, row after row
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (k + e < K) part[k + e] = (begun ? part[k + e] : 0.0f) + g[e] * u[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] *= wk[e];
                finish(k, g, u, mean);
            }
            begun = true;
        }
    }
    if constexpr (C > 0) {
        if (!part) return;
        if constexpr (ROWS > 1) {   // the workgroup's rows side by side, added in order
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) side[(c * 8 + e) * THREADS + threadIdx.x] = dw[c][e];
            __syncthreads();
            if (threadIdx.x >= T) return;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    for (int i = 1; i < ROWS; ++i) dw[c][e] += side[(c * 8 + e) * THREADS + i * T + t];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = 8 * (t + c * T);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K) part[k + e] = dw[c][e];
        }
    }
}

// dw[k] = sum over the parts: 64 columns to a workgroup, whose 16 waves take
// consecutive runs of parts and meet in LDS, in order.  FAR: the parts are `stride`
// apart, and the workgroups of blockIdx.y take kSumGroup each and write as far apart;
// else they are the rows of one array, all taken (8192 x 4096: 1.2 us less).
constexpr int kSumWaves = 16, kSumGroup = kSumWaves * 64;

template <int KIND, bool FAR>
__global__ __launch_bounds__(64 * kSumWaves) void norm_weight_grad_kernel(const float* parts, int nparts, int K, int64_t stride, void* dw) {
    __shared__ float sums[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    int64_t first = 0;
    if constexpr (FAR) {
        const int from = static_cast<int>(blockIdx.y) * kSumGroup;
        first = from * stride;
        nparts = nparts - from < kSumGroup ? nparts - from : kSumGroup;
    }
    auto place = [&](int p) { return FAR ? first + p * stride : static_cast<int64_t>(p) * K; };
    const int run = (nparts + kSumWaves - 1) / kSumWaves;
    const int stop = (wave + 1) * run < nparts ? (wave + 1) * run : nparts;
    float v = 0.0f;
    if (k < K)
        for (int p = wave * run; p < stop; p += 8) {
            float part[8];   // eight in flight (past the last one: that one again, not added)
#pragma unroll
            for (int i = 0; i < 8; ++i) part[i] = parts[place(p + i < stop ? p + i : stop - 1) + k];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p + i < stop) v += part[i];
        }
    sums[wave][lane] = v;
    __syncthreads();
    if (wave != 0 || k >= K) return;
    for (int i = 1; i < kSumWaves; ++i) v += sums[i][lane];
    if constexpr (KIND == 2) static_cast<float*>(dw)[first + k] = v;
    else static_cast<uint16_t*>(dw)[first + k] = narrow<KIND == 1>(v);
}

// Threads and chunks of 8 to a row of K, by measurement (us of quantization, norm
// with residual, the same into int8; a CU holds 2048 threads, and wants several
// rows, of which one waits for memory while another is worked on):
//   8192 x 4096    256 x 2  21, 45, 46    512 x 1  26, 45, 48    256 x 4   25, 51, 68
//   4096 x 8192    512 x 2  22, 46, 47    256 x 4  21, 48, 53    1024 x 1  30, 50, 49
//   4096 x 14336   512 x 4  33, 91, 94    256 x 8  33, 99, 127   1024 x 2  39, 93, 100
//   16384 x 2048   256 x 1  25, 46, 46    64 x 4   21, 48, 51    512 x 1   37, 54, 70
// (a copy's rate: 20, 54, 48 us for the first two and the last, 36, 95, 83 for the
// third).  Few rows want more threads to each:
//   1 x 4096       512 x 1  2.8, 2.8, 3.3   256 x 2  3.0, 3.5, 4.1
//   16 x 14336     1024 x 2  4.5, 4.4, 5.7  512 x 4  4.5, 5.4, 6.8
struct Shape {
    int t, c;
};
Shape shape_of(int64_t R, int64_t K) {
    if (K < 8) return {16, 0};
    if (K <= 128) return {16, 1};
    if (K <= 512) return {64, 1};
    if (K <= 1024) return {64, 2};
    if (K <= 2048) return {256, 1};
    if (K <= 4096) return R <= 512 ? Shape{512, 1} : Shape{256, 2};
    if (K <= 8192) return {512, 2};
    if (K <= 16384) return R <= 256 ? Shape{1024, 2} : Shape{512, 4};
    if (K <= 32768) return {1024, 4};
    return {1024, 0};
}
// Of the gradient, whose sums for dw take registers, too: 8192 x 4096 with a
// residual 53.0 us for 512 x 1 (256 x 2: 56, 1024 x 1: 68; a copy's rate: 54).
Shape grad_shape_of(int64_t K) {
    if (K <= 128) return {16, 1};
    if (K <= 512) return {64, 1};
    if (K <= 1024) return {64, 2};
    if (K <= 2048) return {256, 1};
    if (K <= 4096) return {512, 1};
    if (K <= 8192) return {1024, 1};
    if (K <= 16384) return {1024, 2};
    return {1024, 0};
}

#define DTG_SHAPE(T, C) \
    if (s.t == T && s.c == C) return fn(std::integral_constant<int, T>{}, std::integral_constant<int, C>{});
template <typename Fn>
hipError_t with_shape(Shape s, Fn&& fn) {
    DTG_SHAPE(16, 0)
    DTG_SHAPE(16, 1)
    DTG_SHAPE(64, 1)
    DTG_SHAPE(64, 2)
    DTG_SHAPE(256, 1)
    DTG_SHAPE(256, 2)
    DTG_SHAPE(512, 1)
    DTG_SHAPE(512, 2)
    DTG_SHAPE(512, 4)
    DTG_SHAPE(1024, 2)
    DTG_SHAPE(1024, 4)
    DTG_SHAPE(1024, 0)
    return hipErrorInvalidValue;
}
template <typename Fn>
hipError_t with_grad_shape(Shape s, Fn&& fn) {
    DTG_SHAPE(16, 1)
    DTG_SHAPE(64, 1)
    DTG_SHAPE(64, 2)
    DTG_SHAPE(256, 1)
    DTG_SHAPE(512, 1)
    DTG_SHAPE(1024, 1)
    DTG_SHAPE(1024, 2)
    DTG_SHAPE(1024, 0)
    return hipErrorInvalidValue;
}
#undef DTG_SHAPE

constexpr int64_t kMostGroups = int64_t(1) << 20;   // workgroups of a launch; each then takes several rows

template <bool BF16, bool NORM, bool QUANT>
hipError_t launch_rows_as(const RowsArgs& a, hipStream_t stream) {
    const Shape again = {a.K <= 512 ? 16 : 1024, 0};
    return with_shape(a.by != 1.0f ? again : shape_of(a.R, a.K), [&](auto t_tag, auto c_tag) {
        constexpr int T = decltype(t_tag)::value, C = decltype(c_tag)::value;
        constexpr int THREADS = T < 256 ? 256 : T, ROWS = THREADS / T;
        const int64_t need = (a.R + ROWS - 1) / ROWS;
        hipLaunchKernelGGL((rows_kernel<BF16, T, C, NORM, QUANT>), dim3(static_cast<unsigned>(need < kMostGroups ? need : kMostGroups)),
                           dim3(THREADS), 0, stream, a);
        return hipGetLastError();
    });
}

// Workgroups of the gradient over R rows of K, in one launch.  Each has a part, K floats
// written and read again, so a workgroup takes four rows and more, down to one
// workgroup to a CU; up to as many as keep the memory busy (1024 x 4096: 256 parts
// 15.6 us, 512 17.2; 8192 x 4096: 53.0 with 512, 1024 63.6; 16384 x 1024: 768 30.3,
// 1024 31.5).
int64_t grad_rows(Shape s) { return s.t < 256 ? 256 / s.t : 1; }
int64_t most_groups(Shape s) { return s.t >= 1024 ? 256 : s.t == 512 ? 512 : s.t == 64 ? 768 : 1024; }
int64_t grad_groups(Shape s, int64_t R) {
    const int64_t need = (R + grad_rows(s) - 1) / grad_rows(s);
    int64_t n = (need + 3) / 4;
    if (n < 256) n = 256;
    if (n > most_groups(s)) n = most_groups(s);
    return need < n ? need : n;
}

// Rows of a launch: in a longer one a thread's running fp32 sum for dw would take more
// than 128 rows and lose the last bits of its terms.  An element of dw goes through at
// most 128 + 15 additions in a row here, and 64 + 15 in each pass over the parts (one up
// to 1024 parts, three at 2^31 rows).  (More workgroups in one launch take longer:
// 262144 x 4096 1857 us in one of 2048, 1585 in four of 512, 1608 in one of 512.)
int64_t grad_launch(Shape s) { return 128 * grad_rows(s) * most_groups(s); }

template <bool FAR>
void launch_sum(const float* parts, int n, int K, int64_t stride, void* dw, int kind, unsigned groups, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>((K + 63) / 64), groups), block(64 * kSumWaves);
    if (kind == 2) hipLaunchKernelGGL((norm_weight_grad_kernel<2, FAR>), grid, block, 0, stream, parts, n, K, stride, dw);
    else if (kind == 1) hipLaunchKernelGGL((norm_weight_grad_kernel<1, FAR>), grid, block, 0, stream, parts, n, K, stride, dw);
    else hipLaunchKernelGGL((norm_weight_grad_kernel<0, FAR>), grid, block, 0, stream, parts, n, K, stride, dw);
}

}  // namespace

hipError_t launch_rows(const RowsArgs& given, int bf16, hipStream_t stream) {
    RowsArgs a = given;
    a.by = 1.0f;
    if (a.w && bf16 && a.eps < kLeastEps) {
        a.by = kLarger;
        a.eps *= kLarger * kLarger;
    }
    if (!a.w) return bf16 ? launch_rows_as<true, false, true>(a, stream) : launch_rows_as<false, false, true>(a, stream);
    if (a.q) return bf16 ? launch_rows_as<true, true, true>(a, stream) : launch_rows_as<false, true, true>(a, stream);
    return bf16 ? launch_rows_as<true, true, false>(a, stream) : launch_rows_as<false, true, false>(a, stream);
}

int64_t norm_grad_parts(int64_t R, int64_t K) {
    const Shape s = grad_shape_of(K);
    const int64_t rows = grad_launch(s);
    return R / rows * grad_groups(s, rows) + grad_groups(s, R % rows);
}

hipError_t launch_norm_grad(const NormGradArgs& given, int bf16, hipStream_t stream) {
    const Shape s = grad_shape_of(given.K);
    return with_grad_shape(s, [&](auto t_tag, auto c_tag) {
        constexpr int T = decltype(t_tag)::value, C = decltype(c_tag)::value;
        NormGradArgs a = given;
        for (int64_t left = given.R; left > 0; left -= a.R) {
            a.R = left < grad_launch(s) ? left : grad_launch(s);
            const int64_t groups = grad_groups(s, a.R);
            const dim3 grid(static_cast<unsigned>(groups)), block(T < 256 ? 256 : T);
            if (bf16) hipLaunchKernelGGL((norm_grad_kernel<true, T, C>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((norm_grad_kernel<false, T, C>), grid, block, 0, stream, a);
            a.dy += a.R * a.sy;
            a.h += a.R * a.sh;
            if (a.dh) a.dh += a.R * a.sr;
            a.dx += a.R * a.sx;
            a.rstd += a.R;
            if (a.parts) a.parts += groups * a.K;
        }
        return hipGetLastError();
    });
}

hipError_t launch_norm_weight_grad(float* parts, int64_t nparts, int64_t K, void* dw, int kind, hipStream_t stream) {
    int n = static_cast<int>(nparts);
    const int k = static_cast<int>(K);
    if (n <= kSumGroup) {
        launch_sum<false>(parts, n, k, K, dw, kind, 1, stream);
        return hipGetLastError();
    }
    int64_t stride = K;
    while (n > kSumGroup) {   // groups of parts, each into its first one
        const int groups = (n + kSumGroup - 1) / kSumGroup;
        launch_sum<true>(parts, n, k, stride, parts, 2, static_cast<unsigned>(groups), stream);
        n = groups;
        stride *= kSumGroup;
    }
    launch_sum<true>(parts, n, k, stride, dw, kind, 1, stream);
    return hipGetLastError();
}

}  // namespace dtg
