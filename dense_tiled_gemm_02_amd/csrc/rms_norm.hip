// RMS norm with the residual's addition, rows in 8 bits, and the norm's
// gradients, for gfx950.  One row of K values:
//
//     h = x + r (rounded to the stream's type),  n = sqrt(mean h^2 + eps)
//     y = h w / n                                      (16-bit output)
//     s = max |y| / 127,  q = y / s to the nearest     (int8 output)
//
// All of it from one read: T threads hold the row in registers, C chunks of 8
// values each, with the sums across them through the wave's lanes and, where a
// row takes more than a wave, one LDS word per wave and one barrier.  Bound by
// memory: x, r are read and y or q (and h) are written once.  Rows longer than
// the registers hold are read again for each pass (C = 0).
//
// The quotient y / s is an IEEE division and the scale that it is divided by is
// the stored one, so q is the nearest step of the scale that a product uses.
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

// Elements k .. k + 7 of the weights.
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

// 1 / sqrt(sum / K + eps).  A sum of squares that overflows (bf16 values past
// 1e19) is taken again, scaled by 2^-200.
constexpr float kSmaller = 0x1p-100f;

template <bool BF16, int T, int C, bool NORM, bool QUANT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rows_kernel(RowsArgs a) {
    constexpr int THREADS = T < 256 ? 256 : T, ROWS = THREADS / T;
    __shared__ uint32_t meet_words[T > 64 ? 2 * (T / 64) : 1];
    Meet<T> meet{meet_words};
    const int t = threadIdx.x % T, K = a.K;

    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < a.R; first += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t row = first + threadIdx.x / T;
        const bool live = row < a.R;
        const int Kr = live ? K : 0;   // lanes past the last row touch nothing
        const uint16_t* x = a.x + (live ? row : 0) * a.sx;
        const uint16_t* r = a.r ? a.r + (live ? row : 0) * a.sr : nullptr;
        uint16_t* h = a.r ? a.h + (live ? row : 0) * a.sh : nullptr;

        // the row's values at k .. k + 7, summed and rounded to the stream's type
        auto fetch = [&](int k, float (&v)[8]) {
            const u32x4 ux = load8(x, k, Kr);
            widen8<BF16>(ux, v);
            if (r) {
                float v2[8];
                widen8<BF16>(load8(r, k, Kr), v2);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += v2[e];
                const u32x4 u = narrow8<BF16>(v);
                store8(h, k, Kr, u);
                widen8<BF16>(u, v);
            }
        };
        float keep[C > 0 ? C : 1][8];
        // fn(k, values) over this thread's chunks; `again`: the row has been summed
        auto chunks = [&](bool again, auto&& fn) {
            if constexpr (C > 0) {
#pragma unroll
                for (int c = 0; c < C; ++c) fn(8 * (t + c * T), keep[c]);
            } else {
                for (int k = 8 * t; k < Kr; k += 8 * T) {
                    float v[8];
                    if (!again) fetch(k, v);
                    else widen8<BF16>(load8(r ? h : x, k, Kr), v);
                    fn(k, v);
                }
            }
        };
        if constexpr (C > 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) fetch(8 * (t + c * T), keep[c]);
        }

        float rstd = 1.0f;
        if constexpr (NORM) {
            float ss = 0.0f;
            chunks(false, [&](int, float (&v)[8]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
            });
            ss = meet.sum(ss);
            if (__builtin_expect(ss == kInf && BF16, 0)) {
                float small = 0.0f;
                chunks(true, [&](int, float (&v)[8]) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) small = fmaf(v[e] * kSmaller, v[e] * kSmaller, small);
                });
                // rows of one wave meet by lanes alone; of several, every thread of the workgroup is here
                rstd = kSmaller / sqrtf(meet.sum(small) / static_cast<float>(K));
            } else {
                rstd = 1.0f / sqrtf(ss / static_cast<float>(K) + a.eps);
            }
            if (a.rstd && live && t == 0) a.rstd[row] = rstd;
        }
        auto normed = [&](int k, float (&v)[8]) {
            if constexpr (NORM) {
                float w[8];
                weights8<BF16>(a.w, a.w32, k, Kr, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * rstd * w[e];
            }
        };
        if constexpr (!QUANT) {
            uint16_t* y = a.y + (live ? row : 0) * a.sy;
            chunks(true, [&](int k, float (&v)[8]) {
                normed(k, v);
                store8(y, k, Kr, narrow8<BF16>(v));
            });
        } else {
            float most = 0.0f;
            chunks(NORM, [&](int k, float (&v)[8]) {
                normed(k, v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    most = __uint_as_float(Max()(__float_as_uint(most), __float_as_uint(fabsf(v[e]))));
            });
            most = meet.most(most);
            // a row with an infinity or a NaN has no steps: its scale says so
            const bool fine = __float_as_uint(most) < __float_as_uint(kInf);
            const float s = fine ? most / 127.0f : __builtin_nanf("");
            const bool steps = s > 0.0f;
            if (live && t == 0) a.scale[row] = s;
            int8_t* q = a.q + (live ? row : 0) * a.sy;
            chunks(true, [&](int k, float (&v)[8]) {
                if constexpr (C == 0) normed(k, v);
                int i[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = rintf(v[e] / s);   // in the smallest scales past 127
                    i[e] = steps ? static_cast<int>(fminf(fmaxf(n, -127.0f), 127.0f)) : 0;
                }
                u32x2 u;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    u[e] = (i[4 * e] & 255) | (i[4 * e + 1] & 255) << 8 | (i[4 * e + 2] & 255) << 16 |
                           static_cast<uint32_t>(i[4 * e + 3]) << 24;
                if (k + 8 <= Kr) {
                    reinterpret_cast<Loose8*>(q + k)->v = u;
                } else if (k < Kr) {
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
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(g[e] * wk[e], u[e], dot);
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
// consecutive runs of parts and meet in LDS, in order.
constexpr int kSumWaves = 16;

template <int KIND>
__global__ __launch_bounds__(64 * kSumWaves) void norm_weight_grad_kernel(const float* parts, int nparts, int K, void* dw) {
    __shared__ float sums[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    const int run = (nparts + kSumWaves - 1) / kSumWaves;
    const int stop = (wave + 1) * run < nparts ? (wave + 1) * run : nparts;
    float v = 0.0f;
    if (k < K)
        for (int p = wave * run; p < stop; p += 8) {
            float part[8];   // eight in flight (past the last one: that one again, not added)
#pragma unroll
            for (int i = 0; i < 8; ++i) part[i] = parts[static_cast<int64_t>(p + i < stop ? p + i : stop - 1) * K + k];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (p + i < stop) v += part[i];
        }
    sums[wave][lane] = v;
    __syncthreads();
    if (wave != 0 || k >= K) return;
    for (int i = 1; i < kSumWaves; ++i) v += sums[i][lane];
    if constexpr (KIND == 2) static_cast<float*>(dw)[k] = v;
    else static_cast<uint16_t*>(dw)[k] = narrow<KIND == 1>(v);
}

// Threads and chunks of 8 to a row of K.
struct Shape {
    int t, c;
};
Shape shape_of(int64_t K) {
    if (K <= 128) return {16, 1};
    if (K <= 512) return {64, 1};
    if (K <= 1024) return {64, 2};
    if (K <= 2048) return {256, 1};
    if (K <= 4096) return {256, 2};
    if (K <= 8192) return {1024, 1};
    if (K <= 16384) return {1024, 2};
    return {1024, 0};
}

template <typename Fn>
hipError_t with_shape(int64_t K, Fn&& fn) {
    const Shape s = shape_of(K);
#define DTG_SHAPE(T, C) \
    if (s.t == T && s.c == C) return fn(std::integral_constant<int, T>{}, std::integral_constant<int, C>{});
    DTG_SHAPE(16, 1)
    DTG_SHAPE(64, 1)
    DTG_SHAPE(64, 2)
    DTG_SHAPE(256, 1)
    DTG_SHAPE(256, 2)
    DTG_SHAPE(1024, 1)
    DTG_SHAPE(1024, 2)
    DTG_SHAPE(1024, 0)
#undef DTG_SHAPE
    return hipErrorInvalidValue;
}

constexpr int64_t kMostGroups = int64_t(1) << 20;   // workgroups of a launch; each then takes several rows

template <bool BF16, bool NORM, bool QUANT>
hipError_t launch_rows_as(const RowsArgs& a, hipStream_t stream) {
    return with_shape(a.K, [&](auto t_tag, auto c_tag) {
        constexpr int T = decltype(t_tag)::value, C = decltype(c_tag)::value;
        constexpr int THREADS = T < 256 ? 256 : T, ROWS = THREADS / T;
        const int64_t need = (a.R + ROWS - 1) / ROWS;
        hipLaunchKernelGGL((rows_kernel<BF16, T, C, NORM, QUANT>), dim3(static_cast<unsigned>(need < kMostGroups ? need : kMostGroups)),
                           dim3(THREADS), 0, stream, a);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_rows(const RowsArgs& a, int bf16, hipStream_t stream) {
    if (!a.w) return bf16 ? launch_rows_as<true, false, true>(a, stream) : launch_rows_as<false, false, true>(a, stream);
    if (a.q) return bf16 ? launch_rows_as<true, true, true>(a, stream) : launch_rows_as<false, true, true>(a, stream);
    return bf16 ? launch_rows_as<true, true, false>(a, stream) : launch_rows_as<false, true, false>(a, stream);
}

int64_t norm_grad_parts(int64_t R, int64_t K) {
    const Shape s = shape_of(K);
    const int64_t rows = s.t < 256 ? 256 / s.t : 1, need = (R + rows - 1) / rows;
    const int64_t most = s.t > 256 ? 256 : 1024;   // a CU's worth of threads each
    return need < most ? need : most;
}

hipError_t launch_norm_grad(const NormGradArgs& a, int bf16, hipStream_t stream) {
    return with_shape(a.K, [&](auto t_tag, auto c_tag) {
        constexpr int T = decltype(t_tag)::value, C = decltype(c_tag)::value;
        const dim3 grid(static_cast<unsigned>(norm_grad_parts(a.R, a.K))), block(T < 256 ? 256 : T);
        if (bf16) hipLaunchKernelGGL((norm_grad_kernel<true, T, C>), grid, block, 0, stream, a);
        else hipLaunchKernelGGL((norm_grad_kernel<false, T, C>), grid, block, 0, stream, a);
        return hipGetLastError();
    });
}

hipError_t launch_norm_weight_grad(const float* parts, int64_t nparts, int64_t K, void* dw, int kind, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>((K + 63) / 64)), block(64 * kSumWaves);
    const int n = static_cast<int>(nparts), k = static_cast<int>(K);
    if (kind == 2) hipLaunchKernelGGL((norm_weight_grad_kernel<2>), grid, block, 0, stream, parts, n, k, dw);
    else if (kind == 1) hipLaunchKernelGGL((norm_weight_grad_kernel<1>), grid, block, 0, stream, parts, n, k, dw);
    else hipLaunchKernelGGL((norm_weight_grad_kernel<0>), grid, block, 0, stream, parts, n, k, dw);
    return hipGetLastError();
}

}  // namespace dtg
