// Device helpers of the fused operators.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_f32_fused.h"
#include "device_common.h"
#include "fused.h"
#include "gemm_internal.h"

namespace gemm_f32_impl {
namespace fused {

typedef float float2u __attribute__((ext_vector_type(2), aligned(4)));  // 8 bytes at any word

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kRoot2OverPi = 0.79788456080286535588f;
constexpr float kRootHalfOverPi = 0.39894228040143267794f;  // 1 / sqrt(2 pi)
constexpr float kCubic = 0.044715f;

// exp(x) by the hardware's power of two; results below 2^-126 are zero.
__device__ __forceinline__ float quick_exp(float x) { return __builtin_amdgcn_exp2f(x * kLog2E); }

// exp(x) for x <= 0, held below 2^-126 too.
__device__ __forceinline__ float tail_exp(float x) {
    const float y = x * kLog2E;
    const bool low = y < -120.0f;
    return __builtin_amdgcn_exp2f(low ? y + 64.0f : y) * (low ? 0x1p-64f : 1.0f);
}

// 1 / (1 + exp(-u)), by the exponential that cannot overflow.
__device__ __forceinline__ float logistic(float u) {
    const float t = tail_exp(-fabsf(u));
    return (u < 0.0f ? t : 1.0f) * __builtin_amdgcn_rcpf(1.0f + t);
}

// (1 + erf(z / sqrt 2)) / 2 and e = exp(-z^2 / 2).  For z <= 0 it is e t P(t)
// with t = 1 / (1 + 0.35 |z|), P a polynomial fitted to exp(z^2 / 2) erfc(|z| /
// sqrt 2) / (2 t) over |z| <= 15.2 by reweighted least squares (3.3e-8 of the
// value at most).  Roundings of FP32 move it by at most 20 2^-24 of the value, and those of
// the exponential's argument by 1.2 z^2 2^-24 besides: 5e-7 as a rule for |z| < 1, 7e-6 at z = -11.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    e = tail_exp(-0.5f * z * z);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.35f, fabsf(z), 1.0f));
    float q = -2.916558145e-02f;
    q = fmaf(q, t, 1.440686386e-01f);
    q = fmaf(q, t, -2.559176254e-01f);
    q = fmaf(q, t, 1.594104647e-01f);
    q = fmaf(q, t, -2.327564113e-02f);
    q = fmaf(q, t, 1.055796992e-01f);
    q = fmaf(q, t, 1.198142779e-01f);
    q = fmaf(q, t, 1.398645026e-01f);
    q = fmaf(q, t, 1.396212489e-01f);
    q *= t * e;
    return z > 0.0f ? 1.0f - q : q;
}

// Beyond these |z| the value of a tail is below FP32's range; z itself may be
// infinite there, and 0 times it would be NaN.
__device__ __forceinline__ float activate(int kind, float z) {
    float e;
    switch (kind) {
        case GEMM_F32_ACT_RELU: return z < 0.0f ? 0.0f : z;
        case GEMM_F32_ACT_GELU: return z < -15.0f ? 0.0f : z * normal_cdf(z, e);
        // (1 + tanh u) / 2 is the logistic function of 2 u
        case GEMM_F32_ACT_GELU_TANH:
            return z < -15.0f ? 0.0f : z * logistic(2.0f * kRoot2OverPi * (z + kCubic * z * z * z));
        case GEMM_F32_ACT_SILU: return z < -200.0f ? 0.0f : z * logistic(z);
        default: return z;
    }
}

__device__ __forceinline__ float slope(int kind, float z) {
    switch (kind) {
        case GEMM_F32_ACT_RELU: return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
        case GEMM_F32_ACT_GELU: {
            if (fabsf(z) > 15.0f) return z > 0.0f ? 1.0f : 0.0f;
            float e;
            const float q = normal_cdf(z, e);
            return fmaf(z * kRootHalfOverPi, e, q);
        }
        case GEMM_F32_ACT_GELU_TANH: {
            if (fabsf(z) > 15.0f) return z > 0.0f ? 1.0f : 0.0f;
            const float q = logistic(2.0f * kRoot2OverPi * (z + kCubic * z * z * z));
            return q + z * q * (1.0f - q) * (2.0f * kRoot2OverPi) * (1.0f + 3.0f * kCubic * z * z);
        }
        case GEMM_F32_ACT_SILU: {
            if (fabsf(z) > 200.0f) return z > 0.0f ? 1.0f : 0.0f;
            const float q = logistic(z);
            return q + z * q * (1.0f - q);
        }
        default: return 1.0f;
    }
}

// The value of a lane of the same 16 by a data-parallel move: quads turned by 1
// and 2 lanes, rows of 16 by 4 and 8.
template <int CONTROL>
__device__ __forceinline__ int moved(int x) {
    return __builtin_amdgcn_update_dpp(0, x, CONTROL, 0xf, 0xf, false);
}
// op over the 4 (16) lanes that share a quad (row), in every one of them.
template <int LANES, class F>
__device__ __forceinline__ float over_lanes(float x, F op) {
    static_assert(LANES == 4 || LANES == 16, "");
    auto at = [](int v) { return __builtin_bit_cast(float, v); };
    auto of = [](float v) { return __builtin_bit_cast(int, v); };
    x = op(x, at(moved<0xb1>(of(x))));
    x = op(x, at(moved<0x4e>(of(x))));
    if constexpr (LANES == 16) {
        x = op(x, at(moved<0x124>(of(x))));
        x = op(x, at(moved<0x128>(of(x))));
    }
    return x;
}

// The three bf16 parts of four values x = h + m + l, rounded to nearest each:
// h takes 8 of the 24 bits, m 8 of the at most 16 left, and what is then left
// has no more than 8, so the sum is exact (down to bf16's least value, 2^-133).
struct Parts {
    u32x2 p[3];
};
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ Parts split4(float x0, float x1, float x2, float x3) {
    Parts r;
    float x[4] = {x0, x1, x2, x3};
#pragma unroll
    for (int c = 0; c < 3; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = pack_bf16(x[2 * i], x[2 * i + 1]);
            r.p[c][i] = v;
            x[2 * i] -= __builtin_bit_cast(float, v << 16);
            x[2 * i + 1] -= __builtin_bit_cast(float, v & 0xffff0000u);
        }
    return r;
}

// Two fp16 parts of four values times a power of two that brings their row's
// largest below 2^15: h has 11 bits of the 24, l 11 of the 12 and a sign that are
// left, so h + l is off by at most 2^-23 of the value, or 2^-25, half the last place of
// fp16: 2^-40 of the power of two above the row's largest, so 2^-39 of the largest.
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
struct Halves {
    u32x2 p[2];
};
__device__ __forceinline__ Halves split4_half(const float (&x)[4], float scale) {
    Halves r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const half2v h = __builtin_convertvector(f32x2{x[2 * i] * scale, x[2 * i + 1] * scale}, half2v);
        const half2v l = __builtin_convertvector(
            f32x2{fmaf(x[2 * i], scale, -static_cast<float>(h[0])), fmaf(x[2 * i + 1], scale, -static_cast<float>(h[1]))}, half2v);
        r.p[0][i] = __builtin_bit_cast(uint32_t, h);
        r.p[1][i] = __builtin_bit_cast(uint32_t, l);
    }
    return r;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// What a row's exponentials are taken relative to: its maximum, so that they and their
// sum stay in range, but 0 where that is infinite (x - maximum would be NaN): no word at all
// has a sum of 0, a logit of +inf one of +inf.
__device__ __forceinline__ float base_of(float top) { return finite(top) ? top : 0.0f; }

// Two running (maximum, sum of exp(x - base_of(maximum))) as one.  An empty piece is
// (-inf, 0).  Maxima pass over NaN, which makes the sum NaN.
__device__ __forceinline__ void merge_stats(float &m, float &s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    const float base = base_of(top);
    s = s * quick_exp(m - base) + s2 * quick_exp(m2 - base);
    m = top;
}

}  // namespace fused
}  // namespace gemm_f32_impl
