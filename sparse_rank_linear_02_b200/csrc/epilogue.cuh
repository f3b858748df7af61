// epilogue.cuh -- bias, activation and residual of the layer's epilogue, and
// the activation's slope for its backward pass (internal).
//
//   Z = X S^T + T U^T + b          (fp32)
//   Y = act(Z) + R                 (fp32, rounded to bf16 once)
//
// The activations, with u = sqrt(2/pi) (z + 0.044715 z^3):
//   relu       max(z, 0)                        slope [z > 0]
//   gelu       z Phi(z)                         slope Phi(z) + z phi(z)
//   gelu_tanh  z (1 + tanh u)/2 = z / (1 + e^-2u)
//   silu       z / (1 + e^-z)
// The quotient forms have no cancellation for negative z, where 1 + tanh u
// would lose every digit.  NaN stays NaN in every one of them.
//
// Phi: for a >= 0 the tail 1 - Phi(a) is e^(-a^2/2) times a smooth function of
// t = 1 / (1 + 0.35 a), here t times a polynomial of degree 8 in t, fitted to
// the least largest relative error (3.2e-8 for a <= 13.5).  It costs one
// reciprocal, one exponential and ten multiply-adds, shares the exponential
// with the slope's density, and keeps the tail's relative accuracy; erfcf took
// 160 us where this takes the tanh form's 134 (14336 x 4096, 2048 tokens).
#pragma once

#include "common.cuh"

namespace slr {

// Operands of the epilogue (device pointers; bias, res and pre may be null).
struct Epilogue {
    const uint16_t *bias;   // bf16 [d_out]
    const uint16_t *res;    // bf16 [M, ldr]: R, which may be Y itself
    int64_t ldr;
    uint16_t *pre;          // bf16 [M, d_out]: Z, out
    int32_t act;            // slr_act
};

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// Phi(z), given e = exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float e) {
    const float t = __fdividef(1.0f, fmaf(0.35f, fabsf(z), 1.0f));
    float q = -0.029125869274139404f;
    q = fmaf(q, t, 0.1438722461462021f);
    q = fmaf(q, t, -0.2555046081542969f);
    q = fmaf(q, t, 0.15892933309078217f);
    q = fmaf(q, t, -0.022937165573239326f);
    q = fmaf(q, t, 0.10543294996023178f);
    q = fmaf(q, t, 0.11985243111848831f);
    q = fmaf(q, t, 0.13985908031463623f);
    q = fmaf(q, t, 0.1396215707063675f);
    const float tail = q * t * e;
    return z < 0.f ? tail : 1.0f - tail;
}

__device__ __forceinline__ float act_gelu(float z) { return z * normal_cdf(z, __expf(-0.5f * z * z)); }
__device__ __forceinline__ float act_gelu_tanh(float z) {
    const float u = kGeluC * fmaf(0.044715f * z, z * z, z);
    return __fdividef(z, 1.0f + __expf(-2.0f * u));
}
__device__ __forceinline__ float act_silu(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

// z within [-c, c], NaN kept.  The slopes are at their limits, 0 and 1, well
// inside the bounds used below, where no product of a zero and an infinity
// arises.
__device__ __forceinline__ float clamp_keep_nan(float z, float c) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;\n\t}" : "=f"(r) : "f"(z), "f"(-c), "f"(c));
    return r;
}
__device__ __forceinline__ float slope_gelu(float z) {
    z = clamp_keep_nan(z, 40.f);
    const float e = __expf(-0.5f * z * z);
    return fmaf(z * kInvSqrt2Pi, e, normal_cdf(z, e));
}
__device__ __forceinline__ float slope_gelu_tanh(float z) {
    z = clamp_keep_nan(z, 40.f);
    const float z2 = z * z;
    const float s = __fdividef(1.0f, 1.0f + __expf(-2.0f * kGeluC * fmaf(0.044715f * z, z2, z)));
    return fmaf(z * s * (1.0f - s), 2.0f * kGeluC * fmaf(0.134145f, z2, 1.0f), s);
}
__device__ __forceinline__ float slope_silu(float z) {
    z = clamp_keep_nan(z, 200.f);
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    return s * fmaf(z, 1.0f - s, 1.0f);
}

// z becomes act'(z) over N values.
template <int N>
__device__ __forceinline__ void slope_values(float (&z)[N], int act) {
    switch (act) {
        case SLR_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] > 0.f ? 1.f : 0.f;
            break;
        case SLR_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = slope_gelu(z[i]);
            break;
        case SLR_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = slope_gelu_tanh(z[i]);
            break;
        case SLR_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = slope_silu(z[i]);
            break;
        default:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = 1.f;
            break;
    }
}

// act over N values; the switch is uniform and outside the loops.
template <int N>
__device__ __forceinline__ void act_values(float (&z)[N], int act) {
    switch (act) {
        case SLR_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] <= 0.f ? 0.f : z[i];
            break;
        case SLR_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = act_gelu(z[i]);
            break;
        case SLR_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = act_gelu_tanh(z[i]);
            break;
        case SLR_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = act_silu(z[i]);
            break;
        default: break;
    }
}

// One bf16 of R: an ordinary coherent load (R may be written by the grid
// before a chained call, or be the Y that this grid writes), kept in order with
// griddepcontrol.wait by being volatile.
__device__ __forceinline__ uint32_t ld_res(const uint16_t *p) {
    uint16_t v;
    asm volatile("ld.global.cg.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

// N tokens of R for one output row, two packed per word.  Tokens and rows past
// the problem read its last ones (their outputs are not stored): without
// branches the loads go out together.
template <int N>
__device__ __forceinline__ void load_res_row(const Epilogue &ep, int tok0, int M, int row, int d_out,
                                             uint32_t (&r)[N / 2]) {
    const uint16_t *p = ep.res + min(row, d_out - 1);
    uint32_t v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = ld_res(p + (int64_t)min(tok0 + j, M - 1) * ep.ldr);
#pragma unroll
    for (int j = 0; j < N / 2; ++j) r[j] = v[2 * j] | (v[2 * j + 1] << 16);
}

// N tokens of one output row: z += bias, Z stored (where wanted), act, + R
// (packed as load_res_row gives it; null: none).
template <int N>
__device__ __forceinline__ void epilogue_row(const Epilogue &ep, float (&z)[N], float bias, const uint32_t *r,
                                             int tok0, int M, int row, int d_out) {
#pragma unroll
    for (int j = 0; j < N; ++j) z[j] += bias;
    if (ep.pre != nullptr && row < d_out) {
        uint16_t *p = ep.pre + (int64_t)tok0 * d_out + row;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (tok0 + j < M) p[(int64_t)j * d_out] = f32_to_bf16_bits(z[j]);
    }
    act_values<N>(z, ep.act);
    if (r != nullptr) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] += (j & 1) ? bf16hi_to_f32(r[j / 2]) : bf16lo_to_f32(r[j / 2]);
    }
}

}  // namespace slr
