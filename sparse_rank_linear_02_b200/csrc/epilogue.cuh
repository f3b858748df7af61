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
// the least largest relative error: 6.4e-8 for a <= 13.5 with the fp32 coefficients
// below.  Its evaluation in fp32 adds the roundings of the exponent, which grow with
// a^2 / 2: the tail is within 1e-6 up to a = 2, 2e-6 up to 4, 1e-5 up to 13, always
// far inside the bf16 that it ends in.  It costs one reciprocal, one exponential
// and ten multiply-adds, and shares the exponential with the slope's density;
// erfcf took 160 us where this takes the tanh form's 134 (14336 x 4096, 2048
// tokens).
#pragma once

#include "common.cuh"
#include "f32x2.cuh"

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
__device__ __forceinline__ f32x2 normal_cdf2(f32x2 z, f32x2 e) {
    float a, b;
    unpack2(z, a, b);
    const f32x2 t = rcp2(fma2(dup2(0.35f), pack2(fabsf(a), fabsf(b)), dup2(1.0f)));
    f32x2 q = dup2(-0.029125869274139404f);
    q = fma2(q, t, dup2(0.1438722461462021f));
    q = fma2(q, t, dup2(-0.2555046081542969f));
    q = fma2(q, t, dup2(0.15892933309078217f));
    q = fma2(q, t, dup2(-0.022937165573239326f));
    q = fma2(q, t, dup2(0.10543294996023178f));
    q = fma2(q, t, dup2(0.11985243111848831f));
    q = fma2(q, t, dup2(0.13985908031463623f));
    q = fma2(q, t, dup2(0.1396215707063675f));
    float ta, tb;
    unpack2(mul2(mul2(q, t), e), ta, tb);
    return pack2(a < 0.f ? ta : 1.0f - ta, b < 0.f ? tb : 1.0f - tb);
}
// exp(-z^2 / 2); 1 / (1 + exp(-2u)), u the tanh form's argument, z2 = z^2; 1 / (1 + exp(-z)).
__device__ __forceinline__ f32x2 gauss2(f32x2 z) { return exp2_2(mul2(mul2(z, dup2(-0.5f * kLog2e)), z)); }
__device__ __forceinline__ f32x2 sigma_tanh2(f32x2 z, f32x2 z2) {
    const f32x2 w = mul2(fma2(dup2(-2.0f * kGeluC * kLog2e * 0.044715f), z2, dup2(-2.0f * kGeluC * kLog2e)), z);
    return rcp2(add2(exp2_2(w), dup2(1.0f)));
}
__device__ __forceinline__ f32x2 sigma2(f32x2 z) { return rcp2(add2(exp2_2(mul2(z, dup2(-kLog2e))), dup2(1.0f))); }

// act(z) of two values (not SLR_ACT_NONE).
template <int ACT>
__device__ __forceinline__ f32x2 act2(f32x2 z) {
    if constexpr (ACT == SLR_ACT_GELU) return mul2(z, normal_cdf2(z, gauss2(z)));
    if constexpr (ACT == SLR_ACT_GELU_TANH) return mul2(z, sigma_tanh2(z, mul2(z, z)));
    if constexpr (ACT == SLR_ACT_SILU) return mul2(z, sigma2(z));
    float a, b;
    unpack2(z, a, b);
    return pack2(a <= 0.f ? 0.f : a, b <= 0.f ? 0.f : b);
}

// act'(z) of two values; |z| <= 200, where every slope is at its limit.
template <int ACT>
__device__ __forceinline__ f32x2 slope2(f32x2 z) {
    const f32x2 neg = dup2(-1.0f);
    if constexpr (ACT == SLR_ACT_GELU) {
        const f32x2 e = gauss2(z);
        return fma2(mul2(z, dup2(kInvSqrt2Pi)), e, normal_cdf2(z, e));
    }
    if constexpr (ACT == SLR_ACT_GELU_TANH) {
        const f32x2 z2 = mul2(z, z), s = sigma_tanh2(z, z2), p = mul2(z, s);
        const f32x2 w = fma2(mul2(p, neg), s, p);   // z s (1 - s)
        return fma2(w, fma2(dup2(2.0f * kGeluC * 0.134145f), z2, dup2(2.0f * kGeluC)), s);
    }
    if constexpr (ACT == SLR_ACT_SILU) {
        const f32x2 s = sigma2(z), p = mul2(z, s);
        return add2(s, fma2(mul2(p, neg), s, p));
    }
    if constexpr (ACT == SLR_ACT_RELU) {
        float a, b;
        unpack2(z, a, b);
        return pack2(a > 0.f ? 1.f : 0.f, b > 0.f ? 1.f : 0.f);
    }
    return dup2(1.0f);
}

// act over N values; the switch is uniform and outside the loops.
template <int ACT, int N>
__device__ __forceinline__ void act_values_of(float (&z)[N]) {
    if constexpr (N == 1) {
        float unused;
        unpack2(act2<ACT>(dup2(z[0])), z[0], unused);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) unpack2(act2<ACT>(pack2(z[i], z[i + 1])), z[i], z[i + 1]);
    }
}
template <int N>
__device__ __forceinline__ void act_values(float (&z)[N], int act) {
    switch (act) {
        case SLR_ACT_RELU: act_values_of<SLR_ACT_RELU>(z); break;
        case SLR_ACT_GELU: act_values_of<SLR_ACT_GELU>(z); break;
        case SLR_ACT_GELU_TANH: act_values_of<SLR_ACT_GELU_TANH>(z); break;
        case SLR_ACT_SILU: act_values_of<SLR_ACT_SILU>(z); break;
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
