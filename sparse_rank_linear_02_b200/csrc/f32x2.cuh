// f32x2.cuh -- packed pairs of fp32 values (internal).
#pragma once

#include <stdint.h>

namespace slr {

// Two fp32 values in one register pair: arithmetic on fma.rn.f32x2 and its
// kin takes one issue slot for two results.  (Written one value at a time, the
// slopes of the epilogue's backward bound that kernel by instruction issue:
// 51.6 us where the pairs take 36.5, 2048 x 14336, tanh GELU.)
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f32x2 dup2(float a) { return pack2(a, a); }
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 2^a and 1/a of both values: one special-function operation each.
__device__ __forceinline__ f32x2 exp2_2(f32x2 v) {
    float a, b;
    unpack2(v, a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pack2(a, b);
}
__device__ __forceinline__ f32x2 rcp2(f32x2 v) {
    float a, b;
    unpack2(v, a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return pack2(a, b);
}
constexpr float kLog2e = 1.4426950408889634f;


}  // namespace slr
