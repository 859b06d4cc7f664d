// Packed float32 arithmetic and the approximate units, for the kernels that instructions bound.
#pragma once

#include "common.cuh"

namespace hla2 {
namespace {

// Two float32 values in a register pair: one packed instruction for both halves a kernel's instructions.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v)); }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma_(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sum_of(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ float sum_of(float a) { return a; }

// e^x and 1 / x by the approximate units.  1 / x is good to an ulp; e^x to about 2^-22 + 2^-24 |x| relative, the latter from
// rounding x log2 e, which shows in a sigmoid only where it is e^z, small itself (float32 gates of -20: 6e-7 relative).
// Subnormal results are 0, and overflow is infinity, as with the exact ones.
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_exp(float x) { return fast_exp2(x * 1.4426950408889634f); }
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
}  // namespace
}  // namespace hla2
