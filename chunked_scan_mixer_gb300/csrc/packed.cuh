// Vectors of a row as pairs of float32 values, packed arithmetic on them, and the approximate units, for the kernels that
// instructions bound beside the memory.
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

// A vector of a row in memory
template <typename T, int VEC>
struct Vec;
template <typename T>
struct Vec<T, 1> {
    T v;
};
template <>
struct Vec<bf16, 2> {
    uint32_t v;
};
template <>
struct Vec<bf16, 4> {
    uint2 v;
};
template <>
struct Vec<bf16, 8> {
    uint4 v;
};
template <>
struct Vec<float, 4> {
    float4 v;
};

// VEC values in float32 as N of P: pairs, or a single float
template <int VEC>
struct Lanes {
    using P = F2;
    static constexpr int N = VEC / 2;
    static __device__ __forceinline__ P all(float f) { return pair(f, f); }
};
template <>
struct Lanes<1> {
    using P = float;
    static constexpr int N = 1;
    static __device__ __forceinline__ P all(float f) { return f; }
};

template <typename T>
__device__ __forceinline__ void unpack(const Vec<T, 1>& a, float (&f)[1]) { f[0] = to_f32(a.v); }
__device__ __forceinline__ F2 unpack2(uint32_t u) { return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)); }
__device__ __forceinline__ void unpack(const Vec<bf16, 2>& a, F2 (&f)[1]) { f[0] = unpack2(a.v); }
__device__ __forceinline__ void unpack(const Vec<bf16, 4>& a, F2 (&f)[2]) { f[0] = unpack2(a.v.x), f[1] = unpack2(a.v.y); }
__device__ __forceinline__ void unpack(const Vec<bf16, 8>& a, F2 (&f)[4]) {
    f[0] = unpack2(a.v.x), f[1] = unpack2(a.v.y), f[2] = unpack2(a.v.z), f[3] = unpack2(a.v.w);
}
__device__ __forceinline__ void unpack(const Vec<float, 4>& a, F2 (&f)[2]) {
    f[0] = pair(a.v.x, a.v.y), f[1] = pair(a.v.z, a.v.w);
}
template <typename T>
__device__ __forceinline__ void pack(Vec<T, 1>& a, const float (&f)[1]) { a.v = from_f32<T>(f[0]); }
__device__ __forceinline__ uint32_t pack2(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ void pack(Vec<bf16, 2>& a, const F2 (&f)[1]) { a.v = pack2(f[0]); }
__device__ __forceinline__ void pack(Vec<bf16, 4>& a, const F2 (&f)[2]) { a.v = make_uint2(pack2(f[0]), pack2(f[1])); }
__device__ __forceinline__ void pack(Vec<bf16, 8>& a, const F2 (&f)[4]) {
    a.v = make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
__device__ __forceinline__ void pack(Vec<float, 4>& a, const F2 (&f)[2]) {
    split(f[0], a.v.x, a.v.y);
    split(f[1], a.v.z, a.v.w);
}

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> ldvec(const T* p) { return *reinterpret_cast<const Vec<T, VEC>*>(p); }
template <typename T, int VEC, typename P, int N>
__device__ __forceinline__ void stvec(T* p, const P (&f)[N]) {
    Vec<T, VEC> a;
    pack(a, f);
    *reinterpret_cast<Vec<T, VEC>*>(p) = a;
}

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
// act(z), and act'(z) into slope: with s = sigmoid(z) and t = 1 - s, act = p s and act' = s (t p + e),
// where p = z, e = 1 for the SiLU and p = 1, e = 0 for the sigmoid
__device__ __forceinline__ float gate_of(float z, bool silu, float& slope) {
    const float s = fast_rcp(1.f + fast_exp(-z)), t = 1.f - s, p = silu ? z : 1.f;
    slope = s * fmaf(t, p, silu ? 1.f : 0.f);
    return p * s;
}
__device__ __forceinline__ F2 gate_of(F2 z, bool silu, F2& slope) {
    float lo, hi;
    const F2 one = pair(1.f, 1.f);
    split(z * pair(-1.4426950408889634f, -1.4426950408889634f), lo, hi);
    split(fma_(pair(fast_exp2(lo), fast_exp2(hi)), one, one), lo, hi);
    const F2 s = pair(fast_rcp(lo), fast_rcp(hi)), t = fma_(s, pair(-1.f, -1.f), one);
    const F2 p = silu ? z : one;
    slope = s * fma_(t, p, silu ? one : pair(0.f, 0.f));
    return p * s;
}

}  // namespace
}  // namespace hla2
