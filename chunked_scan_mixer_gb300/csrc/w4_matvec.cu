// Matrix-vector products with 4-bit weights and group scales (include/hla2.h,
// hla2_w4_matvec):  y[m, n] = sum_k x[m, k] (q[n, k] - z[n, k / group]) s[n, k / group] + bias[n].
//
// Bound by reading the weights: half a byte each.  The products run on mma.sync.m16n8k16 with 16
// weight rows as A and up to eight columns of x as B, which turns the 4-bit values into operands at a
// shift and a logic instruction a pair: (w << 3) & 0x00780078 | 0x41804180 is the bf16 pair
// (16 + q_i, 16 + q_{i+4}), exactly, and so is its difference from (16 + z, 16 + z).  (To sum 16 + q and take (16 + z)
// sum x off would round at the size of 24 sum |x|, whatever is left of it: more than the output's own rounding
// where most weights sit at their zero point.)  A group of k is summed unscaled in float32, and the row's scale
// multiplies there.  A float32 x is split into three bf16 columns (8 + 8 + 8 bits) whose sums meet at the end.
//
// Within a group of G values of k, lane (g, c) = (lane / 4, lane % 4) owns k = c G / 4 ..
// (c + 1) G / 4 - 1 of rows g and g + 8: one load of G / 8 bytes of each row, so a warp reads whole
// 32-byte sectors from G = 64 on.  The order of k inside a product is free as long as A and B agree;
// a word's pairs are (k, k + 4), and x is paired the same way.
//
// Measured: 1 x 8192 x 2048, groups of 128: 4.7 to 7.8 us a call (8.8 MB; floor 1.3).  12 x 10001 x 8192, groups of 64, no
// zero points: 26 us (44 MB; floor 6.5), bound by its instructions (84 for each 512 weights) and by x, which every CTA
// reads: 123 MB through the L2.  Copies of x in shared memory, 32 outputs a CTA and three batches in flight were slower
// (38, 37 and 35 us against 32, with sums of x from a product with ones, since replaced by the exact subtraction).
//
// A CTA forms 16 outputs; its eight warps take every eighth batch of k, the next batch's weights in
// flight while one is computed, and their sums meet in shared memory in a fixed order.
#include "common.cuh"

namespace hla2 {
int set_last_error(int code, const char* fmt, ...);

namespace {

constexpr int kWarps = 8;

struct W4Args {
    const void* x;
    long long x_stride;
    const uint8_t* w;
    const void* scales;
    const uint8_t* zeros;
    const void* bias;
    void* y;
    int M, N, K, group;
};

// x of 8 consecutive k as four bf16 pairs (k, k + 4)
__device__ __forceinline__ void pair_x(const uint4& v, uint32_t (&b)[4]) {
    b[0] = __byte_perm(v.x, v.z, 0x5410);
    b[1] = __byte_perm(v.x, v.z, 0x7632);
    b[2] = __byte_perm(v.y, v.w, 0x5410);
    b[3] = __byte_perm(v.y, v.w, 0x7632);
}

// piece 0, 1, 2 of a float as bf16, x = p0 + p1 + p2 exactly: 8 bits each, cut off rather than rounded
// so that large values do not overflow.  An infinity is its first piece.
__device__ __forceinline__ float cut8(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
__device__ __forceinline__ float piece(float x, int p) {
    const float h = cut8(x), r = x == h ? 0.f : x - h;
    if (p == 0) return h;
    const float m = cut8(r);
    return p == 1 ? m : r - m;
}

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

constexpr int kBatch = 128;  // k per warp step

// U consecutive values of a row's scales or zero points
template <typename T, int U>
struct Few {
    T v[U];
};
template <int B>
struct Bytes;
template <> struct Bytes<1> { using type = uint8_t; };
template <> struct Bytes<2> { using type = uint16_t; };
template <> struct Bytes<4> { using type = uint32_t; };
template <> struct Bytes<8> { using type = uint2; };
template <> struct Bytes<16> { using type = uint4; };
template <typename T, int U>
__device__ __forceinline__ void load_few(Few<T, U>& f, const T* p, int count, bool aligned) {
    constexpr int kBytes = U * (int)sizeof(T);
    if (aligned && count >= U) {
        if constexpr (kBytes <= 16) {
            using V = typename Bytes<kBytes>::type;
            *reinterpret_cast<V*>(f.v) = *reinterpret_cast<const V*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                reinterpret_cast<uint4*>(f.v)[i] = reinterpret_cast<const uint4*>(p)[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < U; ++i) f.v[i] = i < count ? p[i] : T{};
    }
}

// What a warp reads of 16 rows for one batch
template <typename T, int G>
struct Weights {
    static constexpr int U = kBatch / G, J = G / 32;  // groups, words of a row and group
    uint32_t w[2][U][J];
    alignas(16) Few<T, U> s[2];
    alignas(16) Few<uint8_t, U> z[2];
};

template <typename T, int NT, int G>
__global__ void __launch_bounds__(kWarps * 32, NT <= 2 ? 3 : 2) w4_kernel(const W4Args a, const bool aligned) {
    constexpr int kPieces = sizeof(T) == 4 ? 3 : 1, U = kBatch / G, J = G / 32;
    __shared__ float red[kWarps][16][NT * 8 + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * 16, gpr = a.K / G;
    const T* scales = static_cast<const T*>(a.scales);
    const int row[2] = {min(n0 + g, a.N - 1), min(n0 + g + 8, a.N - 1)};
    const int cols = a.M * kPieces;
    float sum[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t][0] = sum[t][1] = sum[t][2] = sum[t][3] = 0.f;

    auto load = [&](Weights<T, G>& b, int k0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* p = a.w + (size_t)row[h] * (a.K / 2) + (k0 + c * (G / 4)) / 2;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = k0 + u * G < a.K;
                    if constexpr (J == 4) {
                        const uint4 v = in ? __ldcs(reinterpret_cast<const uint4*>(p + u * G / 2)) : make_uint4(0, 0, 0, 0);
                        b.w[h][u][0] = v.x, b.w[h][u][1] = v.y, b.w[h][u][2] = v.z, b.w[h][u][3] = v.w;
                    } else if constexpr (J == 2) {
                        const uint2 v = in ? __ldcs(reinterpret_cast<const uint2*>(p + u * G / 2)) : make_uint2(0, 0);
                        b.w[h][u][0] = v.x, b.w[h][u][1] = v.y;
                    } else {
                        b.w[h][u][0] = in ? __ldcs(reinterpret_cast<const uint32_t*>(p + u * G / 2)) : 0u;
                    }
                }
                const size_t at = (size_t)row[h] * gpr + k0 / G;
                const int count = min(U, gpr - k0 / G);
                load_few<T, U>(b.s[h], scales + at, count, aligned);
                if (a.zeros) load_few<uint8_t, U>(b.z[h], a.zeros + at, count, aligned);
            }
    };
    auto compute = [&](const Weights<T, G>& b, int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k0 + u * G >= a.K) break;
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
            uint32_t zz[2];  // the pair (16 + z, 16 + z)
#pragma unroll
            for (int h = 0; h < 2; ++h) zz[h] = 0x41804180u | ((a.zeros ? b.z[h].v[u] : 8u) * 0x00080008u);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint32_t x[NT][4];
                const int k = k0 + u * G + c * (G / 4) + 8 * j;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int col = t * 8 + g;
                    x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0u;
                    if (col < cols) {
                        const T* xp = static_cast<const T*>(a.x) + (col / kPieces) * a.x_stride + k;
                        if constexpr (kPieces == 1) {
                            pair_x(*reinterpret_cast<const uint4*>(xp), x[t]);
                        } else {
                            const float4 l = *reinterpret_cast<const float4*>(xp), h = *reinterpret_cast<const float4*>(xp + 4);
                            const int p = col % 3;
                            x[t][0] = pack_bf16x2(piece(l.x, p), piece(h.x, p));
                            x[t][1] = pack_bf16x2(piece(l.y, p), piece(h.y, p));
                            x[t][2] = pack_bf16x2(piece(l.z, p), piece(h.z, p));
                            x[t][3] = pack_bf16x2(piece(l.w, p), piece(h.w, p));
                        }
                    }
                }
                {
                    uint32_t q[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w = b.w[h][u][j];
                        q[h][0] = ((w << 3) & 0x00780078u) | 0x41804180u;
                        q[h][1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
                        q[h][2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
                        q[h][3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
#pragma unroll
                        for (int i = 0; i < 4; ++i) q[h][i] = sub2(q[h][i], zz[h]);
                    }
                    const uint32_t A0[4] = {q[0][0], q[1][0], q[0][1], q[1][1]}, A1[4] = {q[0][2], q[1][2], q[0][3], q[1][3]};
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma_16816(acc[t], A0, x[t][0], x[t][1]);
                        mma_16816(acc[t], A1, x[t][2], x[t][3]);
                    }
                }
            }
            {
                const float f0 = to_f32(b.s[0].v[u]), f1 = to_f32(b.s[1].v[u]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    sum[t][0] = fmaf(f0, acc[t][0], sum[t][0]);
                    sum[t][1] = fmaf(f0, acc[t][1], sum[t][1]);
                    sum[t][2] = fmaf(f1, acc[t][2], sum[t][2]);
                    sum[t][3] = fmaf(f1, acc[t][3], sum[t][3]);
                }
            }
        }
    };
    pdl_wait();
    Weights<T, G> b0, b1;
    const int step = kWarps * kBatch;
    int k0 = warp * kBatch;
    if (k0 < a.K) load(b0, k0);
    for (; k0 < a.K; k0 += 2 * step) {
        if (k0 + step < a.K) load(b1, k0 + step);
        compute(b0, k0);
        if (k0 + step >= a.K) break;
        if (k0 + 2 * step < a.K) load(b0, k0 + 2 * step);
        compute(b1, k0 + step);
    }
    // Not earlier: the next kernel's CTAs would crowd on the SMs that are free while this one runs (128 CTAs, K = 8192:
    // 9.7 us became 12.2).
    pdl_trigger();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float* p = &red[warp][g][t * 8 + 2 * c];
            p[0] = sum[t][0];
            p[1] = sum[t][1];
            p = &red[warp][g + 8][t * 8 + 2 * c];
            p[0] = sum[t][2];
            p[1] = sum[t][3];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * a.M; e += kWarps * 32) {
        const int r = e & 15, m = e >> 4;
        if (n0 + r >= a.N) continue;
        float t = 0.f;
#pragma unroll
        for (int p = kPieces - 1; p >= 0; --p)
            for (int w = 0; w < kWarps; ++w) t += red[w][r][m * kPieces + p];
        if (a.bias) t += to_f32(static_cast<const T*>(a.bias)[n0 + r]);
        static_cast<T*>(a.y)[(size_t)m * a.N + n0 + r] = from_f32<T>(t);
    }
}

template <typename T, int NT, int G>
int launch_w4_g(const W4Args& a, cudaStream_t st) {
    const bool aligned = (a.K / G) % (kBatch / G) == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 15u) == 0 &&
                         (reinterpret_cast<uintptr_t>(a.zeros) & 15u) == 0;
    return launch_pdl(w4_kernel<T, NT, G>, dim3((a.N + 15) / 16), dim3(kWarps * 32), 0, st, a, aligned) == cudaSuccess ? 0 : -1;
}
template <typename T, int NT>
int launch_w4(const W4Args& a, cudaStream_t st) {
    switch (a.group) {
        case 32: return launch_w4_g<T, NT, 32>(a, st);
        case 64: return launch_w4_g<T, NT, 64>(a, st);
        default: return launch_w4_g<T, NT, 128>(a, st);
    }
}

int w4_ok() { return set_last_error(HLA2_OK, "%s", ""); }

}  // namespace
}  // namespace hla2

using namespace hla2;

extern "C" int hla2_w4_matvec(const void* x, long long x_stride, const void* qweight, const void* scales,
                              const void* zeros, const void* bias, void* y, int M, int N, int K, int group, int dtype,
                              hla2_stream_t stream) {
    static const char* const fn = "hla2_w4_matvec";
    if (dtype != HLA2_F32 && dtype != HLA2_BF16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dtype must be HLA2_F32 or HLA2_BF16", fn);
    if (group != 32 && group != 64 && group != 128)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: group must be 32, 64 or 128 (got %d)", fn, group);
    if (M < 0 || N < 0 || K < 0 || K % group)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: M, N, K must not be negative and K a multiple of the group", fn);
    if (M > 16) return set_last_error(HLA2_ERR_UNSUPPORTED, "%s: at most 16 rows of x (got %d)", fn, M);
    if (M == 0 || N == 0) return w4_ok();
    auto al = [](const void* p, size_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; };
    const size_t es = dtype == HLA2_BF16 ? 2 : 4;
    if (!y || (K > 0 && (!x || !qweight || !scales)))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: x, qweight, scales and y must not be NULL", fn);
    if (!al(x, 16) || (M > 1 && (x_stride * (long long)es) % 16) || !al(qweight, 16))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: x, its rows and qweight must be 16-byte aligned", fn);
    if (!al(scales, es) || !al(bias, es) || !al(y, es))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    const Extent ey = extent_of(y, (size_t)M * N * es);
    for (const Extent& i : {extent_of(x, (size_t)((M - 1) * x_stride + K) * es), extent_of(qweight, (size_t)N * (K / 2)),
                            extent_of(scales, (size_t)N * (K / group) * es), extent_of(zeros, (size_t)N * (K / group)),
                            extent_of(bias, N * es)})
        if (meet(ey, i)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: y overlaps an input", fn);
    const W4Args a{x, x_stride, static_cast<const uint8_t*>(qweight), scales, static_cast<const uint8_t*>(zeros),
                   bias, y, M, N, K, group};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int rc = -1;
    if (dtype == HLA2_BF16) {
        rc = M <= 8 ? launch_w4<bf16, 1>(a, st) : launch_w4<bf16, 2>(a, st);
    } else {
        rc = M <= 2 ? launch_w4<float, 1>(a, st) : M <= 5 ? launch_w4<float, 2>(a, st)
             : M <= 8 ? launch_w4<float, 3>(a, st) : launch_w4<float, 6>(a, st);
    }
    if (rc) return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return w4_ok();
}
