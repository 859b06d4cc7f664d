// Matrix-vector products with 4-bit weights and group scales (include/hla2.h,
// hla2_w4_matvec):  y[m, n] = sum_k x[m, k] (q[n, k] - z[n, k / group]) s[n, k / group] + bias[n].
//
// Bound by reading the weights: half a byte each.  The products run on mma.sync.m16n8k16 with 16
// weight rows as A and up to eight columns of x as B, which turns the 4-bit values into operands at
// one logic instruction a pair: (w >> 4 i) & 0x000f000f | 0x43004300 is the bf16 pair (128 + q_i, 128 +
// q_{i+4}), and subtracting the pair (128 + z) is exact.  bf16 products are exact in float32,
// so the only roundings are the float32 sums: one group of k is summed unscaled in the
// accumulator, then scaled by the row's float32 scale and added.  A float32 x is split into three
// bf16 columns (8 + 8 + 8 bits), summed at the end.
//
// Within 32 values of k, lane (g, c) = (lane / 4, lane % 4) owns k = 8 c .. 8 c + 7 of rows g and g + 8:
// one 32-bit word of each row.  The order of k inside a product is free as long as A and B agree; the
// word's pairs are (k, k + 4), so x is paired the same way.
//
// One CTA forms 16 outputs; its warps take every kWarps-th block of 128 k and the partial sums meet in
// shared memory, in a fixed order.
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

template <typename T, int NT>
__global__ void __launch_bounds__(kWarps * 32) w4_kernel(const W4Args a) {
    constexpr int kPieces = sizeof(T) == 4 ? 3 : 1;
    __shared__ float red[kWarps][16][NT * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int n0 = blockIdx.x * 16;
    const int r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
    const int gpr = a.K / a.group;
    const uint8_t *w0 = a.w + (size_t)r0 * (a.K / 2), *w1 = a.w + (size_t)r1 * (a.K / 2);
    const T *s0 = static_cast<const T*>(a.scales) + (size_t)r0 * gpr, *s1 = static_cast<const T*>(a.scales) + (size_t)r1 * gpr;
    const uint8_t *z0 = a.zeros + (size_t)r0 * gpr, *z1 = a.zeros + (size_t)r1 * gpr;
    const int cols = a.M * kPieces;
    float sum[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t][0] = sum[t][1] = sum[t][2] = sum[t][3] = 0.f;

    const int step = a.group;  // one group at a time, groups dealt out to the warps
    for (int k0 = warp * step; k0 < a.K; k0 += kWarps * step) {
        const int gi = k0 / a.group;
        const float f0 = to_f32(s0[gi]), f1 = to_f32(s1[gi]);
        const uint32_t q0 = 0x43004300u | (a.zeros ? z0[gi] * 0x00010001u : 0x00080008u);
        const uint32_t q1 = 0x43004300u | (a.zeros ? z1[gi] * 0x00010001u : 0x00080008u);
        float acc[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
        for (int k = k0; k < k0 + step; k += 32) {
            const uint32_t u0 = *reinterpret_cast<const uint32_t*>(w0 + k / 2 + 4 * c);
            const uint32_t u1 = *reinterpret_cast<const uint32_t*>(w1 + k / 2 + 4 * c);
            uint32_t a0[4], a1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a0[i] = sub2(((u0 >> (4 * i)) & 0x000f000fu) | 0x43004300u, q0);
                a1[i] = sub2(((u1 >> (4 * i)) & 0x000f000fu) | 0x43004300u, q1);
            }
            const uint32_t A0[4] = {a0[0], a1[0], a0[1], a1[1]}, A1[4] = {a0[2], a1[2], a0[3], a1[3]};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int col = t * 8 + g;
                uint32_t b[4] = {0u, 0u, 0u, 0u};
                if (col < cols) {
                    const T* xp = static_cast<const T*>(a.x) + (col / kPieces) * a.x_stride + k + 8 * c;
                    if constexpr (kPieces == 1) {
                        pair_x(*reinterpret_cast<const uint4*>(xp), b);
                    } else {
                        const float4 l = *reinterpret_cast<const float4*>(xp), h = *reinterpret_cast<const float4*>(xp + 4);
                        const int p = col % 3;
                        b[0] = pack_bf16x2(piece(l.x, p), piece(h.x, p));
                        b[1] = pack_bf16x2(piece(l.y, p), piece(h.y, p));
                        b[2] = pack_bf16x2(piece(l.z, p), piece(h.z, p));
                        b[3] = pack_bf16x2(piece(l.w, p), piece(h.w, p));
                    }
                }
                mma_16816(acc[t], A0, b[0], b[1]);
                mma_16816(acc[t], A1, b[2], b[3]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sum[t][0] = fmaf(f0, acc[t][0], sum[t][0]);
            sum[t][1] = fmaf(f0, acc[t][1], sum[t][1]);
            sum[t][2] = fmaf(f1, acc[t][2], sum[t][2]);
            sum[t][3] = fmaf(f1, acc[t][3], sum[t][3]);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        red[warp][g][t * 8 + 2 * c] = sum[t][0];
        red[warp][g][t * 8 + 2 * c + 1] = sum[t][1];
        red[warp][g + 8][t * 8 + 2 * c] = sum[t][2];
        red[warp][g + 8][t * 8 + 2 * c + 1] = sum[t][3];
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

template <typename T, int NT>
int launch_w4(const W4Args& a, cudaStream_t st) {
    w4_kernel<T, NT><<<(a.N + 15) / 16, kWarps * 32, 0, st>>>(a);
    return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
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
    const W4Args a{x, x_stride, static_cast<const uint8_t*>(qweight), scales, static_cast<const uint8_t*>(zeros),
                   bias, y, M, N, K, group};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int rc = -1;
    if (dtype == HLA2_BF16) {
        rc = M <= 8 ? launch_w4<bf16, 1>(a, st) : launch_w4<bf16, 2>(a, st);
    } else {
        switch ((3 * M + 7) / 8) {
            case 1: rc = launch_w4<float, 1>(a, st); break;
            case 2: rc = launch_w4<float, 2>(a, st); break;
            case 3: rc = launch_w4<float, 3>(a, st); break;
            case 4: rc = launch_w4<float, 4>(a, st); break;
            case 5: rc = launch_w4<float, 5>(a, st); break;
            default: rc = launch_w4<float, 6>(a, st); break;
        }
    }
    if (rc) return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return w4_ok();
}
