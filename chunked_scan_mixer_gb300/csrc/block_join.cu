// The norms before and after a block, fused with the block's gate and residual scale, forward
// and backward (include/hla2.h, hla2_block_join).  Per row of D values:
//   ny = y / sqrt(mean(y^2) + eps),  u = ny w_post,  r = x + s a u  (a = act(gate)),
//   nr = r / sqrt(mean(r^2) + eps),  h = nr w_next
// and for the gradients dr, dh:
//   R = dr + inv_r (dh w_next - nr mean(dh w_next nr)),   dx = R,   dw_next += dh nr,
//   ds += R a u,   dgate = R s u act'(gate),   dw_post += R s a ny,
//   dy = inv_y (R s a w_post - ny mean(R s a w_post ny)).
// The backward forms the statistics again from x, y and the gate: nothing is kept from the
// forward, and r enters unrounded.
//
// Bound by memory: 5 tensors forward, 8 backward.  A row stays in the registers of its threads
// (NV vectors of VEC values each) from the one read to the one write.  Rows of at most 32 vectors
// take a part of a warp (TPR threads), longer ones a whole CTA.  Backward CTAs take rows in a fixed
// stride and keep their three weight gradients in registers; each writes one partial row, which a
// second kernel sums in a fixed order.
#include <type_traits>

#include "common.cuh"

namespace hla2 {
int set_last_error(int code, const char* fmt, ...);

namespace {

constexpr int kMaxD = 8192;
constexpr int kSmallThreads = 256;  // CTA size of the sub-warp mapping

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
struct Vec<bf16, 8> {
    uint4 v;
};
template <>
struct Vec<float, 4> {
    float4 v;
};

template <typename T>
__device__ __forceinline__ void unpack(const Vec<T, 1>& a, float (&f)[1]) { f[0] = to_f32(a.v); }
__device__ __forceinline__ void unpack2(uint32_t u, float* f) {
    f[0] = __uint_as_float(u << 16);
    f[1] = __uint_as_float(u & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack(const Vec<bf16, 2>& a, float (&f)[2]) { unpack2(a.v, f); }
__device__ __forceinline__ void unpack(const Vec<bf16, 8>& a, float (&f)[8]) {
    unpack2(a.v.x, f);
    unpack2(a.v.y, f + 2);
    unpack2(a.v.z, f + 4);
    unpack2(a.v.w, f + 6);
}
__device__ __forceinline__ void unpack(const Vec<float, 4>& a, float (&f)[4]) {
    f[0] = a.v.x, f[1] = a.v.y, f[2] = a.v.z, f[3] = a.v.w;
}
template <typename T>
__device__ __forceinline__ void pack(Vec<T, 1>& a, const float (&f)[1]) { a.v = from_f32<T>(f[0]); }
__device__ __forceinline__ void pack(Vec<bf16, 2>& a, const float (&f)[2]) { a.v = pack_bf16x2(f[0], f[1]); }
__device__ __forceinline__ void pack(Vec<bf16, 8>& a, const float (&f)[8]) {
    a.v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void pack(Vec<float, 4>& a, const float (&f)[4]) { a.v = make_float4(f[0], f[1], f[2], f[3]); }

template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> ldvec(const T* p) { return *reinterpret_cast<const Vec<T, VEC>*>(p); }
template <typename T, int VEC>
__device__ __forceinline__ void stvec(T* p, const float (&f)[VEC]) {
    Vec<T, VEC> a;
    pack(a, f);
    *reinterpret_cast<Vec<T, VEC>*>(p) = a;
}

// Sums of N values over the threads of a row: TPR lanes of a warp, or (TPR == 0) the CTA.
// `red` alternates between two halves, so one barrier a call is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[32][N], int& turn) {
#pragma unroll
    for (int o = (TPR ? TPR : 32) / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (TPR == 0) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[turn][warp][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = lane < nw ? red[turn][lane][i] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        turn ^= 1;
    }
}

// act(z) and act'(z)
__device__ __forceinline__ float sigmoidf(float z) { return 1.f / (1.f + __expf(-z)); }
__device__ __forceinline__ float act_of(float z, int act) {
    const float s = sigmoidf(z);
    return act == HLA2_GATE_SILU ? z * s : s;
}
__device__ __forceinline__ float act_slope(float z, int act) {
    const float s = sigmoidf(z);
    return act == HLA2_GATE_SILU ? s * (1.f + z * (1.f - s)) : s * (1.f - s);
}

template <typename T, int VEC, int NV, int TPR, int MAXT>
__global__ void __launch_bounds__(MAXT) join_kernel(const hla2_block_args a, T* __restrict__ r_out, T* __restrict__ h_out) {
    __shared__ float red[2][32][1];
    int turn = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr;
    const long long row = TPR ? (long long)blockIdx.x * (kSmallThreads / (TPR ? TPR : 1)) + threadIdx.x / tpr : blockIdx.x;
    const bool live = row < a.rows;  // whole sub-warps: lanes of a dead row take part in the shuffles
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    const T *x = static_cast<const T*>(a.x) + (live ? row * a.x_stride : 0),
            *y = static_cast<const T*>(a.y) + (live ? row * a.y_stride : 0),
            *z = static_cast<const T*>(a.gate) + (live ? row * a.gate_stride : 0);
    const T *pw = static_cast<const T*>(a.post_weight), *sc = static_cast<const T*>(a.scale),
            *nw = static_cast<const T*>(a.next_weight);
    Vec<T, VEC> xv[NV], yv[NV], zv[NV];
    const bool full = a.gate && a.gate_cols != 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + t) * VEC;
        if (live && c < D) {
            xv[j] = ldvec<T, VEC>(x + c);
            if (a.y) yv[j] = ldvec<T, VEC>(y + c);
            if (full) zv[j] = ldvec<T, VEC>(z + c);
        }
    }
    float r[NV][VEC], sum[1] = {0.f};
    if (a.y) {
        const float a_row = a.gate && !full && live ? act_of(to_f32(z[0]), a.gate_act) : 1.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && (j * tpr + t) * VEC < D) {
                float f[VEC];
                unpack(yv[j], f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[0] += f[i] * f[i];
            }
        row_sum<TPR, 1>(sum, red, turn);
        const float inv = rsqrtf(sum[0] * inv_d + a.eps);
        sum[0] = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * tpr + t) * VEC;
            if (live && c < D) {
                float fx[VEC], fy[VEC], fz[VEC], fw[VEC], fs[VEC];
                unpack(xv[j], fx);
                unpack(yv[j], fy);
                unpack(ldvec<T, VEC>(pw + c), fw);
                if (full) unpack(zv[j], fz);
                if (sc) unpack(ldvec<T, VEC>(sc + c), fs);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float u = fy[i] * inv * fw[i], g = full ? act_of(fz[i], a.gate_act) : a_row;
                    r[j][i] = fx[i] + (sc ? fs[i] * g * u : g * u);
                    sum[0] += r[j][i] * r[j][i];
                }
                stvec<T, VEC>(r_out + row * D + c, r[j]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && (j * tpr + t) * VEC < D) {
                unpack(xv[j], r[j]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[0] += r[j][i] * r[j][i];
            }
    }
    if (!h_out) return;
    row_sum<TPR, 1>(sum, red, turn);
    const float inv = rsqrtf(sum[0] * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * tpr + t) * VEC;
        if (live && c < D) {
            float fw[VEC], o[VEC];
            unpack(ldvec<T, VEC>(nw + c), fw);
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = r[j][i] * inv * fw[i];
            stvec<T, VEC>(h_out + row * D + c, o);
        }
    }
}

struct JoinGrads {
    const void *dr, *dh;
    void *dx, *dy, *dgate;
    float* partial;  // [partials][3][D]: post_weight, scale, next_weight
    int partials;
};

template <typename T, int VEC, int NV, int TPR, int MAXT>
__global__ void __launch_bounds__(MAXT) join_backward_kernel(const hla2_block_args a, const JoinGrads g) {
    __shared__ float red1[2][32][1], red2[2][32][2];
    extern __shared__ float acc_sm[];  // sub-warp mapping: [3][D]
    int turn1 = 0, turn2 = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr;
    const int per = TPR ? kSmallThreads / (TPR ? TPR : 1) : 1, mine = threadIdx.x / tpr;
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    const T *pw = static_cast<const T*>(a.post_weight), *sc = static_cast<const T*>(a.scale),
            *nw = static_cast<const T*>(a.next_weight);
    const bool full = a.gate && a.gate_cols != 1;
    float gp[NV][VEC], gs[NV][VEC], gn[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) gp[j][i] = gs[j][i] = gn[j][i] = 0.f;

    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += (long long)gridDim.x * per) {
        const long long row = row0 + mine;
        const bool live = row < a.rows;
        const long long at = live ? row : 0;
        const T *x = static_cast<const T*>(a.x) + at * a.x_stride, *y = static_cast<const T*>(a.y) + at * a.y_stride,
                *z = static_cast<const T*>(a.gate) + at * a.gate_stride;
        const T *dr = static_cast<const T*>(g.dr) + at * D, *dh = static_cast<const T*>(g.dh) + at * D;
        Vec<T, VEC> xv[NV], yv[NV], zv[NV], rv[NV], hv[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * tpr + t) * VEC;
            if (live && c < D) {
                xv[j] = ldvec<T, VEC>(x + c);
                if (a.y) yv[j] = ldvec<T, VEC>(y + c);
                if (full) zv[j] = ldvec<T, VEC>(z + c);
                if (g.dr) rv[j] = ldvec<T, VEC>(dr + c);
                if (g.dh) hv[j] = ldvec<T, VEC>(dh + c);
            }
        }
        const float z_row = a.gate && !full && live ? to_f32(z[0]) : 0.f;
        const float a_row = a.gate && !full ? act_of(z_row, a.gate_act) : 1.f;
        float inv_y = 0.f;
        if (a.y) {
            float s1[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (live && (j * tpr + t) * VEC < D) {
                    float f[VEC];
                    unpack(yv[j], f);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s1[0] += f[i] * f[i];
                }
            row_sum<TPR, 1>(s1, red1, turn1);
            inv_y = rsqrtf(s1[0] * inv_d + a.eps);
        }
        // r again, sum r^2 and sum (dh w) r
        float R[NV][VEC], inv_r = 0.f, dot = 0.f;
        if (g.dh) {
            float s2[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * tpr + t) * VEC;
                if (live && c < D) {
                    float fx[VEC], fh[VEC], fn[VEC];
                    unpack(xv[j], fx);
                    unpack(hv[j], fh);
                    unpack(ldvec<T, VEC>(nw + c), fn);
                    if (a.y) {
                        float fy[VEC], fz[VEC], fw[VEC], fs[VEC];
                        unpack(yv[j], fy);
                        unpack(ldvec<T, VEC>(pw + c), fw);
                        if (full) unpack(zv[j], fz);
                        if (sc) unpack(ldvec<T, VEC>(sc + c), fs);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float u = fy[i] * inv_y * fw[i], ga = full ? act_of(fz[i], a.gate_act) : a_row;
                            fx[i] += sc ? fs[i] * ga * u : ga * u;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        R[j][i] = fx[i];
                        s2[0] += fx[i] * fx[i];
                        s2[1] += fh[i] * fn[i] * fx[i];
                    }
                }
            }
            row_sum<TPR, 2>(s2, red2, turn2);
            inv_r = rsqrtf(s2[0] * inv_d + a.eps);
            dot = s2[1] * inv_r * inv_d;
        }
        // the gradient of r; of the gate, the scale and y's norm
        float s3[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * tpr + t) * VEC;
            if (live && c < D) {
                float f[VEC], fr[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) fr[i] = 0.f;
                if (g.dr) unpack(rv[j], fr);
                if (g.dh) {
                    float fn[VEC];
                    unpack(hv[j], f);
                    unpack(ldvec<T, VEC>(nw + c), fn);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float nr = R[j][i] * inv_r;
                        gn[j][i] += f[i] * nr;
                        fr[i] += inv_r * (f[i] * fn[i] - nr * dot);
                    }
                }
                stvec<T, VEC>(static_cast<T*>(g.dx) + row * D + c, fr);
                if (a.y) {
                    float fy[VEC], fz[VEC], fw[VEC], fs[VEC], dz[VEC];
                    unpack(yv[j], fy);
                    unpack(ldvec<T, VEC>(pw + c), fw);
                    if (full) unpack(zv[j], fz);
                    if (sc) unpack(ldvec<T, VEC>(sc + c), fs);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float ny = fy[i] * inv_y, u = ny * fw[i], ga = full ? act_of(fz[i], a.gate_act) : a_row;
                        const float Rs = sc ? fr[i] * fs[i] : fr[i];
                        gs[j][i] += fr[i] * ga * u;
                        const float du = Rs * ga;
                        gp[j][i] += du * ny;
                        if (full) dz[i] = Rs * u * act_slope(fz[i], a.gate_act);
                        else s3[1] += Rs * u;
                        R[j][i] = du * fw[i];  // gradient of ny
                        s3[0] += R[j][i] * ny;
                    }
                    if (full) stvec<T, VEC>(static_cast<T*>(g.dgate) + row * D + c, dz);
                }
            }
        }
        if (a.y) {
            row_sum<TPR, 2>(s3, red2, turn2);
            const float m = s3[0] * inv_d;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * tpr + t) * VEC;
                if (live && c < D) {
                    float fy[VEC], o[VEC];
                    unpack(yv[j], fy);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o[i] = inv_y * (R[j][i] - fy[i] * inv_y * m);
                    stvec<T, VEC>(static_cast<T*>(g.dy) + row * D + c, o);
                }
            }
            if (a.gate && !full && live && t == 0)
                static_cast<T*>(g.dgate)[row] = from_f32<T>(s3[1] * act_slope(z_row, a.gate_act));
        }
    }
    float* dst = g.partial + (size_t)blockIdx.x * 3 * D;
    if (TPR) {  // the CTA's row groups one after another, so that the order is fixed
        for (int who = 0; who < per; ++who) {
            if (mine == who) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int c = (j * tpr + t) * VEC + i;
                        if (c < D) {
                            acc_sm[c] = (who ? acc_sm[c] : 0.f) + gp[j][i];
                            acc_sm[D + c] = (who ? acc_sm[D + c] : 0.f) + gs[j][i];
                            acc_sm[2 * D + c] = (who ? acc_sm[2 * D + c] : 0.f) + gn[j][i];
                        }
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 3 * D; c += kSmallThreads) dst[c] = acc_sm[c];
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = (j * tpr + t) * VEC + i;
                if (c < D) {
                    dst[c] = gp[j][i];
                    dst[D + c] = gs[j][i];
                    dst[2 * D + c] = gn[j][i];
                }
            }
    }
}

// Sums the partial rows: 32 columns a CTA, 32 row lanes, then a tree over them in a fixed order.
__global__ void __launch_bounds__(1024) partial_sum_kernel(const float* __restrict__ partial, int partials, int D,
                                                           float* __restrict__ d0, float* __restrict__ d1,
                                                           float* __restrict__ d2) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
    float* dst = which == 0 ? d0 : which == 1 ? d1 : d2;
    if (!dst) return;
    float s = 0.f;
    if (c < D)
        for (int p = w; p < partials; p += 32) s += partial[((size_t)p * 3 + which) * D + c];
    sm[w][lane] = s;
    __syncthreads();
    for (int o = 16; o; o >>= 1) {
        if (w < o) sm[w][lane] += sm[w + o][lane];
        __syncthreads();
    }
    if (w == 0 && c < D) dst[c] = sm[0][lane];
}

// ---- launch choice ------------------------------------------------------------------------

bool al(const void* p, size_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }

// Elements per vector: 16 bytes where every row and vector allows it; else pairs of bf16 in 4 bytes; else
// single elements.
int vec_of(const hla2_block_args* a, const void* const* more, int nmore) {
    auto fits = [&](int vec) {
        const size_t b = (size_t)vec * (a->dtype == HLA2_BF16 ? 2 : 4);
        if (a->D % vec || !al(a->x, b) || !al(a->next_weight, b) || a->x_stride % vec) return false;
        if (a->y && (!al(a->y, b) || !al(a->post_weight, b) || !al(a->scale, b) || a->y_stride % vec)) return false;
        if (a->y && a->gate && a->gate_cols != 1 && (!al(a->gate, b) || a->gate_stride % vec)) return false;
        for (int i = 0; i < nmore; ++i)
            if (!al(more[i], b)) return false;
        return true;
    };
    const int wide = a->dtype == HLA2_BF16 ? 8 : 4;
    if (fits(wide)) return wide;
    if (a->dtype == HLA2_BF16 && fits(2)) return 2;
    return 1;
}

struct Shape {
    int tpr;      // threads per row in a sub-warp mapping, 0: a CTA per row
    int threads;  // CTA size
    int nv;       // vectors per thread
};
// At most 256 threads and 8 values a thread up to D = 2048 (the registers of the backward, which
// keeps five inputs, three weight gradients and one intermediate per value), then 512 threads.
constexpr int kNarrowD = 2048;
Shape shape_of(int D, int vec) {
    const int nvec = (D + vec - 1) / vec;
    if (nvec <= 32) {
        int t = 4;
        while (t < nvec) t *= 2;
        return {t, kSmallThreads, 1};
    }
    const int most = D <= kNarrowD ? 256 : 512;
    int nv = 1;
    while ((nvec + nv - 1) / nv > most) nv *= 2;
    return {0, ((nvec + nv - 1) / nv + 31) / 32 * 32, nv};
}

// f(NV, TPR, MAXT) as integral constants for the shape
template <int VEC, class F>
int with_shape(int D, const Shape& s, F&& f) {
    using std::integral_constant;
    auto go = [&](auto nv, auto tpr, auto maxt) { return f(integral_constant<int, VEC>{}, nv, tpr, maxt); };
    const integral_constant<int, 1> one{};
    const integral_constant<int, 0> cta{};
    const integral_constant<int, kSmallThreads> small{};
    const integral_constant<int, 512> large{};
    switch (s.tpr) {
        case 4: return go(one, integral_constant<int, 4>{}, small);
        case 8: return go(one, integral_constant<int, 8>{}, small);
        case 16: return go(one, integral_constant<int, 16>{}, small);
        case 32: return go(one, integral_constant<int, 32>{}, small);
        default: break;
    }
    if (D <= kNarrowD) {
        if (s.nv == 1) return go(one, cta, small);
        if constexpr (VEC < 8) {
            if (s.nv == 2) return go(integral_constant<int, 2>{}, cta, small);
        }
        if constexpr (VEC < 4) {
            if (s.nv == 4) return go(integral_constant<int, 4>{}, cta, small);
        }
        if constexpr (VEC < 2) {
            if (s.nv == 8) return go(integral_constant<int, 8>{}, cta, small);
        }
        return -1;
    }
    if (s.nv == 8 / VEC) return go(integral_constant<int, 8 / VEC>{}, cta, large);
    if (s.nv == 16 / VEC) return go(integral_constant<int, 16 / VEC>{}, cta, large);
    return -1;
}
template <class F>
int with_vec(int D, int vec, const Shape& s, F&& f) {
    switch (vec) {
        case 8: return with_shape<8>(D, s, f);
        case 4: return with_shape<4>(D, s, f);
        case 2: return with_shape<2>(D, s, f);
        default: return with_shape<1>(D, s, f);
    }
}

int join_ok() { return set_last_error(HLA2_OK, "%s", ""); }

// Whether the call has a block output; without rows there is no address to go by.
bool has_y(const hla2_block_args* a) { return a->rows > 0 ? a->y != nullptr : a->post_weight != nullptr; }

int check_join(const char* fn, const hla2_block_args* a) {
    if (!a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: args must not be NULL", fn);
    if (a->dtype != HLA2_F32 && a->dtype != HLA2_BF16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dtype must be HLA2_F32 or HLA2_BF16", fn);
    if (a->D < 1 || a->D > kMaxD)
        return set_last_error(a->D < 1 ? HLA2_ERR_INVALID_ARG : HLA2_ERR_UNSUPPORTED, "%s: D must be 1 .. %d (got %d)",
                              fn, kMaxD, a->D);
    if (a->rows < 0 || a->rows > 0x7fffffffLL)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: rows must be 0 .. 2^31 - 1", fn);
    if (!has_y(a) && !a->next_weight)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: nothing to form without y and next_weight", fn);
    if (a->y && !a->post_weight) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: y needs post_weight", fn);
    if (!has_y(a) && (a->gate || a->scale || a->post_weight))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: gate, scale and post_weight need y", fn);
    if (a->gate && (a->gate_act != HLA2_GATE_SIGMOID && a->gate_act != HLA2_GATE_SILU))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: unknown gate_act %d", fn, a->gate_act);
    if (a->gate && a->gate_cols != 1 && a->gate_cols != a->D)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: gate_cols must be 1 or D", fn);
    const size_t es = a->dtype == HLA2_BF16 ? 2 : 4;
    if (!al(a->x, es) || !al(a->y, es) || !al(a->gate, es) || !al(a->post_weight, es) || !al(a->scale, es) ||
        !al(a->next_weight, es))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    if (a->rows > 0) {
        if (!a->x) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: x must not be NULL", fn);
        if (a->rows > 1 && (a->x_stride < 0 || (a->y && a->y_stride < 0) || (a->gate && a->gate_stride < 0)))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
    }
    return HLA2_OK;
}

int sms() {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    return v;
}

// CTAs of the backward: at most four per SM, no more than there are rows for.
int backward_ctas(const hla2_block_args* a, const Shape& s) {
    const int per = s.tpr ? kSmallThreads / s.tpr : 1;
    long long need = (a->rows + per - 1) / per;
    const long long most = 4LL * sms();
    return (int)(need < most ? need : most);
}

}  // namespace
}  // namespace hla2

using namespace hla2;

extern "C" {

int hla2_block_join(const hla2_block_args* a, void* r, void* h, hla2_stream_t stream) {
    static const char* const fn = "hla2_block_join";
    if (int rc = check_join(fn, a)) return rc;
    if ((a->y != nullptr) != (r != nullptr) || (a->next_weight != nullptr) != (h != nullptr))
        return (a->rows == 0) ? join_ok()
                              : set_last_error(HLA2_ERR_INVALID_ARG,
                                               "%s: r is needed with y, h with next_weight, and neither without", fn);
    if (a->rows == 0) return join_ok();
    const size_t es = a->dtype == HLA2_BF16 ? 2 : 4;
    if (!al(r, es) || !al(h, es)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: misaligned output", fn);
    if (r && r == h) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: r and h must be distinct", fn);
    const void* outs[2] = {r, h};
    const int vec = vec_of(a, outs, 2);
    const Shape s = shape_of(a->D, vec);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto launch = [&](auto v, auto nv, auto tpr, auto maxt) {
        constexpr int VEC = decltype(v)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value,
                      MAXT = decltype(maxt)::value;
        const unsigned grid = TPR ? (unsigned)((a->rows + kSmallThreads / TPR - 1) / (kSmallThreads / TPR)) : (unsigned)a->rows;
        if constexpr (VEC == 8 || VEC == 2) {
            join_kernel<bf16, VEC, NV, TPR, MAXT><<<grid, s.threads, 0, st>>>(*a, static_cast<bf16*>(r), static_cast<bf16*>(h));
        } else if constexpr (VEC == 4) {
            join_kernel<float, VEC, NV, TPR, MAXT><<<grid, s.threads, 0, st>>>(*a, static_cast<float*>(r), static_cast<float*>(h));
        } else if (a->dtype == HLA2_BF16) {
            join_kernel<bf16, 1, NV, TPR, MAXT><<<grid, s.threads, 0, st>>>(*a, static_cast<bf16*>(r), static_cast<bf16*>(h));
        } else {
            join_kernel<float, 1, NV, TPR, MAXT><<<grid, s.threads, 0, st>>>(*a, static_cast<float*>(r), static_cast<float*>(h));
        }
        return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
    };
    if (with_vec(a->D, vec, s, launch))
        return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return join_ok();
}

size_t hla2_block_join_backward_workspace_bytes(const hla2_block_args* a) {
    if (check_join("hla2_block_join_backward_workspace_bytes", a) != HLA2_OK) return (size_t)-1;
    join_ok();
    size_t most = 0;
    const int wide = a->dtype == HLA2_BF16 ? 8 : 4;
    for (int vec : {1, 2, wide}) {  // whichever the addresses allow
        const size_t c = (size_t)backward_ctas(a, shape_of(a->D, vec));
        if (c > most) most = c;
    }
    return most * 3 * (size_t)a->D * sizeof(float);
}

int hla2_block_join_backward(const hla2_block_args* a, const void* dr, const void* dh, void* dx, void* dy, void* dgate,
                             float* dpost_weight, float* dscale, float* dnext_weight, void* workspace,
                             size_t workspace_bytes, hla2_stream_t stream) {
    static const char* const fn = "hla2_block_join_backward";
    if (int rc = check_join(fn, a)) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t es = a->dtype == HLA2_BF16 ? 2 : 4;
    if ((has_y(a) && !dpost_weight) || (a->scale && !dscale) || (a->next_weight && !dnext_weight))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a weight's gradient is missing", fn);
    if ((!has_y(a) && (dpost_weight || dy)) || (!a->scale && dscale) || (!a->next_weight && (dnext_weight || dh)) ||
        (!a->gate && dgate))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient is asked for without its input", fn);
    if (a->rows > 0) {
        if (!dx || (a->y && !dy) || (a->gate && !dgate) || (a->next_weight && !dh) || (!dr && !dh))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient of rows is missing", fn);
        if (!al(dr, es) || !al(dh, es) || !al(dx, es) || !al(dy, es) || !al(dgate, es) || !al(dpost_weight, 4) ||
            !al(dscale, 4) || !al(dnext_weight, 4))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    }
    const size_t need = hla2_block_join_backward_workspace_bytes(a);
    if (need > 0 && (!workspace || workspace_bytes < need || !al(workspace, 16)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    JoinGrads g{dr, dh, dx, dy, dgate, static_cast<float*>(workspace), 0};
    if (a->rows > 0) {
        const void* outs[5] = {dr, dh, dx, dy, a->gate_cols != 1 ? dgate : nullptr};
        const int vec = vec_of(a, outs, 5);
        const Shape s = shape_of(a->D, vec);
        g.partials = backward_ctas(a, s);
        auto launch = [&](auto v, auto nv, auto tpr, auto maxt) {
            constexpr int VEC = decltype(v)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value,
                      MAXT = decltype(maxt)::value;
            const size_t smem = TPR ? 3 * (size_t)a->D * sizeof(float) : 0;
            if constexpr (VEC == 8 || VEC == 2) {
                join_backward_kernel<bf16, VEC, NV, TPR, MAXT><<<g.partials, s.threads, smem, st>>>(*a, g);
            } else if constexpr (VEC == 4) {
                join_backward_kernel<float, VEC, NV, TPR, MAXT><<<g.partials, s.threads, smem, st>>>(*a, g);
            } else if (a->dtype == HLA2_BF16) {
                join_backward_kernel<bf16, 1, NV, TPR, MAXT><<<g.partials, s.threads, smem, st>>>(*a, g);
            } else {
                join_backward_kernel<float, 1, NV, TPR, MAXT><<<g.partials, s.threads, smem, st>>>(*a, g);
            }
            return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
        };
        if (with_vec(a->D, vec, s, launch))
            return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    }
    partial_sum_kernel<<<dim3((a->D + 31) / 32, 3), 1024, 0, st>>>(g.partial, g.partials, a->D, dpost_weight, dscale,
                                                                   dnext_weight);
    if (cudaPeekAtLastError() != cudaSuccess)
        return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return join_ok();
}

}  // extern "C"
