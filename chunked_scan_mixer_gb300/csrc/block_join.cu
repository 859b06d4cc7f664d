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
// Bound by memory: 5 tensors forward, 8 backward.  Persistent CTAs take rows in a fixed stride.  A thread
// owns NV vectors of VEC values of every row; it copies them ahead with cp.async into a ring of kStages
// rows in shared memory that nobody else reads, so the ring needs no barrier, and the bytes in flight do
// not cost registers (plain loads into registers held 152 of them, one CTA per SM, 1.2 TB/s).
// Rows of at most 32 vectors take a part of a warp (TPR threads), longer ones a whole CTA.  The backward
// keeps its three weight gradients in registers; each CTA writes one partial row, which a second
// kernel sums in a fixed order.
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
// (the approximate reciprocal is good to an ulp, and 0 at infinity)
__device__ __forceinline__ float sigmoidf(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ float act_of(float z, int act) {
    const float s = sigmoidf(z);
    return act == HLA2_GATE_SILU ? z * s : s;
}
__device__ __forceinline__ float act_slope(float z, int act) {
    const float s = sigmoidf(z);
    return act == HLA2_GATE_SILU ? s * (1.f + z * (1.f - s)) : s * (1.f - s);
}

// One thread's ring: slot (stage, tensor, j) holds its j-th vector of that tensor's row.
template <typename T, int VEC, int NV>
struct Ring {
    static constexpr int kBytes = VEC * (int)sizeof(T);
    char* base;       // this thread's first slot
    uint32_t step;    // bytes between slots: the CTA's threads side by side
    int tensors;
    __device__ __forceinline__ Ring(char* sm, int n) : base(sm + threadIdx.x * kBytes), step(blockDim.x * kBytes), tensors(n) {}
    __device__ __forceinline__ char* at(int stage, int tensor, int j) const {
        return base + (uint32_t)((stage * tensors + tensor) * NV + j) * step;
    }
    __device__ __forceinline__ void copy(int stage, int tensor, int j, const T* p) const {
        char* d = at(stage, tensor, j);
        if constexpr (kBytes == 16) {
            cp_async16(d, p);
        } else if constexpr (kBytes == 4) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem_u32(d)), "l"(p));
        } else {
            *reinterpret_cast<T*>(d) = *p;
        }
    }
    __device__ __forceinline__ void get(int stage, int tensor, int j, float (&f)[VEC]) const {
        unpack(*reinterpret_cast<const Vec<T, VEC>*>(at(stage, tensor, j)), f);
    }
};
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N)); }

// The newest `ahead` (0 .. 3) groups may still be in flight.
__device__ __forceinline__ void cp_async_wait_but(int ahead) {
    switch (ahead) {
        case 0: cp_async_wait<0>(); break;
        case 1: cp_async_wait<1>(); break;
        case 2: cp_async_wait<2>(); break;
        default: cp_async_wait<3>(); break;
    }
}

template <typename T, int VEC, int NV, int TPR, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 4 : 2)
    join_kernel(const hla2_block_args a, T* __restrict__ r_out, T* __restrict__ h_out, int stages) {
    extern __shared__ __align__(16) char ring_sm[];
    __shared__ float red[2][32][1];
    int turn = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr, mine = threadIdx.x / tpr;
    const int per = TPR ? kSmallThreads / (TPR ? TPR : 1) : 1;
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    const bool full = a.gate && a.gate_cols != 1;
    const T *pw = static_cast<const T*>(a.post_weight), *sc = static_cast<const T*>(a.scale),
            *nw = static_cast<const T*>(a.next_weight);
    const Ring<T, VEC, NV> ring(ring_sm, 1 + (a.y ? 1 : 0) + (full ? 1 : 0));
    const long long stride = (long long)gridDim.x * per;
    auto fetch = [&](long long row, int stage) {
        if (row < a.rows) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * tpr + t) * VEC;
                if (c < D) {
                    ring.copy(stage, 0, j, static_cast<const T*>(a.x) + row * a.x_stride + c);
                    if (a.y) ring.copy(stage, 1, j, static_cast<const T*>(a.y) + row * a.y_stride + c);
                    if (full) ring.copy(stage, 2, j, static_cast<const T*>(a.gate) + row * a.gate_stride + c);
                }
            }
        }
        cp_async_commit();
    };
    const long long row_first = (long long)blockIdx.x * per + mine;
    for (int i = 0; i + 1 < stages; ++i) fetch(row_first + i * stride, i);
    int stage = 0;
    // whole sub-warps: lanes of a row past the last take part in the shuffles
    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += stride) {
        const long long row = row0 + mine;
        const bool live = row < a.rows;
        const int next = stage == 0 ? stages - 1 : stage - 1;  // the slot of the row before
        fetch(row + (stages - 1) * stride, next);
        const float a_row = a.y && a.gate && !full && live
                                ? act_of(to_f32(static_cast<const T*>(a.gate)[row * a.gate_stride]), a.gate_act) : 1.f;
        cp_async_wait_but(stages - 1);
        float r[NV][VEC], sum[1] = {0.f};
        if (a.y) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (live && (j * tpr + t) * VEC < D) {
                    ring.get(stage, 1, j, r[j]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum[0] += r[j][i] * r[j][i];
                }
            row_sum<TPR, 1>(sum, red, turn);
            const float inv = rsqrtf(sum[0] * inv_d + a.eps);
            sum[0] = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * tpr + t) * VEC;
                if (live && c < D) {
                    float fx[VEC], fz[VEC], fw[VEC], fs[VEC];
                    ring.get(stage, 0, j, fx);
                    unpack(ldvec<T, VEC>(pw + c), fw);
                    if (full) ring.get(stage, 2, j, fz);
                    if (sc) unpack(ldvec<T, VEC>(sc + c), fs);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float u = r[j][i] * inv * fw[i], g = full ? act_of(fz[i], a.gate_act) : a_row;
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
                    ring.get(stage, 0, j, r[j]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum[0] += r[j][i] * r[j][i];
                }
        }
        if (h_out) {
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
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
}

struct JoinGrads {
    const void *dr, *dh;
    void *dx, *dy, *dgate;
    float* partial;  // [partials][3][D]: post_weight, scale, next_weight
    int partials;
};

template <typename T, int VEC, int NV, int TPR, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 2 : 1)
    join_backward_kernel(const hla2_block_args a, const JoinGrads g, int stages) {
    extern __shared__ __align__(16) char ring_sm[];  // the ring; at the end, in a sub-warp mapping, [3][D] sums
    __shared__ float red1[2][32][1], red2[2][32][2];
    int turn1 = 0, turn2 = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr, mine = threadIdx.x / tpr;
    const int per = TPR ? kSmallThreads / (TPR ? TPR : 1) : 1;
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    const T *pw = static_cast<const T*>(a.post_weight), *sc = static_cast<const T*>(a.scale),
            *nw = static_cast<const T*>(a.next_weight);
    const bool full = a.gate && a.gate_cols != 1;
    // ring slots of the tensors that are there
    int slots = 1;
    const int ky = a.y ? slots++ : 0, kz = full ? slots++ : 0, kr = g.dr ? slots++ : 0, kh = g.dh ? slots++ : 0;
    const Ring<T, VEC, NV> ring(ring_sm, slots);
    float gp[NV][VEC], gs[NV][VEC], gn[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) gp[j][i] = gs[j][i] = gn[j][i] = 0.f;

    const long long stride = (long long)gridDim.x * per;
    auto fetch = [&](long long row, int stage) {
        if (row < a.rows) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (j * tpr + t) * VEC;
                if (c < D) {
                    ring.copy(stage, 0, j, static_cast<const T*>(a.x) + row * a.x_stride + c);
                    if (a.y) ring.copy(stage, ky, j, static_cast<const T*>(a.y) + row * a.y_stride + c);
                    if (full) ring.copy(stage, kz, j, static_cast<const T*>(a.gate) + row * a.gate_stride + c);
                    if (g.dr) ring.copy(stage, kr, j, static_cast<const T*>(g.dr) + row * D + c);
                    if (g.dh) ring.copy(stage, kh, j, static_cast<const T*>(g.dh) + row * D + c);
                }
            }
        }
        cp_async_commit();
    };
    const long long row_first = (long long)blockIdx.x * per + mine;
    for (int i = 0; i + 1 < stages; ++i) fetch(row_first + i * stride, i);
    int stage = 0;
    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += stride) {
        const long long row = row0 + mine;
        const bool live = row < a.rows;
        fetch(row + (stages - 1) * stride, stage == 0 ? stages - 1 : stage - 1);
        const float z_row = a.gate && !full && live ? to_f32(static_cast<const T*>(a.gate)[row * a.gate_stride]) : 0.f;
        const float a_row = a.gate && !full ? act_of(z_row, a.gate_act) : 1.f;
        cp_async_wait_but(stages - 1);
        float inv_y = 0.f;
        if (a.y) {
            float s1[1] = {0.f};
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (live && (j * tpr + t) * VEC < D) {
                    float f[VEC];
                    ring.get(stage, ky, j, f);
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
                    ring.get(stage, 0, j, R[j]);
                    if (a.y) {
                        float fy[VEC], fz[VEC], fw[VEC], fs[VEC];
                        ring.get(stage, ky, j, fy);
                        unpack(ldvec<T, VEC>(pw + c), fw);
                        if (full) ring.get(stage, kz, j, fz);
                        if (sc) unpack(ldvec<T, VEC>(sc + c), fs);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float u = fy[i] * inv_y * fw[i], ga = full ? act_of(fz[i], a.gate_act) : a_row;
                            R[j][i] += sc ? fs[i] * ga * u : ga * u;
                        }
                    }
                    float fh[VEC], fn[VEC];
                    ring.get(stage, kh, j, fh);
                    unpack(ldvec<T, VEC>(nw + c), fn);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        s2[0] += R[j][i] * R[j][i];
                        s2[1] += fh[i] * fn[i] * R[j][i];
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
                float fr[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) fr[i] = 0.f;
                if (g.dr) ring.get(stage, kr, j, fr);
                if (g.dh) {
                    float f[VEC], fn[VEC];
                    ring.get(stage, kh, j, f);
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
                    ring.get(stage, ky, j, fy);
                    unpack(ldvec<T, VEC>(pw + c), fw);
                    if (full) ring.get(stage, kz, j, fz);
                    if (sc) unpack(ldvec<T, VEC>(sc + c), fs);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float ny = fy[i] * inv_y, u = ny * fw[i];
                        float ga = a_row, slope = 0.f;
                        if (full) {
                            const float sg = sigmoidf(fz[i]);
                            ga = a.gate_act == HLA2_GATE_SILU ? fz[i] * sg : sg;
                            slope = a.gate_act == HLA2_GATE_SILU ? sg * (1.f + fz[i] * (1.f - sg)) : sg * (1.f - sg);
                        }
                        const float Rs = sc ? fr[i] * fs[i] : fr[i];
                        gs[j][i] += fr[i] * ga * u;
                        const float du = Rs * ga;
                        gp[j][i] += du * ny;
                        if (full) dz[i] = Rs * u * slope;
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
                    ring.get(stage, ky, j, fy);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) o[i] = inv_y * (R[j][i] - fy[i] * inv_y * m);
                    stvec<T, VEC>(static_cast<T*>(g.dy) + row * D + c, o);
                }
            }
            if (a.gate && !full && live && t == 0)
                static_cast<T*>(g.dgate)[row] = from_f32<T>(s3[1] * act_slope(z_row, a.gate_act));
        }
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    cp_async_wait_all();
    // this CTA's partial sums: post_weight and scale with y, next_weight with dh
    float* dst = g.partial + (size_t)blockIdx.x * 3 * D;
    if (TPR) {  // the CTA's row groups one after another, so that the order is fixed
        float* acc = reinterpret_cast<float*>(ring_sm);
        for (int who = 0; who < per; ++who) {
            __syncthreads();
            if (mine == who) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int c = (j * tpr + t) * VEC + i;
                        if (c < D) {
                            acc[c] = (who ? acc[c] : 0.f) + gp[j][i];
                            acc[D + c] = (who ? acc[D + c] : 0.f) + gs[j][i];
                            acc[2 * D + c] = (who ? acc[2 * D + c] : 0.f) + gn[j][i];
                        }
                    }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 3 * D; c += kSmallThreads) dst[c] = acc[c];
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = (j * tpr + t) * VEC + i;
                if (c < D) {
                    if (a.y) dst[c] = gp[j][i];
                    if (sc) dst[D + c] = gs[j][i];
                    if (g.dh) dst[2 * D + c] = gn[j][i];
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
    if (c < D) {
        const float* src = partial + (size_t)which * D + c;
        int p = w;
        for (; p + 7 * 32 < partials; p += 8 * 32) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = src[(size_t)(p + 32 * i) * 3 * D];
            s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        for (; p < partials; p += 32) s += src[(size_t)p * 3 * D];
    }
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

// Persistent CTAs and their ring.  Stages: as many rows ahead as fit in the SM's shared memory beside
// the CTAs that the registers allow (512 threads of the backward, 1024 of the forward), at most
// four; one stage copies and waits.
struct Work {
    int ctas, stages;
    size_t smem;
};
Work work_of(const hla2_block_args* a, const Shape& s, int vec, int tensors, int threads_per_sm, size_t least) {
    const size_t slot = (size_t)vec * (a->dtype == HLA2_BF16 ? 2 : 4);
    const size_t stage = slot * s.threads * s.nv * tensors, room = 220 * 1024;
    int each = threads_per_sm / s.threads;
    if (each < 1) each = 1;
    if (each > 16) each = 16;
    Work w;
    w.stages = 4;
    while (w.stages > 1 && (w.stages * stage + 2048) * each > room && !(each == 1 && w.stages * stage <= room)) --w.stages;
    while (each > 1 && (w.stages * stage + 2048) * each > room) --each;
    w.smem = w.stages * stage > least ? w.stages * stage : least;
    const int per = s.tpr ? kSmallThreads / s.tpr : 1;
    const long long need = (a->rows + per - 1) / per, most = (long long)each * sms();
    w.ctas = (int)(need < most ? need : most);
    return w;
}
constexpr int kFwdThreadsPerSm = 1024, kBwdThreadsPerSm = 512;

Work backward_work(const hla2_block_args* a, const Shape& s, int vec, int tensors) {
    return work_of(a, s, vec, tensors, kBwdThreadsPerSm, s.tpr ? 3 * (size_t)a->D * sizeof(float) : 0);
}

template <class K>
bool set_smem(K kernel, size_t bytes) {
    return bytes <= 40 * 1024 ||  // 48 KB with the static part
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
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
    const int tensors = 1 + (a->y ? 1 : 0) + (a->y && a->gate && a->gate_cols != 1 ? 1 : 0);
    const Work w = work_of(a, s, vec, tensors, kFwdThreadsPerSm, 0);
    auto launch = [&](auto v, auto nv, auto tpr, auto maxt) {
        constexpr int VEC = decltype(v)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value,
                      MAXT = decltype(maxt)::value;
        auto go = [&](auto zero) {
            using T = decltype(zero);
            auto k = join_kernel<T, VEC, NV, TPR, MAXT>;
            if (!set_smem(k, w.smem)) return -1;
            k<<<w.ctas, s.threads, w.smem, st>>>(*a, static_cast<T*>(r), static_cast<T*>(h), w.stages);
            return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
        };
        if constexpr (VEC == 8 || VEC == 2) return go(bf16{});
        else if constexpr (VEC == 4) return go(float{});
        else return a->dtype == HLA2_BF16 ? go(bf16{}) : go(float{});
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
        for (int tensors = 2; tensors <= 5; ++tensors) {
            const size_t c = (size_t)backward_work(a, shape_of(a->D, vec), vec, tensors).ctas;
            if (c > most) most = c;
        }
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
        const int tensors = 1 + (a->y ? 1 : 0) + (a->y && a->gate && a->gate_cols != 1 ? 1 : 0) + (dr ? 1 : 0) + (dh ? 1 : 0);
        const Work w = backward_work(a, s, vec, tensors);
        g.partials = w.ctas;
        auto launch = [&](auto v, auto nv, auto tpr, auto maxt) {
            constexpr int VEC = decltype(v)::value, NV = decltype(nv)::value, TPR = decltype(tpr)::value,
                          MAXT = decltype(maxt)::value;
            auto go = [&](auto zero) {
                using T = decltype(zero);
                auto k = join_backward_kernel<T, VEC, NV, TPR, MAXT>;
                if (!set_smem(k, w.smem)) return -1;
                k<<<w.ctas, s.threads, w.smem, st>>>(*a, g, w.stages);
                return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
            };
            if constexpr (VEC == 8 || VEC == 2) return go(bf16{});
            else if constexpr (VEC == 4) return go(float{});
            else return a->dtype == HLA2_BF16 ? go(bf16{}) : go(float{});
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
