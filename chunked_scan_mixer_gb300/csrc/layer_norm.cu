// Layer norm on rows of D values, forward and backward, and its C ABI (include/hla2.h, hla2_layer_norm*).  Per row
//   m = mean(x),  inv = 1 / sqrt(mean((x - m)^2) + eps),  nx = (x - m) inv,  y = nx w + bias
// and for the gradient g = dy w of nx
//   dx = inv (g - mean(g) - nx mean(g nx)),  dw += dy nx,  dbias += dy.
//
// Bytes bound it: two tensors forward, three backward, whose statistics are formed again.  A row has RW warps, few of them,
// so that the two sums over it (the squares are summed about the mean: the difference of plain sums would lose the variance of
// rows far from zero) cost little beside up to 64 values a lane; with one warp they need no barrier.  The next row's values
// are on their way in registers while a row is worked on.  The backward's two sums over rows stay in registers; each
// CTA writes one partial row, which a second kernel sums in a fixed order.
#include <type_traits>

#include "packed.cuh"
#include "rows.h"

namespace hla2 {
namespace {

constexpr int kMaxNormD = 8192;

struct NormGrads {
    const void* dout;
    void* dx;
    float* partial;  // [CTAs][2][D]: weight, bias
};

// a b, which the compiler may not put into a sum that follows
__device__ __forceinline__ float rounded_product(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ F2 rounded_product(F2 a, F2 b) { return a * b; }

// Rows of RW warps, as many of them to a CTA as make four warps
template <int RW>
struct NormShape {
    static constexpr int rows = RW < 4 ? 4 / RW : 1, threads = 32 * RW * rows;
};

// Sums of K values over a row's warps; `red` alternates between two halves, so that one barrier a call is enough
template <int RW, int K>
__device__ __forceinline__ void norm_sum(float (&v)[K], float (*red)[NormShape<RW>::rows][RW][2], int& turn) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (RW > 1) {
        const int warp = threadIdx.x >> 5, w = warp % RW, row = warp / RW;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) red[turn][row][w][k] = v[k];
        if constexpr (NormShape<RW>::rows == 1) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(row + 1), "n"(32 * RW) : "memory");
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = red[turn][row][0][k];
#pragma unroll
            for (int i = 1; i < RW; ++i) v[k] += red[turn][row][i][k];
        }
        turn ^= 1;
    }
}

// A lane's columns of a row: vectors t, t + 32 RW, ... of VEC values, NV of them
template <typename T, int VEC, int NV, int RW>
struct NormRow {
    Vec<T, VEC> v[NV];
    static __device__ __forceinline__ int column(int j) { return ((int)(threadIdx.x % (32 * RW)) + j * 32 * RW) * VEC; }
    __device__ __forceinline__ void load(const T* p, int D) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j] = Vec<T, VEC>{};
            if (column(j) < D) v[j] = ldvec<T, VEC>(p + column(j));
        }
    }
};

// A lane's columns of the weight or the bias, which are the same in all its rows: held in registers where eight are enough, read
// again with every row elsewhere.  (5000 float32 rows of 999 with gradients: 26.5 us without, 22.8 so; 16384 bf16 rows of 2047:
// 123 and 105.)
template <typename T, int VEC, int NV, int RW>
struct NormParam {
    static constexpr bool kept = NV * (VEC * sizeof(T) < 4 ? 4 : VEC * sizeof(T)) <= 32;
    const T* p;
    NormRow<T, VEC, kept ? NV : 1, RW> v;
    __device__ __forceinline__ NormParam(const T* from, int D) : p(from) {
        if (kept && p) v.load(p, D);
    }
    template <typename P, int N>
    __device__ __forceinline__ void get(int j, P (&f)[N]) const {
        if constexpr (kept) unpack(v.v[j], f);
        else unpack(ldvec<T, VEC>(p + NormRow<T, VEC, NV, RW>::column(j)), f);
    }
};

template <typename T, int VEC, int NV, int RW>
__global__ void __launch_bounds__(NormShape<RW>::threads) layer_norm_kernel(const hla2_norm_args a, T* __restrict__ out) {
    using L = Lanes<VEC>;
    using P = typename L::P;
    using Row = NormRow<T, VEC, NV, RW>;
    constexpr int N = L::N, rows = NormShape<RW>::rows;
    __shared__ float red[2][rows][RW][2];
    int turn = 0;
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    const T* x = static_cast<const T*>(a.x);
    const long long stride = (long long)gridDim.x * rows;
    long long r = (long long)blockIdx.x * rows + threadIdx.x / (32 * RW);
    pdl_wait();
    using Param = NormParam<T, VEC, NV, RW>;
    const Param w(static_cast<const T*>(a.weight), D), bias(static_cast<const T*>(a.bias), D);
    Row next;
    if (r < a.rows) next.load(x + r * a.x_stride, D);
    for (; r < a.rows; r += stride) {  // a row's warps stay together
        P f[NV][N], acc = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            unpack(next.v[j], f[j]);
#pragma unroll
            for (int i = 0; i < N; ++i) acc = fma_(f[j][i], L::all(1.f), acc);
        }
        if (r + stride < a.rows) next.load(x + (r + stride) * a.x_stride, D);
        float s[1] = {sum_of(acc)};
        norm_sum<RW, 1>(s, red, turn);
        const P mean = L::all(-s[0] * inv_d);
        acc = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (Row::column(j) < D) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    f[j][i] = fma_(f[j][i], L::all(1.f), mean);
                    acc = fma_(f[j][i], f[j][i], acc);
                }
            }
        s[0] = sum_of(acc);
        norm_sum<RW, 1>(s, red, turn);
        const P inv = L::all(rsqrtf(s[0] * inv_d + a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (Row::column(j) < D) {
                P fw[N], fb[N], o[N];
                w.get(j, fw);
                if (bias.p) bias.get(j, fb);
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = fma_(f[j][i] * inv, fw[i], bias.p ? fb[i] : L::all(0.f));
                stvec<T, VEC>(out + r * D + Row::column(j), o);
            }
    }
    pdl_trigger();
}

// Two vectors of eight a lane are held to 128 registers, 16 warps an SM: 16384 x 4096 113 -> 91 us (with 64 bytes of spills), 16384 x 2560
// 101 -> 72, 32768 x 2048 95 -> 89, 200000 x 512 127 -> 115; rows that do not fill the GPU lose by it, 1000 x 4096 21 -> 25.  Shapes
// without the bound: four float32 vectors of four take 158 to 174 registers, four bf16 vectors of eight 218, all others at most 128.
template <typename T, int VEC, int NV, int RW>
__global__ void __launch_bounds__(NormShape<RW>::threads, VEC == 8 && NV == 2 ? 512 / NormShape<RW>::threads : 1)
    layer_norm_backward_kernel(const hla2_norm_args a, const NormGrads g) {
    using L = Lanes<VEC>;
    using P = typename L::P;
    using Row = NormRow<T, VEC, NV, RW>;
    constexpr int N = L::N, rows = NormShape<RW>::rows;
    __shared__ float red[2][rows][RW][2];
    extern __shared__ float sums[];  // [2][D], where a CTA has several rows
    int turn = 0;
    const int D = a.D, mine = threadIdx.x / (32 * RW);
    const float inv_d = 1.f / (float)D;
    const T *x = static_cast<const T*>(a.x), *dout = static_cast<const T*>(g.dout);
    T* dx = static_cast<T*>(g.dx);
    const long long stride = (long long)gridDim.x * rows;
    long long r = (long long)blockIdx.x * rows + mine;
    P gw[NV][N], gb[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) gw[j][i] = gb[j][i] = L::all(0.f);
    pdl_wait();
    const NormParam<T, VEC, NV, RW> w(static_cast<const T*>(a.weight), D);
    Row nx_, nd;
    if (r < a.rows) nx_.load(x + r * a.x_stride, D), nd.load(dout + r * D, D);
    for (; r < a.rows; r += stride) {
        P f[NV][N], d[NV][N], sx = L::all(0.f), sg = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            unpack(nx_.v[j], f[j]);
            unpack(nd.v[j], d[j]);
            if (Row::column(j) < D) {
                P fw[N];
                w.get(j, fw);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    sx = fma_(f[j][i], L::all(1.f), sx);
                    sg = fma_(d[j][i], fw[i], sg);
                }
            }
        }
        if (r + stride < a.rows) nx_.load(x + (r + stride) * a.x_stride, D), nd.load(dout + (r + stride) * D, D);
        float s[2] = {sum_of(sx), sum_of(sg)};
        norm_sum<RW, 2>(s, red, turn);
        const P mean = L::all(-s[0] * inv_d), minus = L::all(-s[1] * inv_d);
        P xx = L::all(0.f), gx = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (Row::column(j) < D) {
                P fw[N];
                w.get(j, fw);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    f[j][i] = fma_(f[j][i], L::all(1.f), mean);
                    xx = fma_(f[j][i], f[j][i], xx);
                    gx = fma_(d[j][i] * fw[i], f[j][i], gx);
                }
            }
        s[0] = sum_of(xx), s[1] = sum_of(gx);
        norm_sum<RW, 2>(s, red, turn);
        const float inv = rsqrtf(s[0] * inv_d + a.eps);
        const P dot = L::all(-s[1] * inv * inv_d), pinv = L::all(inv);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (Row::column(j) < D) {
                P o[N], fw[N];
                w.get(j, fw);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const P nx = f[j][i] * pinv;
                    gw[j][i] = fma_(d[j][i], nx, gw[j][i]);
                    gb[j][i] = fma_(d[j][i], L::all(1.f), gb[j][i]);
                    // the mean is taken off a rounded g, as it has been summed, and before the factor inv: in rows of one value that
                    // is large and the difference nothing
                    o[i] = pinv * fma_(nx, dot, fma_(rounded_product(d[j][i], fw[i]), L::all(1.f), minus));
                }
                stvec<T, VEC>(dx + r * D + Row::column(j), o);
            }
    }
    pdl_trigger();
    auto at_of = [](const P (&v)[N], int i) {
        if constexpr (VEC == 1) {
            return v[0];
        } else {
            float lo, hi;
            split(v[i / 2], lo, hi);
            return i % 2 ? hi : lo;
        }
    };
    float* dst = g.partial + (size_t)blockIdx.x * 2 * D;
    if constexpr (rows > 1) {  // the CTA's rows one after another, so that the order is fixed
        for (int who = 0; who < rows; ++who) {
            if (mine == who) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int c = Row::column(j) + i;
                        if (c < D) {
                            sums[c] = (who ? sums[c] : 0.f) + at_of(gw[j], i);
                            sums[D + c] = (who ? sums[D + c] : 0.f) + at_of(gb[j], i);
                        }
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * D; c += NormShape<RW>::threads) dst[c] = sums[c];
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = Row::column(j) + i;
                if (c < D) dst[c] = at_of(gw[j], i), dst[D + c] = at_of(gb[j], i);
            }
    }
}

// Sums the partial rows: 32 columns a CTA, 32 row lanes, then a tree over them in a fixed order.
__global__ void __launch_bounds__(1024)
    norm_sums_kernel(const float* __restrict__ partial, int partials, int cols, int D, float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    pdl_wait();
    float s = 0.f;
    if (c < cols) {
        const float* src = partial + c;
#pragma unroll 8
        for (int p = w; p < partials; p += 32) s += src[(size_t)p * cols];
    }
    sm[w][lane] = s;
    __syncthreads();
    for (int o = 16; o; o >>= 1) {
        if (w < o) sm[w][lane] += sm[w + o][lane];
        __syncthreads();
    }
    if (w == 0 && c < cols) {
        if (c < D) dweight[c] = sm[0][lane];
        else if (dbias) dbias[c - D] = sm[0][lane];
    }
}

// ---- launch ----------------------------------------------------------------------------------

int check_norm(const char* fn, const hla2_norm_args* a) {
    if (!a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: args must not be NULL", fn);
    if (a->dtype != HLA2_F32 && a->dtype != HLA2_BF16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dtype must be HLA2_F32 or HLA2_BF16", fn);
    if (a->D < 1 || a->D > kMaxNormD)
        return set_last_error(a->D < 1 ? HLA2_ERR_INVALID_ARG : HLA2_ERR_UNSUPPORTED, "%s: D must be 1 .. %d (got %d)", fn,
                              kMaxNormD, a->D);
    if (a->rows < 0 || a->rows > 0x7fffffffLL)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: rows must be 0 .. 2^31 - 1", fn);
    if (!a->weight) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: weight must not be NULL", fn);
    const int es = elem_size(a->dtype);
    if (!al(a->x, es) || !al(a->weight, es) || !al(a->bias, es))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    if (a->rows > 0 && !a->x) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: x must not be NULL", fn);
    if (a->rows > 1 && a->x_stride < 0) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
    return HLA2_OK;
}
Extent norm_rows(const hla2_norm_args* a, const void* p, long long stride) {
    return extent_of(p, (size_t)((a->rows - 1) * stride + a->D) * elem_size(a->dtype));
}
// Whether contiguous rows that are written overlap other rows in another way than as exactly the same ones: a row is read whole
// before it is written, but its neighbours may be read earlier or later.
bool norm_spoils(const hla2_norm_args* a, const void* out, const void* in, long long stride) {
    return meet(norm_rows(a, out, a->D), norm_rows(a, in, stride)) && !(out == in && (stride == a->D || a->rows == 1));
}
// Elements a vector: 16 bytes where every row allows it, else one
int norm_vec(const hla2_norm_args* a, const void* const* more, int count) {
    const int v = 16 / elem_size(a->dtype);
    bool fits = a->D % v == 0 && al(a->x, 16) && (a->rows <= 1 || a->x_stride % v == 0) && al(a->weight, 16);
    for (int i = 0; i < count; ++i) fits = fits && al(more[i], 16);
    return fits ? v : 1;
}

template <int V> using Int = std::integral_constant<int, V>;
// f(VEC, NV, RW, zero of the type) for the first shape that holds a row: one warp with 1, 2, .. MOST vectors a lane, then 2, 4, ..
// CAP warps, then more vectors
template <int VEC, int MOST, int CAP, int NV = 1, int RW = 1, class T, class F>
int norm_shape(int D, T zero, F&& f) {
    if constexpr (32 * NV * RW * VEC >= kMaxNormD) {
        return f(Int<VEC>{}, Int<NV>{}, Int<RW>{}, zero);
    } else {
        if (D <= 32 * NV * RW * VEC) return f(Int<VEC>{}, Int<NV>{}, Int<RW>{}, zero);
        if constexpr (NV < MOST) return norm_shape<VEC, MOST, CAP, 2 * NV, RW>(D, zero, f);
        else if constexpr (RW < CAP) return norm_shape<VEC, MOST, CAP, NV, 2 * RW>(D, zero, f);
        else return norm_shape<VEC, MOST, CAP, 2 * NV, RW>(D, zero, f);
    }
}
// Forward: up to 64 bf16 or 32 float32 values a lane (32768 bf16 rows of 2048: 45 us, 64 with a CTA of one vector a lane).  Rows
// that do not give every SM two of them are latency: one vector a lane, up to eight warps (4 x 2048: 3.7 -> 2.2 us).
// Backward, whose sums are held too: 16 values (32768 x 2048: 81 us, 93 with 32, and 4 CTAs an SM instead of 2).
// Single elements: 8 (5000 float32 rows of 999: 7.3 us, 10.5 with 16; backward 15.3 and 17.2, before the weight was held).
template <bool BACK, class F>
int with_norm(const hla2_norm_args* a, int vec, F&& f) {
    const bool bf = a->dtype == HLA2_BF16;
    if (vec == 1) return bf ? norm_shape<1, 8, 16>(a->D, bf16{}, f) : norm_shape<1, 8, 16>(a->D, 0.f, f);
    if constexpr (BACK) {
        return bf ? norm_shape<8, 2, 8>(a->D, bf16{}, f) : norm_shape<4, 4, 16>(a->D, 0.f, f);
    } else {
        if (a->rows <= 2 * sm_count()) return bf ? norm_shape<8, 1, 8>(a->D, bf16{}, f) : norm_shape<4, 1, 8>(a->D, 0.f, f);
        return bf ? norm_shape<8, 8, 8>(a->D, bf16{}, f) : norm_shape<4, 8, 8>(a->D, 0.f, f);
    }
}

// CTAs of a call: what the GPU holds at once
template <class K>
int norm_ctas(K kernel, int threads, size_t smem, long long rows, int rows_each) {
    const long long need = (rows + rows_each - 1) / rows_each;
    if (need <= sm_count()) return (int)need;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess || per_sm < 1) {
        cudaGetLastError();
        per_sm = 1;
    }
    const long long most = (long long)per_sm * sm_count();
    return (int)(need < most ? need : most);
}
// that a backward has at most, whatever its shape
constexpr int kMostCtasPerSm = 8;

}  // namespace
}  // namespace hla2

using namespace hla2;

extern "C" {

int hla2_layer_norm(const hla2_norm_args* a, void* out, hla2_stream_t stream) {
    static const char* const fn = "hla2_layer_norm";
    Range range(fn);
    if (int rc = check_norm(fn, a)) return rc;
    if (a->rows == 0) return ok();
    const size_t es = elem_size(a->dtype);
    if (!out || !al(out, es)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out must be an aligned address", fn);
    const Extent eo = norm_rows(a, out, a->D);
    if (norm_spoils(a, out, a->x, a->x_stride) || meet(eo, extent_of(a->weight, a->D * es)) || meet(eo, extent_of(a->bias, a->D * es)))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out overlaps an input other than in its place", fn);
    const void* more[2] = {out, a->bias};
    const int rc = with_norm<false>(a, norm_vec(a, more, 2), [&](auto v, auto nv, auto rw, auto zero) {
        using T = decltype(zero);
        constexpr int RW = decltype(rw)::value;
        auto k = layer_norm_kernel<T, decltype(v)::value, decltype(nv)::value, RW>;
        const int ctas = norm_ctas(k, NormShape<RW>::threads, 0, a->rows, NormShape<RW>::rows);
        return launch_pdl(k, dim3(ctas), dim3(NormShape<RW>::threads), 0, reinterpret_cast<cudaStream_t>(stream), *a,
                          static_cast<T*>(out)) == cudaSuccess ? 0 : -1;
    });
    return rc ? launch_failed("layer norm") : ok();
}

size_t hla2_layer_norm_backward_workspace_bytes(const hla2_norm_args* a) {
    if (check_norm("hla2_layer_norm_backward_workspace_bytes", a) != HLA2_OK) return (size_t)-1;
    ok();
    const long long most = (long long)kMostCtasPerSm * sm_count();
    return (size_t)(a->rows < most ? a->rows : most) * 2 * (size_t)a->D * sizeof(float);
}

int hla2_layer_norm_backward(const hla2_norm_args* a, const void* dout, void* dx, float* dweight, float* dbias,
                             void* workspace, size_t workspace_bytes, hla2_stream_t stream) {
    static const char* const fn = "hla2_layer_norm_backward";
    Range range(fn);
    if (int rc = check_norm(fn, a)) return rc;
    const size_t es = elem_size(a->dtype), vb = (size_t)a->D * sizeof(float);
    if (!dweight || !al(dweight, 4) || !al(dbias, 4))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dweight is needed, and each sum aligned to its type", fn);
    const Extent sums[2] = {extent_of(dweight, vb), extent_of(dbias, vb)};
    bool bad = meet(sums[0], sums[1]);
    for (const Extent& e : sums) bad |= meet(e, extent_of(a->weight, a->D * es)) || meet(e, extent_of(a->bias, a->D * es));
    if (a->rows > 0) {
        if (!dout || !dx || !al(dout, es) || !al(dx, es))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dout and dx must be aligned addresses", fn);
        const Extent eo = norm_rows(a, dx, a->D);
        bad |= norm_spoils(a, dx, a->x, a->x_stride) || norm_spoils(a, dx, dout, a->D);
        bad |= meet(eo, extent_of(a->weight, a->D * es)) || meet(eo, extent_of(a->bias, a->D * es));
        for (const Extent& e : sums)
            bad |= meet(e, eo) || meet(e, norm_rows(a, a->x, a->x_stride)) || meet(e, norm_rows(a, dout, a->D));
    }
    if (bad) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient overlaps another tensor other than in its place", fn);
    const size_t need = hla2_layer_norm_backward_workspace_bytes(a);
    if (need > 0 && (!workspace || workspace_bytes < need || !al(workspace, 16)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    NormGrads g{dout, dx, static_cast<float*>(workspace)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int partials = 0;
    if (a->rows > 0) {
        const void* more[2] = {dout, dx};
        const int rc = with_norm<true>(a, norm_vec(a, more, 2), [&](auto v, auto nv, auto rw, auto zero) {
            using T = decltype(zero);
            constexpr int RW = decltype(rw)::value;
            auto k = layer_norm_backward_kernel<T, decltype(v)::value, decltype(nv)::value, RW>;
            const size_t smem = NormShape<RW>::rows > 1 ? 2 * vb : 0;  // such rows have 1024 values at most
            partials = norm_ctas(k, NormShape<RW>::threads, smem, a->rows, NormShape<RW>::rows);
            if (partials > kMostCtasPerSm * sm_count()) partials = kMostCtasPerSm * sm_count();
            return launch_pdl(k, dim3(partials), dim3(NormShape<RW>::threads), smem, st, *a, g) == cudaSuccess ? 0 : -1;
        });
        if (rc) return launch_failed("layer norm gradients");
    }
    if (launch_pdl(norm_sums_kernel, dim3((2 * a->D + 31) / 32), dim3(1024), 0, st, g.partial, partials, 2 * a->D, a->D, dweight,
                   dbias) != cudaSuccess)
        return launch_failed("layer norm gradients");
    return ok();
}

}  // extern "C"
