// Layer norm on rows of D values, forward and backward, and its C ABI (include/hla2.h, hla2_layer_norm*).  Per row
//   m = mean(x),  inv = 1 / sqrt(mean((x - m)^2) + eps),  nx = (x - m) inv,  y = nx w + bias
// and for the gradient g = dy w of nx
//   dx = inv (g - mean(g) - nx mean(g nx)),  dw += dy nx,  dbias += dy.
//
// The rows go through the ring and the launch shapes of the block norms (block_join.cuh): persistent CTAs, a thread with the
// same columns of every row, copied ahead.  The squares are summed about the mean, in a second sum over the row in registers:
// the difference of sums would lose the variance of rows far from zero.  The backward forms the statistics again; its two
// sums over rows stay in registers, and each CTA writes one partial row, which a second kernel sums in a fixed order.
#include "block_join.cuh"

namespace hla2 {
namespace {

struct NormGrads {
    const void* dout;
    void* dx;
    float* partial;  // [partials][2][D]: weight, bias
    int partials;
};

// a b, which the compiler may not put into a sum that follows
__device__ __forceinline__ float rounded_product(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ F2 rounded_product(F2 a, F2 b) { return a * b; }

template <typename T, int VEC, int NV, int TPR, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 4 : 2)
    layer_norm_kernel(const hla2_norm_args a, T* __restrict__ out, int stages) {
    using L = Lanes<VEC>;
    using P = typename L::P;
    constexpr int N = L::N;
    extern __shared__ __align__(16) char ring_sm[];
    __shared__ float red[2][16][1];
    int turn = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr, mine = threadIdx.x / tpr;
    constexpr int per = TPR ? kSmallThreads / (TPR ? TPR : 1) : 1;
    const float inv_d = 1.f / (float)a.D;
    const int d_left = a.D - t * VEC;
    const Ring<T, VEC, NV> ring(ring_sm, 1);
    const long long stride = (long long)gridDim.x * per, row_first = (long long)blockIdx.x * per + mine;
    const T* xf = static_cast<const T*>(a.x) + row_first * a.x_stride + t * VEC;
    long long left = row_first < a.rows ? (a.rows - 1 - row_first) / stride + 1 : 0;
    auto fetch = [&](int stage) {
        if (left > 0) {
            --left;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * tpr * VEC < d_left) ring.copy(stage, 0, j, xf + j * tpr * VEC);
            xf += stride * a.x_stride;
        }
        cp_async_commit();
    };
    pdl_wait();
    for (int i = 0; i + 1 < stages; ++i) fetch(i);
    const T *w = static_cast<const T*>(a.weight) + t * VEC, *bias = a.bias ? static_cast<const T*>(a.bias) + t * VEC : nullptr;
    int stage = 0;
    long long at = row_first * a.D + t * VEC;
    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += stride, at += stride * a.D) {
        const int cols = row0 + mine < a.rows ? d_left : 0;
        fetch(stage == 0 ? stages - 1 : stage - 1);
        cp_async_wait_but(stages - 1);
        P x[NV][N], acc = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * tpr * VEC < cols) {
                ring.get(stage, 0, j, x[j]);
#pragma unroll
                for (int i = 0; i < N; ++i) acc = fma_(x[j][i], L::all(1.f), acc);
            }
        float sum[1] = {sum_of(acc)};
        row_sum<TPR, 1>(sum, red, turn);
        const P mean = L::all(-sum[0] * inv_d);
        acc = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * tpr * VEC < cols) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    x[j][i] = fma_(x[j][i], L::all(1.f), mean);
                    acc = fma_(x[j][i], x[j][i], acc);
                }
            }
        sum[0] = sum_of(acc);
        row_sum<TPR, 1>(sum, red, turn);
        const P inv = L::all(rsqrtf(sum[0] * inv_d + a.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * tpr * VEC;
            if (c < cols) {
                P fw[N], fb[N], o[N];
                unpack(ldvec<T, VEC>(w + c), fw);
                if (bias) unpack(ldvec<T, VEC>(bias + c), fb);
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = fma_(x[j][i] * inv, fw[i], bias ? fb[i] : L::all(0.f));
                stvec<T, VEC>(out + at + c, o);
            }
        }
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    pdl_trigger();
}

template <typename T, int VEC, int NV, int TPR, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 256 ? 1 : 3)
    layer_norm_backward_kernel(const hla2_norm_args a, const NormGrads g, int stages) {
    using L = Lanes<VEC>;
    using P = typename L::P;
    constexpr int N = L::N;
    extern __shared__ __align__(16) char ring_sm[];  // the ring; at the end, in a sub-warp mapping, [2][D] sums
    __shared__ float red[2][16][2];
    int turn = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr, mine = threadIdx.x / tpr;
    constexpr int per = TPR ? kSmallThreads / (TPR ? TPR : 1) : 1;
    const int D = a.D, d_left = D - t * VEC;
    const float inv_d = 1.f / (float)D;
    const Ring<T, VEC, NV> ring(ring_sm, 2);
    P gw[NV][N], gb[NV][N], w[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) gw[j][i] = gb[j][i] = L::all(0.f);
    const long long stride = (long long)gridDim.x * per, row_first = (long long)blockIdx.x * per + mine;
    const T *xf = static_cast<const T*>(a.x) + row_first * a.x_stride + t * VEC, *df = static_cast<const T*>(g.dout) + row_first * D + t * VEC;
    long long left = row_first < a.rows ? (a.rows - 1 - row_first) / stride + 1 : 0;
    auto fetch = [&](int stage) {
        if (left > 0) {
            --left;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * tpr * VEC;
                if (c < d_left) ring.copy(stage, 0, j, xf + c), ring.copy(stage, 1, j, df + c);
            }
            xf += stride * a.x_stride, df += stride * D;
        }
        cp_async_commit();
    };
    pdl_wait();
    for (int i = 0; i + 1 < stages; ++i) fetch(i);
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (j * tpr * VEC < d_left) unpack(ldvec<T, VEC>(static_cast<const T*>(a.weight) + (j * tpr + t) * VEC), w[j]);
    int stage = 0;
    long long at = row_first * D + t * VEC;
    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += stride, at += stride * D) {
        const int cols = row0 + mine < a.rows ? d_left : 0;
        fetch(stage == 0 ? stages - 1 : stage - 1);
        cp_async_wait_but(stages - 1);
        // sums of x and of g
        P x[NV][N], d[NV][N], sx = L::all(0.f), sg = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * tpr * VEC < cols) {
                ring.get(stage, 0, j, x[j]);
                ring.get(stage, 1, j, d[j]);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    sx = fma_(x[j][i], L::all(1.f), sx);
                    sg = fma_(d[j][i], w[j][i], sg);
                }
            }
        float s[2] = {sum_of(sx), sum_of(sg)};
        row_sum<TPR, 2>(s, red, turn);
        const P mean = L::all(-s[0] * inv_d);
        const float mean_g = s[1] * inv_d;
        // sums of the squares about the mean, and of g times them
        P xx = L::all(0.f), gx = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * tpr * VEC < cols) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    x[j][i] = fma_(x[j][i], L::all(1.f), mean);
                    xx = fma_(x[j][i], x[j][i], xx);
                    gx = fma_(d[j][i] * w[j][i], x[j][i], gx);
                }
            }
        s[0] = sum_of(xx), s[1] = sum_of(gx);
        row_sum<TPR, 2>(s, red, turn);
        const float inv = rsqrtf(s[0] * inv_d + a.eps);
        const P dot = L::all(-s[1] * inv * inv_d), minus = L::all(-mean_g), pinv = L::all(inv);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * tpr * VEC;
            if (c < cols) {
                P o[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const P nx = x[j][i] * pinv;
                    gw[j][i] = fma_(d[j][i], nx, gw[j][i]);
                    gb[j][i] = fma_(d[j][i], L::all(1.f), gb[j][i]);
                    // the mean is taken off a rounded g, as it has been summed, and before the factor inv: in rows of one value that
                    // is large and the difference nothing
                    o[i] = pinv * fma_(nx, dot, fma_(rounded_product(d[j][i], w[j][i]), L::all(1.f), minus));
                }
                stvec<T, VEC>(static_cast<T*>(g.dx) + at + c, o);
            }
        }
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    cp_async_wait_all();
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
    if (TPR && TPR <= 32) {  // the CTA's row groups one after another, so that the order is fixed
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
                            acc[c] = (who ? acc[c] : 0.f) + at_of(gw[j], i);
                            acc[D + c] = (who ? acc[D + c] : 0.f) + at_of(gb[j], i);
                        }
                    }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * D; c += kSmallThreads) dst[c] = acc[c];
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = (j * tpr + t) * VEC + i;
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

// The arguments as the block norms' launch choice has them: one row tensor, the weight, and what else has columns
hla2_block_args as_block(const hla2_norm_args* a) {
    hla2_block_args b{};
    b.dtype = a->dtype, b.rows = a->rows, b.D = a->D, b.eps = a->eps;
    b.x = a->x, b.x_stride = a->x_stride, b.next_weight = a->weight;
    return b;
}

int check_norm(const char* fn, const hla2_norm_args* a) {
    if (!a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: args must not be NULL", fn);
    if (!a->weight) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: weight must not be NULL", fn);
    const hla2_block_args b = as_block(a);
    if (int rc = check_join(fn, &b)) return rc;
    if (!al(a->bias, a->dtype == HLA2_BF16 ? 2 : 4))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    return HLA2_OK;
}

Work norm_backward_work(const hla2_block_args* b, const Shape& s, int vec, int sms) {
    return work_of(b, s, vec, 2, kNormBwdThreadsPerSm, s.tpr && s.tpr <= 32 ? 2 * (size_t)b->D * sizeof(float) : 0, sms);
}

// f(VEC, NV, TPR, MAXT, zero of the type) as integral constants
template <class F>
int dispatch_norm(const hla2_block_args* b, int vec, const Shape& s, F&& f) {
    return with_vec(b->D, vec, s, [&](auto v, auto nv, auto tpr, auto maxt) {
        constexpr int VEC = decltype(v)::value;
        if constexpr (VEC == 8 || VEC == 2) return f(v, nv, tpr, maxt, bf16{});
        else if constexpr (VEC == 4) return f(v, nv, tpr, maxt, 0.f);
        else return b->dtype == HLA2_BF16 ? f(v, nv, tpr, maxt, bf16{}) : f(v, nv, tpr, maxt, 0.f);
    });
}

}  // namespace
}  // namespace hla2

using namespace hla2;

extern "C" {

int hla2_layer_norm(const hla2_norm_args* a, void* out, hla2_stream_t stream) {
    static const char* const fn = "hla2_layer_norm";
    if (int rc = check_norm(fn, a)) return rc;
    if (a->rows == 0) return join_ok();
    const hla2_block_args b = as_block(a);
    const size_t es = a->dtype == HLA2_BF16 ? 2 : 4;
    if (!out || !al(out, es)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out must be an aligned address", fn);
    const RowsOf o{out, a->D, a->D};
    if (spoils(&b, o, nullptr, 0) || meet(rows_extent(&b, o), extent_of(a->bias, a->D * es)))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out overlaps an input other than in its place", fn);
    const void* more[2] = {out, a->bias};
    const int vec = vec_of(&b, more, 2);
    const Shape s = shape_of(a->D, vec);
    const Work w = work_of(&b, s, vec, 1, kFwdThreadsPerSm, 0, sm_count());
    auto launch = [&](auto v, auto nv, auto tpr, auto maxt, auto zero) {
        using T = decltype(zero);
        auto k = layer_norm_kernel<T, decltype(v)::value, decltype(nv)::value, decltype(tpr)::value, decltype(maxt)::value>;
        if (!set_smem(k, w.smem)) return -1;
        return launch_pdl(k, dim3(w.ctas), dim3(s.threads), w.smem, reinterpret_cast<cudaStream_t>(stream), *a, static_cast<T*>(out),
                          w.stages) == cudaSuccess ? 0 : -1;
    };
    if (dispatch_norm(&b, vec, s, launch))
        return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return join_ok();
}

size_t hla2_layer_norm_backward_workspace_bytes(const hla2_norm_args* a) {
    if (check_norm("hla2_layer_norm_backward_workspace_bytes", a) != HLA2_OK) return (size_t)-1;
    join_ok();
    const hla2_block_args b = as_block(a);
    size_t most = 0;
    for (int vec : {1, 2, a->dtype == HLA2_BF16 ? 8 : 4}) {  // whichever the addresses allow
        const size_t c = (size_t)norm_backward_work(&b, shape_of(a->D, vec), vec, sm_count()).ctas;
        if (c > most) most = c;
    }
    return most * 2 * (size_t)a->D * sizeof(float);
}

int hla2_layer_norm_backward(const hla2_norm_args* a, const void* dout, void* dx, float* dweight, float* dbias,
                             void* workspace, size_t workspace_bytes, hla2_stream_t stream) {
    static const char* const fn = "hla2_layer_norm_backward";
    if (int rc = check_norm(fn, a)) return rc;
    const hla2_block_args b = as_block(a);
    const size_t es = a->dtype == HLA2_BF16 ? 2 : 4, vb = (size_t)a->D * sizeof(float);
    if (!dweight || !al(dweight, 4) || !al(dbias, 4))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dweight is needed, and each sum aligned to its type", fn);
    const Extent sums[2] = {extent_of(dweight, vb), extent_of(dbias, vb)};
    bool bad = meet(sums[0], sums[1]);
    for (const Extent& e : sums) bad |= meet(e, extent_of(a->weight, a->D * es)) || meet(e, extent_of(a->bias, a->D * es));
    if (a->rows > 0) {
        if (!dout || !dx || !al(dout, es) || !al(dx, es))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dout and dx must be aligned addresses", fn);
        const RowsOf o{dx, a->D, a->D}, more[1] = {{dout, a->D, a->D}};
        bad |= spoils(&b, o, more, 1) || meet(rows_extent(&b, o), extent_of(a->bias, a->D * es));
        for (const RowsOf& t : {RowsOf{a->x, a->x_stride, a->D}, more[0], o})
            for (const Extent& e : sums) bad |= meet(e, rows_extent(&b, t));
    }
    if (bad) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient overlaps another tensor other than in its place", fn);
    const size_t need = hla2_layer_norm_backward_workspace_bytes(a);
    if (need > 0 && (!workspace || workspace_bytes < need || !al(workspace, 16)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    NormGrads g{dout, dx, static_cast<float*>(workspace), 0};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a->rows > 0) {
        const void* more[2] = {dout, dx};
        const int vec = vec_of(&b, more, 2);
        const Shape s = shape_of(a->D, vec);
        const Work w = norm_backward_work(&b, s, vec, sm_count());
        g.partials = w.ctas;
        auto launch = [&](auto v, auto nv, auto tpr, auto maxt, auto zero) {
            using T = decltype(zero);
            auto k = layer_norm_backward_kernel<T, decltype(v)::value, decltype(nv)::value, decltype(tpr)::value, decltype(maxt)::value>;
            if (!set_smem(k, w.smem)) return -1;
            return launch_pdl(k, dim3(w.ctas), dim3(s.threads), w.smem, st, *a, g, w.stages) == cudaSuccess ? 0 : -1;
        };
        if (dispatch_norm(&b, vec, s, launch))
            return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    }
    if (launch_pdl(norm_sums_kernel, dim3((2 * a->D + 31) / 32), dim3(1024), 0, st, g.partial, g.partials, 2 * a->D, a->D, dweight,
                   dbias) != cudaSuccess)
        return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return join_ok();
}

}  // extern "C"
