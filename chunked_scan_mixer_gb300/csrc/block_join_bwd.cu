// The backward of the block norms; the mathematics is in block_join.cu.  The gradients of post_weight
// and scale are one sum over the rows, V = sum R a ny, times the other of the two: a thread keeps V and
// dw_next of its columns.
#include "block_join.cuh"

namespace hla2 {
namespace {

struct JoinGrads {
    const void *dr, *dh;
    void *dx, *dy, *dgate;
    float* partial;  // [partials][2][D]: V, next_weight
    int partials;
};

template <typename T, int VEC, int NV, int TPR, int MAXT, int MODE>
__global__ void __launch_bounds__(MAXT, MAXT > 256 ? 1 : MODE == kNormOnly ? 3 : 2)
    join_backward_kernel(const hla2_block_args a, const JoinGrads g, int stages) {
    using L = Lanes<VEC>;
    using P = typename L::P;
    constexpr int N = L::N;
    extern __shared__ __align__(16) char ring_sm[];  // the ring; at the end, in a sub-warp mapping, [2][D] sums
    __shared__ float red1[2][16][1], red2[2][16][2];
    int turn1 = 0, turn2 = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr, mine = threadIdx.x / tpr;
    constexpr int per = TPR ? kSmallThreads / (TPR ? TPR : 1) : 1;
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    constexpr bool has_y = MODE != kNormOnly;
    const bool full = MODE == kAll || (MODE == kAny && a.gate && a.gate_cols != 1);
    const bool scaled = MODE == kAll || (MODE == kAny && a.scale);
    const bool has_dr = MODE == kAll || g.dr, has_dh = MODE != kAny || g.dh;
    const bool silu = a.gate_act == HLA2_GATE_SILU;
    const T *pw = static_cast<const T*>(a.post_weight) + t * VEC, *sc = static_cast<const T*>(a.scale) + t * VEC,
            *nw = static_cast<const T*>(a.next_weight) + t * VEC;
    // ring slots of the tensors that are there
    int slots = 1;
    const int ky = has_y ? slots++ : 0, kz = full ? slots++ : 0, kr = has_dr ? slots++ : 0, kh = has_dh ? slots++ : 0;
    const Ring<T, VEC, NV> ring(ring_sm, slots);
    P gv[NV][N], gn[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) gv[j][i] = gn[j][i] = L::all(0.f);

    const long long stride = (long long)gridDim.x * per, row_first = (long long)blockIdx.x * per + mine;
    const T *xf = static_cast<const T*>(a.x) + row_first * a.x_stride + t * VEC,
            *yf = static_cast<const T*>(a.y) + row_first * a.y_stride + t * VEC,
            *zf = static_cast<const T*>(a.gate) + row_first * a.gate_stride + t * VEC;
    const long long xs = stride * a.x_stride, ys = stride * a.y_stride, zs = stride * a.gate_stride;
    long long left = row_first < a.rows ? (a.rows - 1 - row_first) / stride + 1 : 0;  // rows still to copy
    long long af = row_first * D + t * VEC;
    const int d_left = D - t * VEC;
    constexpr bool holds = kHolds<T, VEC, NV>;
    T held_in[5][holds ? NV : 1];
    int held_stage = -1;
    auto put_held = [&]() {
        if (!holds || held_stage < 0) return;
#pragma unroll
        for (int j = 0; j < (holds ? NV : 1); ++j)
            if (j * tpr * VEC < d_left) {
                ring.put(held_stage, 0, j, held_in[0][j]);
                if (has_y) ring.put(held_stage, ky, j, held_in[1][j]);
                if (full) ring.put(held_stage, kz, j, held_in[2][j]);
                if (has_dr) ring.put(held_stage, kr, j, held_in[3][j]);
                if (has_dh) ring.put(held_stage, kh, j, held_in[4][j]);
            }
        held_stage = -1;
    };
    auto fetch = [&](int stage) {
        put_held();
        if (left > 0) {
            --left;
            if (holds) held_stage = stage;
            const T *drf = static_cast<const T*>(g.dr) + af, *dhf = static_cast<const T*>(g.dh) + af;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * tpr * VEC;
                if (c < d_left) {
                    if constexpr (holds) {
                        held_in[0][j] = xf[c];
                        if (has_y) held_in[1][j] = yf[c];
                        if (full) held_in[2][j] = zf[c];
                        if (has_dr) held_in[3][j] = drf[c];
                        if (has_dh) held_in[4][j] = dhf[c];
                    } else {
                        ring.copy(stage, 0, j, xf + c);
                        if (has_y) ring.copy(stage, ky, j, yf + c);
                        if (full) ring.copy(stage, kz, j, zf + c);
                        if (has_dr) ring.copy(stage, kr, j, drf + c);
                        if (has_dh) ring.copy(stage, kh, j, dhf + c);
                    }
                }
            }
            xf += xs;
            if (has_y) yf += ys;
            if (full) zf += zs;
            af += stride * D;
        }
        cp_async_commit();
    };
    pdl_wait();
    for (int i = 0; i + 1 < stages; ++i) fetch(i);
    // the norm alone has registers for its weights, and for dh until its second use
    P kept[has_y ? 1 : NV][N], held[has_y ? 1 : NV][N];
    if (!has_y) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * tpr * VEC < d_left) unpack(ldvec<T, VEC>(nw + j * tpr * VEC), kept[has_y ? 0 : j]);
    }
    // dh and next_weight of a vector
    auto get_h = [&](int stage, int j, int c, bool again, P (&f)[N], P (&w)[N]) {
        if constexpr (has_y) {
            ring.get(stage, kh, j, f);
            unpack(ldvec<T, VEC>(nw + c), w);
        } else {
            if (!again) ring.get(stage, kh, j, held[j]);
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = held[j][i], w[i] = kept[j][i];
        }
    };
    int stage = 0;
    long long at = row_first * D + t * VEC;
    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += stride, at += stride * D) {
        const bool live = row0 + mine < a.rows;
        const int cols = live ? d_left : 0;
        fetch(stage == 0 ? stages - 1 : stage - 1);
        if (stages == 1) put_held();
        float a_row = 1.f, slope_row = 0.f;
        if (MODE == kAny && a.gate && !full && live)
            a_row = gate_of(to_f32(static_cast<const T*>(a.gate)[(row0 + mine) * a.gate_stride]), silu, slope_row);
        cp_async_wait_but(stages - 1);
        // norm(y), act(gate), scale act'(gate) u; with 16 values a thread they are formed again from the ring where
        // they are used: kept, they spill (4000 bf16 rows of 5001, forward and backward: 1030 us, 658 so)
        constexpr bool again = NV * VEC >= 16;
        P ny[again ? 1 : NV][N], ga[again ? 1 : NV][N], dz[again ? 1 : NV][N], acc = L::all(0.f);
        float inv_y = 0.f;
        auto gates = [&](int j, int c, P (&n)[N], P (&act)[N], P (&d)[N], P (&w)[N], P (&s)[N]) {  // n: y on entry
            P z[N];
            unpack(ldvec<T, VEC>(pw + c), w);
            if (full) ring.get(stage, kz, j, z);
            if (scaled) unpack(ldvec<T, VEC>(sc + c), s);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!scaled) s[i] = L::all(1.f);
                n[i] = n[i] * L::all(inv_y);
                P slope = L::all(1.f);
                act[i] = full ? gate_of(z[i], silu, slope) : L::all(a_row);
                d[i] = slope * (n[i] * w[i]) * s[i];
            }
        };
        if (has_y) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * tpr * VEC < cols) {
                    P(&n)[N] = ny[again ? 0 : j];
                    ring.get(stage, ky, j, n);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc = fma_(n[i], n[i], acc);
                }
            float s1[1] = {sum_of(acc)};
            row_sum<TPR, 1>(s1, red1, turn1);
            inv_y = rsqrtf(s1[0] * inv_d + a.eps);
        }
        // r again, sum r^2 and sum (dh w) r
        P R[NV][N], rr = L::all(0.f), hr = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * tpr * VEC;
            if (c < cols) {
                ring.get(stage, 0, j, R[j]);
                if (has_y) {
                    P fw[N], fs[N], (&n)[N] = ny[again ? 0 : j], (&act)[N] = ga[again ? 0 : j];
                    if (again) ring.get(stage, ky, j, n);
                    gates(j, c, n, act, dz[again ? 0 : j], fw, fs);
#pragma unroll
                    for (int i = 0; i < N; ++i) R[j][i] = fma_(fs[i] * act[i], n[i] * fw[i], R[j][i]);
                }
                if (has_dh) {
                    P fh[N], fn[N];
                    get_h(stage, j, c, false, fh, fn);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        rr = fma_(R[j][i], R[j][i], rr);
                        hr = fma_(fh[i] * fn[i], R[j][i], hr);
                    }
                }
            }
        }
        float inv_r = 0.f, dot = 0.f;
        if (has_dh) {
            float s2[2] = {sum_of(rr), sum_of(hr)};
            row_sum<TPR, 2>(s2, red2, turn2);
            inv_r = rsqrtf(s2[0] * inv_d + a.eps);
            dot = s2[1] * inv_r * inv_d;
        }
        // the gradient of r; of the gate, the scale and y's norm
        P dn = L::all(0.f), dg = L::all(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = j * tpr * VEC;
            if (c < cols) {
                P fr[N];
#pragma unroll
                for (int i = 0; i < N; ++i) fr[i] = L::all(0.f);
                if (has_dr) ring.get(stage, kr, j, fr);
                if (has_dh) {
                    P fh[N], fn[N];
                    get_h(stage, j, c, true, fh, fn);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const P nr = R[j][i] * L::all(inv_r);
                        gn[j][i] = fma_(fh[i], nr, gn[j][i]);
                        fr[i] = fma_(L::all(inv_r), fma_(nr, L::all(-dot), fh[i] * fn[i]), fr[i]);
                    }
                }
                stvec<T, VEC>(static_cast<T*>(g.dx) + at + c, fr);
                if (has_y) {
                    P fw[N], fs[N], (&n)[N] = ny[again ? 0 : j], (&act)[N] = ga[again ? 0 : j], (&d)[N] = dz[again ? 0 : j];
                    if (again) {
                        ring.get(stage, ky, j, n);
                        gates(j, c, n, act, d, fw, fs);
                    } else {
                        unpack(ldvec<T, VEC>(pw + c), fw);
                        if (scaled) unpack(ldvec<T, VEC>(sc + c), fs);
                    }
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (!scaled) fs[i] = L::all(1.f);
                        const P rg = fr[i] * act[i];
                        gv[j][i] = fma_(rg, n[i], gv[j][i]);
                        d[i] = d[i] * fr[i];
                        R[j][i] = rg * (fs[i] * fw[i]);  // gradient of ny
                        dn = fma_(R[j][i], n[i], dn);
                        if (MODE == kAny) dg = fma_(d[i], L::all(1.f), dg);
                    }
                    if (full) stvec<T, VEC>(static_cast<T*>(g.dgate) + at + c, d);
                }
            }
        }
        if (has_y) {
            float s3[2] = {sum_of(dn), sum_of(dg)};
            if (MODE == kAny) {
                row_sum<TPR, 2>(s3, red2, turn2);
            } else {
                float s4[1] = {s3[0]};
                row_sum<TPR, 1>(s4, red1, turn1);
                s3[0] = s4[0];
            }
            const P m = L::all(-s3[0] * inv_d);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * tpr * VEC;
                if (c < cols) {
                    P o[N], (&n)[N] = ny[again ? 0 : j];
                    if (again) {
                        ring.get(stage, ky, j, n);
#pragma unroll
                        for (int i = 0; i < N; ++i) n[i] = n[i] * L::all(inv_y);
                    }
#pragma unroll
                    for (int i = 0; i < N; ++i) o[i] = L::all(inv_y) * fma_(n[i], m, R[j][i]);
                    stvec<T, VEC>(static_cast<T*>(g.dy) + at + c, o);
                }
            }
            if (MODE == kAny && a.gate && !full && live && t == 0)
                static_cast<T*>(g.dgate)[row0 + mine] = from_f32<T>(s3[1] * slope_row);
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
    // this CTA's partial sums: V with y, next_weight with dh
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
                            acc[c] = (who ? acc[c] : 0.f) + at_of(gv[j], i);
                            acc[D + c] = (who ? acc[D + c] : 0.f) + at_of(gn[j], i);
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
                if (c < D) {
                    if (has_y) dst[c] = at_of(gv[j], i);
                    if (has_dh) dst[D + c] = at_of(gn[j], i);
                }
            }
    }
}

// Sums the partial rows: 32 columns a CTA, 32 row lanes, then a tree over them in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024)
    partial_sum_kernel(const float* __restrict__ partial, int partials, int D, const T* __restrict__ post_weight,
                       const T* __restrict__ scale, float* __restrict__ d_post, float* __restrict__ d_scale,
                       float* __restrict__ d_next) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
    pdl_wait();
    if (!(which == 0 ? d_post : d_next)) return;
    float s = 0.f;
    if (c < D) {
        const float* src = partial + (size_t)which * D + c;
        int p = w;
        for (; p + 7 * 32 < partials; p += 8 * 32) {  // eight loads in flight
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = src[(size_t)(p + 32 * i) * 2 * D];
            s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        for (; p < partials; p += 32) s += src[(size_t)p * 2 * D];
    }
    sm[w][lane] = s;
    __syncthreads();
    for (int o = 16; o; o >>= 1) {
        if (w < o) sm[w][lane] += sm[w + o][lane];
        __syncthreads();
    }
    if (w == 0 && c < D) {
        if (which == 1) {
            d_next[c] = sm[0][lane];
        } else {
            d_post[c] = scale ? sm[0][lane] * to_f32(scale[c]) : sm[0][lane];
            if (d_scale) d_scale[c] = sm[0][lane] * to_f32(post_weight[c]);
        }
    }
}

Work backward_work(const hla2_block_args* a, const Shape& s, int vec, int tensors, int sms) {
    return work_of(a, s, vec, tensors, has_y(a) ? kBwdThreadsPerSm : kNormBwdThreadsPerSm, s.tpr && s.tpr <= 32 ? 2 * (size_t)a->D * sizeof(float) : 0, sms);
}

}  // namespace
}  // namespace hla2

using namespace hla2;

extern "C" {

size_t hla2_block_join_backward_workspace_bytes(const hla2_block_args* a) {
    if (check_join("hla2_block_join_backward_workspace_bytes", a) != HLA2_OK) return (size_t)-1;
    join_ok();
    size_t most = 0;
    const int sms = sm_count();
    const int wide = a->dtype == HLA2_BF16 ? 8 : 4;
    for (int vec : {1, 2, wide}) {  // whichever the addresses allow
        for (int tensors = 2; tensors <= 5; ++tensors) {
            const size_t c = (size_t)backward_work(a, shape_of(a->D, vec), vec, tensors, sms).ctas;
            if (c > most) most = c;
        }
    }
    return most * 2 * (size_t)a->D * sizeof(float);
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
    {
        const RowsOf grads[2] = {{dr, a->D, a->D}, {dh, a->D, a->D}};
        const RowsOf out[3] = {{dx, a->D, a->D}, {dy, a->D, a->D}, {dgate, a->gate_cols, a->gate_cols}};
        const size_t vb = (size_t)a->D * sizeof(float);
        const Extent sums[3] = {extent_of(dpost_weight, vb), extent_of(dscale, vb), extent_of(dnext_weight, vb)};
        bool bad = false;
        for (int i = 0; i < 3; ++i) {
            for (int j = 0; j < i; ++j) bad |= meet(sums[i], sums[j]);
            for (const void* w : {a->post_weight, a->scale, a->next_weight}) bad |= meet(sums[i], extent_of(w, a->D * es));
            if (a->rows == 0) continue;
            for (const RowsOf& t : {RowsOf{a->x, a->x_stride, a->D}, RowsOf{a->y, a->y_stride, a->D},
                                    RowsOf{a->gate, a->gate_stride, a->gate_cols}, grads[0], grads[1], out[0], out[1], out[2]})
                bad |= t.p && meet(sums[i], rows_extent(a, t));
            if (!out[i].p) continue;
            bad |= spoils(a, out[i], grads, 2);
            for (int j = 0; j < i; ++j) bad |= out[j].p && meet(rows_extent(a, out[i]), rows_extent(a, out[j]));
        }
        if (bad) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient overlaps another tensor other than in its place", fn);
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
        const Work w = backward_work(a, s, vec, tensors, sm_count());
        g.partials = w.ctas;
        auto launch = [&](auto v, auto nv, auto tpr, auto maxt, auto mode, auto zero) {
            using T = decltype(zero);
            auto k = join_backward_kernel<T, decltype(v)::value, decltype(nv)::value, decltype(tpr)::value,
                                          decltype(maxt)::value, decltype(mode)::value>;
            if (!set_smem(k, w.smem)) return -1;
            return launch_pdl(k, dim3(w.ctas), dim3(s.threads), w.smem, st, *a, g, w.stages) == cudaSuccess ? 0 : -1;
        };
        if (dispatch(a, mode_of(a, dr), vec, s, launch))
            return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    }
    auto join_sums = [&](auto zero) {
        using T = decltype(zero);
        return launch_pdl(partial_sum_kernel<T>, dim3((a->D + 31) / 32, 2), dim3(1024), 0, st, g.partial, g.partials, a->D,
                          static_cast<const T*>(a->post_weight), static_cast<const T*>(a->scale), dpost_weight, dscale,
                          dnext_weight);
    };
    if ((a->dtype == HLA2_BF16 ? join_sums(bf16{}) : join_sums(0.f)) != cudaSuccess)
        return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return join_ok();
}

}  // extern "C"
