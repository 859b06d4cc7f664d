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
// Memory floor: 5 tensors forward, 8 backward.  Persistent CTAs take rows in a fixed stride.  A thread
// owns NV vectors of VEC values of every row; it copies them ahead with cp.async into a ring of rows
// in shared memory that nobody else reads, so the ring needs no barrier, and the bytes in flight do
// not cost registers (plain loads into registers held 152 of them, one CTA per SM, 1.2 TB/s).
// Rows of at most 32 vectors take a part of a warp (TPR threads), longer ones a whole CTA.  The backward
// keeps its two sums over rows in registers; each CTA writes one partial row, which a second kernel
// sums in a fixed order.
//
// 32768 bf16 rows of 2048, gate, scale and next norm: 112 us forward (6.0 TB/s, 89 % of the measured
// copy), 223 us backward (4.8 TB/s).  What is left is instructions and the latency of the row sums: 41 and
// 68 instructions a value (82 backward before packed arithmetic and the shared sum), of which unpacking
// bf16 takes a quarter, at two (backward) to four CTAs an SM.  5000 float32 rows of 999, the norm alone, single
// elements: 11 us forward, 15.7 us backward and 6 us for the partial rows.
#include "block_join.cuh"

namespace hla2 {
namespace {

template <typename T, int VEC, int NV, int TPR, int MAXT, int MODE>
__global__ void __launch_bounds__(MAXT, MAXT <= 256 ? 4 : 2)
    join_kernel(const hla2_block_args a, T* __restrict__ r_out, T* __restrict__ h_out, int stages) {
    using L = Lanes<VEC>;
    using P = typename L::P;
    constexpr int N = L::N;
    extern __shared__ __align__(16) char ring_sm[];
    __shared__ float red[2][16][1];
    int turn = 0;
    const int tpr = TPR ? TPR : blockDim.x, t = threadIdx.x % tpr, mine = threadIdx.x / tpr;
    constexpr int per = TPR ? kSmallThreads / (TPR ? TPR : 1) : 1;
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    constexpr bool has_y = MODE != kNormOnly;
    const bool full = MODE == kAll || (MODE == kAny && a.gate && a.gate_cols != 1);
    const bool scaled = MODE == kAll || (MODE == kAny && a.scale), normed = MODE != kAny || h_out;
    const bool silu = a.gate_act == HLA2_GATE_SILU;
    const T *pw = static_cast<const T*>(a.post_weight) + t * VEC, *sc = static_cast<const T*>(a.scale) + t * VEC,
            *nw = static_cast<const T*>(a.next_weight) + t * VEC;
    const Ring<T, VEC, NV> ring(ring_sm, 1 + (has_y ? 1 : 0) + (full ? 1 : 0));
    const long long stride = (long long)gridDim.x * per, row_first = (long long)blockIdx.x * per + mine;
    // the next row to copy: this thread's first value of it
    const T *xf = static_cast<const T*>(a.x) + row_first * a.x_stride + t * VEC,
            *yf = static_cast<const T*>(a.y) + row_first * a.y_stride + t * VEC,
            *zf = static_cast<const T*>(a.gate) + row_first * a.gate_stride + t * VEC;
    const long long xs = stride * a.x_stride, ys = stride * a.y_stride, zs = stride * a.gate_stride;
    long long left = row_first < a.rows ? (a.rows - 1 - row_first) / stride + 1 : 0;  // rows still to copy
    const int d_left = D - t * VEC;  // columns from this thread's first on
    constexpr bool holds = kHolds<T, VEC, NV>;
    T held[3][holds ? NV : 1];
    int held_stage = -1;
    auto put_held = [&]() {
        if (!holds || held_stage < 0) return;
#pragma unroll
        for (int j = 0; j < (holds ? NV : 1); ++j)
            if (j * tpr * VEC < d_left) {
                ring.put(held_stage, 0, j, held[0][j]);
                if (has_y) ring.put(held_stage, 1, j, held[1][j]);
                if (full) ring.put(held_stage, 2, j, held[2][j]);
            }
        held_stage = -1;
    };
    auto fetch = [&](int stage) {
        put_held();
        if (left > 0) {
            --left;
            if (holds) held_stage = stage;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * tpr * VEC;
                if (c < d_left) {
                    if constexpr (holds) {
                        held[0][j] = xf[c];
                        if (has_y) held[1][j] = yf[c];
                        if (full) held[2][j] = zf[c];
                    } else {
                        ring.copy(stage, 0, j, xf + c);
                        if (has_y) ring.copy(stage, 1, j, yf + c);
                        if (full) ring.copy(stage, 2, j, zf + c);
                    }
                }
            }
            xf += xs;
            if (has_y) yf += ys;
            if (full) zf += zs;
        }
        cp_async_commit();
    };
    pdl_wait();
    for (int i = 0; i + 1 < stages; ++i) fetch(i);
    // the norm alone has registers for its weights
    P kept[has_y ? 1 : NV][N];
    if (!has_y) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * tpr * VEC < d_left) unpack(ldvec<T, VEC>(nw + j * tpr * VEC), kept[has_y ? 0 : j]);
    }
    int stage = 0;
    long long at = row_first * D + t * VEC;
    // whole sub-warps: lanes of a row past the last take part in the shuffles
    for (long long row0 = (long long)blockIdx.x * per; row0 < a.rows; row0 += stride, at += stride * D) {
        const bool live = row0 + mine < a.rows;
        const int cols = live ? d_left : 0;
        fetch(stage == 0 ? stages - 1 : stage - 1);  // into the slot of the row before
        if (stages == 1) put_held();
        float a_row = 1.f, slope;
        if (MODE == kAny && a.gate && !full && live)
            a_row = gate_of(to_f32(static_cast<const T*>(a.gate)[(row0 + mine) * a.gate_stride]), silu, slope);
        cp_async_wait_but(stages - 1);
        P r[NV][N], acc = L::all(0.f);
        float sum[1];
        if (has_y) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * tpr * VEC < cols) {
                    ring.get(stage, 1, j, r[j]);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc = fma_(r[j][i], r[j][i], acc);
                }
            sum[0] = sum_of(acc);
            row_sum<TPR, 1>(sum, red, turn);
            const P inv = L::all(rsqrtf(sum[0] * inv_d + a.eps));
            acc = L::all(0.f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * tpr * VEC;
                if (c < cols) {
                    P fx[N], fz[N], fw[N], fs[N], slope_;
                    ring.get(stage, 0, j, fx);
                    unpack(ldvec<T, VEC>(pw + c), fw);
                    if (full) ring.get(stage, 2, j, fz);
                    if (scaled) unpack(ldvec<T, VEC>(sc + c), fs);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        P u = r[j][i] * inv * fw[i];
                        u = u * (full ? gate_of(fz[i], silu, slope_) : L::all(a_row));
                        r[j][i] = fma_(scaled ? fs[i] : L::all(1.f), u, fx[i]);
                        acc = fma_(r[j][i], r[j][i], acc);
                    }
                    stvec<T, VEC>(r_out + at + c, r[j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * tpr * VEC < cols) {
                    ring.get(stage, 0, j, r[j]);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc = fma_(r[j][i], r[j][i], acc);
                }
        }
        if (normed) {
            sum[0] = sum_of(acc);
            row_sum<TPR, 1>(sum, red, turn);
            const P inv = L::all(rsqrtf(sum[0] * inv_d + a.eps));
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = j * tpr * VEC;
                if (c < cols) {
                    P o[N];
                    if (!has_y) {
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = r[j][i] * inv * kept[has_y ? 0 : j][i];
                    } else {
                        P fw[N];
                        unpack(ldvec<T, VEC>(nw + c), fw);
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = r[j][i] * inv * fw[i];
                    }
                    stvec<T, VEC>(h_out + at + c, o);
                }
            }
        }
        stage = stage + 1 == stages ? 0 : stage + 1;
    }
    // At the end (as the backward): from the start on, CTAs of the next kernel crowd on the SMs that are free
    // first (32768 rows of 2048, forward and backward: 357 us, 339 now, 344 without).
    pdl_trigger();
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
    const RowsOf ro{r, a->D, a->D}, ho{h, a->D, a->D};
    if (r && h && meet(rows_extent(a, ro), rows_extent(a, ho)))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: r and h must be distinct", fn);
    if ((r && spoils(a, ro, nullptr, 0)) || (h && spoils(a, ho, nullptr, 0)))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: an output overlaps an input other than in its place", fn);
    const void* outs[2] = {r, h};
    const int vec = vec_of(a, outs, 2);
    const Shape s = shape_of(a->D, vec);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int tensors = 1 + (a->y ? 1 : 0) + (a->y && a->gate && a->gate_cols != 1 ? 1 : 0);
    const Work w = work_of(a, s, vec, tensors, kFwdThreadsPerSm, 0, sm_count());
    auto launch = [&](auto v, auto nv, auto tpr, auto maxt, auto mode, auto zero) {
        using T = decltype(zero);
        auto k = join_kernel<T, decltype(v)::value, decltype(nv)::value, decltype(tpr)::value, decltype(maxt)::value,
                             decltype(mode)::value>;
        if (!set_smem(k, w.smem)) return -1;
        return launch_pdl(k, dim3(w.ctas), dim3(s.threads), w.smem, st, *a, static_cast<T*>(r), static_cast<T*>(h),
                          w.stages) == cudaSuccess
                   ? 0
                   : -1;
    };
    if (dispatch(a, mode_of(a, h), vec, s, launch))
        return set_last_error(HLA2_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(cudaGetLastError()));
    return join_ok();
}

}  // extern "C"
