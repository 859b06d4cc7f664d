// First-order linear attention with a decay for each head: the chunk passes in float32
// arithmetic (SIMT), the scan over segments, and the step of single tokens.  The mathematics
// of a pass is in linattn_pass.h.
//
// Chunk pass.  One CTA runs the chunks of one segment of one state head.  Per chunk of W rows
// (Wc of them valid) and state Sig at the chunk's entry, forward:
//     A = (X K^T) * [j <= i] g^(i-j)          Y = s_fin (s_col A V + diag(g^(i+1)) X Sig)
//     Sig <- g^Wc Sig + s_state (diag(g^(Wc-1-j)) K)^T V
// and in reverse [j >= i] g^(j-i), g^(Wc-i) and g^j.  X, K^T, V, A and Sig stay in shared memory;
// every product is register-tiled (simt_tile.cuh).
#include "linattn_pass.h"
#include "simt_tile.cuh"

namespace hla2 {

namespace {

using simt::kThreads;
using simt::pad;

struct LinSmem {
    int X, Kt, V, A, S, Y, gp, total;
};
__host__ __device__ inline LinSmem lin_smem(int dx, int dy, int W, bool keep_y) {
    LinSmem L;
    int o = 0;
    L.X = o;  o += W * pad(dx);
    L.Kt = o; o += dx * pad(W);
    L.V = o;  o += W * dy;
    L.A = o;  o += W * pad(W);
    L.S = o;  o += dx * dy;
    L.Y = o;  o += keep_y ? W * dy : 0;
    L.gp = o; o += W + 4;
    L.total = o;
    return L;
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ const float* row_ptr(const hla2_view& w, int b, int h, int row) {
    return static_cast<const float*>(w.p) + b * w.sb + h * w.sh + row * w.sn;
}

// rows [row0, row0 + Wc) of a view as W x D floats (leading dimension ld), the rest zero; W and D are
// powers of two
__device__ __forceinline__ void load_rows(float* dst, int ld, const hla2_view& w, int b, int h, int row0, int W, int Wc,
                                          int D) {
    const int sh = 29 - __clz(D);  // log2(D / 4)
    for (int e = threadIdx.x; e < W << sh; e += kThreads) {
        const int i = e >> sh, f = (e - (i << sh)) * 4;
        const float4 t = i < Wc ? load4(row_ptr(w, b, h, row0 + i) + f) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + i * ld + f) = t;
    }
}
// the same, transposed, row i times weight(i)
template <class Weight>
__device__ __forceinline__ void load_rows_t(float* dst, int ld, const hla2_view& w, int b, int h, int row0, int W,
                                            int Wc, int D, Weight weight) {
    const int sh = 31 - __clz(W);
    for (int e = threadIdx.x; e < (D >> 2) << sh; e += kThreads) {
        const int i = e & (W - 1), f = (e >> sh) * 4;  // lanes on rows: the transposed stores fall in distinct banks
        const float4 t = i < Wc ? load4(row_ptr(w, b, h, row0 + i) + f) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float m = weight(i);
        dst[f * ld + i] = m * t.x;
        dst[(f + 1) * ld + i] = m * t.y;
        dst[(f + 2) * ld + i] = m * t.z;
        dst[(f + 3) * ld + i] = m * t.w;
    }
}
// the rows' lines towards the L2, for the loads of the next chunk
__device__ __forceinline__ void prefetch_rows(const hla2_view& w, int b, int h, int row0, int rows, int D) {
    const int sh = D > 32 ? 26 - __clz(D) : 0;  // log2 of a row's 128-byte lines
    for (int e = threadIdx.x; e < rows << sh; e += kThreads)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row_ptr(w, b, h, row0 + (e >> sh)) + (e & ((1 << sh) - 1)) * 32));
}

// MANY: several passes in one launch.  Their fields are loaded by an index at every use then (231 against
// 198 us for 32 heads x 4000 rows of 64), so one pass goes by a constant address.
template <bool SUMMARY, bool MANY>
__global__ void __launch_bounds__(kThreads, 3) lin_simt_kernel(const __grid_constant__ LinPasses all) {
    const LinPass& a = all.p[MANY ? blockIdx.z : 0];
    extern __shared__ __align__(16) float sm[];
    const int dx = a.dx, dy = a.dy, W = a.W;
    const bool keep_y = !SUMMARY && a.rk > 1;
    const LinSmem L = lin_smem(dx, dy, W, keep_y);
    float *Xs = sm + L.X, *Kt = sm + L.Kt, *Vs = sm + L.V, *As = sm + L.A, *S = sm + L.S, *Ys = sm + L.Y,
          *gp = sm + L.gp;
    const int tid = threadIdx.x;
    const int seg = blockIdx.y, bs = blockIdx.x, b = bs / a.Hs, s = bs % a.Hs;
    pdl_wait();
    const int len = lin_len(a.lengths, b, a.n);
    const int c0 = seg * a.seg_chunks, c1 = min(c0 + a.seg_chunks, a.nchunks);
    const float log2g = log2f(lin_decay(a, s));
    const bool rev = a.rev != 0;
    const float s_in = a.s_fin * a.s_col;
    for (int i = tid; i <= W; i += kThreads) gp[i] = pow_decay(log2g, (float)i);
    const float* carry = SUMMARY || !a.carry ? nullptr : a.carry + ((size_t)bs * a.nseg + seg) * dx * dy;
    for (int e = tid; e < dx * dy; e += kThreads)
        S[e] = !carry ? 0.f : a.carry_t ? carry[(e % dy) * dx + e / dy] : carry[e];

    const int items = a.rx > a.rk ? a.rx : a.rk;
    for (int cc = c0; cc < c1; ++cc) {
        const int c = rev ? c0 + c1 - 1 - cc : cc;
        const int row0 = c * W, Wn = min(W, a.n - row0), Wc = max(0, min(Wn, len - row0));
        if (Wc == 0 && SUMMARY) continue;
        for (int r = 0; r < items; ++r) {
            const bool x_new = r == 0 || a.rx > 1, kv_new = r == 0 || a.rk > 1;
            const bool y_last = a.rx > 1 || r == items - 1, s_now = a.rk > 1 || r == items - 1;
            const int hx = s * a.rx + (a.rx > 1 ? r : 0), hk = s * a.rk + (a.rk > 1 ? r : 0);
            __syncthreads();
            if (!SUMMARY && x_new) load_rows(Xs, pad(dx), a.x, b, hx, row0, W, Wc, dx);
            if (kv_new) {
                load_rows_t(Kt, pad(W), a.k, b, hk, row0, W, Wc, dx,
                            [&](int i) { return !SUMMARY || i >= Wc ? 1.f : a.s_state * gp[rev ? i : Wc - 1 - i]; });
                load_rows(Vs, dy, a.v, b, hk, row0, W, Wc, dy);
            }
            __syncthreads();
            if (r == items - 1 && cc + 1 < c1) {  // (of the first heads, where there are several)
                const int next = (rev ? c - 1 : c + 1) * W, rows = min(W, len - next);
                if (!SUMMARY) prefetch_rows(a.x, b, s * a.rx, next, rows, dx);
                prefetch_rows(a.k, b, s * a.rk, next, rows, dx);
                prefetch_rows(a.v, b, s * a.rk, next, rows, dy);
            }
            if (!SUMMARY) {
                simt::with_rm(W, W, [&](auto RMc) {
                    constexpr int RM = decltype(RMc)::value;
                    simt::for_blocks<RM>(W, W, [&](int m0, int n0) {
                        simt::Acc<RM> acc;
                        simt::zero<RM>(acc);
                        const bool any = rev ? n0 + 3 >= m0 : n0 <= m0 + RM - 1;
                        if (any) simt::mac_r<RM>(acc, Xs + m0 * pad(dx), pad(dx), Kt + n0, pad(W), dx);
#pragma unroll
                        for (int i = 0; i < RM; ++i) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int e = rev ? n0 + j - m0 - i : m0 + i - n0 - j;
                                acc[i][j] = e >= 0 ? acc[i][j] * gp[e] : 0.f;
                            }
                            simt::st4(As + (m0 + i) * pad(W) + n0, acc[i]);
                        }
                    });
                });
                __syncthreads();
                simt::with_rm(W, dy, [&](auto RMc) {
                    constexpr int RM = decltype(RMc)::value;
                    simt::for_blocks<RM>(W, dy, [&](int m0, int n0) {
                        simt::Acc<RM> acc;
                        simt::zero<RM>(acc);
                        if (x_new) {
                            simt::mac_r<RM>(acc, Xs + m0 * pad(dx), pad(dx), S + n0, dy, dx);
#pragma unroll
                            for (int i = 0; i < RM; ++i) {
                                const int e = rev ? max(Wc - m0 - i, 0) : m0 + i + 1;
                                simt::scale_row<RM>(acc, i, a.s_fin * gp[e]);
                            }
                        }
                        simt::Acc<RM> in;
                        simt::zero<RM>(in);
                        if (rev) {
                            const int j0 = m0 & ~3;
                            simt::mac_r<RM>(in, As + m0 * pad(W) + j0, pad(W), Vs + j0 * dy + n0, dy, W - j0);
                        } else {
                            simt::mac_r<RM>(in, As + m0 * pad(W), pad(W), Vs + n0, dy, m0 + RM);
                        }
#pragma unroll
                        for (int i = 0; i < RM; ++i) {
                            const int row = m0 + i;
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[i][j] += s_in * in[i][j];
                            if (keep_y) {
                                float* p = Ys + row * dy + n0;
                                if (r > 0) {
#pragma unroll
                                    for (int j = 0; j < 4; ++j) acc[i][j] += p[j];
                                }
                                simt::st4(p, acc[i]);
                            }
                            if (y_last && row < Wn) {
                                if (row >= Wc) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
                                simt::store4(const_cast<float*>(row_ptr(a.y, b, hx, row0 + row)) + n0, acc[i]);
                            }
                        }
                    });
                });
            }
            if (s_now && Wc > 0 && (SUMMARY || cc + 1 < c1)) {  // no row reads the state after the last chunk
                __syncthreads();  // Sig has been read
                const float rho = r == 0 || a.rk == 1 ? gp[Wc] : 1.f;
                simt::with_rm(dx, dy, [&](auto RMc) {
                    constexpr int RM = decltype(RMc)::value;
                    simt::for_blocks<RM>(dx, dy, [&](int m0, int n0) {
                        simt::Acc<RM> acc;
                        simt::zero<RM>(acc);
                        if (SUMMARY)
                            simt::mac_r<RM>(acc, Kt + m0 * pad(W), pad(W), Vs + n0, dy, Wc);
                        else
                            simt::mac_r<RM>(acc, Kt + m0 * pad(W), pad(W), Vs + n0, dy, Wc,
                                            [&](int j) { return a.s_state * gp[rev ? j : Wc - 1 - j]; });
#pragma unroll
                        for (int i = 0; i < RM; ++i) simt::decay_add4(S + (m0 + i) * dy + n0, rho, acc[i]);
                    });
                });
            }
        }
    }
    pdl_trigger();  // at the end: CTAs of the next kernel would crowd on the SMs that are free before
    if (SUMMARY) {
        __syncthreads();
        float* dst = a.sums + ((size_t)bs * a.nseg + seg) * dx * dy;
        for (int e = tid; e < dx * dy; e += kThreads) dst[e] = S[e];
    }
}

// ---- scan over the segments -----------------------------------------------------------
//
// A thread owns four state elements.  PARTS threads share them where there are many segments: each
// sums its run of segments, they pass the runs' sums on through shared memory, and each then scans its
// run.  Up to kScanAhead segments a run stay in registers between the two.  Bound by latency: 2 heads x
// 64 segments of 32 x 64 states take 6.8 us (12.4 us with one thread an element and serial runs), 64
// heads x 2 segments of 128 x 128 take 6.5 us (14 us with one element a thread).
constexpr int kScanAhead = 8, kScanParts = 8;

template <int PARTS>
__global__ void __launch_bounds__(kThreads)
    lin_scan_kernel(const LinScan s0, const LinScan s1, const float* __restrict__ gamma,
                    const int* __restrict__ lengths, int Hs, int n, int seg_rows, int nseg, int elems) {
    const bool second = blockIdx.z > 0;
    const float* __restrict__ sums = second ? s1.sums : s0.sums;
    float* __restrict__ carry = second ? s1.carry : s0.carry;
    const float* __restrict__ init = second ? s1.init : s0.init;
    float* __restrict__ fin = second ? s1.final_state : s0.final_state;
    const int rev = second ? s1.rev : s0.rev;
    constexpr int kOwners = kThreads / PARTS;
    __shared__ float4 run_sum[PARTS][kOwners];
    const int bs = blockIdx.x, b = bs / Hs, owner = threadIdx.x % kOwners, part = threadIdx.x / kOwners;
    const int e = (blockIdx.y * kOwners + owner) * 4;
    const bool live = e < elems;
    pdl_trigger();
    pdl_wait();
    const float g = gamma ? __ldg(gamma + bs % Hs) : 1.f;
    const float log2g = log2f(g);
    const int len = lin_len(lengths, b, n);
    auto rows_before = [&](int i) { return lin_rows_before(len, rev, i, nseg, seg_rows); };
    auto decay = [&](int from, int to) { return pow_decay(log2g, (float)(rows_before(to) - rows_before(from))); };
    auto step = [](float4& c, float f, const float4& v) {
        c = make_float4(fmaf(f, c.x, v.x), fmaf(f, c.y, v.y), fmaf(f, c.z, v.z), fmaf(f, c.w, v.w));
    };
    const size_t base = (size_t)bs * nseg * elems + e;
    const int steps = fin ? nseg : nseg - 1;  // the last sum only enters the final state
    const int run = (nseg + PARTS - 1) / PARTS, lo = min(nseg, part * run), hi = min(nseg, lo + run);
    float4 v[kScanAhead];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j) {
            const int i = i0 + j;
            v[j] = live && i < hi && i < steps
                       ? *reinterpret_cast<const float4*>(sums + base + (size_t)(rev ? nseg - 1 - i : i) * elems)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init && live) {
        cur = *reinterpret_cast<const float4*>(init + (size_t)bs * elems + e);
        if (rev) cur = make_float4(cur.x / g, cur.y / g, cur.z / g, cur.w / g);
    }
    if (PARTS > 1) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = lo; i0 < hi; i0 += kScanAhead) {
            fetch(i0);
#pragma unroll
            for (int j = 0; j < kScanAhead; ++j)
                if (i0 + j < hi) step(sum, decay(i0 + j, i0 + j + 1), v[j]);
        }
        run_sum[part][owner] = sum;
        __syncthreads();
#pragma unroll
        for (int p = 0; p < PARTS - 1; ++p)
            if (p < part) step(cur, decay(min(nseg, p * run), min(nseg, (p + 1) * run)), run_sum[p][owner]);
    }
    if (!live) return;
    for (int i0 = lo; i0 < hi; i0 += kScanAhead) {
        if (PARTS == 1 || run > kScanAhead) fetch(i0);
#pragma unroll
        for (int j = 0; j < kScanAhead; ++j) {
            const int i = i0 + j;
            if (i >= hi) break;
            if (carry) *reinterpret_cast<float4*>(carry + base + (size_t)(rev ? nseg - 1 - i : i) * elems) = cur;
            if (i < steps) step(cur, decay(i, i + 1), v[j]);
        }
    }
    if (fin && part == PARTS - 1) {
        if (rev) cur = make_float4(g * cur.x, g * cur.y, g * cur.z, g * cur.w);
        *reinterpret_cast<float4*>(fin + (size_t)bs * elems + e) = cur;
    }
}

// ---- step of single tokens -----------------------------------------------------------------
//
// One CTA per state; thread t holds the float4 column t % (dv / 4) of every (threads / (dv / 4))-th
// row, all RP of its loads in flight at once.  The state is read and written once.
template <typename T, int RP>
__global__ void __launch_bounds__(kThreads)
    lin_step_kernel(float* __restrict__ state, const T* __restrict__ q, const T* __restrict__ k,
                    const T* __restrict__ v, T* __restrict__ out, int Hk, int group, int d, int dv,
                    const float* __restrict__ gamma, float scale) {
    __shared__ __align__(16) float qs[128], ks[128], red[kThreads / 32][128];
    const int head = blockIdx.x, tid = threadIdx.x, NT = blockDim.x;
    const int lpr = dv >> 2, col = (tid % lpr) * 4, row = tid / lpr, step = NT / lpr;
    float* P = state + (size_t)head * d * dv;
    pdl_trigger();
    pdl_wait();
    float4 p[RP];
#pragma unroll
    for (int j = 0; j < RP; ++j) p[j] = __ldcs(reinterpret_cast<const float4*>(P + (size_t)(row + j * step) * dv + col));
    const float g = gamma ? __ldg(gamma + head % Hk) : 1.f;
    for (int i = tid; i < d; i += NT) ks[i] = to_f32(k[(size_t)head * d + i]);
    float vv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) vv[j] = to_f32(v[(size_t)head * dv + col + j]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < RP; ++j) {
        const float kk = ks[row + j * step];
        p[j].x = fmaf(g, p[j].x, kk * vv[0]);
        p[j].y = fmaf(g, p[j].y, kk * vv[1]);
        p[j].z = fmaf(g, p[j].z, kk * vv[2]);
        p[j].w = fmaf(g, p[j].w, kk * vv[3]);
        __stcs(reinterpret_cast<float4*>(P + (size_t)(row + j * step) * dv + col), p[j]);
    }
    for (int r = 0; r < group; ++r) {
        const size_t hq = (size_t)head * group + r;
        for (int i = tid; i < d; i += NT) qs[i] = to_f32(q[hq * d + i]);
        __syncthreads();
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < RP; ++j) {
            const float qq = qs[row + j * step];
            s.x = fmaf(qq, p[j].x, s.x);
            s.y = fmaf(qq, p[j].y, s.y);
            s.z = fmaf(qq, p[j].z, s.z);
            s.w = fmaf(qq, p[j].w, s.w);
        }
        for (int o = lpr; o < 32; o <<= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
            s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
            s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
        }
        const int warp = tid >> 5, lane = tid & 31;
        if (lane < lpr) *reinterpret_cast<float4*>(&red[warp][col]) = s;
        __syncthreads();
        for (int c = tid; c < dv; c += NT) {
            float t = 0.f;
            for (int w = 0; w < NT / 32; ++w) t += red[w][c];
            out[hq * dv + c] = from_f32<T>(scale * t);
        }
    }
}

template <typename T>
int launch_step_t(float* state, const void* q, const void* k, const void* v, void* out, int N, int Hk, int group, int d,
                  int dv, const float* gamma, float scale, cudaStream_t st) {
    const int vecs = d * dv / 4, threads = vecs < kThreads ? vecs : kThreads, rp = vecs / threads;
    const unsigned grid = (unsigned)N * (unsigned)Hk;
    auto go = [&](auto kfn) {
        return launch_pdl(kfn, dim3(grid), dim3(threads), 0, st, state, static_cast<const T*>(q), static_cast<const T*>(k),
                          static_cast<const T*>(v), static_cast<T*>(out), Hk, group, d, dv, gamma, scale) == cudaSuccess
                   ? 0
                   : -1;
    };
    switch (rp) {
        case 1: return go(lin_step_kernel<T, 1>);
        case 2: return go(lin_step_kernel<T, 2>);
        case 4: return go(lin_step_kernel<T, 4>);
        case 8: return go(lin_step_kernel<T, 8>);
        case 16: return go(lin_step_kernel<T, 16>);
        default: return -1;
    }
}

}  // namespace

int lin_simt_width(int dx, int dy, long long heads, int n, int sms) {
    int W = dx > 64 || dy > 64 ? 32 : 64;
    while (W > 16 && heads * ((n + W - 1) / W) < sms) W /= 2;
    return W;
}
int lin_simt_ctas(int dx, int dy, int W) {
    return simt::min_ctas(3, simt::ctas_per_sm(lin_smem(dx, dy, W, false).total * sizeof(float)));
}

int launch_lin_simt(const LinPass* passes, int count, bool summary, cudaStream_t st) {
    const LinPass& a = passes[0];  // they share the sizes of the grid
    if (count == 0 || a.B * a.Hs == 0 || a.nseg == 0) return 0;
    // one launch where the GPU holds all its CTAs at once, else it would gain nothing
    if (count > 1 && (long long)a.B * a.Hs * a.nseg * count > 3LL * sm_count()) {
        for (int i = 0; i < count; ++i)
            if (launch_lin_simt(passes + i, 1, summary, st)) return -1;
        return 0;
    }
    LinPasses all{};
    size_t smem = 0;
    for (int i = 0; i < count; ++i) {
        all.p[i] = passes[i];
        const LinPass& s = passes[i];
        const size_t b = lin_smem(s.dx, s.dy, s.W, !summary && s.rk > 1).total * sizeof(float);
        if (b > smem) smem = b;
    }
    auto kfn = count > 1 ? summary ? lin_simt_kernel<true, true> : lin_simt_kernel<false, true>
                         : summary ? lin_simt_kernel<true, false> : lin_simt_kernel<false, false>;
    if (raise_smem(kfn, smem) != cudaSuccess) return -1;
    return launch_pdl(kfn, dim3(a.B * a.Hs, a.nseg, count), dim3(kThreads), smem, st, all) == cudaSuccess ? 0 : -1;
}

int launch_lin_scan(const LinScan* scans, int count, const float* gamma, const int* lengths, int B, int Hs, int n,
                    int seg_rows, int nseg, int elems, cudaStream_t st) {
    if (count == 0 || B * Hs == 0) return 0;
    auto go = [&](auto kernel, int parts) {
        const int each = kThreads / parts * 4;  // elements of a CTA; a head's are a multiple of four
        return launch_pdl(kernel, dim3(B * Hs, (elems + each - 1) / each, count), dim3(kThreads), 0, st, scans[0],
                          scans[count - 1], gamma, lengths, Hs, n, seg_rows, nseg, elems) == cudaSuccess
                   ? 0
                   : -1;
    };
    return nseg > kScanAhead ? go(lin_scan_kernel<kScanParts>, kScanParts) : go(lin_scan_kernel<1>, 1);
}

int launch_lin_step(float* state, const void* q, const void* k, const void* v, void* out, int N, int H, int Hk, int d,
                    int dv, const float* gamma, float scale, bool is_bf16, cudaStream_t st) {
    if (N * Hk == 0) return 0;
    return is_bf16 ? launch_step_t<bf16>(state, q, k, v, out, N, Hk, H / Hk, d, dv, gamma, scale, st)
                   : launch_step_t<float>(state, q, k, v, out, N, Hk, H / Hk, d, dv, gamma, scale, st);
}

}  // namespace hla2
