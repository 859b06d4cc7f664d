// The short causal convolution of each channel with W = 2, 3 or 4 taps, forward, backward and single tokens, and its C ABI
// (include/hla2.h, hla2_short_conv_*):
//   p_t = bias + sum_j w_j x_{t - W + 1 + j},  y_t = act(p_t)
//   dp = dy act'(p),  dx_s = sum_j w_j dp_{s + W - 1 - j},  dw_j = sum_t dp_t x_{t - W + 1 + j},  dbias = sum_t dp_t.
//
// Bytes are the floor of all of them: x read and y written once, x and dy read and dx written in the backward, which forms p again.
// A thread has one vector of channels and walks over a run of tokens with the last W - 1 inputs (and dp's) in registers,
// several tokens' loads ahead; the runs' edges are read twice.  The backward's sums of a thread go through shared memory to
// one partial row a CTA, which a second kernel adds in a fixed order.
//
// 65536 x 2048 bf16, W = 4: 93 us (5.7 TB/s, 85 % of the measured copy).  Four tokens a block without conditions, the inputs of a block
// in place instead of a window that moves: 132 us before, with 35 instructions for two values instead of 16.  Backward of 8 x 4096 x 2048,
// bf16: 102 us (4.0 TB/s), 100 of them this kernel, at two CTAs an SM (137 with one, 325 with three): 128 registers of which W = 4 spills
// 88 bytes (164 read back), float32 252 (588; W = 3 84 and 204), and 2.0 warp instructions a cycle and SM at 14 warps (float32 1.3).
#include <type_traits>

#include "packed.cuh"
#include "rows.h"

namespace hla2 {
namespace {

struct ConvPass {
    int B, n, D, W, silu;
    int cols, run, runs;  // vectors of a row, tokens of a run, runs of a sequence
    long long x_sb, x_sn, o_sb, o_sn, g_sb, g_sn;
    const void *x, *weight, *bias, *init;
    const int* lengths;
    void* out;    // y, or dx
    void* fin;    // the state after the last token, or the gradient of the one before the first
    const void *dout, *dfinal;
    float* partial;  // [rows][D][W + 1]
};

constexpr int kAhead = 4;  // tokens of a block, whose loads go out while the block before is worked on

__device__ __forceinline__ int length_of(const int* lengths, int b, int n) {
    return lengths ? max(0, min(__ldg(lengths + b), n)) : n;
}

// A thread's channels: VEC side by side, moved as a vector, or at odd widths and places (APART) two that are 32 apart, so that a warp
// moves 32 neighbours with each single element.  Either way they are worked on as pairs.  (One channel a thread at odd widths: bf16 8 x
// 4096 x 2047 92 us and with gradients 245, 74 and 226 so; a step of 256 x 4095 12.5 and 8.5.  Four channels 32 apart: 70, 213 and 8.5,
// but 1.5 us more in calls of 10, and spills in the gradients.  Four neighbours moved one by one: 153 and 418.)
template <typename T, int VEC, bool APART>
struct ConvChannels {
    static constexpr int N = VEC / 2, step = APART ? 32 : 1;
    using Raw = Vec<T, VEC>;
    explicit __device__ __forceinline__ ConvChannels(int) {}
    // the first channel of thread q of a row
    static __device__ __forceinline__ int first(int q) { return q * VEC; }
    __device__ __forceinline__ Raw load(const T* p) const { return ldvec<T, VEC>(p); }
    __device__ __forceinline__ void store(T* p, const Raw& a) const { *reinterpret_cast<Raw*>(p) = a; }
    __device__ __forceinline__ void store(T* p, const F2 (&f)[N]) const { stvec<T, VEC>(p, f); }
    static __device__ __forceinline__ void values(const Raw& a, F2 (&f)[N]) { unpack(a, f); }
    // the weights of each tap; a channel's lie side by side
    template <int W>
    __device__ __forceinline__ void taps(const T* w, F2 (&t)[W][N]) const {
        float f[VEC * W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            F2 v[N];
            unpack(ldvec<T, VEC>(w + k * VEC), v);
#pragma unroll
            for (int i = 0; i < N; ++i) split(v[i], f[k * VEC + 2 * i], f[k * VEC + 2 * i + 1]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) t[j][i] = pair(f[2 * i * W + j], f[(2 * i + 1) * W + j]);
    }
};
template <typename T, int VEC>
struct ConvChannels<T, VEC, true> {
    static constexpr int N = VEC / 2, step = 32;
    struct Raw {  // as they come, so that nothing waits for them
        T e[VEC];
    };
    int at[VEC];  // of each from the first; those that are not there read it again
    int count;    // channels from the first on
    explicit __device__ __forceinline__ ConvChannels(int count) : count(count) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) at[k] = 32 * k < count ? 32 * k : 0;
    }
    static __device__ __forceinline__ int first(int q) { return q / 32 * (32 * VEC) + q % 32; }
    __device__ __forceinline__ Raw load(const T* p) const {
        Raw r;
#pragma unroll
        for (int k = 0; k < VEC; ++k) r.e[k] = p[at[k]];
        return r;
    }
    __device__ __forceinline__ void store(T* p, const Raw& a) const {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (32 * k < count) p[32 * k] = a.e[k];
    }
    __device__ __forceinline__ void store(T* p, const F2 (&f)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float lo, hi;
            split(f[i], lo, hi);
            if (64 * i < count) p[64 * i] = from_f32<T>(lo);
            if (64 * i + 32 < count) p[64 * i + 32] = from_f32<T>(hi);
        }
    }
    static __device__ __forceinline__ void values(const Raw& a, F2 (&f)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = pair(to_f32(a.e[2 * i]), to_f32(a.e[2 * i + 1]));
    }
    template <int W>
    __device__ __forceinline__ void taps(const T* w, F2 (&t)[W][N]) const {
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) t[j][i] = pair(to_f32(w[at[2 * i] * W + j]), to_f32(w[at[2 * i + 1] * W + j]));
    }
};

template <typename T, int VEC, bool APART, int W>
__global__ void __launch_bounds__(128, 4) conv_kernel(const ConvPass a) {
    using C = ConvChannels<T, VEC, APART>;
    using P = F2;
    constexpr int N = C::N, U = kAhead;
    pdl_wait();
    const long long i0 = (long long)blockIdx.x * 128 + threadIdx.x, i1 = i0 / a.cols;
    const int c = C::first((int)(i0 - i1 * a.cols)), b = (int)(i1 / a.runs), run = (int)(i1 - (long long)b * a.runs);
    if (b >= a.B || c >= a.D) return;
    const C mine(a.D - c);
    const int len = length_of(a.lengths, b, a.n);
    const int t0 = run * a.run, t1 = min(t0 + a.run, a.n);
    const T* x = static_cast<const T*>(a.x) + b * a.x_sb + c;
    T* out = static_cast<T*>(a.out) + b * a.o_sb + c;
    const T* init = a.init ? static_cast<const T*>(a.init) + (long long)b * (W - 1) * a.D + c : nullptr;
    auto input = [&](int t) {  // at a token that may be before the first, as the state has it
        typename C::Raw v{};
        if (t >= 0) v = mine.load(x + t * a.x_sn);
        else if (init) v = mine.load(init + (long long)(t + W - 1) * a.D);
        return v;
    };
    P taps[W][N], bias[N], in[W - 1 + U][N];  // in: the last W - 1 inputs, and those of a block
    mine.template taps<W>(static_cast<const T*>(a.weight) + (long long)c * W, taps);
#pragma unroll
    for (int i = 0; i < N; ++i) bias[i] = pair(0.f, 0.f);
    if (a.bias) C::values(mine.load(static_cast<const T*>(a.bias) + c), bias);
    if (t0 < len) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) C::values(input(t0 - (W - 1) + j), in[j]);
    }
    const int live = min(len, t1);
    typename C::Raw next[U];
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < live) next[u] = mine.load(x + (t + u) * a.x_sn);
    };
    // U tokens from t on; `whole`: all of them are there
    auto block = [&](int t, auto whole) {
        constexpr bool all = decltype(whole)::value;
#pragma unroll
        for (int u = 0; u < U; ++u) C::values(next[u], in[W - 1 + u]);
        fetch(t + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!all && t + u >= live) break;
            P y[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                y[i] = bias[i];
#pragma unroll
                for (int j = 0; j < W; ++j) y[i] = fma_(taps[j][i], in[u + j][i], y[i]);
                P slope;
                if (a.silu) y[i] = gate_of(y[i], true, slope);
            }
            mine.store(out + (t + u) * a.o_sn, y);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) in[j][i] = in[U + j][i];
    };
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = typename C::Raw{};
    fetch(t0);
    int t = t0;
    for (; t + U <= live; t += U) block(t, std::true_type{});
    if (t < live) block(t, std::false_type{});
    P zero[N];
#pragma unroll
    for (int i = 0; i < N; ++i) zero[i] = pair(0.f, 0.f);
    for (t = max(t0, live); t < t1; ++t) mine.store(out + t * a.o_sn, zero);
    pdl_trigger();
    if (run == 0 && a.fin) {
        T* fin = static_cast<T*>(a.fin) + (long long)b * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            mine.store(fin + (long long)j * a.D, input(len - (W - 1) + j));
    }
}

// Eight runs a CTA at a time, 32 vectors of channels
template <typename T, int VEC, bool APART, int W>
__global__ void __launch_bounds__(256, 2) conv_backward_kernel(const ConvPass a, int rows) {
    using C = ConvChannels<T, VEC, APART>;
    using P = F2;
    constexpr int N = C::N;
    __shared__ float sums[8][32 * VEC + 1];
    pdl_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = C::first(blockIdx.y * 32 + lane), per_b = (a.runs + 7) / 8;
    const C mine(a.D - c);
    P taps[W][N], bias[N], dw[W][N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        bias[i] = db[i] = pair(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = pair(0.f, 0.f);
    }
    if (c < a.D) {
        mine.template taps<W>(static_cast<const T*>(a.weight) + (long long)c * W, taps);
        if (a.bias) C::values(mine.load(static_cast<const T*>(a.bias) + c), bias);
    }
    for (int row = blockIdx.x; row < rows; row += gridDim.x) {
        const int b = row / per_b, run = (row - b * per_b) * 8 + w;
        if (c >= a.D || run >= a.runs) continue;
        const int len = length_of(a.lengths, b, a.n), t0 = run * a.run, t1 = min(t0 + a.run, a.n);
        const T *x = static_cast<const T*>(a.x) + b * a.x_sb + c, *dout = static_cast<const T*>(a.dout) + b * a.g_sb + c;
        T* dx = static_cast<T*>(a.out) + b * a.o_sb + c;
        const long long at = (long long)b * (W - 1) * a.D + c;
        const T *init = a.init ? static_cast<const T*>(a.init) + at : nullptr,
                *dfin = a.dfinal ? static_cast<const T*>(a.dfinal) + at : nullptr;
        T* dinit = a.fin ? static_cast<T*>(a.fin) + at : nullptr;
        constexpr int U = kAhead;
        P in[W - 1 + U][N], dp[W - 1 + U][N];  // inputs and dp's: the last W - 1, and those of a block
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) in[j][i] = dp[j][i] = pair(0.f, 0.f);
        if (t0 < len) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const int t = t0 - (W - 1) + j;
                if (t >= 0) C::values(mine.load(x + t * a.x_sn), in[j]);
                else if (init) C::values(mine.load(init + (long long)(t + W - 1) * a.D), in[j]);
            }
        }
        // dx_s is there with dp_t, t = s + W - 1
        const int first = run == 0 ? -(W - 1) : t0, last = t1 + W - 1, live = min(len, last);
        // the sums take this run's valid tokens: one past the length would add 0 times inputs before it, which may be infinite
        const int own_end = min(t1, live);
        typename C::Raw vx[U], vg[U];
        auto fetch = [&](int t) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < live) vx[u] = mine.load(x + (t + u) * a.x_sn), vg[u] = mine.load(dout + (t + u) * a.g_sn);
        };
        // U tokens from t on; `inner`: all of them are this run's own, and so are the dx's
        auto block = [&](int t, auto inner) {
            constexpr bool all = decltype(inner)::value;
            P g[U][N];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                C::values(vx[u], in[W - 1 + u]);
                C::values(vg[u], g[u]);
                if (!all && t + u >= live) {
#pragma unroll
                    for (int i = 0; i < N; ++i) in[W - 1 + u][i] = g[u][i] = pair(0.f, 0.f);
                }
            }
            fetch(t + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool own = all || t + u < own_end;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    P p = bias[i], slope = pair(1.f, 1.f);
                    if (a.silu) {
#pragma unroll
                        for (int j = 0; j < W; ++j) p = fma_(taps[j][i], in[u + j][i], p);
                        gate_of(p, true, slope);
                    }
                    const P d = !all && t + u >= live ? pair(0.f, 0.f) : g[u][i] * slope;
                    dp[W - 1 + u][i] = d;
                    if (own) {
                        db[i] = fma_(d, pair(1.f, 1.f), db[i]);
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][i] = fma_(d, in[u + j][i], dw[j][i]);
                    }
                }
                const int s = t + u - (W - 1);
                if (!all && (s < first || s >= t1)) continue;
                P o[N];
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = taps[0][i] * dp[W - 1 + u][i];
                if (!all) {
                    const int k = s - (len - (W - 1));  // its place in the state after the last token
                    if (dfin && k >= 0 && s < len) {
                        P f[N];
                        C::values(mine.load(dfin + (long long)k * a.D), f);
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = fma_(f[i], pair(1.f, 1.f), o[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 1; j < W; ++j) o[i] = fma_(taps[j][i], dp[W - 1 + u - j][i], o[i]);
                if (!all && s >= len) {
#pragma unroll
                    for (int i = 0; i < N; ++i) o[i] = pair(0.f, 0.f);
                }
                if (all || s >= 0) mine.store(dx + s * a.o_sn, o);
                else if (dinit) mine.store(dinit + (long long)(s + W - 1) * a.D, o);
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < N; ++i) in[j][i] = in[U + j][i], dp[j][i] = dp[U + j][i];
        };
#pragma unroll
        for (int u = 0; u < U; ++u) vx[u] = vg[u] = typename C::Raw{};
        fetch(t0);
        block(t0, std::false_type{});
        int t = t0 + U;
        for (; t + U <= min(live, t1); t += U) block(t, std::true_type{});
        for (; t < last; t += U) block(t, std::false_type{});
    }
    pdl_trigger();
    // the eight runs' sums, one tap after another
    float* dst = a.partial + (long long)blockIdx.x * a.D * (W + 1);
#pragma unroll
    for (int j = 0; j <= W; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float lo, hi;
            split(j < W ? dw[j < W ? j : 0][i / 2] : db[i / 2], lo, hi);
            sums[w][i * 32 + lane] = i % 2 ? hi : lo;
        }
        __syncthreads();
        for (int k = threadIdx.x; k < 32 * VEC; k += 256) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r) s += sums[r][k];
            const int ch = C::first(blockIdx.y * 32 + k % 32) + k / 32 * C::step;
            if (ch < a.D) dst[(long long)j * a.D + ch] = s;
        }
        __syncthreads();
    }
}

// dweight [D, W] and dbias [D]: the partial rows [W + 1][D], 32 columns a CTA with 16 row lanes
__global__ void __launch_bounds__(512) conv_sums_kernel(const ConvPass a, int rows, float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float sm[16][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long cols = (long long)a.D * (a.W + 1), c = (long long)blockIdx.x * 32 + lane;
    pdl_wait();
    float s = 0.f;
    if (c < cols) {
#pragma unroll 8
        for (int r = w; r < rows; r += 16) s += a.partial[r * cols + c];
    }
    sm[w][lane] = s;
    __syncthreads();
    for (int o = 8; o; o >>= 1) {
        if (w < o) sm[w][lane] += sm[w + o][lane];
        __syncthreads();
    }
    if (w || c >= cols) return;
    const int j = (int)(c / a.D), d = (int)(c - (long long)j * a.D);
    if (j < a.W) dweight[(long long)d * a.W + j] = sm[0][lane];
    else if (dbias) dbias[d] = sm[0][lane];
}

// One token: the state moves up by one
template <typename T, int VEC, bool APART, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvPass a, T* __restrict__ state) {
    using C = ConvChannels<T, VEC, APART>;
    using P = F2;
    constexpr int N = C::N;
    pdl_trigger();
    pdl_wait();
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    const int b = (int)(i / a.cols), c = C::first((int)(i - (long long)b * a.cols));
    if (b >= a.B || c >= a.D) return;
    const C mine(a.D - c);
    T* st = state + (long long)b * (W - 1) * a.D + c;
    typename C::Raw v[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) v[j] = mine.load(st + (long long)j * a.D);
    v[W - 1] = mine.load(static_cast<const T*>(a.x) + b * a.x_sb + c);
    P taps[W][N], y[N];
    mine.template taps<W>(static_cast<const T*>(a.weight) + (long long)c * W, taps);
#pragma unroll
    for (int k = 0; k < N; ++k) y[k] = pair(0.f, 0.f);
    if (a.bias) C::values(mine.load(static_cast<const T*>(a.bias) + c), y);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        P x[N];
        C::values(v[j], x);
#pragma unroll
        for (int k = 0; k < N; ++k) y[k] = fma_(taps[j][k], x[k], y[k]);
        if (j > 0) mine.store(st + (long long)(j - 1) * a.D, v[j]);
    }
    P slope;
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (a.silu) y[k] = gate_of(y[k], true, slope);
    mine.store(static_cast<T*>(a.out) + b * a.o_sb + c, y);
}

// ---- launch ----------------------------------------------------------------------------------

constexpr int kWide = 8, kWideBack = 4;  // bf16 elements of a vector, forward and backward
constexpr int kApart = 2;                // channels of a thread without vectors

// f(zero of the type, VEC, APART, W) as integral constants: BF_VEC bf16 or 4 float32 channels a thread where the tensors allow vectors
// of them
template <int V> using Int = std::integral_constant<int, V>;
template <int BF_VEC, class F>
int with_conv(int dtype, bool vec, int W, F&& f) {
    auto taps = [&](auto zero, auto v, auto apart) {
        switch (W) {
            case 2: return f(zero, v, apart, Int<2>{});
            case 3: return f(zero, v, apart, Int<3>{});
            default: return f(zero, v, apart, Int<4>{});
        }
    };
    if (dtype == HLA2_BF16) return vec ? taps(bf16{}, Int<BF_VEC>{}, std::false_type{}) : taps(bf16{}, Int<kApart>{}, std::true_type{});
    return vec ? taps(0.f, Int<4>{}, std::false_type{}) : taps(0.f, Int<kApart>{}, std::true_type{});
}

int check_conv(const char* fn, const hla2_conv_args* a) {
    if (!a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: args must not be NULL", fn);
    if (a->dtype != HLA2_F32 && a->dtype != HLA2_BF16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dtype must be HLA2_F32 or HLA2_BF16", fn);
    if (a->B < 0 || a->n < 0 || a->D < 0)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: B, n and D must not be negative", fn);
    if (a->W < 2 || a->W > 4) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: W must be 2, 3 or 4 (got %d)", fn, a->W);
    if (a->silu != 0 && a->silu != 1) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: silu must be 0 or 1", fn);
    // the grids' limits: columns of 64 channels, and rows of at least 64 tokens or a sequence
    if ((long long)a->B * a->D > 0x7fffffffLL || a->D > 1 << 20 || a->n > 1 << 30 || (long long)a->B * ((a->n + 63LL) / 64) > 0x7fffffffLL)
        return set_last_error(HLA2_ERR_UNSUPPORTED, "%s: B * D and B * n / 64 must fit in 31 bits, D be at most 2^20 and n 2^30", fn);
    return HLA2_OK;
}

// Tokens of a run: as many as leave `threads` threads an SM, 8 to 128
int run_of(const hla2_conv_args* a, int vec, int threads) {
    const long long all = (long long)a->B * ((a->D + vec - 1) / vec) * a->n, want = (long long)threads * sm_count();
    const long long run = (all / want + 7) / 8 * 8;
    return run < 8 ? 8 : run > 128 ? 128 : (int)run;
}
// Threads of a row
int conv_cols(const hla2_conv_args* a, bool vec, int wide) { return vec ? a->D / wide : (a->D + 32 * kApart - 1) / (32 * kApart) * 32; }
// The backward's runs, rows of eight of them, and the partial rows of its CTAs, who take several rows where there are more than
// fill the GPU four times (two CTAs an SM): the partial rows would be larger than the inputs with many short sequences.
struct ConvRows {
    int run, runs, rows, partials;
};
ConvRows backward_rows(const hla2_conv_args* a) {
    ConvRows r{};
    r.run = run_of(a, 4, 768);
    r.runs = (int)(((long long)a->n + r.run - 1) / r.run);
    const long long rows = (long long)a->B * ((r.runs + 7) / 8), tiles = (a->D + 127) / 128;
    const long long most = tiles ? (8LL * sm_count() + tiles - 1) / tiles : 0;
    r.rows = (int)rows;
    r.partials = (int)(rows < most ? rows : most);
    return r;
}

struct ConvInputs {
    int es, wide;  // bytes of an element, elements of a vector
    Places read;
    bool vec = true;
    ConvInputs(const hla2_conv_args* a, int bf_vec) : es(elem_size(a->dtype)), wide(es == 2 ? bf_vec : 4), read(es) {}
    // a contiguous tensor, whose vectors are read or written
    void vectors(const void* p, int D) {
        if (p) vec = vec && al(p, wide * es) && D % wide == 0;
    }
    void add(const void* p, size_t elems, int D) {
        read.add(extent_of(p, elems * es));
        vectors(p, D);
    }
    int rows(const char* fn, const Tensor& t, bool written) {
        if (int rc = check_tensor(fn, t, es, written)) return rc;
        vec = vec && t.vec(wide, es);
        if (!written) read.add(t);
        return HLA2_OK;
    }
    int params(const char* fn, const hla2_conv_args* a) {
        if (!a->weight) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: weight must not be NULL", fn);
        if (!al(a->weight, es) || !al(a->bias, es) || !al(a->init_state, es) || !al(a->lengths, 4))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
        add(a->weight, (size_t)a->D * a->W, a->D);
        add(a->bias, a->D, a->D);
        add(a->init_state, (size_t)a->B * (a->W - 1) * a->D, a->D);
        read.add(extent_of(a->lengths, (size_t)a->B * sizeof(int)));
        return HLA2_OK;
    }
};

ConvPass base_pass(const hla2_conv_args* a) {
    ConvPass p{};
    p.B = a->B, p.n = a->n, p.D = a->D, p.W = a->W, p.silu = a->silu;
    p.x = a->x.p, p.weight = a->weight, p.bias = a->bias, p.init = a->init_state;
    p.x_sb = a->x.sb, p.x_sn = a->x.sn;
    p.lengths = a->lengths;
    return p;
}

}  // namespace
}  // namespace hla2

using namespace hla2;

extern "C" {

int hla2_short_conv_forward(const hla2_conv_args* a, hla2_rows out, void* final_state, hla2_stream_t stream) {
    static const char* const fn = "hla2_short_conv_forward";
    Range range(fn);
    if (int rc = check_conv(fn, a)) return rc;
    if (a->B == 0 || a->D == 0) return ok();
    ConvInputs in(a, kWide);
    if (int rc = in.params(fn, a)) return rc;
    const Tensor o = rows("out", out, a->B, a->n, a->D);
    const Extent fin = extent_of(final_state, (size_t)a->B * (a->W - 1) * a->D * in.es);
    if (!al(final_state, in.es)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    in.vectors(final_state, a->D);
    if (a->n > 0) {
        if (int rc = in.rows(fn, rows("x", a->x, a->B, a->n, a->D), false)) return rc;
        if (int rc = in.rows(fn, o, true)) return rc;
        if (in.read.meets(o) || meet(o.extent(in.es), fin))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out overlaps another tensor", fn);
    } else if (!final_state) {
        return ok();
    }
    if (in.read.meets(fin)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: final_state overlaps an input", fn);
    ConvPass p = base_pass(a);
    p.out = const_cast<void*>(out.p), p.o_sb = out.sb, p.o_sn = out.sn;
    p.fin = final_state;
    const int v = in.vec ? in.wide : kApart;
    p.run = run_of(a, v, 1024);
    p.runs = a->n > 0 ? (int)(((long long)a->n + p.run - 1) / p.run) : 1;
    p.cols = conv_cols(a, in.vec, in.wide);
    const long long threads = (long long)p.cols * p.runs * a->B;
    if ((threads + 127) / 128 > 0x7fffffffLL) return set_last_error(HLA2_ERR_UNSUPPORTED, "%s: too many values", fn);
    const int rc = with_conv<kWide>(a->dtype, in.vec, a->W, [&](auto zero, auto vec, auto apart, auto taps) {
        using T = decltype(zero);
        return launch_pdl(conv_kernel<T, decltype(vec)::value, decltype(apart)::value, decltype(taps)::value>, dim3((unsigned)((threads + 127) / 128)),
                          dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), p) == cudaSuccess ? 0 : -1;
    });
    return rc ? launch_failed("short convolution") : ok();
}

size_t hla2_short_conv_backward_workspace_bytes(const hla2_conv_args* a) {
    if (check_conv("hla2_short_conv_backward_workspace_bytes", a) != HLA2_OK) return (size_t)-1;
    ok();
    return (size_t)backward_rows(a).partials * a->D * (a->W + 1) * sizeof(float);
}

int hla2_short_conv_backward(const hla2_conv_args* a, hla2_rows dout, const void* dfinal_state, hla2_rows dx, float* dweight,
                             float* dbias, void* dinit_state, hla2_stream_t stream) {
    static const char* const fn = "hla2_short_conv_backward";
    Range range(fn);
    if (int rc = check_conv(fn, a)) return rc;
    if (a->D == 0) return ok();
    ConvInputs in(a, kWideBack);
    if (int rc = in.params(fn, a)) return rc;
    const size_t state = (size_t)a->B * (a->W - 1) * a->D;
    if (!al(dfinal_state, in.es) || !al(dinit_state, in.es) || !al(dweight, 4) || !al(dbias, 4))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    if (!dweight || (a->bias != nullptr) != (dbias != nullptr))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dweight is needed, dbias with bias, and only then", fn);
    in.add(dfinal_state, state, a->D);
    in.vectors(dinit_state, a->D);
    const Extent written[3] = {extent_of(dweight, (size_t)a->D * a->W * sizeof(float)), extent_of(dbias, (size_t)a->D * sizeof(float)),
                               extent_of(dinit_state, state * in.es)};
    if (a->n > 0 && a->B > 0) {
        if (int rc = in.rows(fn, rows("x", a->x, a->B, a->n, a->D), false)) return rc;
        if (int rc = in.rows(fn, rows("dout", dout, a->B, a->n, a->D), false)) return rc;
        const Tensor o = rows("dx", dx, a->B, a->n, a->D);
        if (int rc = in.rows(fn, o, true)) return rc;
        if (in.read.meets(o)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient overlaps an input", fn);
        for (const Extent& e : written)
            if (meet(e, o.extent(in.es))) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: gradients overlap", fn);
    }
    for (int i = 0; i < 3; ++i) {
        if (in.read.meets(written[i])) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient overlaps an input", fn);
        for (int j = 0; j < i; ++j)
            if (meet(written[i], written[j])) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: gradients overlap", fn);
    }
    const size_t need = hla2_short_conv_backward_workspace_bytes(a);
    if (need > 0 && (!a->workspace || a->workspace_bytes < need || !al(a->workspace, 16)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    ConvPass p = base_pass(a);
    p.out = const_cast<void*>(dx.p), p.o_sb = dx.sb, p.o_sn = dx.sn;
    p.dout = dout.p, p.g_sb = dout.sb, p.g_sn = dout.sn;
    p.fin = dinit_state, p.dfinal = dfinal_state;
    p.partial = static_cast<float*>(a->workspace);
    const ConvRows r = backward_rows(a);
    p.run = r.run, p.runs = r.runs;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    int rc = 0;
    if (r.partials > 0)
        rc = with_conv<kWideBack>(a->dtype, in.vec, a->W, [&](auto zero, auto vec, auto apart, auto taps) {
            using T = decltype(zero);
            constexpr int V = decltype(vec)::value;
            return launch_pdl(conv_backward_kernel<T, V, decltype(apart)::value, decltype(taps)::value>, dim3(r.partials, (a->D + 32 * V - 1) / (32 * V)),
                              dim3(256), 0, st, p, r.rows) == cudaSuccess ? 0 : -1;
        });
    else if (dinit_state && a->B > 0)  // no tokens: the state after the last is the one before the first
        rc = (dfinal_state ? cudaMemcpyAsync(dinit_state, dfinal_state, state * in.es, cudaMemcpyDeviceToDevice, st)
                           : cudaMemsetAsync(dinit_state, 0, state * in.es, st)) == cudaSuccess ? 0 : -1;
    const long long cols = (long long)a->D * (a->W + 1);
    if (rc == 0)
        rc = launch_pdl(conv_sums_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(512), 0, st, p, r.partials, dweight, dbias) == cudaSuccess
                 ? 0 : -1;
    return rc ? launch_failed("short convolution gradients") : ok();
}

int hla2_short_conv_decode_step(const hla2_conv_args* a, void* state, hla2_rows out, hla2_stream_t stream) {
    static const char* const fn = "hla2_short_conv_decode_step";
    Range range(fn);
    hla2_conv_args one;  // n is not looked at
    if (a) one = *a, one.n = 1, a = &one;
    if (int rc = check_conv(fn, a)) return rc;
    if (a->B == 0 || a->D == 0) return ok();
    if (a->lengths || a->init_state)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: lengths and init_state must be NULL", fn);
    ConvInputs in(a, kWide);
    if (int rc = in.params(fn, a)) return rc;
    if (int rc = in.rows(fn, rows("x", a->x, a->B, 1, a->D), false)) return rc;
    const Tensor o = rows("out", out, a->B, 1, a->D);
    if (int rc = in.rows(fn, o, true)) return rc;
    if (!state || !al(state, in.es))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: the state must be an address aligned to its type", fn);
    in.vectors(state, a->D);
    const Extent est = extent_of(state, (size_t)a->B * (a->W - 1) * a->D * in.es);
    if (meet(o.extent(in.es), est) || in.read.meets(o) || in.read.meets(est))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out or the state overlaps another tensor", fn);
    ConvPass p = base_pass(a);
    p.out = const_cast<void*>(out.p), p.o_sb = out.sb;
    p.cols = conv_cols(a, in.vec, in.wide);
    const long long threads = (long long)p.cols * a->B;
    const int rc = with_conv<kWide>(a->dtype, in.vec, a->W, [&](auto zero, auto vec, auto apart, auto taps) {
        using T = decltype(zero);
        return launch_pdl(conv_step_kernel<T, decltype(vec)::value, decltype(apart)::value, decltype(taps)::value>, dim3((unsigned)((threads + 127) / 128)),
                          dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), p, static_cast<T*>(state)) == cudaSuccess ? 0 : -1;
    });
    return rc ? launch_failed("short convolution step") : ok();
}

}  // extern "C"
