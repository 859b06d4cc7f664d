// Shared by the passes of the selective scan (ssm.cu, ssm_bwd.cu): what a pass gets, how a CTA's threads share its
// channels and states, and the values of a token and channel.
#pragma once

#include "packed.cuh"

namespace hla2 {

constexpr int kSsmChannels = 64;  // of a CTA
constexpr int kSsmTokens = 16;    // segments are multiples of it

// One tensor [B, n, D]: address and the element strides of batch and token
struct SsmRows {
    const void* p;
    long long sb, sn;
};

struct SsmPass {
    int B, n, D, N, G;
    int per;           // channels of a group
    int tiles;         // CTAs of a group's channels
    int nseg, seg_tokens;  // segments of the sequence, and their tokens (a multiple of kSsmTokens)
    int softplus;
    SsmRows x, dt, gate, out;
    hla2_view b, c;
    const float *a, *skip, *dt_bias;
    const int* lengths;
    const float* init;
    float* fin;
    float *sums, *steps;  // of the segments: states from zero, and the sums of the steps
};

// What a backward has beside the inputs.  Scratch `marks` and `mark_steps`: the state before each sixteen tokens of a
// segment (from zero where there are several segments) and the sum of the steps up to there.
struct SsmGrads {
    SsmRows dout, dx, ddt, dgate;
    hla2_view db, dc;
    float *da, *dskip, *ddt_bias, *dinit;
    const float* dfinal;
    float *marks, *mark_steps;
    float* rsums;   // of the segments: the gradient of the state before it, from zero after it
    float* bc;      // [B, n, G, tiles, 2 N] the tiles' parts of db and dc
    float* params;  // parts of da [B, segments, D, N], then of dskip and ddt_bias [B, segments, 2, D]
    int macros;     // marks of a segment
};

// Launchers; 0, or -1 where a launch failed.
int launch_ssm_backward(const SsmPass& p, const SsmGrads& g, bool is_bf16, bool vec, cudaStream_t st);
int launch_ssm_forward(const SsmPass& p, bool is_bf16, bool vec, cudaStream_t st);
int launch_ssm_step(const SsmPass& p, float* state, bool is_bf16, bool vec, cudaStream_t st);

namespace {

// A CTA has 64 channels of one group and 4 N threads: thread t holds states 4 (t % (N / 4)) .. + 3 of channels
// 4 (t / (N / 4)) .. + 3.  The channels of a thread are pairs for the packed instructions; b and c are in shared memory
// twice, so that they are pairs there.  Sixteen recurrences a thread hide the latency of each, a token's steps, inputs and
// b, c are read once for them, and a sum over states or channels starts with four in the thread itself.
template <int N>
struct SsmShape {
    static constexpr int lanes = N / 4;  // threads of a channel's states
    static constexpr int threads = kSsmChannels / 4 * lanes;
    static constexpr int tokens = N < 16 ? kSsmTokens / 2 : kSsmTokens;  // staged at a time: 16 values a thread, or fewer
};

struct SsmPair2 {  // four values as pairs
    F2 lo, hi;
};
__device__ __forceinline__ SsmPair2 ld4(const float* p) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    return {{v.x}, {v.y}};
}
__device__ __forceinline__ void st4(float* p, SsmPair2 a) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(a.lo.v, a.hi.v);
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 ex2_(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return pair(fast_exp2(lo), fast_exp2(hi));
}

constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// e^-|x| to about 2^-22 relative: x log2 e in two parts, as its rounding alone would cost |x| 2^-24
__device__ __forceinline__ float exp_neg_abs(float x) {
    const float m = -fabsf(x), t = m * kLog2E;
    if (!(t > -126.f)) return x != x ? x : 0.f;
    const float lo = fmaf(m, 1.925963033500e-8f, fmaf(m, kLog2E, -t));
    const float e = fast_exp2(t);
    return fmaf(e, lo * kLn2, e);
}
// 1 / (1 + e^-x)
__device__ __forceinline__ float sigmoid_of(float x) {
    const float e = exp_neg_abs(x), r = fast_rcp(1.f + e);
    return x < 0.f ? e * r : r;
}
// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x|; log(1 + e) = 2 artanh(s), s = e / (2 + e) <= 1/3, by its series up
// to s^15, which leaves 2e-8 relative.  (log of a rounded 1 + e would lose the small steps that such layers start with.)
__device__ __forceinline__ float softplus_of(float x) {
    const float e = exp_neg_abs(x), s = e * fast_rcp(2.f + e), q = s * s;
    float p = 2.f / 15;
    p = fmaf(p, q, 2.f / 13);
    p = fmaf(p, q, 2.f / 11);
    p = fmaf(p, q, 2.f / 9);
    p = fmaf(p, q, 2.f / 7);
    p = fmaf(p, q, 2.f / 5);
    p = fmaf(p, q, 2.f / 3);
    p = fmaf(p, q, 2.f);
    return fmaf(p, s, x < 0.f ? 0.f : x);
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> ld_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void clear(Pack<T, V>& a) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] = from_f32<T>(0.f);
}

// A thread's parts of `rows` tokens of a tile of `cols` columns, V columns at a time
template <typename T, int V, int ROWS, int COLS, int THREADS>
struct Tile {
    static constexpr int vecs = COLS / V, all = ROWS * vecs, each = (all + THREADS - 1) / THREADS;
    Pack<T, V> v[each];
    // f(k, row, column) for the parts that there are
    template <class F>
    static __device__ __forceinline__ void parts(F&& f) {
#pragma unroll
        for (int k = 0; k < each; ++k) {
            const int i = threadIdx.x + k * THREADS;
            if (all % THREADS == 0 || i < all) f(k, i / vecs, i % vecs * V);
        }
    }
    // rows t0 .. t_end of p, columns up to `cols`; zeros elsewhere
    __device__ __forceinline__ void load(const T* p, long long sn, int t0, int t_end, int cols) {
        parts([&](int k, int r, int c) {
            if (t0 + r < t_end && c < cols) v[k] = ld_pack<T, V>(p + (long long)(t0 + r) * sn + c);
            else clear(v[k]);
        });
    }
};

// Sum over a channel's state lanes of the values of a thread's four channels; lane sl has channel sl % 4's, with two
// lanes both of its two's in r[0], r[1].
template <int SL>
__device__ __forceinline__ void state_sum(F2 a01, F2 a23, int sl, float (&r)[2]) {
    const bool up = SL == 2 ? sl & 1 : sl & 2;
    float g0, g1, k0, k1;
    split(up ? a01 : a23, g0, g1);
    split(up ? a23 : a01, k0, k1);
    constexpr int o = SL == 2 ? 1 : 2;
    k0 += __shfl_xor_sync(0xffffffffu, g0, o);
    k1 += __shfl_xor_sync(0xffffffffu, g1, o);
    if constexpr (SL == 2) {
        r[0] = k0, r[1] = k1;
    } else {
        const bool odd = sl & 1;
        float s = (odd ? k1 : k0) + __shfl_xor_sync(0xffffffffu, odd ? k0 : k1, 1);
#pragma unroll
        for (int m = 4; m < SL; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        r[0] = s;
    }
}
template <int SL>
__device__ __forceinline__ void put_state_sum(float* row, int cg, int sl, const float (&r)[2]) {
    if constexpr (SL == 2) *reinterpret_cast<float2*>(row + 4 * cg + 2 * sl) = make_float2(r[0], r[1]);
    else if (SL == 4 || sl < 4) row[4 * cg + (sl & 3)] = r[0];
}

// The state of a thread's tile: [state][pair of channels]
struct SsmState {
    F2 v[4][2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s][0] = v[s][1] = pair(0.f, 0.f);
    }
    // of [.., D, N] float32, `chans` of the thread's four channels being there
    __device__ __forceinline__ void load(const float* p, int N, int chans) {
        float4 f[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            f[c] = c < chans ? *reinterpret_cast<const float4*>(p + (long long)c * N) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[0][0] = pair(f[0].x, f[1].x), v[0][1] = pair(f[2].x, f[3].x);
        v[1][0] = pair(f[0].y, f[1].y), v[1][1] = pair(f[2].y, f[3].y);
        v[2][0] = pair(f[0].z, f[1].z), v[2][1] = pair(f[2].z, f[3].z);
        v[3][0] = pair(f[0].w, f[1].w), v[3][1] = pair(f[2].w, f[3].w);
    }
    __device__ __forceinline__ void store(float* p, int N, int chans) const {
        float f[4][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) split(v[s][0], f[0][s], f[1][s]), split(v[s][1], f[2][s], f[3][s]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < chans) *reinterpret_cast<float4*>(p + (long long)c * N) = make_float4(f[c][0], f[c][1], f[c][2], f[c][3]);
    }
    // in scratch, a CTA's threads side by side
    __device__ __forceinline__ void get(const float* p, int threads) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const SsmPair2 a = ld4(p + ((long long)s * threads + threadIdx.x) * 4);
            v[s][0] = a.lo, v[s][1] = a.hi;
        }
    }
    __device__ __forceinline__ void put(float* p, int threads) const {
#pragma unroll
        for (int s = 0; s < 4; ++s) st4(p + ((long long)s * threads + threadIdx.x) * 4, {v[s][0], v[s][1]});
    }
    __device__ __forceinline__ void scale(float f) {
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s][0] = v[s][0] * pair(f, f), v[s][1] = v[s][1] * pair(f, f);
    }
};

// Where a CTA stands: blockIdx = (sequence and tile of all groups, segment)
struct SsmPlace {
    int group, tile, c0, cols, b, seg, t0, t_end, live_end;
    __device__ __forceinline__ SsmPlace(const SsmPass& p) {
        const int tiles = p.G * p.tiles;
        b = blockIdx.x / tiles;
        tile = blockIdx.x - b * tiles;
        group = tile / p.tiles;
        const int in = (tile - group * p.tiles) * kSsmChannels;
        c0 = group * p.per + in;
        cols = min(kSsmChannels, p.per - in);
        seg = blockIdx.y;
        t0 = (int)min((long long)seg * p.seg_tokens, (long long)p.n);
        t_end = (int)min((long long)t0 + p.seg_tokens, (long long)p.n);
        const int len = p.lengths ? max(0, min(__ldg(p.lengths + b), p.n)) : p.n;
        live_end = max(t0, min(len, t_end));
    }
    // of this sequence and tile, segment s
    __device__ __forceinline__ long long slot(const SsmPass& p, int s) const { return (long long)blockIdx.x * p.nseg + s; }
};

}  // namespace
}  // namespace hla2
