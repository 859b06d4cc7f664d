// Shared by the passes of the selective scan (ssm.cu, ssm_bwd.cu): what a pass gets, how a CTA's threads share its
// channels and states, and the values of a token and channel.
#pragma once

#include "packed.cuh"

namespace hla2 {

constexpr int kSsmChannels = 64;  // of a CTA
constexpr int kSsmTokens = 16;    // segments are multiples of it
constexpr int kSsmMark = 16;      // tokens between the marks of a backward

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
// The segments' sums become the states before them; with rsums also the gradients of the states after them, dfinal after the last
int launch_ssm_carry(const SsmPass& p, float* rsums, const float* dfinal, cudaStream_t st);
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
template <typename P>
__device__ __forceinline__ P all_(float f) {
    if constexpr (sizeof(P) == sizeof(float)) return f;
    else return pair(f, f);
}
__device__ __forceinline__ float ex2_(float a) { return fast_exp2(a); }
__device__ __forceinline__ F2 ex2_(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return pair(fast_exp2(lo), fast_exp2(hi));
}

constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// a log2(e), finite where a is -inf or as low: the tokens that fill up a tile have delta 0, and 0 times -inf would make their decay NaN
// instead of 1, and a gradient of the step NaN where the decay is 0
__device__ __forceinline__ float exponent_of(float a) {
    float r;
    asm("max.NaN.f32 %0, %1, 0fFF7FFFFF;" : "=f"(r) : "f"(a * kLog2E));
    return r;
}
// A token's decay exp(delta a), from a log2(e).  The instruction's results are a little low: for exponents of -4e-6 .. -2e-3 by 5e-9 to
// 1e-8 on average (measured), which a product over thousands of tokens adds up.  1e-8 more in the exponent leaves 3e-9 there and
// less than before everywhere, and 1 for an exponent of 0.
template <typename P>
__device__ __forceinline__ P decay_of(P delta, P a) {
    return ex2_(fma_(delta, a, all_<P>(1e-8f)));
}

// max(x, 0), NaN where x is
__device__ __forceinline__ float positive_part(float x) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ F2 positive_part(F2 x) {
    float lo, hi;
    split(x, lo, hi);
    return pair(positive_part(lo), positive_part(hi));
}
__device__ __forceinline__ float rcp_(float x) { return fast_rcp(x); }
__device__ __forceinline__ F2 rcp_(F2 x) {
    float lo, hi;
    split(x, lo, hi);
    return pair(fast_rcp(lo), fast_rcp(hi));
}
__device__ __forceinline__ float neg_abs(float x) { return fmaxf(-fabsf(x), -120.f); }
__device__ __forceinline__ F2 neg_abs(F2 x) {
    float lo, hi;
    split(x, lo, hi);
    return pair(neg_abs(lo), neg_abs(hi));
}
__device__ __forceinline__ float ex2_neg(float x) { return fast_exp2(-x); }
__device__ __forceinline__ F2 ex2_neg(F2 x) {
    float lo, hi;
    split(x, lo, hi);
    return pair(fast_exp2(-lo), fast_exp2(-hi));
}

// e^-|x| (e^-120 below that), to 2^-22 + 1.25 2^-24 |x| relative: the unit's error, and |x| log2 e, whose product and constant are rounded
// (softplus_of by it: 2.4e-7 off at most for x above -1, 1.8e-6 down to -40).  P: a float, or a pair of them
template <typename P>
__device__ __forceinline__ P exp_neg_abs(P x) {
    return ex2_neg(neg_abs(x) * all_<P>(-kLog2E));
}
// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x|; log(1 + e) = 2 artanh(s), s = e / (2 + e) <= 1/3: s times a polynomial
// in s^2 fitted to 2 artanh(s) / s over that range, 8e-9 off at most.  (log of a rounded 1 + e would lose the small
// steps that such layers start with.)
template <typename P>
__device__ __forceinline__ P softplus_of(P x) {
    const P e = exp_neg_abs(x), s = e * rcp_(fma_(e, all_<P>(1.f), all_<P>(2.f))), q = s * s;
    P p = all_<P>(0.2817833423614502f);
    p = fma_(p, q, all_<P>(0.27960601449012756f));
    p = fma_(p, q, all_<P>(0.40024909377098083f));
    p = fma_(p, q, all_<P>(0.6666631698608398f));
    p = fma_(p, q, all_<P>(2.f));
    return fma_(p, s, positive_part(x));
}
// 1 / (1 + e^-x)
__device__ __forceinline__ F2 sigmoid_of(F2 x) {
    const F2 e = exp_neg_abs(x), r = rcp_(fma_(e, pair(1.f, 1.f), pair(1.f, 1.f))), er = e * r;
    float x0, x1, r0, r1, e0, e1;
    split(x, x0, x1), split(r, r0, r1), split(er, e0, e1);
    return pair(x0 < 0.f ? e0 : r0, x1 < 0.f ? e1 : r1);
}
// x silu(z)
template <typename P>
__device__ __forceinline__ P times_silu(P x, P z) {
    P slope;
    return x * gate_of(z, true, slope);
}

// Four elements of a row, of which `count` are there (zeros for the others).  M: elements moved at a time, 4 where all of a call's rows
// are aligned to them and its groups' channels a multiple, else 1.  The values are worked on by four either way: with single ones
// bf16 2 x 2048 x 2047 took 149 us, 109 so, and with gradients 550 and 495.
template <typename T, int M>
__device__ __forceinline__ Vec<T, 4> ldrow(const T* p, int count) {
    if constexpr (M == 4) {
        return ldvec<T, 4>(p);
    } else {
        Vec<T, 4> r;
        if constexpr (sizeof(T) == 2) {
            const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
            uint32_t e[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) e[k] = k < count ? q[k] : 0;
            r.v = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
        } else {
            r.v.x = 0 < count ? p[0] : 0.f, r.v.y = 1 < count ? p[1] : 0.f;
            r.v.z = 2 < count ? p[2] : 0.f, r.v.w = 3 < count ? p[3] : 0.f;
        }
        return r;
    }
}
template <typename T, int M>
__device__ __forceinline__ void strow(T* p, const F2 (&v)[2], int count) {
    if constexpr (M == 4) {
        stvec<T, 4>(p, v);
    } else {
        float f[4];
        split(v[0], f[0], f[1]), split(v[1], f[2], f[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < count) p[k] = from_f32<T>(f[k]);
    }
}

// A thread's parts of `rows` tokens of a tile of `cols` columns, four columns at a time
template <typename T, int M, int ROWS, int COLS, int THREADS>
struct Tile {
    static constexpr int vecs = COLS / 4, all = ROWS * vecs, each = (all + THREADS - 1) / THREADS;
    Vec<T, 4> v[each];
    // f(k, row, column) for the parts that there are
    template <class F>
    static __device__ __forceinline__ void parts(F&& f) {
#pragma unroll
        for (int k = 0; k < each; ++k) {
            const int i = threadIdx.x + k * THREADS;
            if (all % THREADS == 0 || i < all) f(k, i / vecs, i % vecs * 4);
        }
    }
    // Rows t0 .. t_end of p, columns up to `cols`; zeros elsewhere.  SPLIT: whole tiles without conditions, a path of its own.  The
    // backward gains by it, 4 x 4096 x 2048 937 -> 910 us; where the loads run ahead of the work, as in the forward, it costs: one
    // segment of 2 x 2048 x 2048 350 -> 360, two 289 -> 340.
    template <bool SPLIT>
    __device__ __forceinline__ void load(const T* p, long long sn, int t0, int t_end, int cols) {
        const T* at = p + t0 * sn;
        if (SPLIT && t0 + ROWS <= t_end && cols == COLS) {  // the same for the whole CTA
            parts([&](int k, int r, int c) { v[k] = ldrow<T, M>(at + r * sn + c, 4); });
        } else {
            parts([&](int k, int r, int c) {
                v[k] = Vec<T, 4>{};
                if (t0 + r < t_end && c < cols) v[k] = ldrow<T, M>(at + r * sn + c, cols - c);
            });
        }
    }
};

// Four values to and from shared memory
__device__ __forceinline__ void put_values(float* p, const F2 (&f)[2]) { st4(p, {f[0], f[1]}); }
__device__ __forceinline__ void get_values(const float* p, F2 (&f)[2]) {
    const SsmPair2 a = ld4(p);
    f[0] = a.lo, f[1] = a.hi;
}
// each of them twice
__device__ __forceinline__ void put_twice(float* p, const F2 (&f)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float lo, hi;
        split(f[i], lo, hi);
        *reinterpret_cast<float4*>(p + 4 * i) = make_float4(lo, lo, hi, hi);
    }
}

// delta, delta x and, with DY, dout silu(gate) of a thread's part of a tile; delta 0 where there is no token or channel (`on`).  Channels
// of such a part that are not there have zeros for x and dout, so that their states and gradients stay zero.
template <typename T, bool DY>
__device__ __forceinline__ void stage(const Vec<T, 4>& x, const Vec<T, 4>& dt, const Vec<T, 4>& dout, const Vec<T, 4>& z, bool gated,
                                      bool softplus, bool on, const float* bias, float* sd, float* su, float* sy) {
    F2 fx[2], v[2], fb[2], d[2], u[2];
    unpack(x, fx);
    unpack(dt, v);
    get_values(bias, fb);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        v[i] = v[i] + fb[i];
        d[i] = !on ? pair(0.f, 0.f) : softplus ? softplus_of(v[i]) : v[i];
        u[i] = d[i] * fx[i];
    }
    put_values(sd, d);
    put_values(su, u);
    if constexpr (DY) {
        F2 g[2], fz[2];
        unpack(dout, g);
        if (gated) {
            unpack(z, fz);
#pragma unroll
            for (int i = 0; i < 2; ++i) g[i] = times_silu(g[i], fz[i]);
        }
        put_values(sy, g);
    }
}

// Sums over the state lanes of a channel go through shared memory: each thread leaves the values of its four channels in a
// row of its lane (of at most four; with more lanes they first exchange halves), and the readers add the rows.  The rows are 8
// floats more than the channels apart, which keeps the writers of two channel groups and four lanes on different banks.
template <int N>
struct LaneRows {
    static constexpr int lanes = SsmShape<N>::lanes, rows = lanes < 4 ? lanes : 4, stride = kSsmChannels + 8, token = rows * stride;
    static __device__ __forceinline__ void put(float* sums, int cg, int sl, F2 a01, F2 a23) {
        if constexpr (lanes <= 4) {
            st4(sums + sl * stride + 4 * cg, {a01, a23});
        } else {
            const bool up = sl & 4;
            float g0, g1, k0, k1;
            split(up ? a01 : a23, g0, g1);
            split(up ? a23 : a01, k0, k1);
            k0 += __shfl_xor_sync(0xffffffffu, g0, 4);
            k1 += __shfl_xor_sync(0xffffffffu, g1, 4);
            float* at = sums + (sl & 3) * stride + 4 * cg + (up ? 2 : 0);
            if constexpr (lanes == 8) {
                *reinterpret_cast<float2*>(at) = make_float2(k0, k1);
            } else {
                const bool second = sl & 8;
                at[second] = (second ? k1 : k0) + __shfl_xor_sync(0xffffffffu, second ? k0 : k1, 8);
            }
        }
    }
    // the sums of four channels
    static __device__ __forceinline__ void get(const float* sums, F2 (&f)[2]) {
        get_values(sums, f);
#pragma unroll
        for (int r = 1; r < rows; ++r) {
            F2 w[2];
            get_values(sums + r * stride, w);
            f[0] = f[0] + w[0], f[1] = f[1] + w[1];
        }
    }
};

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
    // of a, exponents of the decays
    __device__ __forceinline__ void exponents() {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float lo, hi;
                split(v[s][i], lo, hi);
                v[s][i] = pair(exponent_of(lo), exponent_of(hi));
            }
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

// Up to this many segments a CTA joins those before (or after) its own itself; more are joined by a scan of their own, which
// writes each segment's state in the place of its sum.  (2 x 2048 x 2048, forward, 16 segments: 88 us and 93 with the scan; 32: 87
// and 89; 1 x 8192 x 64, 128 segments: 42 and 25, which is 22 with the 256 that it has now.)
constexpr int kSsmJoin = 32;

// The state s before segment `last` from those of the segments between, `first` on in the direction dir: sums from zero of each,
// and its decay exp(a steps).  Four segments' loads are in flight together.
template <int N>
__device__ __forceinline__ void join_segments(const SsmPass& p, const SsmPlace& at, SsmState& s, const SsmState& a, const float* sums,
                                              int cg, int first, int last, int dir) {
    constexpr int NT = SsmShape<N>::threads, CT = kSsmChannels;
    auto step = [&](const SsmPair2& steps, const SsmState& w) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s.v[k][0] = fma_(ex2_(steps.lo * a.v[k][0]), s.v[k][0], w.v[k][0]);
            s.v[k][1] = fma_(ex2_(steps.hi * a.v[k][1]), s.v[k][1], w.v[k][1]);
        }
    };
    int i = first;
    if (p.nseg > kSsmJoin) {
        i = last;
        s.get(sums + at.slot(p, last) * (CT * N), NT);
    }
    for (; (last - i) * dir >= 4; i += 4 * dir) {
        SsmState w[4];
        SsmPair2 steps[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const long long slot = at.slot(p, i + q * dir);
            steps[q] = ld4(p.steps + slot * CT + 4 * cg);
            w[q].get(sums + slot * (CT * N), NT);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) step(steps[q], w[q]);
    }
    for (; i != last; i += dir) {
        const long long slot = at.slot(p, i);
        SsmState w;
        w.get(sums + slot * (CT * N), NT);
        step(ld4(p.steps + slot * CT + 4 * cg), w);
    }
}

}  // namespace
}  // namespace hla2
