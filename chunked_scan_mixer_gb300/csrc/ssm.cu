// The selective scan, forward: per channel d with states n = 0 .. N - 1, and per token t
//   delta = softplus(dt + dt_bias),  h = exp(delta a) h + delta x b,  y = sum_n c h + skip x,  out = y silu(gate).
//
// A CTA (ssm.cuh) walks over the tokens of one segment with its states in registers.  Sixteen tokens at a time are
// staged: delta, delta x and the pairs of b and c in shared memory; x and the gate wait in registers for the output.
// Where the channels alone do not fill the GPU the sequence is cut into segments: a first pass forms each segment's state
// from zero and its sum of steps, and the output pass starts from exp(a sum) of those before (ssm_api.cu has the rule).
#include "ssm.cuh"

namespace hla2 {
namespace {

template <typename T, int V, int N, bool SUMS>
__global__ void __launch_bounds__(SsmShape<N>::threads, 512 / SsmShape<N>::threads) ssm_kernel(const SsmPass p) {
    constexpr int SL = SsmShape<N>::lanes, NT = SsmShape<N>::threads, TT = SsmShape<N>::tokens, CT = kSsmChannels;
    using L = Lanes<V>;
    using P = typename L::P;
    using Sums = LaneRows<N>;
    __shared__ __align__(16) float sd[TT][CT], su[TT][CT], sy[SUMS ? 1 : TT][Sums::token], sb[TT][2 * N], sc[SUMS ? 1 : TT][2 * N],
        sskip[CT], sbias[CT];
    const int tid = threadIdx.x, sl = tid % SL, cg = tid / SL;
    pdl_wait();
    const SsmPlace at(p);
    const int chans = at.cols - 4 * cg;  // of the thread's four, those that there are
    const T *x = static_cast<const T*>(p.x.p) + at.b * p.x.sb + at.c0, *dt = static_cast<const T*>(p.dt.p) + at.b * p.dt.sb + at.c0,
            *z = p.gate.p ? static_cast<const T*>(p.gate.p) + at.b * p.gate.sb + at.c0 : nullptr,
            *b = static_cast<const T*>(p.b.p) + at.b * p.b.sb + at.group * p.b.sh,
            *c = static_cast<const T*>(p.c.p) + at.b * p.c.sb + at.group * p.c.sh;
    T* out = SUMS ? nullptr : static_cast<T*>(const_cast<void*>(p.out.p)) + at.b * p.out.sb + at.c0;
    using Chan = Tile<T, V, TT, CT, NT>;
    using Stat = Tile<T, V, TT, N, NT>;
    Chan xn, dn, xc, zc;
    Stat bn, cn;
    auto fetch = [&](int t0) {
        xn.load(x, p.x.sn, t0, at.live_end, at.cols);
        dn.load(dt, p.dt.sn, t0, at.live_end, at.cols);
        bn.load(b, p.b.sn, t0, at.live_end, N);
        if (!SUMS) cn.load(c, p.c.sn, t0, at.live_end, N);
    };
    fetch(at.t0);
    for (int i = tid; i < CT; i += NT) {
        sskip[i] = p.skip && i < at.cols ? p.skip[at.c0 + i] : 0.f;
        sbias[i] = p.dt_bias && i < at.cols ? p.dt_bias[at.c0 + i] : 0.f;
    }
    SsmState a, h;
    a.load(p.a + (long long)(at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    a.scale(kLog2E);
    h.zero();
    if (!SUMS) {
        if (p.init) h.load(p.init + ((long long)at.b * p.D + at.c0 + 4 * cg) * N + 4 * sl, N, chans);
        join_segments<N>(p, at, h, a, p.sums, cg, 0, at.seg, 1);
    }
    F2 sum01 = pair(0.f, 0.f), sum23 = sum01;
    __syncthreads();
    for (int t0 = at.t0; t0 < at.live_end; t0 += TT) {
        Chan::parts([&](int k, int r, int ch) {
            stage<T, V, false>(xn.v[k], dn.v[k], xn.v[k], xn.v[k], false, p.softplus, t0 + r < at.live_end && ch < at.cols, sbias + ch,
                               &sd[r][ch], &su[r][ch], nullptr);
        });
        Stat::parts([&](int k, int r, int s) {
            P f[L::N];
            unpack(bn.v[k], f);
            put_twice<V>(&sb[r][2 * s], f);
            if (!SUMS) {
                unpack(cn.v[k], f);
                put_twice<V>(&sc[r][2 * s], f);
            }
        });
        if (!SUMS) {
            xc = xn;
            if (z) zc.load(z, p.gate.sn, t0, at.live_end, at.cols);
        }
        fetch(t0 + TT);
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const SsmPair2 d = ld4(&sd[t][4 * cg]), u = ld4(&su[t][4 * cg]);
            F2 y01 = pair(0.f, 0.f), y23 = y01;
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const SsmPair2 bb = ld4(&sb[t][8 * sl + 2 * k]);
                SsmPair2 cc{};
                if (!SUMS) cc = ld4(&sc[t][8 * sl + 2 * k]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    F2(&hk)[2] = h.v[k + j];
                    const F2 bk = j ? bb.hi : bb.lo, ck = j ? cc.hi : cc.lo;
                    hk[0] = fma_(ex2_(d.lo * a.v[k + j][0]), hk[0], u.lo * bk);
                    hk[1] = fma_(ex2_(d.hi * a.v[k + j][1]), hk[1], u.hi * bk);
                    if (!SUMS) y01 = k + j ? fma_(hk[0], ck, y01) : hk[0] * ck, y23 = k + j ? fma_(hk[1], ck, y23) : hk[1] * ck;
                }
            }
            if (SUMS) sum01 = sum01 + d.lo, sum23 = sum23 + d.hi;
            else Sums::put(sy[t], cg, sl, y01, y23);
        }
        __syncthreads();
        if (!SUMS)
            Chan::parts([&](int k, int r, int ch) {
                if (t0 + r >= at.t_end || ch >= at.cols) return;
                P y[L::N], fx[L::N], fs[L::N];
                Sums::template get<V>(&sy[r][ch], y);
                unpack(xc.v[k], fx);
                get_values<V>(sskip + ch, fs);
#pragma unroll
                for (int i = 0; i < L::N; ++i) y[i] = fma_(fs[i], fx[i], y[i]);
                if (z) {
                    unpack(zc.v[k], fx);
#pragma unroll
                    for (int i = 0; i < L::N; ++i) y[i] = times_silu(y[i], fx[i]);
                }
                if (t0 + r >= at.live_end) {
#pragma unroll
                    for (int i = 0; i < L::N; ++i) y[i] = L::all(0.f);
                }
                stvec<T, V>(out + (long long)(t0 + r) * p.out.sn + ch, y);
            });
    }
    pdl_trigger();
    if (SUMS) {
        const long long slot = at.slot(p, at.seg);
        h.put(p.sums + slot * (CT * N), NT);
        if (sl == 0) st4(p.steps + slot * CT + 4 * cg, {sum01, sum23});
        return;
    }
    // padding past the last staged token
    P zero[L::N];
#pragma unroll
    for (int i = 0; i < L::N; ++i) zero[i] = L::all(0.f);
    const int first = at.t0 + (at.live_end - at.t0 + TT - 1) / TT * TT;
    for (long long i = tid; i < (long long)(at.t_end - first) * (CT / V); i += NT) {
        const int t = first + (int)(i / (CT / V)), ch = (int)(i % (CT / V)) * V;
        if (ch < at.cols) stvec<T, V>(out + (long long)t * p.out.sn + ch, zero);
    }
    if (p.fin && at.seg == p.nseg - 1) h.store(p.fin + ((long long)at.b * p.D + at.c0 + 4 * cg) * N + 4 * sl, N, chans);
}

template <typename T, int V, int N>
int forward_n(const SsmPass& p, cudaStream_t st) {
    const dim3 block(SsmShape<N>::threads);
    if (p.nseg > 1 &&
        launch_pdl(ssm_kernel<T, V, N, true>, dim3(p.B * p.G * p.tiles, p.nseg - 1), block, 0, st, p) != cudaSuccess)
        return -1;
    return launch_pdl(ssm_kernel<T, V, N, false>, dim3(p.B * p.G * p.tiles, p.nseg), block, 0, st, p) == cudaSuccess ? 0 : -1;
}
template <typename T, int V>
int forward_v(const SsmPass& p, cudaStream_t st) {
    switch (p.N) {
        case 8: return forward_n<T, V, 8>(p, st);
        case 16: return forward_n<T, V, 16>(p, st);
        case 32: return forward_n<T, V, 32>(p, st);
        case 64: return forward_n<T, V, 64>(p, st);
        default: return -1;
    }
}

// ---- step of single tokens -----------------------------------------------------------------
//
// A thread holds four states of J channels, N / 4 threads apart in a row of blockDim: the state is read and written once,
// all J loads in flight together, and bounds the step.
template <typename T, int V>
__device__ __forceinline__ void four(const T* p, float (&f)[4]) {
    if constexpr (V == 4) {
        F2 a[2];
        unpack(ldvec<T, 4>(p), a);
        split(a[0], f[0], f[1]), split(a[1], f[2], f[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = to_f32(p[k]);
    }
}

template <typename T, int V, int N, int J>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmPass p, float* __restrict__ state) {
    constexpr int SL = N / 4, PC = 256 / SL;  // channels of one round of the CTA
    const int sl = threadIdx.x % SL, row = threadIdx.x / SL;
    const long long rows = (long long)p.B * p.D, first = (long long)blockIdx.x * (PC * J) + row;
    const T *x = static_cast<const T*>(p.x.p), *dt = static_cast<const T*>(p.dt.p), *z = static_cast<const T*>(p.gate.p),
            *b = static_cast<const T*>(p.b.p), *c = static_cast<const T*>(p.c.p);
    T* out = static_cast<T*>(const_cast<void*>(p.out.p));
    pdl_trigger();
    pdl_wait();
    float4 h[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
        if (first + j * PC < rows) h[j] = __ldcs(reinterpret_cast<const float4*>(state + (first + j * PC) * N + 4 * sl));
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const long long i = first + j * PC;
        if (i >= rows) break;  // the same for the lanes of a channel, which alone meet in the sum
        const int s = (int)(i / p.D), d = (int)(i - (long long)s * p.D), g = d / p.per;
        const float xv = to_f32(x[s * p.x.sb + d]), v = to_f32(dt[s * p.dt.sb + d]) + (p.dt_bias ? p.dt_bias[d] : 0.f);
        const float delta = p.softplus ? softplus_of(v) : v, u = delta * xv;
        const float4 a = *reinterpret_cast<const float4*>(p.a + (long long)d * N + 4 * sl);
        const T *bp = b + s * p.b.sb + g * p.b.sh + 4 * sl, *cp = c + s * p.c.sb + g * p.c.sh + 4 * sl;
        float bv[4], cv[4];
        four<T, V>(bp, bv);
        four<T, V>(cp, cv);
        const float e = delta * kLog2E;
        h[j].x = fmaf(fast_exp2(e * a.x), h[j].x, u * bv[0]);
        h[j].y = fmaf(fast_exp2(e * a.y), h[j].y, u * bv[1]);
        h[j].z = fmaf(fast_exp2(e * a.z), h[j].z, u * bv[2]);
        h[j].w = fmaf(fast_exp2(e * a.w), h[j].w, u * bv[3]);
        __stcs(reinterpret_cast<float4*>(state + i * N + 4 * sl), h[j]);
        float y = fmaf(h[j].x, cv[0], h[j].y * cv[1]) + fmaf(h[j].z, cv[2], h[j].w * cv[3]);
        const unsigned lanes = (SL == 32 ? 0xffffffffu : (1u << SL) - 1) << (threadIdx.x & 31 & ~(SL - 1));
#pragma unroll
        for (int m = 1; m < SL; m <<= 1) y += __shfl_xor_sync(lanes, y, m);
        if (sl == 0) {
            y = fmaf(p.skip ? p.skip[d] : 0.f, xv, y);
            if (z) {
                const float gv = to_f32(z[s * p.gate.sb + d]);
                y *= gv * sigmoid_of(gv);
            }
            out[s * p.out.sb + d] = from_f32<T>(y);
        }
    }
}

template <typename T, int V, int N>
int step_n(const SsmPass& p, float* state, cudaStream_t st) {
    constexpr int PC = 256 / (N / 4);
    const long long rows = (long long)p.B * p.D;
    auto go = [&](auto kernel, int j) {
        const long long ctas = (rows + PC * j - 1) / (PC * j);
        return launch_pdl(kernel, dim3((unsigned)ctas), dim3(256), 0, st, p, state) == cudaSuccess ? 0 : -1;
    };
    return rows / PC >= 8LL * 4 * sm_count() ? go(ssm_step_kernel<T, V, N, 4>, 4) : go(ssm_step_kernel<T, V, N, 1>, 1);
}
template <typename T, int V>
int step_v(const SsmPass& p, float* state, cudaStream_t st) {
    switch (p.N) {
        case 8: return step_n<T, V, 8>(p, state, st);
        case 16: return step_n<T, V, 16>(p, state, st);
        case 32: return step_n<T, V, 32>(p, state, st);
        case 64: return step_n<T, V, 64>(p, state, st);
        default: return -1;
    }
}

}  // namespace

int launch_ssm_forward(const SsmPass& p, bool is_bf16, bool vec, cudaStream_t st) {
    if (is_bf16) return vec ? forward_v<bf16, 4>(p, st) : forward_v<bf16, 1>(p, st);
    return vec ? forward_v<float, 4>(p, st) : forward_v<float, 1>(p, st);
}

int launch_ssm_step(const SsmPass& p, float* state, bool is_bf16, bool vec, cudaStream_t st) {
    if (is_bf16) return vec ? step_v<bf16, 4>(p, state, st) : step_v<bf16, 1>(p, state, st);
    return vec ? step_v<float, 4>(p, state, st) : step_v<float, 1>(p, state, st);
}

}  // namespace hla2
