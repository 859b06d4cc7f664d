// The selective scan, forward: per channel d with states n = 0 .. N - 1, and per token t
//   delta = softplus(dt + dt_bias),  h = exp(delta a) h + delta x b,  y = sum_n c h + skip x,  out = y silu(gate).
//
// A CTA (ssm.cuh) walks over the tokens of one segment with its states in registers.  Sixteen tokens at a time are
// staged: delta, delta x and the pairs of b and c in shared memory; x and the gate wait in registers for the output.
// Where the channels alone do not fill the GPU the sequence is cut into segments: a first pass forms each segment's state
// from zero and its sum of steps, and the output pass starts from those before, h before the next = exp(a sum) h + state
// (ssm_api.cu has the rule).
//
// Instructions bound it, not bytes: a state and token take two products, two multiply-adds and an exponential, whose register reads
// alone take half of the time, and a channel and token about 60 instructions more for its step, gate and staging.  4 x 4096
// tokens of 2048 channels, N = 16, bf16: sums 114 us and outputs 188 (2.9e12 states a second; memory alone 40 us, the
// exponentials 57); one segment of 8 x 4096 x 4096 924 us.
#include "ssm.cuh"

namespace hla2 {
namespace {

template <typename T, int M, int N, bool SUMS>
__global__ void __launch_bounds__(SsmShape<N>::threads, 512 / SsmShape<N>::threads) ssm_kernel(const SsmPass p) {
    constexpr int SL = SsmShape<N>::lanes, NT = SsmShape<N>::threads, TT = SsmShape<N>::tokens, CT = kSsmChannels;
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
    using Chan = Tile<T, M, TT, CT, NT>;
    using Stat = Tile<T, M, TT, N, NT>;
    Chan xn, dn, xc, zc;
    Stat bn, cn;
    auto fetch = [&](int t0) {
        xn.template load<false>(x, p.x.sn, t0, at.live_end, at.cols);
        dn.template load<false>(dt, p.dt.sn, t0, at.live_end, at.cols);
        bn.template load<false>(b, p.b.sn, t0, at.live_end, N);
        if (!SUMS) cn.template load<false>(c, p.c.sn, t0, at.live_end, N);
    };
    for (int i = tid; i < CT; i += NT) {
        sskip[i] = p.skip && i < at.cols ? p.skip[at.c0 + i] : 0.f;
        sbias[i] = p.dt_bias && i < at.cols ? p.dt_bias[at.c0 + i] : 0.f;
    }
    SsmState a, h;
    a.load(p.a + (long long)(at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    a.exponents();
    h.zero();
    if (!SUMS) {
        if (p.init) h.load(p.init + ((long long)at.b * p.D + at.c0 + 4 * cg) * N + 4 * sl, N, chans);
        join_segments<N>(p, at, h, a, p.sums, cg, 0, at.seg, 1);
    }
    fetch(at.t0);
    F2 sum01 = pair(0.f, 0.f), sum23 = sum01;
    __syncthreads();
    for (int t0 = at.t0; t0 < at.live_end; t0 += TT) {
        Chan::parts([&](int k, int r, int ch) {
            stage<T, false>(xn.v[k], dn.v[k], xn.v[k], xn.v[k], false, p.softplus, t0 + r < at.live_end && ch < at.cols, sbias + ch,
                               &sd[r][ch], &su[r][ch], nullptr);
        });
        Stat::parts([&](int k, int r, int s) {
            F2 f[2];
            unpack(bn.v[k], f);
            put_twice(&sb[r][2 * s], f);
            if (!SUMS) {
                unpack(cn.v[k], f);
                put_twice(&sc[r][2 * s], f);
            }
        });
        if (!SUMS) {
            xc = xn;
            if (z) zc.template load<false>(z, p.gate.sn, t0, at.live_end, at.cols);
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
                    hk[0] = fma_(decay_of(d.lo, a.v[k + j][0]), hk[0], u.lo * bk);
                    hk[1] = fma_(decay_of(d.hi, a.v[k + j][1]), hk[1], u.hi * bk);
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
                F2 y[2], fx[2], fs[2];
                Sums::get(&sy[r][ch], y);
                unpack(xc.v[k], fx);
                get_values(sskip + ch, fs);
#pragma unroll
                for (int i = 0; i < 2; ++i) y[i] = fma_(fs[i], fx[i], y[i]);
                if (z) {
                    unpack(zc.v[k], fx);
#pragma unroll
                    for (int i = 0; i < 2; ++i) y[i] = times_silu(y[i], fx[i]);
                }
                if (t0 + r >= at.live_end) y[0] = y[1] = pair(0.f, 0.f);
                strow<T, M>(out + (long long)(t0 + r) * p.out.sn + ch, y, at.cols - ch);
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
    const F2 zero[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
    const int first = at.t0 + (at.live_end - at.t0 + TT - 1) / TT * TT;
    for (long long i = tid; i < (long long)(at.t_end - first) * (CT / 4); i += NT) {
        const int t = first + (int)(i / (CT / 4)), ch = (int)(i % (CT / 4)) * 4;
        if (ch < at.cols) strow<T, M>(out + (long long)t * p.out.sn + ch, zero, at.cols - ch);
    }
    if (p.fin && at.seg == p.nseg - 1) h.store(p.fin + ((long long)at.b * p.D + at.c0 + 4 * cg) * N + 4 * sl, N, chans);
}

// ---- the states before the segments ---------------------------------------------------------
//
// A warp has one state of four channels, a thread's sixteen bytes in the sums, and its lanes are segments: 32 at a time, whose
// pairs (decay, sum) join in five steps.  All loads of a batch are in flight together, where a CTA of the output pass that joins the
// segments before it waits for them four at a time.
template <int N>
__global__ void __launch_bounds__(256) ssm_carry_kernel(const SsmPass p, float* __restrict__ rsums, const float* __restrict__ dfinal) {
    constexpr int NT = SsmShape<N>::threads, SL = SsmShape<N>::lanes, CT = kSsmChannels;
    const int lane = threadIdx.x & 31, unit = blockIdx.y * 8 + (threadIdx.x >> 5), k = unit / NT, t = unit % NT;
    const int sl = t % SL, cg = t / SL, tiles = p.G * p.tiles, b = blockIdx.x / tiles, tile = blockIdx.x - b * tiles, group = tile / p.tiles;
    const int in = (tile - group * p.tiles) * CT + 4 * cg, ch = group * p.per + in;
    const bool rev = blockIdx.z;
    float* sums = (rev ? rsums : p.sums) + ((long long)k * NT + t) * 4;
    const float* from = rev ? dfinal : p.init;
    pdl_wait();
    float a[4], h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool on = in + j < p.per;
        const long long at = (long long)(ch + j) * N + 4 * sl + k;
        a[j] = on ? exponent_of(p.a[at]) : 0.f;
        h[j] = on && from ? from[(long long)b * p.D * N + at] : 0.f;
    }
    for (int first = 0; first < p.nseg; first += 32) {
        const int i = first + lane, seg = rev ? p.nseg - 1 - i : i;
        const long long slot = (long long)blockIdx.x * p.nseg + seg;
        float d[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
        if (i < p.nseg - 1) {  // nothing comes after the last
            const float4 v = *reinterpret_cast<const float4*>(sums + slot * (CT * N));
            const float4 steps = *reinterpret_cast<const float4*>(p.steps + slot * CT + 4 * cg);
            s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
            d[0] = fast_exp2(steps.x * a[0]), d[1] = fast_exp2(steps.y * a[1]), d[2] = fast_exp2(steps.z * a[2]), d[3] = fast_exp2(steps.w * a[3]);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float pd = __shfl_up_sync(0xffffffffu, d[j], o), ps = __shfl_up_sync(0xffffffffu, s[j], o);
                if (lane >= o) s[j] = fmaf(d[j], ps, s[j]), d[j] *= pd;
            }
        float start[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float pd = __shfl_up_sync(0xffffffffu, d[j], 1), ps = __shfl_up_sync(0xffffffffu, s[j], 1);
            start[j] = lane ? fmaf(pd, h[j], ps) : h[j];
            h[j] = fmaf(__shfl_sync(0xffffffffu, d[j], 31), h[j], __shfl_sync(0xffffffffu, s[j], 31));
        }
        if (i < p.nseg) *reinterpret_cast<float4*>(sums + slot * (CT * N)) = make_float4(start[0], start[1], start[2], start[3]);
    }
    pdl_trigger();
}

template <typename T, int M, int N>
int forward_n(const SsmPass& p, cudaStream_t st) {
    const dim3 block(SsmShape<N>::threads);
    if (p.nseg > 1 &&
        (launch_pdl(ssm_kernel<T, M, N, true>, dim3(p.B * p.G * p.tiles, p.nseg - 1), block, 0, st, p) != cudaSuccess ||
         (p.nseg > kSsmJoin && launch_ssm_carry(p, nullptr, nullptr, st))))
        return -1;
    return launch_pdl(ssm_kernel<T, M, N, false>, dim3(p.B * p.G * p.tiles, p.nseg), block, 0, st, p) == cudaSuccess ? 0 : -1;
}
template <typename T, int M>
int forward_v(const SsmPass& p, cudaStream_t st) {
    switch (p.N) {
        case 8: return forward_n<T, M, 8>(p, st);
        case 16: return forward_n<T, M, 16>(p, st);
        case 32: return forward_n<T, M, 32>(p, st);
        case 64: return forward_n<T, M, 64>(p, st);
        default: return -1;
    }
}

// ---- step of single tokens -----------------------------------------------------------------
//
// A thread holds four states of a channel for Q sequences, so that a is read once for them; the state is read and written
// once, all Q loads in flight together, and bounds the step.  The N / 4 threads of a channel share its elementwise
// values: each forms those of one sequence (of two, where there are two threads) and hands them round, and the sums over the
// states come back to it.  (256 x 4096, N = 16: 40 us with every thread on its own, 22.3 so, 6.4 TB/s.)
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

template <typename T, int V, int N, int Q>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmPass p, float* __restrict__ state) {
    constexpr int SL = N / 4, PC = 256 / SL, LQ = SL < 4 ? SL : 4;  // channels of the CTA; lanes with sequences of their own
    constexpr int own = Q >= LQ ? Q / LQ : 1;
    const int sl = threadIdx.x % SL, d = blockIdx.x * PC + threadIdx.x / SL, s0 = blockIdx.y * Q;
    const T *x = static_cast<const T*>(p.x.p), *dt = static_cast<const T*>(p.dt.p), *z = static_cast<const T*>(p.gate.p),
            *b = static_cast<const T*>(p.b.p), *c = static_cast<const T*>(p.c.p);
    T* out = static_cast<T*>(const_cast<void*>(p.out.p));
    pdl_trigger();
    pdl_wait();
    const bool on = d < p.D;
    const int dc = on ? d : 0, g = dc / p.per;
    float* st = state + ((long long)s0 * p.D + dc) * N + 4 * sl;
    const long long step = (long long)p.D * N;
    float4 h[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
        if (on && s0 + q < p.B) h[q] = __ldcs(reinterpret_cast<const float4*>(st + q * step));
        else h[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 a = *reinterpret_cast<const float4*>(p.a + (long long)dc * N + 4 * sl);
    a.x = exponent_of(a.x), a.y = exponent_of(a.y), a.z = exponent_of(a.z), a.w = exponent_of(a.w);
    const float skip = p.skip ? p.skip[dc] : 0.f, bias = p.dt_bias ? p.dt_bias[dc] : 0.f;
    // this lane's sequences: lane + LQ m of the Q (all lanes one, where there is one)
    float delta[own], u[own], xv[own], zv[own];
    const int lane = Q == 1 ? 0 : sl % LQ;
#pragma unroll
    for (int m = 0; m < own; ++m) {
        const int s = s0 + lane + LQ * m < p.B ? s0 + lane + LQ * m : s0;
        xv[m] = to_f32(x[s * p.x.sb + dc]);
        const float v = to_f32(dt[s * p.dt.sb + dc]) + bias;
        zv[m] = z ? to_f32(z[s * p.gate.sb + dc]) : 0.f;
        delta[m] = p.softplus ? softplus_of(v) : v;
        u[m] = delta[m] * xv[m];
    }
    float y[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int s = s0 + q < p.B ? s0 + q : s0;
        const float dq = Q == 1 ? delta[0] : __shfl_sync(0xffffffffu, delta[q / LQ], q % LQ, SL);
        const float uq = Q == 1 ? u[0] : __shfl_sync(0xffffffffu, u[q / LQ], q % LQ, SL);
        float bv[4], cv[4];
        four<T, V>(b + s * p.b.sb + g * p.b.sh + 4 * sl, bv);
        four<T, V>(c + s * p.c.sb + g * p.c.sh + 4 * sl, cv);
        h[q].x = fmaf(decay_of(dq, a.x), h[q].x, uq * bv[0]);
        h[q].y = fmaf(decay_of(dq, a.y), h[q].y, uq * bv[1]);
        h[q].z = fmaf(decay_of(dq, a.z), h[q].z, uq * bv[2]);
        h[q].w = fmaf(decay_of(dq, a.w), h[q].w, uq * bv[3]);
        if (on && s0 + q < p.B) __stcs(reinterpret_cast<float4*>(st + q * step), h[q]);
        y[q] = fmaf(h[q].x, cv[0], h[q].y * cv[1]) + fmaf(h[q].z, cv[2], h[q].w * cv[3]);
    }
    // sums over the lanes, each back to the lane of its sequence
    if constexpr (Q == 4) {
        const bool odd = sl & 1, up = sl & 2;
        float k0 = (odd ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, odd ? y[0] : y[1], 1);
        const float k1 = (odd ? y[3] : y[2]) + __shfl_xor_sync(0xffffffffu, odd ? y[2] : y[3], 1);
        if constexpr (SL == 2) {
            y[0] = k0, y[1] = k1;
        } else {
            k0 = (up ? k1 : k0) + __shfl_xor_sync(0xffffffffu, up ? k0 : k1, 2);
            if constexpr (SL > 4) k0 += __shfl_xor_sync(0xffffffffu, k0, 4);
            if constexpr (SL > 8) k0 += __shfl_xor_sync(0xffffffffu, k0, 8);
            y[0] = k0;
        }
    } else {
#pragma unroll
        for (int m = 1; m < SL; m <<= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], m);
    }
#pragma unroll
    for (int m = 0; m < own; ++m) {
        const int s = s0 + lane + LQ * m;
        if (!on || s >= p.B || (Q == 1 ? sl : sl >= LQ)) continue;
        float o = fmaf(skip, xv[m], y[m]);
        if (z) o = times_silu(o, zv[m]);
        out[s * p.out.sb + d] = from_f32<T>(o);
    }
}

// Four sequences a CTA where there are as many, and CTAs for every SM left
template <typename T, int V, int N>
int step_n(const SsmPass& p, float* state, cudaStream_t st) {
    constexpr int PC = 256 / (N / 4);
    const int tiles = (p.D + PC - 1) / PC;
    auto go = [&](auto kernel, int q) {
        for (SsmPass r = p; r.B > 0;) {  // the grid holds 65535 rows of CTAs
            const int most = 65535 * q, now = r.B < most ? r.B : most;
            SsmPass part = r;
            part.B = now;
            if (launch_pdl(kernel, dim3(tiles, (now + q - 1) / q), dim3(256), 0, st, part, state) != cudaSuccess) return -1;
            r.B -= now;
            auto on = [&](const void*& a, long long sb) {
                if (a) a = static_cast<const T*>(a) + now * sb;
            };
            on(r.x.p, r.x.sb), on(r.dt.p, r.dt.sb), on(r.gate.p, r.gate.sb), on(r.out.p, r.out.sb), on(r.b.p, r.b.sb), on(r.c.p, r.c.sb);
            state += (long long)now * p.D * N;
        }
        return 0;
    };
    return p.B >= 4 && (long long)tiles * (p.B / 4) >= sm_count() ? go(ssm_step_kernel<T, V, N, 4>, 4) : go(ssm_step_kernel<T, V, N, 1>, 1);
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

int launch_ssm_carry(const SsmPass& p, float* rsums, const float* dfinal, cudaStream_t st) {
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(p.B * p.G * p.tiles, 2 * p.N, rsums ? 2 : 1), dim3(256), 0, st, p, rsums, dfinal) == cudaSuccess ? 0 : -1;
    };
    switch (p.N) {
        case 8: return go(ssm_carry_kernel<8>);
        case 16: return go(ssm_carry_kernel<16>);
        case 32: return go(ssm_carry_kernel<32>);
        case 64: return go(ssm_carry_kernel<64>);
        default: return -1;
    }
}

int launch_ssm_forward(const SsmPass& p, bool is_bf16, bool vec, cudaStream_t st) {
    if (is_bf16) return vec ? forward_v<bf16, 4>(p, st) : forward_v<bf16, 1>(p, st);
    return vec ? forward_v<float, 4>(p, st) : forward_v<float, 1>(p, st);
}

int launch_ssm_step(const SsmPass& p, float* state, bool is_bf16, bool vec, cudaStream_t st) {
    if (is_bf16) return vec ? step_v<bf16, 4>(p, state, st) : step_v<bf16, 1>(p, state, st);
    return vec ? step_v<float, 4>(p, state, st) : step_v<float, 1>(p, state, st);
}

}  // namespace hla2
