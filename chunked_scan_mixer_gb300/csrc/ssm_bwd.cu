// The selective scan, backward (the forward is in ssm.cu).  With dy = dout silu(gate) and a_t = exp(delta_t a),
// R_t = c_t dy_t + a_{t+1} R_{t+1} is the gradient of h_t, and per token
//   dc = sum_d h dy,  db = sum_d R delta x,  in = sum_n R b,  E = R a_t h_{t-1},
//   da += E delta,  ddelta = in x + sum_n E a,  ddt = ddelta sigmoid(dt + dt_bias),  dx = in delta + skip dy,
//   dgate = dout (sum_n c h + skip x) silu'(gate),  dskip += x dy,  ddt_bias += ddt.
//
// Nothing is kept from the forward.  A first pass over the segments leaves the state before every sixteen tokens in scratch,
// and with several segments their sums for the states and for R.  The main pass takes sixteen tokens at a time, last ones
// first: it forms the states before each four from the mark, then for four tokens at a time forms the four states again
// into registers and goes back through them.  The products that are summed over states or channels go through
// shared memory: a thread adds its own four, and the others are added column by column, with fewer instructions than
// exchanges between lanes take.  db and dc of a CTA's 64 channels and the parameters' sums go to scratch; two more kernels add
// them in a fixed order.
#include "ssm.cuh"

namespace hla2 {
namespace {

constexpr int kMacro = kSsmTokens;  // tokens between marks
constexpr int kBack = 4;            // tokens whose states are in registers

__device__ __forceinline__ float silu_slope(float z, float s) { return s * fmaf(z, 1.f - s, 1.f); }

// Marks and sums of a segment.  REV: there are several segments, the states start from zero and R's sums are formed too.
template <typename T, int V, int N, bool REV>
__global__ void __launch_bounds__(SsmShape<N>::threads, 512 / SsmShape<N>::threads)
    ssm_marks_kernel(const SsmPass p, const SsmGrads g) {
    constexpr int NT = SsmShape<N>::threads, SL = SsmShape<N>::lanes, TT = SsmShape<N>::tokens, CT = kSsmChannels;
    constexpr int VB = V > N ? N : V;
    __shared__ __align__(16) float sd[TT][CT], su[TT][CT], sy[REV ? TT : 1][CT], sb[TT][2 * N], sc[REV ? TT : 1][2 * N], sbias[CT];
    const int tid = threadIdx.x, sl = tid % SL, cg = tid / SL;
    pdl_wait();
    const SsmPlace at(p);
    const int chans = at.cols - 4 * cg;
    for (int i = tid; i < CT; i += NT) sbias[i] = p.dt_bias && i < at.cols ? p.dt_bias[at.c0 + i] : 0.f;
    SsmState a, h, P, R;
    a.load(p.a + (long long)(at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    a.scale(kLog2E);
    h.zero();
    if (!REV && p.init) h.load(p.init + ((long long)at.b * p.D + at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    R.zero();
#pragma unroll
    for (int k = 0; k < 4; ++k) P.v[k][0] = P.v[k][1] = pair(1.f, 1.f);
    const T *x = static_cast<const T*>(p.x.p) + at.b * p.x.sb + at.c0, *dt = static_cast<const T*>(p.dt.p) + at.b * p.dt.sb + at.c0,
            *z = p.gate.p ? static_cast<const T*>(p.gate.p) + at.b * p.gate.sb + at.c0 : nullptr,
            *dout = static_cast<const T*>(g.dout.p) + at.b * g.dout.sb + at.c0,
            *b = static_cast<const T*>(p.b.p) + at.b * p.b.sb + at.group * p.b.sh,
            *c = static_cast<const T*>(p.c.p) + at.b * p.c.sb + at.group * p.c.sh;
    using Chan = Tile<T, V, TT, CT, NT>;
    using Stat = Tile<T, VB, TT, N, NT>;
    const long long slot = at.slot(p, at.seg);
    F2 sum01 = pair(0.f, 0.f), sum23 = sum01;
    __syncthreads();
    for (int t0 = at.t0; t0 < at.live_end; t0 += TT) {
        const int macro = (t0 - at.t0) / kMacro;
        if ((t0 - at.t0) % kMacro == 0 && macro > 0) {
            h.put(g.marks + (slot * g.macros + macro) * (CT * N), NT);
            if (REV && sl == 0) st4(g.mark_steps + (slot * g.macros + macro) * CT + 4 * cg, {sum01, sum23});
        }
        // the states after the last mark of a lone segment have no reader
        if (!REV && macro == g.macros - 1) break;
        {
            Chan xr, dr, zr, or_;
            Stat br, cr;
            xr.load(x, p.x.sn, t0, at.live_end, at.cols);
            dr.load(dt, p.dt.sn, t0, at.live_end, at.cols);
            br.load(b, p.b.sn, t0, at.live_end, N);
            if (REV) {
                or_.load(dout, g.dout.sn, t0, at.live_end, at.cols);
                if (z) zr.load(z, p.gate.sn, t0, at.live_end, at.cols);
                cr.load(c, p.c.sn, t0, at.live_end, N);
            }
            Chan::parts([&](int k, int r, int ch) {
                const bool on = t0 + r < at.live_end && ch < at.cols;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = to_f32(dr.v[k].v[i]) + sbias[ch + i];
                    const float d = on ? p.softplus ? softplus_of(v) : v : 0.f;
                    sd[r][ch + i] = d;
                    su[r][ch + i] = d * to_f32(xr.v[k].v[i]);
                    if (REV) {
                        float dy = to_f32(or_.v[k].v[i]);
                        if (z) {
                            const float gv = to_f32(zr.v[k].v[i]);
                            dy *= gv * sigmoid_of(gv);
                        }
                        sy[r][ch + i] = dy;
                    }
                }
            });
            Stat::parts([&](int k, int r, int s) {
#pragma unroll
                for (int i = 0; i < VB; ++i) {
                    const float fb = to_f32(br.v[k].v[i]);
                    *reinterpret_cast<float2*>(&sb[r][2 * (s + i)]) = make_float2(fb, fb);
                    if (REV) {
                        const float fc = to_f32(cr.v[k].v[i]);
                        *reinterpret_cast<float2*>(&sc[r][2 * (s + i)]) = make_float2(fc, fc);
                    }
                }
            });
        }
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const SsmPair2 d = ld4(&sd[t][4 * cg]), u = ld4(&su[t][4 * cg]);
            SsmPair2 dy{};
            if (REV) dy = ld4(&sy[t][4 * cg]);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const SsmPair2 bb = ld4(&sb[t][8 * sl + 2 * k]);
                SsmPair2 cc{};
                if (REV) cc = ld4(&sc[t][8 * sl + 2 * k]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const F2 bk = j ? bb.hi : bb.lo, ck = j ? cc.hi : cc.lo;
                    const F2 e0 = ex2_(d.lo * a.v[k + j][0]), e1 = ex2_(d.hi * a.v[k + j][1]);
                    h.v[k + j][0] = fma_(e0, h.v[k + j][0], u.lo * bk);
                    h.v[k + j][1] = fma_(e1, h.v[k + j][1], u.hi * bk);
                    if (REV) {
                        P.v[k + j][0] = P.v[k + j][0] * e0;
                        P.v[k + j][1] = P.v[k + j][1] * e1;
                        R.v[k + j][0] = fma_(P.v[k + j][0], dy.lo * ck, R.v[k + j][0]);
                        R.v[k + j][1] = fma_(P.v[k + j][1], dy.hi * ck, R.v[k + j][1]);
                    }
                }
            }
            if (REV) sum01 = sum01 + d.lo, sum23 = sum23 + d.hi;
        }
        __syncthreads();
    }
    pdl_trigger();
    if (REV) {
        h.put(p.sums + slot * (CT * N), NT);
        R.put(g.rsums + slot * (CT * N), NT);
        if (sl == 0) st4(p.steps + slot * CT + 4 * cg, {sum01, sum23});
    }
}

// Shared memory of the main pass, in floats
template <int N>
struct BackSmem {
    static constexpr int threads = SsmShape<N>::threads;
    static constexpr int d = 0, u = d + kMacro * kSsmChannels, y = u + kMacro * kSsmChannels, b = y + kMacro * kSsmChannels,
                         c = b + kMacro * 2 * N, states = c + kMacro * 2 * N,
                         // the segment's first state, and those before each four tokens but the last
                         sums = states + kMacro / kBack * threads * 16,
                         // five values of four from each thread and token
                         skip = sums + 5 * kBack * threads * 4, bias = skip + kSsmChannels, total = bias + kSsmChannels;
};

template <typename T, int V, int N>
__global__ void __launch_bounds__(SsmShape<N>::threads, 256 / SsmShape<N>::threads)
    ssm_backward_kernel(const SsmPass p, const SsmGrads g) {
    constexpr int NT = SsmShape<N>::threads, SL = SsmShape<N>::lanes, CT = kSsmChannels, MT = kMacro, TC = kBack;
    constexpr int VB = V > N ? N : V, VE = V > 1 ? 4 : 1;  // vectors of the staging of b and c, and of the outputs
    constexpr int items = TC * CT / 4 > NT ? TC * CT / 4 / NT : 1;
    using S = BackSmem<N>;
    extern __shared__ __align__(16) float sm[];
    float *sd = sm + S::d, *su = sm + S::u, *sy = sm + S::y, *sb = sm + S::b, *sc = sm + S::c, *sst = sm + S::states,
          *sskip = sm + S::skip, *sbias = sm + S::bias;
    // [token][thread] four: dc, db of four states; y, in and sum E a of four channels, these as [token][lane][channel]
    float *vdc = sm + S::sums, *vdb = vdc + TC * NT * 4, *vy = vdb + TC * NT * 4, *vin = vy + TC * NT * 4, *ve = vin + TC * NT * 4;
    const int tid = threadIdx.x, sl = tid % SL, cg = tid / SL;
    pdl_wait();
    const SsmPlace at(p);
    const int chans = at.cols - 4 * cg;
    for (int i = tid; i < CT; i += NT) {
        sskip[i] = p.skip && i < at.cols ? p.skip[at.c0 + i] : 0.f;
        sbias[i] = p.dt_bias && i < at.cols ? p.dt_bias[at.c0 + i] : 0.f;
    }
    const long long state_at = ((long long)at.b * p.D + at.c0 + 4 * cg) * N + 4 * sl;
    SsmState a, h, E, da;
    a.load(p.a + (long long)(at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    a.scale(kLog2E);
    da.zero();
    h.zero();
    E.zero();
    if (p.init) h.load(p.init + state_at, N, chans);
    if (g.dfinal) E.load(g.dfinal + state_at, N, chans);
    auto join = [&](SsmState& s, const float* sums, int seg) {
        const long long slot = at.slot(p, seg);
        const SsmPair2 steps = ld4(p.steps + slot * CT + 4 * cg);
        SsmState w;
        w.get(sums + slot * (CT * N), NT);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s.v[k][0] = fma_(ex2_(steps.lo * a.v[k][0]), s.v[k][0], w.v[k][0]);
            s.v[k][1] = fma_(ex2_(steps.hi * a.v[k][1]), s.v[k][1], w.v[k][1]);
        }
    };
    for (int s = 0; s < at.seg; ++s) join(h, p.sums, s);
    for (int s = p.nseg - 1; s > at.seg; --s) join(E, g.rsums, s);
    h.put(sst, NT);
    const T *x = static_cast<const T*>(p.x.p) + at.b * p.x.sb + at.c0, *dt = static_cast<const T*>(p.dt.p) + at.b * p.dt.sb + at.c0,
            *z = p.gate.p ? static_cast<const T*>(p.gate.p) + at.b * p.gate.sb + at.c0 : nullptr,
            *dout = static_cast<const T*>(g.dout.p) + at.b * g.dout.sb + at.c0,
            *b = static_cast<const T*>(p.b.p) + at.b * p.b.sb + at.group * p.b.sh,
            *c = static_cast<const T*>(p.c.p) + at.b * p.c.sb + at.group * p.c.sh;
    auto out = [&](const SsmRows& r) { return static_cast<T*>(const_cast<void*>(r.p)) + at.b * r.sb + at.c0; };
    T *dx = out(g.dx), *ddt = out(g.ddt), *dgate = z ? out(g.dgate) : nullptr;
    using Chan = Tile<T, V, MT, CT, NT>;
    using Stat = Tile<T, VB, MT, N, NT>;
    const long long slot = at.slot(p, at.seg);
    // sums of this thread's items' channels
    float gskip[4] = {0.f, 0.f, 0.f, 0.f}, gbias[4] = {0.f, 0.f, 0.f, 0.f};
    const int quad = tid % (CT / 4) * 4;

    const int macros = (at.live_end - at.t0 + MT - 1) / MT;
    for (int macro = macros - 1; macro >= 0; --macro) {
        const int t0 = at.t0 + macro * MT;
        // the state before these tokens
        if (macro == 0) {
            h.get(sst, NT);
        } else {
            h.get(g.marks + (slot * g.macros + macro) * (CT * N), NT);
            if (p.nseg > 1) {
                const SsmPair2 steps = ld4(g.mark_steps + (slot * g.macros + macro) * CT + 4 * cg);
                SsmState w;
                w.get(sst, NT);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h.v[k][0] = fma_(ex2_(steps.lo * a.v[k][0]), w.v[k][0], h.v[k][0]);
                    h.v[k][1] = fma_(ex2_(steps.hi * a.v[k][1]), w.v[k][1], h.v[k][1]);
                }
            }
        }
        __syncthreads();  // the last macro's readers, and at first sskip and sbias
        {
            Chan xr, dr, zr, or_;
            Stat br, cr;
            xr.load(x, p.x.sn, t0, at.live_end, at.cols);
            dr.load(dt, p.dt.sn, t0, at.live_end, at.cols);
            or_.load(dout, g.dout.sn, t0, at.live_end, at.cols);
            if (z) zr.load(z, p.gate.sn, t0, at.live_end, at.cols);
            br.load(b, p.b.sn, t0, at.live_end, N);
            cr.load(c, p.c.sn, t0, at.live_end, N);
            Chan::parts([&](int k, int r, int ch) {
                const bool on = t0 + r < at.live_end && ch < at.cols;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float v = to_f32(dr.v[k].v[i]) + sbias[ch + i];
                    const float d = on ? p.softplus ? softplus_of(v) : v : 0.f;
                    sd[r * CT + ch + i] = d;
                    su[r * CT + ch + i] = d * to_f32(xr.v[k].v[i]);
                    float dy = to_f32(or_.v[k].v[i]);
                    if (z) {
                        const float gv = to_f32(zr.v[k].v[i]);
                        dy *= gv * sigmoid_of(gv);
                    }
                    sy[r * CT + ch + i] = dy;
                }
            });
            Stat::parts([&](int k, int r, int s) {
#pragma unroll
                for (int i = 0; i < VB; ++i) {
                    const float fb = to_f32(br.v[k].v[i]), fc = to_f32(cr.v[k].v[i]);
                    *reinterpret_cast<float2*>(&sb[r * 2 * N + 2 * (s + i)]) = make_float2(fb, fb);
                    *reinterpret_cast<float2*>(&sc[r * 2 * N + 2 * (s + i)]) = make_float2(fc, fc);
                }
            });
        }
        __syncthreads();
        // the states before each four tokens; the last stays in registers
        for (int t = 0; t < MT - TC; t += TC) {
            h.put(sst + (1 + t / TC) * (NT * 16), NT);
#pragma unroll
            for (int i = 0; i < TC; ++i) {
                const SsmPair2 d = ld4(sd + (t + i) * CT + 4 * cg), u = ld4(su + (t + i) * CT + 4 * cg);
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const SsmPair2 bb = ld4(sb + (t + i) * 2 * N + 8 * sl + 2 * k);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const F2 bk = j ? bb.hi : bb.lo;
                        h.v[k + j][0] = fma_(ex2_(d.lo * a.v[k + j][0]), h.v[k + j][0], u.lo * bk);
                        h.v[k + j][1] = fma_(ex2_(d.hi * a.v[k + j][1]), h.v[k + j][1], u.hi * bk);
                    }
                }
            }
        }
        for (int t = MT - TC; t >= 0; t -= TC) {
            if (t < MT - TC) h.get(sst + (1 + t / TC) * (NT * 16), NT);
            // what the items of these tokens take from memory
            Pack<T, VE> ix[items][4 / VE], id[items][4 / VE], iz[items][4 / VE], io[items][4 / VE];
            auto each_item = [&](auto&& f) {
#pragma unroll
                for (int m = 0; m < items; ++m) {
                    const int i = tid + m * NT, r = i / (CT / 4);
                    if (items == 1 && NT > TC * CT / 4 && i >= TC * CT / 4) continue;
                    f(m, r, t0 + t + r);
                }
            };
            each_item([&](int m, int r, int tok) {
#pragma unroll
                for (int q = 0; q < 4 / VE; ++q) {
                    const int ch = quad + q * VE;
                    if (tok < at.live_end && ch < at.cols) {
                        ix[m][q] = ld_pack<T, VE>(x + (long long)tok * p.x.sn + ch);
                        id[m][q] = ld_pack<T, VE>(dt + (long long)tok * p.dt.sn + ch);
                        if (z) {
                            iz[m][q] = ld_pack<T, VE>(z + (long long)tok * p.gate.sn + ch);
                            io[m][q] = ld_pack<T, VE>(dout + (long long)tok * g.dout.sn + ch);
                        }
                    } else {
                        clear(ix[m][q]), clear(id[m][q]), clear(iz[m][q]), clear(io[m][q]);
                    }
                }
            });
            SsmState kept[TC];  // the states before each of the tokens
#pragma unroll
            for (int i = 0; i < TC; ++i) {
                kept[i] = h;
                const int r = t + i;
                const SsmPair2 d = ld4(sd + r * CT + 4 * cg), u = ld4(su + r * CT + 4 * cg), dy = ld4(sy + r * CT + 4 * cg);
                F2 y01 = pair(0.f, 0.f), y23 = y01;
                float dc[4];
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const SsmPair2 bb = ld4(sb + r * 2 * N + 8 * sl + 2 * k), cc = ld4(sc + r * 2 * N + 8 * sl + 2 * k);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const F2 bk = j ? bb.hi : bb.lo, ck = j ? cc.hi : cc.lo;
                        F2(&hk)[2] = h.v[k + j];
                        hk[0] = fma_(ex2_(d.lo * a.v[k + j][0]), hk[0], u.lo * bk);
                        hk[1] = fma_(ex2_(d.hi * a.v[k + j][1]), hk[1], u.hi * bk);
                        y01 = fma_(hk[0], ck, y01), y23 = fma_(hk[1], ck, y23);
                        dc[k + j] = sum_of(fma_(hk[0], dy.lo, hk[1] * dy.hi));
                    }
                }
                *reinterpret_cast<float4*>(vdc + (i * NT + tid) * 4) = make_float4(dc[0], dc[1], dc[2], dc[3]);
                if (z) st4(vy + (i * SL + sl) * CT + 4 * cg, {y01, y23});
            }
#pragma unroll
            for (int i = TC - 1; i >= 0; --i) {
                const int r = t + i;
                const SsmPair2 d = ld4(sd + r * CT + 4 * cg), u = ld4(su + r * CT + 4 * cg), dy = ld4(sy + r * CT + 4 * cg);
                F2 in01 = pair(0.f, 0.f), in23 = in01, e01 = in01, e23 = in01;
                float db[4];
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const SsmPair2 bb = ld4(sb + r * 2 * N + 8 * sl + 2 * k), cc = ld4(sc + r * 2 * N + 8 * sl + 2 * k);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const F2 bk = j ? bb.hi : bb.lo, ck = j ? cc.hi : cc.lo;
                        F2(&Ek)[2] = E.v[k + j];
                        const F2 R0 = fma_(dy.lo, ck, Ek[0]), R1 = fma_(dy.hi, ck, Ek[1]);
                        db[k + j] = sum_of(fma_(R0, u.lo, R1 * u.hi));
                        in01 = fma_(R0, bk, in01), in23 = fma_(R1, bk, in23);
                        Ek[0] = R0 * ex2_(d.lo * a.v[k + j][0]);
                        Ek[1] = R1 * ex2_(d.hi * a.v[k + j][1]);
                        const F2 q0 = Ek[0] * kept[i].v[k + j][0], q1 = Ek[1] * kept[i].v[k + j][1];
                        da.v[k + j][0] = fma_(q0, d.lo, da.v[k + j][0]);
                        da.v[k + j][1] = fma_(q1, d.hi, da.v[k + j][1]);
                        e01 = fma_(q0, a.v[k + j][0], e01), e23 = fma_(q1, a.v[k + j][1], e23);
                    }
                }
                *reinterpret_cast<float4*>(vdb + (i * NT + tid) * 4) = make_float4(db[0], db[1], db[2], db[3]);
                st4(vin + (i * SL + sl) * CT + 4 * cg, {in01, in23});
                st4(ve + (i * SL + sl) * CT + 4 * cg, {e01, e23});
            }
            __syncthreads();
            // dc and db of these tokens: two threads a column of four states, eight channels' each
            {
                const int col = tid >> 1, lane = col % SL, which = col / SL % 2, r = col / (2 * SL);
                const float* v = (which ? vdc : vdb) + (r * NT + (tid & 1) * SL + lane) * 4;
                SsmPair2 s = ld4(v);
#pragma unroll
                for (int i = 1; i < 8; ++i) {
                    const SsmPair2 w = ld4(v + i * 2 * SL * 4);
                    s.lo = s.lo + w.lo, s.hi = s.hi + w.hi;
                }
                float4 f;
                split(s.lo, f.x, f.y), split(s.hi, f.z, f.w);
                f.x += __shfl_xor_sync(0xffffffffu, f.x, 1), f.y += __shfl_xor_sync(0xffffffffu, f.y, 1);
                f.z += __shfl_xor_sync(0xffffffffu, f.z, 1), f.w += __shfl_xor_sync(0xffffffffu, f.w, 1);
                const int tok = t0 + t + r;
                if (!(tid & 1) && tok < at.live_end)
                    *reinterpret_cast<float4*>(g.bc + (((long long)at.b * p.n + tok) * (p.G * p.tiles) + at.tile) * (2 * N) +
                                               which * N + 4 * lane) = f;
            }
            each_item([&](int m, int r, int tok) {
                float in[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
                auto add = [](float (&s)[4], const float* v) {
                    const float4 f = *reinterpret_cast<const float4*>(v);
                    s[0] += f.x, s[1] += f.y, s[2] += f.z, s[3] += f.w;
                };
#pragma unroll
                for (int l = 0; l < SL; ++l) {
                    add(in, vin + (r * SL + l) * CT + quad);
                    add(e, ve + (r * SL + l) * CT + quad);
                    if (z) add(y, vy + (r * SL + l) * CT + quad);
                }
                if (tok >= at.t_end) return;
                const bool on = tok < at.live_end;
                Pack<T, VE> ox[4 / VE], od[4 / VE], og[4 / VE];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int ch = quad + i;
                    const float xv = to_f32(ix[m][i / VE].v[i % VE]), d = sd[(t + r) * CT + ch], dy = sy[(t + r) * CT + ch];
                    float dd = fmaf(xv, in[i], e[i] * kLn2);
                    if (p.softplus) dd *= sigmoid_of(to_f32(id[m][i / VE].v[i % VE]) + sbias[ch]);
                    dd = on ? dd : 0.f;
                    gbias[i] += dd;
                    gskip[i] = fmaf(xv, dy, gskip[i]);
                    ox[i / VE].v[i % VE] = from_f32<T>(on ? fmaf(d, in[i], sskip[ch] * dy) : 0.f);
                    od[i / VE].v[i % VE] = from_f32<T>(dd);
                    if (z) {
                        const float zv = to_f32(iz[m][i / VE].v[i % VE]), s = sigmoid_of(zv);
                        const float dg = to_f32(io[m][i / VE].v[i % VE]) * fmaf(sskip[ch], xv, y[i]) * silu_slope(zv, s);
                        og[i / VE].v[i % VE] = from_f32<T>(on ? dg : 0.f);
                    }
                }
#pragma unroll
                for (int q = 0; q < 4 / VE; ++q) {
                    const int ch = quad + q * VE;
                    if (ch >= at.cols) continue;
                    *reinterpret_cast<Pack<T, VE>*>(dx + (long long)tok * g.dx.sn + ch) = ox[q];
                    *reinterpret_cast<Pack<T, VE>*>(ddt + (long long)tok * g.ddt.sn + ch) = od[q];
                    if (z) *reinterpret_cast<Pack<T, VE>*>(dgate + (long long)tok * g.dgate.sn + ch) = og[q];
                }
            });
            __syncthreads();
        }
    }
    pdl_trigger();
    if (g.dinit && at.seg == 0) E.store(g.dinit + state_at, N, chans);
    // parts of the parameters' gradients
    const long long row = ((long long)at.b * p.nseg + at.seg) * p.D;
    da.store(g.params + (row + at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    float* per_channel = g.params + (long long)p.B * p.nseg * p.D * N + 2 * row + at.c0;
    // the items of a quad are in threads 16 apart
    constexpr int who = items * NT > TC * CT / 4 ? TC : NT / (CT / 4);
    float* sums = sm + S::sums;
    __syncthreads();
    if (tid < TC * CT / 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sums[(tid / (CT / 4)) * CT + quad + i] = gskip[i];
            sums[(TC + tid / (CT / 4)) * CT + quad + i] = gbias[i];
        }
    }
    __syncthreads();
    for (int i = tid; i < 2 * CT; i += NT) {
        const int which = i / CT, ch = i % CT;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < who; ++k) s += sums[(which * TC + k) * CT + ch];
        if (ch < at.cols) per_channel[(long long)which * p.D + ch] = s;
    }
    // padding past the last tokens gone through
    Pack<T, VE> zero;
    clear(zero);
    const int first = at.t0 + macros * MT;
    for (long long i = tid; i < (long long)(at.t_end - first) * (CT / VE); i += NT) {
        const int tok = first + (int)(i / (CT / VE)), ch = (int)(i % (CT / VE)) * VE;
        if (ch >= at.cols) continue;
        *reinterpret_cast<Pack<T, VE>*>(dx + (long long)tok * g.dx.sn + ch) = zero;
        *reinterpret_cast<Pack<T, VE>*>(ddt + (long long)tok * g.ddt.sn + ch) = zero;
        if (z) *reinterpret_cast<Pack<T, VE>*>(dgate + (long long)tok * g.dgate.sn + ch) = zero;
    }
}

// db and dc: the parts of a group's tiles, four states a thread
template <typename T, int N>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const SsmPass p, const SsmGrads g) {
    constexpr int quads = 2 * N / 4;
    pdl_wait();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, tg = i / quads;
    const int q = (int)(i - tg * quads) * 4, which = q / N, n = q % N;  // db first
    const long long bt = tg / p.G;
    const int gr = (int)(tg - bt * p.G), b = (int)(bt / p.n), t = (int)(bt - (long long)b * p.n);
    if (b >= p.B) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < (p.lengths ? __ldg(p.lengths + b) : p.n)) {
        const float* v = g.bc + tg * p.tiles * (2 * N) + q;
#pragma unroll 8
        for (int k = 0; k < p.tiles; ++k) {
            const float4 f = __ldcs(reinterpret_cast<const float4*>(v + (long long)k * (2 * N)));
            s.x += f.x, s.y += f.y, s.z += f.z, s.w += f.w;
        }
    }
    const hla2_view& o = which ? g.dc : g.db;
    T* d = static_cast<T*>(const_cast<void*>(o.p)) + b * o.sb + gr * o.sh + t * o.sn + n;
    d[0] = from_f32<T>(s.x), d[1] = from_f32<T>(s.y), d[2] = from_f32<T>(s.z), d[3] = from_f32<T>(s.w);
}

// da, dskip and ddt_bias: the parts of the sequences and segments, 32 values a CTA with eight row lanes
__global__ void __launch_bounds__(256) ssm_params_kernel(const SsmPass p, const SsmGrads g) {
    __shared__ float sm[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long cols = (long long)p.D * (p.N + 2), c = (long long)blockIdx.x * 32 + lane;
    const int rows = p.B * p.nseg;
    pdl_wait();
    const long long da = (long long)p.D * p.N;
    float s = 0.f;
    if (c < cols) {
        const float* v = c < da ? g.params + c : g.params + rows * da + (c - da);
        const long long step = c < da ? da : 2LL * p.D;
#pragma unroll 4
        for (int r = w; r < rows; r += 8) s += v[r * step];
    }
    sm[w][lane] = s;
    __syncthreads();
    if (w || c >= cols) return;
    s = ((sm[0][lane] + sm[1][lane]) + (sm[2][lane] + sm[3][lane])) + ((sm[4][lane] + sm[5][lane]) + (sm[6][lane] + sm[7][lane]));
    if (c < da) g.da[c] = s;
    else if (c < da + p.D) { if (g.dskip) g.dskip[c - da] = s; }
    else if (g.ddt_bias) g.ddt_bias[c - da - p.D] = s;
}

template <typename T, int V, int N>
int backward_n(const SsmPass& p, const SsmGrads& g, cudaStream_t st) {
    const long long cols = (long long)p.D * (N + 2), quads = (long long)p.B * p.n * p.G * (2 * N / 4);
    auto params = [&]() {
        return launch_pdl(ssm_params_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, st, p, g) == cudaSuccess ? 0 : -1;
    };
    if (p.B == 0) return params();  // zeros
    const dim3 block(SsmShape<N>::threads), grid(p.B * p.G * p.tiles, p.nseg);
    if (p.nseg > 1) {
        if (launch_pdl(ssm_marks_kernel<T, V, N, true>, grid, block, 0, st, p, g) != cudaSuccess) return -1;
    } else if (g.macros > 1) {
        if (launch_pdl(ssm_marks_kernel<T, V, N, false>, grid, block, 0, st, p, g) != cudaSuccess) return -1;
    }
    auto kernel = ssm_backward_kernel<T, V, N>;
    constexpr size_t smem = BackSmem<N>::total * sizeof(float);
    if (raise_smem(kernel, smem) != cudaSuccess) return -1;
    if (launch_pdl(kernel, grid, block, smem, st, p, g) != cudaSuccess) return -1;
    if (quads > 0 && launch_pdl(ssm_bc_kernel<T, N>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, p, g) != cudaSuccess)
        return -1;
    return params();
}
template <typename T, int V>
int backward_v(const SsmPass& p, const SsmGrads& g, cudaStream_t st) {
    switch (p.N) {
        case 8: return backward_n<T, V, 8>(p, g, st);
        case 16: return backward_n<T, V, 16>(p, g, st);
        case 32: return backward_n<T, V, 32>(p, g, st);
        case 64: return backward_n<T, V, 64>(p, g, st);
        default: return -1;
    }
}

}  // namespace

int launch_ssm_backward(const SsmPass& p, const SsmGrads& g, bool is_bf16, bool vec, cudaStream_t st) {
    if (is_bf16) return vec ? backward_v<bf16, 8>(p, g, st) : backward_v<bf16, 1>(p, g, st);
    return vec ? backward_v<float, 4>(p, g, st) : backward_v<float, 1>(p, g, st);
}

}  // namespace hla2
