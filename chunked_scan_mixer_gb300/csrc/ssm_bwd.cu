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
// exchanges between lanes take.  db and dc of a CTA's 64 channels and the parameters' sums go to scratch; one more kernel adds
// them in a fixed order.
//
// 4 x 4096 tokens of 2048 channels, N = 16, bf16: marks and sums 191 us, main pass 706 (349 instructions for a thread's 16 states of a
// token, 1.7 a cycle and SM with the eight warps that four tokens' states in registers leave room for), parts of db and dc 16 and of
// the parameters 8 before they shared a launch.
#include "ssm.cuh"

namespace hla2 {
namespace {

constexpr int kMacro = kSsmMark;  // tokens between marks
constexpr int kBack = 4;            // tokens whose states are in registers

// Marks and sums of a segment.  REV: there are several segments, the states start from zero and R's sums are formed too.
template <typename T, int M, int N, bool REV>
__global__ void __launch_bounds__(SsmShape<N>::threads, 512 / SsmShape<N>::threads)
    ssm_marks_kernel(const SsmPass p, const SsmGrads g) {
    constexpr int NT = SsmShape<N>::threads, SL = SsmShape<N>::lanes, TT = SsmShape<N>::tokens < kMacro ? SsmShape<N>::tokens : kMacro, CT = kSsmChannels;
    __shared__ __align__(16) float sd[TT][CT], su[TT][CT], sy[REV ? TT : 1][CT], sb[TT][2 * N], sc[REV ? TT : 1][2 * N], sbias[CT];
    const int tid = threadIdx.x, sl = tid % SL, cg = tid / SL;
    pdl_wait();
    const SsmPlace at(p);
    const int chans = at.cols - 4 * cg;
    for (int i = tid; i < CT; i += NT) sbias[i] = p.dt_bias && i < at.cols ? p.dt_bias[at.c0 + i] : 0.f;
    SsmState a, h, W, R;  // W: the decay since the segment's start
    a.load(p.a + (long long)(at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    a.exponents();
    h.zero();
    if (!REV && p.init) h.load(p.init + ((long long)at.b * p.D + at.c0 + 4 * cg) * N + 4 * sl, N, chans);
    R.zero();
#pragma unroll
    for (int k = 0; k < 4; ++k) W.v[k][0] = W.v[k][1] = pair(1.f, 1.f);
    const T *x = static_cast<const T*>(p.x.p) + at.b * p.x.sb + at.c0, *dt = static_cast<const T*>(p.dt.p) + at.b * p.dt.sb + at.c0,
            *z = p.gate.p ? static_cast<const T*>(p.gate.p) + at.b * p.gate.sb + at.c0 : nullptr,
            *dout = static_cast<const T*>(g.dout.p) + at.b * g.dout.sb + at.c0,
            *b = static_cast<const T*>(p.b.p) + at.b * p.b.sb + at.group * p.b.sh,
            *c = static_cast<const T*>(p.c.p) + at.b * p.c.sb + at.group * p.c.sh;
    using Chan = Tile<T, M, TT, CT, NT>;
    using Stat = Tile<T, M, TT, N, NT>;
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
            xr.template load<true>(x, p.x.sn, t0, at.live_end, at.cols);
            dr.template load<true>(dt, p.dt.sn, t0, at.live_end, at.cols);
            br.template load<true>(b, p.b.sn, t0, at.live_end, N);
            if (REV) {
                or_.template load<true>(dout, g.dout.sn, t0, at.live_end, at.cols);
                if (z) zr.template load<true>(z, p.gate.sn, t0, at.live_end, at.cols);
                cr.template load<true>(c, p.c.sn, t0, at.live_end, N);
            }
            Chan::parts([&](int k, int r, int ch) {
                stage<T, REV>(xr.v[k], dr.v[k], or_.v[k], zr.v[k], z, p.softplus, t0 + r < at.live_end && ch < at.cols, sbias + ch,
                                 &sd[r][ch], &su[r][ch], &sy[REV ? r : 0][ch]);
            });
            Stat::parts([&](int k, int r, int n) {
                F2 f[2];
                unpack(br.v[k], f);
                put_twice(&sb[r][2 * n], f);
                if (REV) {
                    unpack(cr.v[k], f);
                    put_twice(&sc[REV ? r : 0][2 * n], f);
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
                    const F2 e0 = decay_of(d.lo, a.v[k + j][0]), e1 = decay_of(d.hi, a.v[k + j][1]);
                    h.v[k + j][0] = fma_(e0, h.v[k + j][0], u.lo * bk);
                    h.v[k + j][1] = fma_(e1, h.v[k + j][1], u.hi * bk);
                    if (REV) {
                        W.v[k + j][0] = W.v[k + j][0] * e0;
                        W.v[k + j][1] = W.v[k + j][1] * e1;
                        R.v[k + j][0] = fma_(W.v[k + j][0], dy.lo * ck, R.v[k + j][0]);
                        R.v[k + j][1] = fma_(W.v[k + j][1], dy.hi * ck, R.v[k + j][1]);
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
    static constexpr int threads = SsmShape<N>::threads, rows = kMacro * kSsmChannels;
    static constexpr int d = 0, u = d + rows, y = u + rows, b = y + rows, c = b + kMacro * 2 * N,
                         // the segment's first state, and those before each four tokens but the last
                         states = c + kMacro * 2 * N,
                         // of four tokens: dc and db of each thread's states, y, in and sum E a by lane rows
                         dc = states + kMacro / kBack * threads * 16, db = dc + kBack * threads * 4, py = db + kBack * threads * 4,
                         in = py + kBack * LaneRows<N>::token, e = in + kBack * LaneRows<N>::token,
                         skip = e + kBack * LaneRows<N>::token, bias = skip + kSsmChannels, total = bias + kSsmChannels;
};

template <typename T, int M, int N>
__global__ void __launch_bounds__(SsmShape<N>::threads, 256 / SsmShape<N>::threads)
    ssm_backward_kernel(const SsmPass p, const SsmGrads g) {
    constexpr int NT = SsmShape<N>::threads, SL = SsmShape<N>::lanes, CT = kSsmChannels, MT = kMacro, TC = kBack;
    using Sums = LaneRows<N>;
    constexpr int items = TC * CT / 4 > NT ? TC * CT / 4 / NT : 1;
    using S = BackSmem<N>;
    extern __shared__ __align__(16) float sm[];
    float *sd = sm + S::d, *su = sm + S::u, *sy = sm + S::y, *sb = sm + S::b, *sc = sm + S::c, *sst = sm + S::states,
          *sskip = sm + S::skip, *sbias = sm + S::bias;
    float *vdc = sm + S::dc, *vdb = sm + S::db, *vy = sm + S::py, *vin = sm + S::in, *ve = sm + S::e;
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
    a.exponents();
    da.zero();
    h.zero();
    E.zero();
    if (p.init) h.load(p.init + state_at, N, chans);
    if (g.dfinal) E.load(g.dfinal + state_at, N, chans);
    if (p.nseg > 1) {
        join_segments<N>(p, at, h, a, p.sums, cg, 0, at.seg, 1);
        join_segments<N>(p, at, E, a, g.rsums, cg, p.nseg - 1, at.seg, -1);
    }
    h.put(sst, NT);
    const T *x = static_cast<const T*>(p.x.p) + at.b * p.x.sb + at.c0, *dt = static_cast<const T*>(p.dt.p) + at.b * p.dt.sb + at.c0,
            *z = p.gate.p ? static_cast<const T*>(p.gate.p) + at.b * p.gate.sb + at.c0 : nullptr,
            *dout = static_cast<const T*>(g.dout.p) + at.b * g.dout.sb + at.c0,
            *b = static_cast<const T*>(p.b.p) + at.b * p.b.sb + at.group * p.b.sh,
            *c = static_cast<const T*>(p.c.p) + at.b * p.c.sb + at.group * p.c.sh;
    auto out = [&](const SsmRows& r) { return static_cast<T*>(const_cast<void*>(r.p)) + at.b * r.sb + at.c0; };
    T *dx = out(g.dx), *ddt = out(g.ddt), *dgate = z ? out(g.dgate) : nullptr;
    using Chan = Tile<T, M, MT, CT, NT>;
    using Stat = Tile<T, M, MT, N, NT>;
    const long long slot = at.slot(p, at.seg);
    // sums of this thread's items' channels
    F2 gskip[2], gbias[2];
    gskip[0] = gskip[1] = gbias[0] = gbias[1] = pair(0.f, 0.f);
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
            xr.template load<true>(x, p.x.sn, t0, at.live_end, at.cols);
            dr.template load<true>(dt, p.dt.sn, t0, at.live_end, at.cols);
            or_.template load<true>(dout, g.dout.sn, t0, at.live_end, at.cols);
            if (z) zr.template load<true>(z, p.gate.sn, t0, at.live_end, at.cols);
            br.template load<true>(b, p.b.sn, t0, at.live_end, N);
            cr.template load<true>(c, p.c.sn, t0, at.live_end, N);
            Chan::parts([&](int k, int r, int ch) {
                stage<T, true>(xr.v[k], dr.v[k], or_.v[k], zr.v[k], z, p.softplus, t0 + r < at.live_end && ch < at.cols, sbias + ch,
                                  sd + r * CT + ch, su + r * CT + ch, sy + r * CT + ch);
            });
            Stat::parts([&](int k, int r, int n) {
                F2 f[2];
                unpack(br.v[k], f);
                put_twice(sb + r * 2 * N + 2 * n, f);
                unpack(cr.v[k], f);
                put_twice(sc + r * 2 * N + 2 * n, f);
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
                        h.v[k + j][0] = fma_(decay_of(d.lo, a.v[k + j][0]), h.v[k + j][0], u.lo * bk);
                        h.v[k + j][1] = fma_(decay_of(d.hi, a.v[k + j][1]), h.v[k + j][1], u.hi * bk);
                    }
                }
            }
        }
        for (int t = MT - TC; t >= 0; t -= TC) {
            if (t < MT - TC) h.get(sst + (1 + t / TC) * (NT * 16), NT);
            // what the items of these tokens take from memory
            Vec<T, 4> ix[items], id[items], iz[items], io[items];
            auto each_item = [&](auto&& f) {  // f(item, token of the four, its place); an item is four channels of a token
#pragma unroll
                for (int m = 0; m < items; ++m) {
                    const int i = tid + m * NT, r = i / (CT / 4);
                    if (NT > TC * CT / 4 && i >= TC * CT / 4) continue;
                    f(m, r, t0 + t + r);
                }
            };
            each_item([&](int m, int, int tok) {
                ix[m] = id[m] = iz[m] = io[m] = Vec<T, 4>{};
                if (tok < at.live_end && quad < at.cols) {
                    const int count = at.cols - quad;
                    ix[m] = ldrow<T, M>(x + (long long)tok * p.x.sn + quad, count);
                    id[m] = ldrow<T, M>(dt + (long long)tok * p.dt.sn + quad, count);
                    if (z) {
                        iz[m] = ldrow<T, M>(z + (long long)tok * p.gate.sn + quad, count);
                        io[m] = ldrow<T, M>(dout + (long long)tok * g.dout.sn + quad, count);
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
                        hk[0] = fma_(decay_of(d.lo, a.v[k + j][0]), hk[0], u.lo * bk);
                        hk[1] = fma_(decay_of(d.hi, a.v[k + j][1]), hk[1], u.hi * bk);
                        y01 = fma_(hk[0], ck, y01), y23 = fma_(hk[1], ck, y23);
                        dc[k + j] = sum_of(fma_(hk[0], dy.lo, hk[1] * dy.hi));
                    }
                }
                *reinterpret_cast<float4*>(vdc + (i * NT + tid) * 4) = make_float4(dc[0], dc[1], dc[2], dc[3]);
                if (z) Sums::put(vy + i * Sums::token, cg, sl, y01, y23);
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
                        Ek[0] = R0 * decay_of(d.lo, a.v[k + j][0]);
                        Ek[1] = R1 * decay_of(d.hi, a.v[k + j][1]);
                        const F2 q0 = Ek[0] * kept[i].v[k + j][0], q1 = Ek[1] * kept[i].v[k + j][1];
                        da.v[k + j][0] = fma_(q0, d.lo, da.v[k + j][0]);
                        da.v[k + j][1] = fma_(q1, d.hi, da.v[k + j][1]);
                        e01 = fma_(q0, a.v[k + j][0], e01), e23 = fma_(q1, a.v[k + j][1], e23);
                    }
                }
                *reinterpret_cast<float4*>(vdb + (i * NT + tid) * 4) = make_float4(db[0], db[1], db[2], db[3]);
                Sums::put(vin + i * Sums::token, cg, sl, in01, in23);
                Sums::put(ve + i * Sums::token, cg, sl, e01, e23);
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
                if (tok >= at.t_end || quad >= at.cols) return;
                F2 in[2], e[2], xv[2], v[2], d[2], dy[2], fb[2], fs[2], dd[2], ox[2];
                Sums::get(vin + r * Sums::token + quad, in);
                Sums::get(ve + r * Sums::token + quad, e);
                unpack(ix[m], xv);
                unpack(id[m], v);
                get_values(sd + (t + r) * CT + quad, d);
                get_values(sy + (t + r) * CT + quad, dy);
                get_values(sbias + quad, fb);
                get_values(sskip + quad, fs);
                const bool on = tok < at.live_end;
                const int count = at.cols - quad;
                const F2 zero = pair(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    dd[i] = fma_(xv[i], in[i], e[i] * pair(kLn2, kLn2));
                    if (p.softplus) dd[i] = dd[i] * sigmoid_of(v[i] + fb[i]);
                    ox[i] = fma_(d[i], in[i], fs[i] * dy[i]);
                    if (!on) dd[i] = ox[i] = zero;
                    gbias[i] = dd[i] + gbias[i];
                    gskip[i] = fma_(xv[i], dy[i], gskip[i]);
                }
                strow<T, M>(dx + (long long)tok * g.dx.sn + quad, ox, count);
                strow<T, M>(ddt + (long long)tok * g.ddt.sn + quad, dd, count);
                if (z) {
                    F2 y[2], fz[2], fo[2];
                    Sums::get(vy + r * Sums::token + quad, y);
                    unpack(iz[m], fz);
                    unpack(io[m], fo);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        F2 slope;
                        gate_of(fz[i], true, slope);
                        y[i] = on ? fo[i] * fma_(fs[i], xv[i], y[i]) * slope : zero;
                    }
                    strow<T, M>(dgate + (long long)tok * g.dgate.sn + quad, y, count);
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
    float* sums = vdc;
    if (tid < TC * CT / 4) {
        float* to = sums + tid / (CT / 4) * CT + quad;
        put_values(to, gskip);
        put_values(to + TC * CT, gbias);
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
    const F2 zero[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
    const int first = at.t0 + macros * MT;
    for (long long i = tid; i < (long long)(at.t_end - first) * (CT / 4); i += NT) {
        const int tok = first + (int)(i / (CT / 4)), ch = (int)(i % (CT / 4)) * 4, count = at.cols - ch;
        if (count <= 0) continue;
        strow<T, M>(dx + (long long)tok * g.dx.sn + ch, zero, count);
        strow<T, M>(ddt + (long long)tok * g.ddt.sn + ch, zero, count);
        if (z) strow<T, M>(dgate + (long long)tok * g.dgate.sn + ch, zero, count);
    }
}

// db and dc: the parts of a group's tiles, four states a thread
template <typename T, int N>
__device__ __forceinline__ void add_bc(const SsmPass& p, const SsmGrads& g, int block) {
    constexpr int quads = 2 * N / 4;
    const long long i = (long long)block * 256 + threadIdx.x, tg = i / quads;
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
__device__ __forceinline__ void add_params(const SsmPass& p, const SsmGrads& g, int block) {
    __shared__ float sm[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long cols = (long long)p.D * (p.N + 2), c = (long long)block * 32 + lane;
    const int rows = p.B * p.nseg;
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

// Both in one launch, the first `params` CTAs and those after them (two launches: 100 tokens of 256 channels, forward and backward,
// 39 us instead of 35.5)
template <typename T, int N>
__global__ void __launch_bounds__(256) ssm_parts_kernel(const SsmPass p, const SsmGrads g, int params) {
    pdl_wait();
    if ((int)blockIdx.x < params) add_params(p, g, blockIdx.x);
    else add_bc<T, N>(p, g, blockIdx.x - params);
}

template <typename T, int M, int N>
int backward_n(const SsmPass& p, const SsmGrads& g, cudaStream_t st) {
    const long long params = ((long long)p.D * (N + 2) + 31) / 32, bc = ((long long)p.B * p.n * p.G * (2 * N / 4) + 255) / 256;
    auto parts = [&]() {
        return launch_pdl(ssm_parts_kernel<T, N>, dim3((unsigned)(params + bc)), dim3(256), 0, st, p, g, (int)params) == cudaSuccess ? 0 : -1;
    };
    if (p.B == 0) return parts();  // zeros
    const dim3 block(SsmShape<N>::threads), grid(p.B * p.G * p.tiles, p.nseg);
    if (p.nseg > 1) {
        if (launch_pdl(ssm_marks_kernel<T, M, N, true>, grid, block, 0, st, p, g) != cudaSuccess ||
            (p.nseg > kSsmJoin && launch_ssm_carry(p, g.rsums, g.dfinal, st)))
            return -1;
    } else if (g.macros > 1) {
        if (launch_pdl(ssm_marks_kernel<T, M, N, false>, grid, block, 0, st, p, g) != cudaSuccess) return -1;
    }
    auto kernel = ssm_backward_kernel<T, M, N>;
    constexpr size_t smem = BackSmem<N>::total * sizeof(float);
    if (raise_smem(kernel, smem) != cudaSuccess) return -1;
    if (launch_pdl(kernel, grid, block, smem, st, p, g) != cudaSuccess) return -1;
    return parts();
}
template <typename T, int M>
int backward_v(const SsmPass& p, const SsmGrads& g, cudaStream_t st) {
    switch (p.N) {
        case 8: return backward_n<T, M, 8>(p, g, st);
        case 16: return backward_n<T, M, 16>(p, g, st);
        case 32: return backward_n<T, M, 32>(p, g, st);
        case 64: return backward_n<T, M, 64>(p, g, st);
        default: return -1;
    }
}

}  // namespace

int launch_ssm_backward(const SsmPass& p, const SsmGrads& g, bool is_bf16, bool vec, cudaStream_t st) {
    if (is_bf16) return vec ? backward_v<bf16, 4>(p, g, st) : backward_v<bf16, 1>(p, g, st);
    return vec ? backward_v<float, 4>(p, g, st) : backward_v<float, 1>(p, g, st);
}

}  // namespace hla2
