// C ABI of the selective scan: argument checks, the segmentation of the sequence and the passes of a call (ssm.cuh).
// The declarations and their documentation are in include/hla2.h.
#include <cmath>

#include "rows.h"
#include "ssm.cuh"

using namespace hla2;

namespace {

// Sizes and types: what the workspace query can check.
int check_sizes(const char* fn, const hla2_ssm_args* a) {
    if (!a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: args must not be NULL", fn);
    if (a->dtype != HLA2_F32 && a->dtype != HLA2_BF16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dtype must be HLA2_F32 or HLA2_BF16", fn);
    if (a->B < 0 || a->n < 0 || a->D < 0)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: B, n and D must not be negative", fn);
    if (a->N != 8 && a->N != 16 && a->N != 32 && a->N != 64)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: N must be 8, 16, 32 or 64 (got %d)", fn, a->N);
    if (a->G < 1 || a->D % a->G != 0)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: D (%d) must be a multiple of G (%d)", fn, a->D, a->G);
    if (a->softplus != 0 && a->softplus != 1)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: softplus must be 0 or 1", fn);
    const long long tiles = a->D ? (long long)a->G * ((a->D / a->G + kSsmChannels - 1) / kSsmChannels) : 0;
    if (tiles * a->B > 0x7fffffffLL || (long long)a->B * a->D > 0x7fffffffLL || a->n > 1 << 30)
        return set_last_error(HLA2_ERR_UNSUPPORTED, "%s: B * D must fit in 31 bits, and n be at most 2^30", fn);
    return HLA2_OK;
}

constexpr int kSsmVec = 4;  // elements that a thread moves at a time, where the tensors allow it

// The inputs of a call, and everything that it reads
struct Inputs {
    Tensor t[5] = {};
    int count = 0;
    Places read;
    explicit Inputs(int es) : read(es) {}
    int check(const char* fn, const hla2_ssm_args* a, int n) {
        const int es = elem_size(a->dtype);
        t[count++] = rows("x", a->x, a->B, n, a->D);
        t[count++] = rows("dt", a->dt, a->B, n, a->D);
        t[count++] = view("b", a->b, a->B, a->G, n, a->N);
        t[count++] = view("c", a->c, a->B, a->G, n, a->N);
        if (a->gate.p) t[count++] = rows("gate", a->gate, a->B, n, a->D);
        for (int i = 0; i < count; ++i) {
            if (int rc = check_tensor(fn, t[i], es, false)) return rc;
            read.add(t[i]);
        }
        return HLA2_OK;
    }
    int check_params(const char* fn, const hla2_ssm_args* a) {
        if (!a->a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a must not be NULL", fn);
        if (!al(a->a, 16) || !al(a->init_state, 16))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a and the states must be 16-byte aligned", fn);
        if (!al(a->skip, 4) || !al(a->dt_bias, 4) || !al(a->lengths, 4))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
        const size_t d = (size_t)a->D * sizeof(float);
        read.add(extent_of(a->a, d * a->N));
        read.add(extent_of(a->skip, d));
        read.add(extent_of(a->dt_bias, d));
        read.add(extent_of(a->lengths, (size_t)a->B * sizeof(int)));
        read.add(extent_of(a->init_state, d * a->B * a->N));
        return HLA2_OK;
    }
    // whether every tensor allows vectors of v elements of the staged rows, within a group's channels too
    bool vec(const hla2_ssm_args* a, int v) const {
        for (int i = 0; i < count; ++i)
            if (!t[i].vec(v, elem_size(a->dtype))) return false;
        return a->D / a->G % v == 0;
    }
};

SsmRows dev(const Tensor& t) { return {t.p, t.sb, t.sn}; }
hla2_view dev4(const Tensor& t) { return {t.p, t.sb, t.sh, t.sn}; }

// ---- plan ----------------------------------------------------------------------------------

struct SsmPlan {
    int tiles, nseg, seg_tokens;
};

// Segments of each sequence, by the time in us of sixteen tokens in a CTA of the main pass: `alone` with the SM to itself,
// and `beside` for each CTA once they fill it (measured at N = 16 over 1 to 128 segments of 32 to 512 tiles of channels;
// the part of it that goes with the states, here 0.55 of it, goes with N).  An SM holds `most` CTAs (of 64 threads): up to
// there the fullest SM counts, above it they follow one another without waves.  More than one segment adds the pass of
// their sums, a launch, and the joining of the segments before, which a CTA reads four at a time; the backward has a pass
// of marks without them too.
// The scaling to other N foretells the forward to an eighth up to N = 32, and too little beyond and in the backward: 4 x 2048 x 2048 with N = 8, 16,
// 32 and 64 takes 115, 155, 275 and 463 us for 123, 162, 245 and 358 foretold, backward 390, 472, 927 and 1980 for 342, 468, 720 and
// 1224.  (The output kernels hold 16, 7, 4 and 2 CTAs an SM there, by threads and shared memory, where `most` has 14, 7, 3 and 1.)
// (2 x 2048 x 2048, N = 16, forward: one segment 363 us, 8 105, 16 89, 64 107; backward 1299, 282, 274, 311.  8 x 4096 x 4096, which
// fills the GPU by itself: forward 939 with one, 1050 with 8.)
struct SsmCost {
    double alone, beside, sums, marks;
    int most;
};
constexpr SsmCost kForwardCost{2.8, 0.9, 0.55, 0.0, 7}, kBackwardCost{9.5, 3.0, 0.4, 0.2, 4};

SsmPlan ssm_plan(const hla2_ssm_args* a, bool backward) {
    SsmPlan p{(a->D / a->G + kSsmChannels - 1) / kSsmChannels, 1, kSsmTokens};
    const SsmCost& c = backward ? kBackwardCost : kForwardCost;
    const int steps = (a->n + kSsmTokens - 1) / kSsmTokens, sms = sm_count();
    const int most = c.most * 16 / a->N > 1 ? c.most * 16 / a->N : 1;
    const double ctas = (double)a->B * a->G * p.tiles, beside = c.beside * (0.45 + 0.55 * a->N / 16);
    double best = 0;
    for (int want = 1; want <= steps && want <= 1024; want = want < 4 ? want + 1 : want * 5 / 4) {
        const int each = (steps + want - 1) / want, nseg = (steps + each - 1) / each;
        const double per_sm = ctas * nseg / sms;
        const double full = per_sm <= most ? std::ceil(per_sm) : 0.87 * per_sm + 1.2;
        const double load = full * beside > c.alone ? full * beside : c.alone;
        const double cost = nseg == 1 ? each * load * (1 + c.marks)
                                      : (each + 0.45) * load * (1 + c.sums) + 6 + (nseg <= kSsmJoin ? 0.2 * nseg : 6.0);
        if (want == 1 || cost < best) best = cost, p.nseg = nseg, p.seg_tokens = each * kSsmTokens;
    }
    return p;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Scratch of the segments, by sequence, tile and segment: states, sums of the steps; for a backward what SsmGrads has
struct Scratch {
    size_t sums, steps, marks, mark_steps, rsums, bc, params, total;
};
Scratch scratch_of(const hla2_ssm_args* a, const SsmPlan& p, bool backward) {
    Scratch s{};
    const size_t slots = (size_t)a->B * a->G * p.tiles * p.nseg;
    if (p.nseg > 1) {
        s.sums = s.total, s.total += up256(slots * kSsmChannels * a->N * sizeof(float));
        s.steps = s.total, s.total += up256(slots * kSsmChannels * sizeof(float));
    }
    if (backward) {
        const size_t marks = slots * (p.seg_tokens / kSsmMark), state = kSsmChannels * a->N * sizeof(float);
        s.marks = s.total, s.total += up256(marks * state);
        if (p.nseg > 1) {
            s.mark_steps = s.total, s.total += up256(marks * kSsmChannels * sizeof(float));
            s.rsums = s.total, s.total += up256(slots * state);
        }
        s.bc = s.total, s.total += up256((size_t)a->B * a->n * a->G * p.tiles * 2 * a->N * sizeof(float));
        s.params = s.total, s.total += up256((size_t)a->B * p.nseg * a->D * (a->N + 2) * sizeof(float));
    }
    return s;
}

SsmPass base_pass(const hla2_ssm_args* a, const Inputs& in, const SsmPlan& pl) {
    SsmPass p{};
    p.B = a->B, p.n = a->n, p.D = a->D, p.N = a->N, p.G = a->G;
    p.per = a->D / a->G;
    p.tiles = pl.tiles, p.nseg = pl.nseg, p.seg_tokens = pl.seg_tokens;
    p.softplus = a->softplus;
    p.x = dev(in.t[0]), p.dt = dev(in.t[1]);
    p.b = dev4(in.t[2]), p.c = dev4(in.t[3]);
    if (a->gate.p) p.gate = dev(in.t[4]);
    p.a = a->a, p.skip = a->skip, p.dt_bias = a->dt_bias;
    p.lengths = a->lengths;
    p.init = a->init_state;
    return p;
}

}  // namespace

extern "C" {

size_t hla2_ssm_workspace_bytes(const hla2_ssm_args* a, int backward) {
    if (check_sizes("hla2_ssm_workspace_bytes", a) != HLA2_OK) return (size_t)-1;
    ok();
    if (a->D == 0 || (a->B == 0 && !backward)) return 0;
    return scratch_of(a, ssm_plan(a, backward != 0), backward != 0).total;
}

int hla2_ssm_forward(const hla2_ssm_args* a, hla2_rows out, float* final_state, hla2_stream_t stream) {
    static const char* const fn = "hla2_ssm_forward";
    Range range(fn);
    if (int rc = check_sizes(fn, a)) return rc;
    if (a->B == 0 || a->D == 0) return ok();
    const int es = elem_size(a->dtype);
    Inputs in(es);
    if (int rc = in.check_params(fn, a)) return rc;
    const Extent fin = extent_of(final_state, (size_t)a->B * a->D * a->N * sizeof(float));
    if (!al(final_state, 16)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a and the states must be 16-byte aligned", fn);
    bool vec = true;
    Tensor o = rows("out", out, a->B, a->n, a->D);
    if (a->n > 0) {
        if (int rc = in.check(fn, a, a->n)) return rc;
        if (int rc = check_tensor(fn, o, es, true)) return rc;
        if (in.read.meets(o) || meet(o.extent(es), fin))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out overlaps another tensor", fn);
        vec = in.vec(a, kSsmVec) && o.vec(kSsmVec, es);
    } else if (!final_state) {
        return ok();
    }
    if (in.read.meets(fin)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: final_state overlaps an input", fn);
    const SsmPlan pl = ssm_plan(a, false);
    const Scratch s = scratch_of(a, pl, false);
    if (s.total > 0 && (!a->workspace || a->workspace_bytes < s.total || !al(a->workspace, 16)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, s.total);
    SsmPass p = base_pass(a, in, pl);
    p.out = dev(o);
    p.fin = final_state;
    char* ws = static_cast<char*>(a->workspace);
    if (pl.nseg > 1) {
        p.sums = reinterpret_cast<float*>(ws + s.sums);
        p.steps = reinterpret_cast<float*>(ws + s.steps);
    }
    if (launch_ssm_forward(p, a->dtype == HLA2_BF16, vec, reinterpret_cast<cudaStream_t>(stream)))
        return launch_failed("selective scan");
    return ok();
}

int hla2_ssm_backward(const hla2_ssm_args* a, hla2_rows dout, const float* dfinal_state, const hla2_ssm_grads* grads,
                      hla2_stream_t stream) {
    static const char* const fn = "hla2_ssm_backward";
    Range range(fn);
    if (int rc = check_sizes(fn, a)) return rc;
    if (!grads) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: grads must not be NULL", fn);
    if (a->D == 0) return ok();
    const int es = elem_size(a->dtype);
    Inputs in(es);
    if (int rc = in.check_params(fn, a)) return rc;
    const size_t db = (size_t)a->D * sizeof(float);
    in.read.add(extent_of(dfinal_state, db * a->B * a->N));
    if (!grads->da || (a->skip != nullptr) != (grads->dskip != nullptr) ||
        (a->dt_bias != nullptr) != (grads->ddt_bias != nullptr))
        return set_last_error(HLA2_ERR_INVALID_ARG,
                              "%s: da is needed, dskip and ddt_bias with their inputs, and neither without", fn);
    if (!al(dfinal_state, 16) || !al(grads->dinit_state, 16))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a and the states must be 16-byte aligned", fn);
    if (!al(grads->da, 4) || !al(grads->dskip, 4) || !al(grads->ddt_bias, 4))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    const Extent sums[4] = {extent_of(grads->da, db * a->N), extent_of(grads->dskip, db), extent_of(grads->ddt_bias, db),
                            extent_of(grads->dinit_state, db * a->B * a->N)};
    bool vec = true;
    Tensor o[6] = {};
    int outs = 0;
    if (a->n > 0 && a->B > 0) {
        if (int rc = in.check(fn, a, a->n)) return rc;
        o[outs++] = rows("dout", dout, a->B, a->n, a->D);
        o[outs++] = rows("dx", grads->dx, a->B, a->n, a->D);
        o[outs++] = rows("ddt", grads->ddt, a->B, a->n, a->D);
        o[outs++] = view("db", grads->db, a->B, a->G, a->n, a->N);
        o[outs++] = view("dc", grads->dc, a->B, a->G, a->n, a->N);
        if (a->gate.p) o[outs++] = rows("dgate", grads->dgate, a->B, a->n, a->D);
        vec = in.vec(a, kSsmVec);
        for (int i = 0; i < outs; ++i) {
            if (int rc = check_tensor(fn, o[i], es, i > 0)) return rc;
            if (i == 0) in.read.add(o[i]);
            vec = vec && o[i].vec(kSsmVec, es);
        }
    }
    if ((a->gate.p != nullptr) != (grads->dgate.p != nullptr) && a->n > 0 && a->B > 0)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dgate is needed with gate, and only then", fn);
    Places written(es);
    int rc = 0;
    auto write = [&](const auto& e) {
        if (rc) return;
        if (in.read.meets(e)) rc = set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient overlaps an input", fn);
        else if (written.meets(e)) rc = set_last_error(HLA2_ERR_INVALID_ARG, "%s: gradients overlap", fn);
        else written.add(e);
    };
    for (const Extent& e : sums) write(e);
    for (int i = 1; i < outs; ++i) write(o[i]);
    if (rc) return rc;
    const SsmPlan pl = ssm_plan(a, true);
    const Scratch s = scratch_of(a, pl, true);
    if (s.total > 0 && (!a->workspace || a->workspace_bytes < s.total || !al(a->workspace, 16)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, s.total);
    SsmPass p = base_pass(a, in, pl);
    SsmGrads g{};
    g.dout = dev(o[0]), g.dx = dev(o[1]), g.ddt = dev(o[2]);
    g.db = dev4(o[3]), g.dc = dev4(o[4]);
    if (a->gate.p) g.dgate = dev(o[5]);
    g.da = grads->da, g.dskip = grads->dskip, g.ddt_bias = grads->ddt_bias, g.dinit = grads->dinit_state;
    g.dfinal = dfinal_state;
    g.macros = pl.seg_tokens / kSsmMark;
    auto at = [&](size_t offset) { return reinterpret_cast<float*>(static_cast<char*>(a->workspace) + offset); };
    g.marks = at(s.marks), g.bc = at(s.bc), g.params = at(s.params);
    if (pl.nseg > 1) p.sums = at(s.sums), p.steps = at(s.steps), g.mark_steps = at(s.mark_steps), g.rsums = at(s.rsums);
    if (launch_ssm_backward(p, g, a->dtype == HLA2_BF16, vec, reinterpret_cast<cudaStream_t>(stream)))
        return launch_failed("selective scan gradients");
    return ok();
}

int hla2_ssm_decode_step(const hla2_ssm_args* a, float* state, hla2_rows out, hla2_stream_t stream) {
    static const char* const fn = "hla2_ssm_decode_step";
    Range range(fn);
    hla2_ssm_args one;  // n is not looked at
    if (a) one = *a, one.n = 1, a = &one;
    if (int rc = check_sizes(fn, a)) return rc;
    if (a->B == 0 || a->D == 0) return ok();
    if (a->lengths || a->init_state)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: lengths and init_state must be NULL", fn);
    const int es = elem_size(a->dtype);
    Inputs in(es);
    if (int rc = in.check_params(fn, a)) return rc;
    if (int rc = in.check(fn, a, 1)) return rc;
    if (!state || !al(state, 16))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: the state must be a 16-byte aligned address", fn);
    const Tensor o = rows("out", out, a->B, 1, a->D);
    if (int rc = check_tensor(fn, o, es, true)) return rc;
    const Extent est = extent_of(state, (size_t)a->B * a->D * a->N * sizeof(float));
    if (meet(o.extent(es), est) || in.read.meets(o) || in.read.meets(est))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out or the state overlaps another tensor", fn);
    SsmPass p = base_pass(a, in, SsmPlan{1, 1, 1});
    p.out = dev(o);
    const bool vec = in.t[2].vec(kSsmVec, es) && in.t[3].vec(kSsmVec, es);  // of b and c
    if (launch_ssm_step(p, state, a->dtype == HLA2_BF16, vec, reinterpret_cast<cudaStream_t>(stream)))
        return launch_failed("selective scan step");
    return ok();
}

}  // extern "C"
