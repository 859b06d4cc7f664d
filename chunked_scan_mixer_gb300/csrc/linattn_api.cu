// C ABI of the first-order linear attention with a decay for each head: argument checks, the
// segmentation of the sequence, and the passes that make up a forward and a backward
// (linattn_pass.h).  The declarations and their documentation are in include/hla2.h.
#include <nvtx3/nvToolsExt.h>

#include "linattn_pass.h"

namespace hla2 {
int set_last_error(int code, const char* fmt, ...);
}

using namespace hla2;

namespace {

constexpr size_t kStatusBytes = 256;

struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;
};

int ok() { return set_last_error(HLA2_OK, "%s", ""); }
int launch_failed(const char* what) {
    return set_last_error(HLA2_ERR_CUDA, "%s: %s", what, cudaGetErrorString(cudaGetLastError()));
}

bool lin_dim(int x) { return x == 16 || x == 32 || x == 64 || x == 128; }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int elem_size(int dtype) { return dtype == HLA2_BF16 ? 2 : 4; }

// Sizes, types: what the workspace query can check.
int check_sizes(const char* fn, const hla2_linattn_args* a) {
    if (!a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: args must not be NULL", fn);
    if (a->dtype != HLA2_F32 && a->dtype != HLA2_BF16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dtype must be HLA2_F32 or HLA2_BF16", fn);
    if (a->B < 0 || a->H < 0 || a->Hk < 0 || a->n < 0)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: B, H, Hk and n must not be negative", fn);
    if (!lin_dim(a->d) || !lin_dim(a->dv))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: d and dv must be 16, 32, 64 or 128 (got %d, %d)", fn, a->d,
                              a->dv);
    if ((a->Hk == 0) != (a->H == 0) || (a->Hk > 0 && a->H % a->Hk != 0))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: H (%d) must be a multiple of Hk (%d)", fn, a->H, a->Hk);
    // grid limits and 32-bit head counts
    if ((long long)a->B * a->H > 0x7fffffff || a->n > 1 << 30)
        return set_last_error(HLA2_ERR_UNSUPPORTED, "%s: B * H must fit in 31 bits, and n be at most 2^30", fn);
    return HLA2_OK;
}

// Strides of dimensions of one element do not matter: they become the packed ones.
int check_view(const char* fn, const char* name, hla2_view& w, int B, int H, int n, int D, int es) {
    if (!w.p) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: %s must not be NULL", fn, name);
    const long long per16 = 16 / es;
    if (n <= 1) w.sn = D;
    if (H <= 1) w.sh = w.sn * (n > 1 ? n : 1);
    if (B <= 1) w.sb = w.sh * (H > 1 ? H : 1);
    if (!al16(w.p) || w.sn % per16 || w.sh % per16 || w.sb % per16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: the address and strides of %s must be multiples of 16 bytes", fn,
                              name);
    if (w.sn < D || w.sh < D || w.sb < D)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: the strides of %s must be at least its last dimension", fn, name);
    return HLA2_OK;
}

Extent extent(const hla2_view& w, int B, int H, int n, int D, int es) {
    return extent_of(w.p, (size_t)((B - 1) * w.sb + (H - 1) * w.sh + (n - 1) * w.sn + D) * es);
}
Extent state_extent(const hla2_linattn_args* a, const float* p) {
    return extent_of(p, (size_t)a->B * a->Hk * a->d * a->dv * sizeof(float));
}

// ---- plan ----------------------------------------------------------------------------------

struct LinPlan {
    int W, nchunks, seg_chunks, nseg;
};

// Whether the output pass joins the segments' sums itself: the last segment's CTA then reads all of them, four
// at a time, where the scan takes 6 to 8 us and a launch.  So: up to 512 KB of states, and 16 of them.
// (Eight segments of 64 x 64: 24.6 -> 20.6 us for the call; nine instead of nineteen and a scan: 180 -> 173.)
bool joins(const hla2_linattn_args* a, int nseg) {
    return a->dtype == HLA2_BF16 && nseg > 0 && nseg <= 16 && (long long)nseg * a->d * a->dv <= 128 * 1024;
}

// Segments per state head.  Unit: the time of one chunk of the output pass.  More than one segment
// adds the summary pass (about half of the output pass: it reads two of four tensors) and, where there is
// one, about two chunks' time for the scan and its launch.  The waves of CTAs count whole, each with about two chunks'
// time to start and to end.
LinPlan lin_plan(const hla2_linattn_args* a, int W, int slots) {
    LinPlan p{W, (a->n + W - 1) / W, 0, 0};
    const long long heads = (long long)a->B * a->Hk;
    if (p.nchunks == 0 || heads == 0) return p;
    double best = 0;
    // one segment, and as many as fill one to four waves
    for (int wave = 0; wave <= 4; ++wave) {
        long long want = wave == 0 ? 1 : (long long)wave * slots / heads;
        if (want < 1) continue;
        if (want > p.nchunks) want = p.nchunks;
        if (want > 4096) want = 4096;
        const int sc = (int)((p.nchunks + want - 1) / want), ns = (p.nchunks + sc - 1) / sc;
        const long long waves = (heads * ns + slots - 1) / slots;
        const double cost = (double)waves * (sc + 2) * (ns > 1 ? 1.5 : 1.0) + (ns > 1 && !joins(a, ns) ? 2.0 : 0.0);
        if (p.nseg == 0 || cost < best) best = cost, p.seg_chunks = sc, p.nseg = ns;
    }
    return p;
}

LinPlan plan_of(const hla2_linattn_args* a) {
    if (a->dtype == HLA2_BF16) return lin_plan(a, 128, sm_count());
    const int sms = sm_count(), W = lin_simt_width(a->d, a->dv, (long long)a->B * a->Hk, a->n, sms);
    return lin_plan(a, W, sms * lin_simt_ctas(a->d, a->dv, W));
}

size_t state_array_bytes(const hla2_linattn_args* a, const LinPlan& p) {
    return ((size_t)a->B * a->Hk * p.nseg * a->d * a->dv * sizeof(float) + 255) & ~size_t(255);
}

// Passes that do not wait for each other
int run_passes(const LinPass* p, int count, bool summary, int dtype, cudaStream_t st) {
    if (dtype != HLA2_BF16) return launch_lin_simt(p, count, summary, st);
    for (int i = 0; i < count; ++i)
        if (launch_lin_tc(p[i], summary, st)) return -1;
    return 0;
}

// Common fields of every pass of one call.
LinPass base_pass(const hla2_linattn_args* a, const LinPlan& p) {
    LinPass s{};
    s.B = a->B;
    s.Hs = a->Hk;
    s.rx = s.rk = 1;
    s.n = a->n;
    s.W = p.W;
    s.nchunks = p.nchunks;
    s.seg_chunks = p.seg_chunks;
    s.nseg = p.nseg;
    s.s_col = s.s_fin = s.s_state = 1.f;
    s.gamma = a->gamma;
    s.lengths = a->lengths;
    s.status = static_cast<int*>(a->workspace);
    return s;
}


// Forward states of k, v, or reverse ones of q, dout, before the output passes: what has to run for them.
struct States {
    LinPass pass;  // of the summaries
    LinScan scan;
    bool sums, scans;
};
// `s` holds the states' fields and gets what the output passes take of them (the final state with the first
// pass that joins them).
States states(const hla2_linattn_args* a, const LinPlan& p, LinPass& s, float* sums, float* carry, const float* init,
              float* final_state) {
    States x{s, {sums, p.nseg > 0 ? carry : nullptr, init, final_state, s.rev}, false, false};
    x.sums = p.nseg > 1 || (final_state && p.nseg > 0);
    x.pass.sums = sums;
    x.pass.exact_sums = final_state != nullptr;
    if (joins(a, p.nseg)) {
        s.prior = sums;
        s.init = init;
        s.fin = final_state;
    } else {
        x.scans = p.nseg > 1 || final_state || init;
        if (p.nseg > 1 || init) s.carry = carry;
    }
    return x;
}
int run_states(const hla2_linattn_args* a, const LinPlan& p, const States* x, int count, cudaStream_t st) {
    LinPass passes[2];
    LinScan scans[2];
    int np = 0, ns = 0;
    for (int i = 0; i < count; ++i) {
        if (x[i].sums) passes[np++] = x[i].pass;
        if (x[i].scans) scans[ns++] = x[i].scan;
    }
    if (run_passes(passes, np, true, a->dtype, st)) return -1;
    return launch_lin_scan(scans, ns, a->gamma, a->lengths, a->B, a->Hk, a->n, p.seg_chunks * p.W, p.nseg, a->d * a->dv, st);
}

}  // namespace

extern "C" {

size_t hla2_linattn_workspace_bytes(const hla2_linattn_args* a, int backward, int want_final) {
    if (check_sizes("hla2_linattn_workspace_bytes", a) != HLA2_OK) return (size_t)-1;
    ok();
    const LinPlan p = plan_of(a);
    if (p.nseg == 0) return 0;
    const bool fwd_states = p.nseg > 1 || a->init_state || (!backward && want_final);
    const bool rev_states = backward && (p.nseg > 1 || want_final);
    return kStatusBytes + 2 * state_array_bytes(a, p) * ((fwd_states ? 1 : 0) + (rev_states ? 1 : 0));
}

int hla2_linattn_forward(const hla2_linattn_args* args, hla2_view out, float* final_state, hla2_stream_t stream) {
    static const char* const fn = "hla2_linattn_forward";
    Range range(fn);
    if (int rc = check_sizes(fn, args)) return rc;
    hla2_linattn_args a = *args;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a.B == 0 || a.H == 0) return ok();
    const int es = elem_size(a.dtype);
    if (!al16(a.init_state) || !al16(final_state))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: states must be 16-byte aligned", fn);
    // the segments' CTAs read the one while the last segment's writes the other
    if (meet(state_extent(&a, final_state), state_extent(&a, a.init_state)))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: final_state overlaps init_state", fn);
    if (a.n > 0) {
        if (int rc = check_view(fn, "q", a.q, a.B, a.H, a.n, a.d, es)) return rc;
        if (int rc = check_view(fn, "k", a.k, a.B, a.Hk, a.n, a.d, es)) return rc;
        if (int rc = check_view(fn, "v", a.v, a.B, a.Hk, a.n, a.dv, es)) return rc;
        if (int rc = check_view(fn, "out", out, a.B, a.H, a.n, a.dv, es)) return rc;
        const Extent eo = extent(out, a.B, a.H, a.n, a.dv, es);
        if (meet(eo, extent(a.q, a.B, a.H, a.n, a.d, es)) || meet(eo, extent(a.k, a.B, a.Hk, a.n, a.d, es)) ||
            meet(eo, extent(a.v, a.B, a.Hk, a.n, a.dv, es)))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out overlaps an input", fn);
    }
    const size_t need = hla2_linattn_workspace_bytes(&a, 0, final_state != nullptr);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need || !al16(a.workspace)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    const LinPlan p = plan_of(&a);
    float* sums = p.nseg ? reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kStatusBytes) : nullptr;
    float* carry = p.nseg ? sums + state_array_bytes(&a, p) / sizeof(float) : nullptr;

    LinPass s = base_pass(&a, p);
    s.x = a.q, s.k = a.k, s.v = a.v, s.y = out;
    s.rx = a.H / a.Hk;
    s.dx = a.d, s.dy = a.dv;
    s.s_fin = a.scale;
    const States x = states(&a, p, s, sums, carry, a.init_state, final_state);
    if (run_states(&a, p, &x, 1, st)) return launch_failed("linear attention states");
    if (p.nseg == 0) return ok();
    if (run_passes(&s, 1, false, a.dtype, st)) return launch_failed("linear attention output pass");
    return ok();
}

int hla2_linattn_backward(const hla2_linattn_args* args, hla2_view dout, hla2_view dq, hla2_view dk, hla2_view dv,
                          const float* dfinal_state, float* dinit_state, hla2_stream_t stream) {
    static const char* const fn = "hla2_linattn_backward";
    Range range(fn);
    if (int rc = check_sizes(fn, args)) return rc;
    hla2_linattn_args a = *args;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a.B == 0 || a.H == 0) return ok();
    const int es = elem_size(a.dtype);
    if (!al16(a.init_state) || !al16(dfinal_state) || !al16(dinit_state))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: states must be 16-byte aligned", fn);
    // several passes read the states, the first of them writes dinit_state
    if (meet(state_extent(&a, dinit_state), state_extent(&a, dfinal_state)) ||
        meet(state_extent(&a, dinit_state), state_extent(&a, a.init_state)))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dinit_state overlaps another state", fn);
    if (a.n > 0) {
        if (int rc = check_view(fn, "q", a.q, a.B, a.H, a.n, a.d, es)) return rc;
        if (int rc = check_view(fn, "k", a.k, a.B, a.Hk, a.n, a.d, es)) return rc;
        if (int rc = check_view(fn, "v", a.v, a.B, a.Hk, a.n, a.dv, es)) return rc;
        if (int rc = check_view(fn, "dout", dout, a.B, a.H, a.n, a.dv, es)) return rc;
        if (int rc = check_view(fn, "dq", dq, a.B, a.H, a.n, a.d, es)) return rc;
        if (int rc = check_view(fn, "dk", dk, a.B, a.Hk, a.n, a.d, es)) return rc;
        if (int rc = check_view(fn, "dv", dv, a.B, a.Hk, a.n, a.dv, es)) return rc;
        const Extent in[4] = {extent(a.q, a.B, a.H, a.n, a.d, es), extent(a.k, a.B, a.Hk, a.n, a.d, es),
                              extent(a.v, a.B, a.Hk, a.n, a.dv, es), extent(dout, a.B, a.H, a.n, a.dv, es)};
        const Extent go[3] = {extent(dq, a.B, a.H, a.n, a.d, es), extent(dk, a.B, a.Hk, a.n, a.d, es),
                              extent(dv, a.B, a.Hk, a.n, a.dv, es)};
        for (const Extent& o : go)
            for (const Extent& i : in)
                if (meet(o, i)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a gradient overlaps an input", fn);
        if (dq.p == dk.p || dq.p == dv.p || dk.p == dv.p)
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dq, dk and dv must be distinct", fn);
    }
    const bool rev_state = dfinal_state || dinit_state;
    const size_t need = hla2_linattn_workspace_bytes(&a, 1, rev_state);
    if (need > 0 && (!a.workspace || a.workspace_bytes < need || !al16(a.workspace)))
        return set_last_error(HLA2_ERR_WORKSPACE, "%s: needs %zu bytes of 16-byte aligned workspace", fn, need);
    const LinPlan p = plan_of(&a);
    const size_t sf = state_array_bytes(&a, p) / sizeof(float);
    float* at = p.nseg ? reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kStatusBytes) : nullptr;
    const int group = a.H / a.Hk;

    // forward states of k, v, for dq; reverse states of q, dout (scaled), for dv and dk
    const bool carried = p.nseg > 1 || a.init_state;
    LinPass q = base_pass(&a, p), v = base_pass(&a, p);
    q.k = a.k, q.v = a.v;
    q.dx = a.d, q.dy = a.dv;
    v.rev = 1;
    v.rk = group;
    v.k = a.q, v.v = dout;
    v.dx = a.d, v.dy = a.dv;
    v.s_col = v.s_state = a.scale;
    States x[2];
    int nx = 0;
    if (p.nseg > 0) x[nx++] = states(&a, p, q, at, at + sf, a.init_state, nullptr);
    if (carried) at += 2 * sf;
    x[nx++] = states(&a, p, v, at, at + sf, dfinal_state, dinit_state);
    if (run_states(&a, p, x, nx, st)) return launch_failed("linear attention states");
    if (p.nseg == 0) return ok();

    q.x = dout, q.k = a.v, q.v = a.k, q.y = dq;
    q.rx = group;
    q.dx = a.dv, q.dy = a.d;
    q.carry_t = 1;
    q.s_fin = a.scale;
    v.x = a.k, v.y = dv;
    LinPass k = v;
    k.fin = nullptr;
    k.x = a.v, k.k = dout, k.v = a.q, k.y = dk;
    k.dx = a.dv, k.dy = a.d;
    k.carry_t = 1;
    const LinPass passes[3] = {q, v, k};
    if (run_passes(passes, 3, false, a.dtype, st)) return launch_failed("linear attention gradients");
    return ok();
}

int hla2_linattn_decode_step(float* state, const void* q, const void* k, const void* v, void* out, int N, int H,
                             int Hk, int d, int dv, const float* gamma, float scale, int dtype,
                             hla2_stream_t stream) {
    static const char* const fn = "hla2_linattn_decode_step";
    Range range(fn);
    hla2_linattn_args a{};
    a.dtype = dtype, a.B = N, a.H = H, a.Hk = Hk, a.n = 1, a.d = d, a.dv = dv;
    if (int rc = check_sizes(fn, &a)) return rc;
    if (N == 0 || H == 0) return ok();
    if (!state || !q || !k || !v || !out)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: pointers must not be NULL", fn);
    if (!al16(state) || !al16(q) || !al16(k) || !al16(v) || !al16(out))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
    const size_t es = elem_size(dtype), nh = (size_t)N * H, nk = (size_t)N * Hk;
    const Extent in[3] = {extent_of(q, nh * d * es), extent_of(k, nk * d * es), extent_of(v, nk * dv * es)};
    const Extent eo = extent_of(out, nh * dv * es), est = extent_of(state, nk * d * dv * sizeof(float));
    if (meet(eo, est)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out overlaps the state", fn);
    for (const Extent& i : in)
        if (meet(i, eo) || meet(i, est))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: out or the state overlaps an input", fn);
    if (launch_lin_step(state, q, k, v, out, N, H, Hk, d, dv, gamma, scale, dtype == HLA2_BF16,
                        reinterpret_cast<cudaStream_t>(stream)))
        return launch_failed("linear attention step");
    return ok();
}

}  // extern "C"
