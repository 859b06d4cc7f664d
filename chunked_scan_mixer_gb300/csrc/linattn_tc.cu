// First-order linear attention with a decay for each head on the 5th-generation tensor cores:
// bf16 rows, chunks of 128 rows, float32 sums.  The mathematics of a pass is in linattn_pass.h.
//
// Tiles are [128 rows][D] bf16 with D = 64 or 128, loaded and stored by TMA straight from and to
// the caller's strided tensors; a smaller dx or dy is filled with zeros by the copy, so one kernel
// covers every pair of sizes.  Per chunk, with Sig the state at its entry (forward; reverse
// mirrors the decays):
//   MMA-G   G = X K^T                                   128 x 128 float32 in tensor memory
//   EPI-1   G~ = mask(G) s_col g^(64-a_j) -> bf16, over G's own columns: A operand of MMA-Y
//   MMA-C   Y = X Sig~ (Sig~ = bf16 of g^64 Sig)   MMA-Y   Y += G~ V
//   EPI-Y   s_fin g^(a_i-64) Y -> bf16 tile -> TMA store
//   KT      K~ = s_state g^(Wc-1-j) K in pieces of bf16, in shared memory
//   MMA-S   dSig = K~^T V;   EPI-S   Sig <- g^Wc Sig + dSig  (float32 registers), publish Sig~
// with a_i = i + 1 (reverse: 128 - i), the distance of row i to the carry (reverse: of a whole chunk; a
// shorter one, which comes first, takes its carry times g^(Wc-128) more).  g^(i-j) = g^(a_i-64) g^(64-a_j):
// the row's factor waits for the end, so both products share one accumulator and EPI-1 needs a
// factor per column only.  Its powers stay within g^(+-64), which float32 and bf16 hold as long as g
// >= 2^(-60/64) = 0.52; a head that decays faster ("steep") takes g^(i-j) itself in EPI-1 and has MMA-C's
// result scaled in tensor memory (EPI-C) before MMA-Y adds to it.
//
// Roundings to bf16.  G~ and Sig~ are operands of one product each and are rounded once, which
// adds to the output about its own rounding (measured against 64 bits: 2.3e-3 to 2.5e-3 relative where
// a float32 form rounded at the end has 1.65e-3).  A second operand for what is cut off would double those
// products, and the state's has no room beside the slots at either size (226 of 227 KB are used).  The decayed keys are cut into two pieces (16
// bits, 2^-17) here, where they only feed Sig~, and into three (24 bits, exact to float32) in the
// summary kernel, whose sums become the states that are returned.  Decays stay float32 and out of
// the operands everywhere else.
//
// Work items.  A state head has rx x / y heads (queries that share a key head) or rk key / value
// heads (their gradients); item (chunk, r) is one product chain.  With rx > 1 the keys, values
// and the state are loaded and formed once per chunk for all its items; with rk > 1 X, Y and the state
// are, and Y and dSig accumulate over the items in tensor memory.
//
// Roles (one CTA per SM): warp 0 allocates tensor memory and issues MMA-G, MMA-C and MMA-Y, warp 3
// MMA-S; warp 1 issues the loads, warp 2 the stores; warps 4..11 (A: a row and half of its columns
// per thread) run EPI-1 and EPI-Y; warps 12.. (B) run KT and EPI-S.  The chains A and B only meet in
// Sig~.  There are two Gram regions: the next item's Gram (at D = 64 also its EPI-1) runs while this one's
// products do.
//
// What a hand-over costs decides the time of a chunk (measured, in SM cycles: issuing one MMA 49, a
// commit 52, a wait on an mbarrier whose phase is already complete 45 to 90 and twice that while
// sixteen warps poll, a named barrier 16).  So: threads meet in named barriers; only commits and copies
// signal mbarriers, which one lane of one warp of A or of B polls for its group; a commit is made where
// someone waits for it, and slots are released by the epilogue that saw the commit.  Every poll is
// bounded; one that gives up records its site in the status word, and every role runs on to its
// end without waiting (each meets the same named barriers on any path).
//
// The loops are kept short on purpose.  The roles run different code side by side, straight through it once a
// chunk, so together they have to fit the SM's instruction cache: fully unrolled they took
// 102 KB, half of all instruction fetches missed, and the epilogues ran at 20 cycles an instruction.
//
// D = 64 stacks the two key pieces as one 128-row A operand (rows 0..63 the high piece's
// features, 64..127 the low one's), so MMA-S has full height; the two halves of the state stay
// apart and MMA-C takes both (K = 128), which costs nothing there.  D = 128 has no shared memory
// for a second piece beside two slots of each tile: the high piece replaces the keys, and once it has
// been multiplied the low one, kept in registers, replaces it.
#include "fo_common.cuh"
#include "linattn_pass.h"

namespace hla2 {

namespace {

namespace lt {

constexpr int kW = 128;
constexpr int kA0 = 4, kAWarps = 8, kB0 = 12;
__host__ __device__ constexpr int b_warps(int D) { return D == 64 ? 8 : 16; }
__host__ __device__ constexpr int threads(int D) { return 32 * (kB0 + b_warps(D)); }
constexpr uint32_t kBlk = la_common::kBlk;  // [128 rows][64 bf16]

struct Maps {
    CUtensorMap x, k, v, y;
};

__device__ __forceinline__ void load_4d(void* dst, const CUtensorMap* m, int x, int row, int h, int b, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
            "r"(smem_u32(dst)), "l"(m), "r"(x), "r"(row), "r"(h), "r"(b), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void store_4d(const CUtensorMap* m, const void* src, int x, int row, int h, int b) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(m), "r"(x),
                 "r"(row), "r"(h), "r"(b), "r"(smem_u32(src))
                 : "memory");
}

// Wait of one thread for the phase of the given parity; after about two seconds it gives up.
constexpr long long kWaitClocks = 4LL * 1000 * 1000 * 1000;
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int where) {
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (clock64() - t0 > kWaitClocks) {
            *abort = 1;
            if (status) atomicCAS(status, 0, where);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int where) {
    return tc::mbar_try_wait(bar, parity) || wait_long(bar, parity, abort, status, where);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Two float32 products in one instruction
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b, float c, float d) {
    uint64_t p, q, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %2};" : "=l"(q) : "f"(c), "f"(d));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(p), "l"(q));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Named barriers (0 is __syncthreads)
enum { kNbSC = 4, kNbGT = 5, kNbKT = 7, kNbSP = 8, kNbVZ = 10, kNbA = 12, kNbB = 13 };
constexpr int kRef = 64;                  // the middle of the row factors
constexpr float kSteep = -60.f / kRef;    // log2 of the decay below which the factors are not split

template <int D>
struct Out {  // shared memory of the output kernel
    static constexpr uint32_t kTile = (uint32_t)(D / 64) * kBlk;
    static constexpr int NS = D == 64 ? 4 : 2;           // slots of each of x, k, v
    static constexpr uint32_t oX = 0, oK = oX + NS * kTile, oV = oK + NS * kTile, oM = oV + NS * kTile,
                              oS = oM + (D == 64 ? kTile : 0);
    static constexpr uint32_t oGp = oS + kTile;          // g^0 .. g^128
    static constexpr uint32_t oCol = oGp + 4 * 132;      // s_col g^(64 - a_j), j = 0 .. 127
    static constexpr uint32_t oBar = oCol + 4 * 128;
    enum { XF = 0, XE = XF + NS, OS = XE + NS, KF = OS + NS, VF = KF + NS, E = VF + NS, BG = E + NS, BGK = BG + 4, BC = BGK + 2, YL, YD,
           YI, SH, SD, kBars };
    static constexpr uint32_t oMisc = oBar + kBars * 8;
    static constexpr uint32_t kBytes = oMisc + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

// Tensor memory columns of the output kernel: two Gram regions, Y, dSig.
template <int D>
struct Cols {
    // Whether the next Gram and its EPI-1 come before this item's products.  At D = 128 its tiles, of
    // which there are two slots only, arrive too late for that.
    static constexpr bool kEarly = D == 64;
    __device__ static constexpr uint32_t G(int i) { return (uint32_t)(i & 1) * 128; }
    static constexpr uint32_t Y = 256, S = Y + D;
};

struct Where {  // the CTA's state head, segment and valid chunks
    int bs, b, s, len, c0, c1, nit;
};
__device__ __forceinline__ Where locate(const LinPass& a) {
    Where w;
    w.bs = blockIdx.x;
    w.b = w.bs / a.Hs;
    w.s = w.bs % a.Hs;
    w.len = lin_len(a.lengths, w.b, a.n);
    w.c0 = blockIdx.y * a.seg_chunks;
    const int end = min(w.c0 + a.seg_chunks, a.nchunks);
    w.c1 = min(end, (w.len + kW - 1) / kW);
    w.nit = max(0, w.c1 - w.c0);
    w.len = uniform(w.len);
    w.c1 = uniform(w.c1);
    w.nit = uniform(w.nit);
    return w;
}

// bf16 pieces of w times eight bf16 values: hi, the rest's high part, and what is left
template <int P>
__device__ __forceinline__ void pieces8(uint4 c, float w, uint4 (&out)[P]) {
    float f[8] = {la_bf_lo(c.x), la_bf_hi(c.x), la_bf_lo(c.y), la_bf_hi(c.y),
                  la_bf_lo(c.z), la_bf_hi(c.z), la_bf_lo(c.w), la_bf_hi(c.w)};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= w;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        out[p] = la_pack8(f);
        if (p + 1 < P) {
            const uint32_t u[4] = {out[p].x, out[p].y, out[p].z, out[p].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] -= la_bf_lo(u[i]);
                f[2 * i + 1] -= la_bf_hi(u[i]);
            }
        }
    }
}

// The state that enters the CTA's segment, into shared memory as it is stored (rows padded by four
// floats), and the state after the scan.  Coalesced, by all threads: read by the threads that keep it, a
// lane to a row, 128 x 128 states took 8 us of each CTA.
__device__ __forceinline__ void stage_carry(const LinPass& a, const Where& w, float* to, float log2g, int tid, int threads) {
    const int elems = a.dx * a.dy, inner = (a.carry_t ? a.dx : a.dy) / 4;
    const int order = a.rev ? a.nseg - 1 - (int)blockIdx.y : blockIdx.y, seg_rows = a.seg_chunks * kW;
    const bool ends = a.fin && order == a.nseg - 1;
    const size_t head = (size_t)w.bs * elems;
    const float g = lin_decay(a, w.s);
    auto decay = [&](int i) {
        return pow_decay(log2g, (float)(lin_rows_before(w.len, a.rev, i + 1, a.nseg, seg_rows) -
                                        lin_rows_before(w.len, a.rev, i, a.nseg, seg_rows)));
    };
    auto step = [](float4& c, float f, const float4& v) {
        c = make_float4(fmaf(f, c.x, v.x), fmaf(f, c.y, v.y), fmaf(f, c.z, v.z), fmaf(f, c.w, v.w));
    };
    auto scaled = [](const float4& c, float f) { return make_float4(f * c.x, f * c.y, f * c.z, f * c.w); };
#pragma unroll 1
    for (int e = tid; e < elems / 4; e += threads) {
        float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.carry) {
            cur = reinterpret_cast<const float4*>(a.carry + (head * a.nseg + (size_t)blockIdx.y * elems))[e];
        } else {
            if (a.init) {
                cur = reinterpret_cast<const float4*>(a.init + head)[e];
                if (a.rev) cur = make_float4(cur.x / g, cur.y / g, cur.z / g, cur.w / g);
            }
            const float4* sums = reinterpret_cast<const float4*>(a.prior + head * a.nseg) + e;
            const int count = order + (ends ? 1 : 0);  // sums to read
            float4 f = cur;
#pragma unroll 1
            for (int i0 = 0; i0 < count; i0 += 4) {
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i0 + i < count) v[i] = sums[(size_t)(a.rev ? a.nseg - 1 - i0 - i : i0 + i) * (elems / 4)];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i0 + i >= count) break;
                    cur = f;
                    step(f, decay(i0 + i), v[i]);
                }
            }
            if (ends) reinterpret_cast<float4*>(a.fin + head)[e] = a.rev ? scaled(f, g) : f;
            else cur = f;
        }
        *reinterpret_cast<float4*>(to + (e / inner) * (inner + 1) * 4 + e % inner * 4) = cur;
    }
}

__device__ __forceinline__ uint64_t kdesc(uint32_t base, int ks) {  // K-major, K step of 16 features
    return tc::smem_desc(base + (uint32_t)(ks >> 2) * kBlk + (uint32_t)(ks & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t mdesc(uint32_t base, int ks, uint32_t lbo = kBlk) {  // MN-major, 16 rows
    return tc::smem_desc(base + 2048u * ks, lbo, 1024);
}

}  // namespace lt

// ----------------------------------------------------------------------------------------
// Output kernel
// ----------------------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(lt::threads(D), 1) lin_out_tc_kernel(const __grid_constant__ lt::Maps maps, const LinPass a) {
    using L = lt::Out<D>;
    using C = lt::Cols<D>;
    constexpr int kW = lt::kW, kThreads = lt::threads(D), kBWarps = lt::b_warps(D);
    constexpr int kBlocks = D / 64;
    constexpr int kSC = D / (kBWarps / 4);  // state columns per B thread
    constexpr int NS = L::NS;
    extern __shared__ unsigned char smem_raw[];
    // an offset, not a rounded pointer: the compiler then still knows the address space
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* gp = reinterpret_cast<float*>(sm + L::oGp);
    float* colf = reinterpret_cast<float*>(sm + L::oCol);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::oMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::oMisc + 4);
    int* status = a.status;

    const int tid = threadIdx.x, warp = lt::uniform(tid >> 5), lane = tid & 31;
    pdl_trigger();
    if (tid == 0) {
        for (int i = 0; i < L::kBars; ++i) {
            const bool by_a = i >= L::OS && i < L::OS + NS;   // one arrival per A warp
            const bool by_two = i >= L::E && i < L::E + NS;   // A (or MMA-Y's commit) and B
            tc::mbar_init(&bars[i], by_a ? lt::kAWarps : by_two ? 2 : 1);
        }
        *abort = 0;
        tc::mbar_fence_init();
    }
    pdl_wait();
    const lt::Where w = lt::locate(a);
    const bool rev = a.rev != 0, mode_a = a.rx > 1, mode_b = a.rk > 1;
    const int items = mode_a ? a.rx : a.rk, total = w.nit * items;
    const float log2g = log2f(lin_decay(a, w.s));

    // rows of the segment past the sequence: zeros
    {
        const int z0 = max(w.c0, w.c1) * kW, z1 = min((w.c0 + a.seg_chunks) * kW, a.n);
        const int per = a.dy / 8, count = max(0, z1 - z0) * per;
#pragma unroll 1
        for (int h = 0; h < a.rx; ++h) {
            bf16* y = static_cast<bf16*>(const_cast<void*>(a.y.p)) + w.b * a.y.sb + (long long)(w.s * a.rx + h) * a.y.sh;
#pragma unroll 1
            for (int e = tid; e < count; e += kThreads)
                *reinterpret_cast<uint4*>(y + (long long)(z0 + e / per) * a.y.sn + (e % per) * 8) = make_uint4(0, 0, 0, 0);
        }
    }
    const bool carried = a.carry || a.init || (a.prior && (rev ? blockIdx.y + 1 < a.nseg : blockIdx.y > 0));
    const bool ends = a.fin && blockIdx.y == (rev ? 0 : a.nseg - 1);
    float* const stage = reinterpret_cast<float*>(sm + L::oX);  // before the first copy arrives there
    if ((carried && w.nit > 0) || ends) lt::stage_carry(a, w, stage, log2g, tid, kThreads);
    if (w.nit == 0) return;

    const bool steep = log2g < lt::kSteep;
    auto dist = [&](int i) { return rev ? kW - i : i + 1; };  // a_i
    if (tid <= kW) gp[tid] = pow_decay(log2g, (float)tid);
    if (tid < kW) colf[tid] = steep ? 0.f : a.s_col * pow_decay(log2g, (float)(lt::kRef - dist(tid)));
    if (warp == 0) tc::tmem_alloc(tmem_holder, 512);

    // B thread: state row sr, columns sc0 .. sc0 + kSC - 1.  D = 64: rows 64.. hold the low pieces' sums.
    const int q4 = warp & 3, part = (warp - lt::kB0) >> 2;
    const int sr = 32 * q4 + lane, sc0 = part * kSC;
    float sig[kSC];
    auto publish = [&](float pub) {  // pub: g^64
#pragma unroll
        for (int j = 0; j < kSC / 8; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = pub * sig[8 * j + i];
            *reinterpret_cast<uint4*>(sm + L::oS + la_off(sc0 / 64, sr, (sc0 % 64) / 8 + j)) = la_pack8(f);
        }
    };
    __syncthreads();
    if (warp >= lt::kB0) {
        // D = 64: dx <= 64, so only the high half takes the carry
        const bool has = carried && sr < a.dx;
        const float* src = stage + (a.carry_t ? sc0 * (a.dx + 4) + sr : sr * (a.dy + 4) + sc0);
        const int step = a.carry_t ? a.dx + 4 : 1;
#pragma unroll
        for (int j = 0; j < kSC; j += 4) {
            const bool in = has && sc0 + (j & ~15) < a.dy;  // dy is a multiple of 16
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in && !a.carry_t) v = *reinterpret_cast<const float4*>(src + j);
            else if (in) v = make_float4(src[j * step], src[(j + 1) * step], src[(j + 2) * step], src[(j + 3) * step]);
            sig[j] = v.x, sig[j + 1] = v.y, sig[j + 2] = v.z, sig[j + 3] = v.w;
        }
        const int first = rev ? w.c1 - 1 : w.c0, Wc = min(kW, w.len - first * kW);
        publish(steep ? 1.f : pow_decay(log2g, (float)(lt::kRef - (rev ? kW - Wc : 0))));
    }
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = (uint32_t)lt::uniform((int)*tmem_holder);
    auto chunk_of = [&](int ci) { return rev ? w.c1 - 1 - ci : w.c0 + ci; };
    auto valid_of = [&](int ci) { return min(kW, w.len - chunk_of(ci) * kW); };
    volatile int never = 0;

    constexpr int kAThreads = 32 * lt::kAWarps, kBThreads = 32 * kBWarps;
    constexpr uint32_t T = L::kTile >> 4;    // descriptor units (16 bytes): a slot, and 16 rows MN-major
    constexpr uint64_t kMK = 2048 >> 4;
    auto kstep = [](int ks) { return (uint64_t)(((ks >> 2) * lt::kBlk + (ks & 3) * 32) >> 4); };  // K-major

    if (warp == 0) {
        // ----------------------------------------------------------- MMA-G, MMA-C, MMA-Y
        constexpr uint32_t I_G = tc::idesc_bf16(128, 128, 0, 0), I_Y = tc::idesc_bf16(128, D, 0, 1);
        const uint64_t dX = lt::kdesc(smem_u32(sm + L::oX), 0), dK = lt::kdesc(smem_u32(sm + L::oK), 0),
                       dV = lt::mdesc(smem_u32(sm + L::oV), 0), dS = lt::mdesc(smem_u32(sm + L::oS), 0);
        int r = -1, ci = 0;
#pragma unroll 1
        for (int it = -1; it < total; ++it) {
            // item it = (chunk ci, r); -1: only the first Gram
            const bool first = r == 0, last = r == items - 1;
            const bool new_y = !mode_b || first, end_y = !mode_b || last;
            const int ki = mode_b ? it : ci, xi = mode_b ? ci : it;
            __syncwarp();
            auto products = [&]() {
                if (first && ci > 0) tc::named_bar(lt::kNbSP, kBThreads + 32);
                tc::named_bar(lt::kNbGT + (it & 1), kAThreads + 32);  // also: Y of the item before is read
                if (lane == 0) {
                    tc::fence_after_sync();
                    if (new_y) {
                        const uint64_t x = dX + (xi % NS) * T;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)  // D = 64: the two halves of the state in turn
                            tc::mma_ss(tmem + C::Y, x + kstep(D == 64 ? ks & 3 : ks), dS + ks * kMK, I_Y, ks > 0);
                        if (steep) tc::mma_commit(&bars[L::BC]);
                    }
                    if (!mode_a || first) lt::wait(&bars[L::VF + ki % NS], (ki / NS) & 1, abort, status, 305);
                }
                __syncwarp();
                if (a.lengths && (!mode_a || first)) tc::named_bar(lt::kNbVZ + (ki & 1), kBThreads + 64);
                if (steep && new_y) tc::named_bar(lt::kNbSC, kAThreads + 32);
                if (lane == 0) {
                    tc::fence_after_sync();
                    const uint64_t v = dV + (ki % NS) * T;
                    const uint32_t tg = tmem + C::G(it);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)  // G~: columns 0..63 of the Gram in its first 32, the rest from 64 on
                        tc::mma_ts(tmem + C::Y, tg + 8 * (ks & 3) + (ks >> 2) * 64, v + ks * kMK, I_Y, 1);
                    if (end_y) tc::mma_commit(&bars[L::YD]);
                    if (mode_a && last) tc::mma_commit(&bars[L::YL]);
                    if (mode_b) {
                        tc::mma_commit(&bars[L::E + ki % NS]);
                        tc::mma_commit(&bars[L::YI]);
                    }
                }
            };
            // (in turn, before the next commit on it: nobody else waits for YI, and the drain would take its phase
            // before the last one for the last)
            if (lane == 0 && it > 0 && (mode_b || it + 1 < total))
                lt::wait(&bars[mode_b ? L::YI : L::YD], (it - 1) & 1, abort, status, 308);
            if (!C::kEarly && it >= 0) products();
            if (lane == 0 && it + 1 < total) {  // MMA-G, into the region that MMA-Y of it - 1 read
                const bool wrap = last || it < 0;  // the next item begins a chunk
                const int rn = wrap ? 0 : r + 1, cn = it < 0 ? 0 : ci + (last ? 1 : 0);
                const int xn = mode_b ? cn : it + 1, kn = mode_a ? cn : it + 1;
                if (!mode_b || rn == 0) lt::wait(&bars[L::XF + xn % NS], (xn / NS) & 1, abort, status, 301);
                if (!mode_a || rn == 0) lt::wait(&bars[L::KF + kn % NS], (kn / NS) & 1, abort, status, 302);
                tc::fence_after_sync();
                const uint64_t x = dX + (xn % NS) * T, k = dK + (kn % NS) * T;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc::mma_ss(tmem + C::G(it + 1), x + kstep(ks), k + kstep(ks), I_G, ks > 0);
                tc::mma_commit(&bars[L::BG + ((it + 1) & 3)]);  // four: B may be three tiles behind
                // two: with two items a chunk, B may be waiting for the chunk before
                if (mode_a && rn == items - 1) tc::mma_commit(&bars[L::BGK + (cn & 1)]);
            }
            __syncwarp();
            if (C::kEarly && it >= 0) products();
            if (++r == items) r = 0, ++ci;
            if (it < 0) r = 0, ci = 0;
        }
        // drain: the last commit covers every MMA of this thread
        if (lane == 0)
            lt::wait(&bars[mode_b ? L::YI : mode_a ? L::YL : L::YD], ((mode_a ? w.nit : total) - 1) & 1, &never, nullptr, 0);
    } else if (warp == 3) {
        // --------------------------------------------------------------------------- MMA-S
        constexpr uint32_t I_S = tc::idesc_bf16(128, D, 1, 1);
        const uint32_t sK = smem_u32(sm + L::oK), sM = smem_u32(sm + L::oM);
        const uint64_t dK = lt::mdesc(sK, 0, D == 64 ? sM - sK : lt::kBlk), dV = lt::mdesc(smem_u32(sm + L::oV), 0);
        const int tiles = mode_a ? w.nit : total, per = mode_a ? 1 : items;
#pragma unroll 1
        for (int ki = 0, r = 0, ci = 0; ki < tiles; ++ki, ci += ++r == per, r = r == per ? 0 : r) {
            const int slot = ki % NS;
            if (a.lengths) tc::named_bar(lt::kNbVZ + (ki & 1), kBThreads + 64);
            if (ci + 1 >= w.nit) continue;  // no state after the last chunk
            const uint64_t v = dV + slot * T;
            // D = 64: the low piece's tile is the second 64-row block of A, at a distance (the block
            // stride field) that shrinks with the slot
            const uint64_t k = dK + slot * T - (D == 64 ? (uint64_t)(slot * T) << 16 : 0);
#pragma unroll 1
            for (int piece = 0; piece < (D == 64 ? 1 : 2); ++piece) {
                tc::named_bar(lt::kNbKT, kBThreads + 32);
                if (lane == 0) {
                    lt::wait(&bars[L::VF + slot], (ki / NS) & 1, abort, status, 306);
                    tc::fence_after_sync();
                    const uint32_t acc = r > 0 || piece > 0;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        tc::mma_ss(tmem + C::S, k + ks * kMK, v + ks * kMK, I_S, ks > 0 ? 1u : acc);
                    tc::mma_commit(&bars[D == 64 || piece > 0 ? L::SD : L::SH]);
                }
                __syncwarp();
            }
        }
        const int done = w.nit > 1 ? (w.nit - 1) * per : 0;
        if (lane == 0 && done > 0) lt::wait(&bars[L::SD], (done - 1) & 1, &never, nullptr, 0);
    } else if (warp == 1) {
        if (lane == 0) {
            // ----------------------------------------------------------------------- loads
            int nx = 0, nkv = 0, nv = 0;
            auto load = [&](uint32_t slot, const CUtensorMap* m, int row, int h, uint64_t* bar) {
                tc::mbar_arrive_expect_tx(bar, L::kTile);
#pragma unroll 1
                for (int i = 0; i < kBlocks; ++i) lt::load_4d(sm + slot + i * lt::kBlk, m, 64 * i, row, h, w.b, bar);
            };
#pragma unroll 1
            for (int it = 0, r = 0, ci = 0; it < total; ++it, ci += ++r == items, r = r == items ? 0 : r) {
                const int row = chunk_of(ci) * kW;
                if (!mode_b || r == 0) {
                    const int slot = nx % NS;
                    if (nx >= NS && !lt::wait(&bars[L::XE + slot], (nx / NS - 1) & 1, abort, status, 311)) break;
                    load(L::oX + slot * L::kTile, &maps.x, row, w.s * a.rx + (mode_a ? r : 0), &bars[L::XF + slot]);
                    ++nx;
                }
                if (!mode_a || r == 0) {
                    const int h = w.s * a.rk + (mode_b ? r : 0), slot = nkv % NS;
                    if (nkv >= NS && !lt::wait(&bars[L::E + slot], (nkv / NS - 1) & 1, abort, status, 312)) break;
                    load(L::oK + slot * L::kTile, &maps.k, row, h, &bars[L::KF + slot]);
                    load(L::oV + slot * L::kTile, &maps.v, row, h, &bars[L::VF + slot]);
                    ++nkv;
                }
            }
            nv = nkv;
            // drain: every load has landed
#pragma unroll 1
            for (int i = max(0, nx - NS); i < nx; ++i) lt::wait(&bars[L::XF + i % NS], (i / NS) & 1, &never, nullptr, 0);
#pragma unroll 1
            for (int i = max(0, nv - NS); i < nv; ++i) {
                lt::wait(&bars[L::KF + i % NS], (i / NS) & 1, &never, nullptr, 0);
                lt::wait(&bars[L::VF + i % NS], (i / NS) & 1, &never, nullptr, 0);
            }
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ---------------------------------------------------------------------- stores
            const int groups = mode_b ? w.nit : total, per = mode_a ? items : 1;
#pragma unroll 1
            for (int g = 0, r = 0, ci = 0; g < groups; ++g, ci += ++r == per, r = r == per ? 0 : r) {
                const int slot = g % NS;
                if (!lt::wait(&bars[L::OS + slot], (g / NS) & 1, abort, status, 321)) break;
                const int row = chunk_of(ci) * kW, h = w.s * a.rx + r;
#pragma unroll 1
                for (int i = 0; i < kBlocks; ++i)
                    if (64 * i < a.dy)
                        lt::store_4d(&maps.y, sm + L::oX + slot * L::kTile + i * lt::kBlk, 64 * i, row, h, w.b);
                tc::bulk_commit();
                tc::bulk_wait_read_all();
                tc::mbar_arrive(&bars[L::XE + slot]);
            }
            tc::bulk_wait_all();
        }
    } else if (warp < lt::kB0) {
        // ------------------------ A: row i of the chunk, half ah of the columns per thread
        const int i = 32 * q4 + lane, row0 = 32 * q4, ah = (warp - lt::kA0) >> 2;
        const uint32_t lanes = (uint32_t)row0 << 16;
        const bool poller = warp == lt::kA0 && lane == 0;
        auto wait_a = [&](int bar, int parity, int where) {
            if (poller) lt::wait(&bars[bar], parity, abort, status, where);
            __syncwarp();
            tc::named_bar(lt::kNbA, kAThreads);
            tc::fence_after_sync();
        };
        // EPI-1 of item it (Wc valid rows): columns 64 ah .. 64 ah + 63, 16 at a time, packed over the first
        // half of them.  Products of masked columns are selected away (past the sequence they may be
        // anything).
        auto epi1 = [&](int it, int Wc) {
            const uint32_t tg = tmem + lanes + C::G(it) + 64 * ah;
            wait_a(L::BG + (it & 3), (it >> 2) & 1, 331);
            const int limit = rev ? Wc : kW;
#pragma unroll 1
            for (int cb = 0; cb < 64; cb += 16) {
                const int c = 64 * ah + cb;
                const bool some = rev ? c + 15 >= row0 : c <= row0 + 31;  // some row keeps some column
                const bool all = (rev ? c > row0 + 31 : c + 15 < row0) && c + 15 < limit;
                uint32_t pk[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                if (some) {
                    uint32_t g[16];
                    float f[16];
                    tc::tmem_ld16(tg + cb, g);
                    if (steep) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) f[j] = a.s_col * gp[abs(i - c - j)];
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<float4*>(f + j) = *reinterpret_cast<const float4*>(colf + c + j);
                    }
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; j += 2)
                        lt::mul2(f[j], f[j + 1], f[j], f[j + 1], __uint_as_float(g[j]), __uint_as_float(g[j + 1]));
                    if (!all) {
                        const int lo = rev ? i - c : 0, hi = rev ? limit - c : i - c + 1;  // kept: lo <= j < hi
#pragma unroll
                        for (int j = 0; j < 16; ++j) f[j] = j >= lo && j < hi ? f[j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) pk[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
                }
                lt::tmem_st8(tg + cb / 2, pk);  // columns that this thread has read
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
        };
        const float fin = a.s_fin * (steep ? 1.f : pow_decay(log2g, (float)(dist(i) - lt::kRef)));
        int groups = 0, r = -1, ci = 0;
#pragma unroll 1
        for (int it = -1; it < total; ++it) {
            // item it = (chunk ci, r); -1: only the first EPI-1
            const bool last = r == items - 1, new_y = it >= 0 && (!mode_b || r == 0), end_y = it >= 0 && (!mode_b || last);
            const int Wc = valid_of(ci), Wn = valid_of(it >= 0 && last ? ci + 1 : ci);
            const uint32_t ty = tmem + lanes + C::Y + ah * (D / 2);
            if (it >= 0) tc::named_arrive(lt::kNbGT + (it & 1), kAThreads + 32);
            if (steep && new_y) {  // EPI-C
                wait_a(L::BC, groups & 1, 332);
                const float f = gp[rev ? max(Wc - i, 0) : i + 1];
#pragma unroll 1
                for (int cb = 0; cb < D / 2; cb += 16) {
                    uint32_t y[16];
                    tc::tmem_ld16(ty + cb, y);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(f * __uint_as_float(y[j]));
                    tc::tmem_st16(ty + cb, y);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::named_arrive(lt::kNbSC, kAThreads + 32);
            }
#pragma unroll 1
            for (int step = 0; step < 2; ++step) {
                if ((step == 0) == C::kEarly) {
                    if (it + 1 < total) epi1(it + 1, Wn);
                } else if (end_y) {
                    // EPI-Y, into the X tile, which the products have read
                    wait_a(L::YD, groups & 1, 333);
                    if (poller && !mode_b && last) tc::mbar_arrive(&bars[L::E + (mode_a ? ci : it) % NS]);
                    unsigned char* st = sm + L::oX + (groups % NS) * L::kTile;
                    const bool live = i < Wc;
                    uint32_t y[16];
                    tc::tmem_ld16(ty, y);
    #pragma unroll 1
                    for (int cb = 0; cb < D / 2; cb += 16) {
                        float o[16];
                        tc::tmem_wait_ld();
    #pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = live ? fin * __uint_as_float(y[j]) : 0.f;
                        if (cb + 16 < D / 2) tc::tmem_ld16(ty + cb + 16, y);
    #pragma unroll
                        for (int j = 0; j < 16; j += 8) {
                            const int col = ah * (D / 2) + cb + j;
                            *reinterpret_cast<uint4*>(st + la_off(col / 64, i, (col % 64) / 8)) = la_pack8(o + j);
                        }
                    }
                    tc::fence_before_sync();
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars[L::OS + groups % NS]);
                    ++groups;
                }
            }
            if (++r == items) r = 0, ++ci;
            if (it < 0) r = 0, ci = 0;
        }
    } else {
        // -------------------------------------------- B: keys' pieces, the values' padding, the state
        const int row = 32 * q4 + lane;             // KT: row of the chunk; 16-byte chunks of it below
        constexpr int kC = D / 8 / (kBWarps / 4);   // 16-byte chunks per thread
        const int c0 = part * kC;                   // chunk index over the whole row: block c / 8, chunk c % 8
        const uint32_t lanes = (uint32_t)(32 * q4) << 16;
        const bool poller = warp == lt::kB0 && lane == 0;
        const float pub = steep ? 1.f : gp[lt::kRef];
        auto meet = [&]() {  // after the poller's waits
            __syncwarp();
            tc::named_bar(lt::kNbB, kBThreads);
        };
        const int tiles = mode_a ? w.nit : total, per = mode_a ? 1 : items;
#pragma unroll 1
        for (int ki = 0, r = 0, ci = 0; ki < tiles; ++ki, ci += ++r == per, r = r == per ? 0 : r) {
            const int Wc = valid_of(ci), slot = ki % NS;
            const bool state_now = ci + 1 < w.nit, last = r == per - 1;
            // The Gram products have to have read K: with shared keys (mode a) those of the chunk's last item, and
            // then the values' padding is cleared before that.
            if (mode_a && a.lengths) {
                if (poller) lt::wait(&bars[L::VF + slot], (ki / NS) & 1, abort, status, 341);
                meet();
            }
            if (!mode_a) {
                if (poller) {
                    lt::wait(&bars[L::KF + slot], (ki / NS) & 1, abort, status, 342);
                    lt::wait(&bars[L::BG + (ki & 3)], (ki >> 2) & 1, abort, status, 343);
                    if (a.lengths) lt::wait(&bars[L::VF + slot], (ki / NS) & 1, abort, status, 341);
                }
                meet();
            }
            if (a.lengths) {
                if (Wc < min(kW, a.n - chunk_of(ci) * kW) && row >= Wc) {
#pragma unroll 1
                    for (int c = c0; c < c0 + kC; ++c)
                        *reinterpret_cast<uint4*>(sm + L::oV + slot * L::kTile + la_off(c >> 3, row, c & 7)) =
                            make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async();
                tc::named_arrive(lt::kNbVZ + (ki & 1), kBThreads + 64);
            }
            if (!state_now) {  // no product of ours reads this tile
                if (poller) tc::mbar_arrive(&bars[L::E + slot]);
                continue;
            }
            if (mode_a) {
                if (poller) {
                    lt::wait(&bars[L::KF + slot], (ki / NS) & 1, abort, status, 342);
                    lt::wait(&bars[L::BGK + (ki & 1)], (ki >> 1) & 1, abort, status, 343);
                }
                meet();
            }
            const float wt = row < Wc ? a.s_state * gp[rev ? row : Wc - 1 - row] : 0.f;
            unsigned char *kt = sm + L::oK + slot * L::kTile, *mt = sm + L::oM;
            uint4 low[D == 64 ? 1 : kC];
#pragma unroll(D == 64 ? 2 : kC)
            for (int c = 0; c < kC; ++c) {
                const uint32_t at = la_off((c0 + c) >> 3, row, (c0 + c) & 7);
                uint4 p[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (row < Wc) lt::pieces8<2>(*reinterpret_cast<const uint4*>(kt + at), wt, p);
                *reinterpret_cast<uint4*>(kt + at) = p[0];
                if (D == 64) *reinterpret_cast<uint4*>(mt + at) = p[1];
                else low[c] = p[1];
            }
            tc::fence_proxy_async();
            tc::named_arrive(lt::kNbKT, kBThreads + 32);
            if (D != 64) {  // the low piece replaces the high one
                if (poller) lt::wait(&bars[L::SH], ki & 1, abort, status, 346);
                meet();
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    *reinterpret_cast<uint4*>(kt + la_off((c0 + c) >> 3, row, (c0 + c) & 7)) = low[c];
                tc::fence_proxy_async();
                tc::named_arrive(lt::kNbKT, kBThreads + 32);
            }
            if (poller) {  // the products are done: the tile is released, the low piece may be overwritten
                lt::wait(&bars[L::SD], ki & 1, abort, status, 345);
                tc::mbar_arrive(&bars[L::E + slot]);
                // MMA-C of this chunk has read the state that publish() overwrites
                if (last) lt::wait(&bars[mode_a ? L::YL : L::YD], ci & 1, abort, status, 347);
            }
            if (!last) continue;
            // EPI-S
            meet();
            tc::fence_after_sync();
            const float rho = gp[Wc];
#pragma unroll
            for (int cb = 0; cb < kSC; cb += 16) {
                uint32_t d[16];
                tc::tmem_ld16(tmem + lanes + C::S + sc0 + cb, d);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) sig[cb + j] = fmaf(rho, sig[cb + j], __uint_as_float(d[j]));
            }
            publish(pub);
            tc::fence_before_sync();
            tc::fence_proxy_async();
            tc::named_arrive(lt::kNbSP, kBThreads + 32);
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------------------------------
// Summary kernel: Sig_B = s_state sum_i g^(distance to the segment's end) k_i v_i^T over the
// segment's rows (all key / value heads of the state).  The weights are relative to the segment, so
// nothing decays from tile to tile.  The decayed keys are cut into P pieces of bf16: three where the sums end in a
// state that is returned (exact to float32), two where they only feed the carries.  A tile's products
// accumulate in tensor memory (two regions in turn) and are added to float32 registers: accumulation
// there cuts bits off at every step, which over thousands of rows would cost a digit of the state.
// ----------------------------------------------------------------------------------------
namespace lt {
template <int D, int P>
struct Sum {
    static constexpr uint32_t kTile = (uint32_t)(D / 64) * kBlk;
    static constexpr int NS = D == 64 ? 4 : 2;               // key / value slots
    static constexpr int NP = D == 128 && P == 3 ? 1 : 2;    // buffers of the lower pieces
    static constexpr uint32_t oK = 0, oV = oK + NS * kTile, oM = oV + NS * kTile, oL = oM + NP * kTile,
                              oZ = oL + (P == 3 ? NP : 0) * kTile;  // D = 64: a tile of zeros beside the third piece
    static constexpr uint32_t oGp = oZ + (D == 64 && P == 3 ? kTile : 0);  // g^0 .. g^127
    static constexpr uint32_t oBar = oGp + 512;
    enum { KF = 0, VF = KF + NS, E = VF + NS, AD = E + NS, kBars = AD + 2 };
    static constexpr uint32_t oMisc = oBar + kBars * 8;
    static constexpr uint32_t kBytes = oMisc + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};
constexpr int kSumThreads = 640, kSumB0 = 4, kSumBWarps = 16;  // warp 0 MMA, warp 1 loads, warps 4..19 pieces and sums
}  // namespace lt

template <int D, int P>
__global__ void __launch_bounds__(lt::kSumThreads, 1) lin_sum_tc_kernel(const __grid_constant__ lt::Maps maps, const LinPass a) {
    using L = lt::Sum<D, P>;
    constexpr int kW = lt::kW, kBlocks = D / 64, kC = D / 32;  // kC: 16-byte chunks per thread and tile
    constexpr int kCols = D / 4;                               // sums per thread
    extern __shared__ unsigned char smem_raw[];
    // an offset, not a rounded pointer: the compiler then still knows the address space
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* gp = reinterpret_cast<float*>(sm + L::oGp);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::oMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::oMisc + 4);
    int* status = a.status;
    const int tid = threadIdx.x, warp = lt::uniform(tid >> 5), lane = tid & 31, q4 = warp & 3;
    pdl_trigger();
    if (tid == 0) {
        for (int i = 0; i < L::kBars; ++i) tc::mbar_init(&bars[i], 1);
        *abort = 0;
        tc::mbar_fence_init();
    }
    pdl_wait();
    const lt::Where w = lt::locate(a);
    const bool rev = a.rev != 0;
    const int items = a.rk, total = w.nit * items;
    float* dst = a.sums + ((size_t)w.bs * a.nseg + blockIdx.y) * a.dx * a.dy;
    if (w.nit == 0) {
        for (int e = tid; e < a.dx * a.dy; e += lt::kSumThreads) dst[e] = 0.f;
        return;
    }
    const float log2g = log2f(lin_decay(a, w.s));
    if (tid < kW) gp[tid] = pow_decay(log2g, (float)tid);
    if (warp == 0) tc::tmem_alloc(tmem_holder, 2 * D);
    if (D == 64 && P == 3) {
        for (int e = tid; e < (int)(L::kTile / 16); e += lt::kSumThreads)
            *reinterpret_cast<uint4*>(sm + L::oZ + 16 * e) = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = (uint32_t)lt::uniform((int)*tmem_holder);
    volatile int never = 0;
    const int seg_rows = min(w.len, w.c1 * kW) - w.c0 * kW;  // valid rows of the segment
    float sum[kCols];
    constexpr int kBThreads = 32 * lt::kSumBWarps;
    enum { kNbAll = 1, kNbKT = 2, kNbDR = 4 };  // named barriers (two of each of KT, DR: by tile parity)

    if (warp == 0) {
        constexpr uint32_t I_S = tc::idesc_bf16(128, D, 1, 1);
        constexpr uint32_t T = L::kTile >> 4;
        constexpr uint64_t kMK = 2048 >> 4;
        const uint32_t sK = smem_u32(sm + L::oK), sM = smem_u32(sm + L::oM), sL = smem_u32(sm + L::oL),
                       sZ = smem_u32(sm + L::oZ);
        // D = 64: the middle piece's tile is the second 64-row block of the high one's A, the tile of zeros
        // that of the third piece's; the distance (the block stride field, bits 16 ..) follows the slots
        const uint64_t dK = lt::mdesc(sK, 0, D == 64 ? sM - sK : lt::kBlk), dV = lt::mdesc(smem_u32(sm + L::oV), 0),
                       dM = lt::mdesc(sM, 0), dL = lt::mdesc(sL, 0, D == 64 ? sZ - sL : lt::kBlk);
#pragma unroll 1
        for (int it = 0; it < total; ++it) {
            const int s = it % L::NS, p = it % L::NP;
            const uint32_t acc = tmem + (it & 1) * D;
            if (lane == 0) lt::wait(&bars[L::VF + s], (it / L::NS) & 1, abort, status, 351);
            __syncwarp();
            if (it >= 2) tc::named_bar(kNbDR + (it & 1), kBThreads + 32);
            tc::named_bar(kNbKT + (it & 1), kBThreads + 32);
            if (lane == 0) {
                tc::fence_after_sync();
                const uint64_t v = dV + s * T;
                const uint64_t k = dK + s * T + (D == 64 ? ((uint64_t)(p * T) << 16) - ((uint64_t)(s * T) << 16) : 0);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) tc::mma_ss(acc, k + ks * kMK, v + ks * kMK, I_S, ks > 0);
                if (D != 64) {
                    const uint64_t m = dM + p * T;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) tc::mma_ss(acc, m + ks * kMK, v + ks * kMK, I_S, 1);
                }
                if (P == 3) {
                    const uint64_t l = dL + p * T - (D == 64 ? (uint64_t)(p * T) << 16 : 0);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) tc::mma_ss(acc, l + ks * kMK, v + ks * kMK, I_S, 1);
                }
                tc::mma_commit(&bars[L::E + s]);
                tc::mma_commit(&bars[L::AD + (it & 1)]);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0;
#pragma unroll 1
            for (; it < total; ++it) {
                const int s = it % L::NS, ci = it / items, h = w.s * a.rk + it % items;
                const int row = (rev ? w.c1 - 1 - ci : w.c0 + ci) * kW;
                if (it >= L::NS && !lt::wait(&bars[L::E + s], (it / L::NS - 1) & 1, abort, status, 353)) break;
                tc::mbar_arrive_expect_tx(&bars[L::KF + s], L::kTile);
                tc::mbar_arrive_expect_tx(&bars[L::VF + s], L::kTile);
#pragma unroll 1
                for (int i = 0; i < kBlocks; ++i) {
                    lt::load_4d(sm + L::oK + s * L::kTile + i * lt::kBlk, &maps.k, 64 * i, row, h, w.b, &bars[L::KF + s]);
                    lt::load_4d(sm + L::oV + s * L::kTile + i * lt::kBlk, &maps.v, 64 * i, row, h, w.b, &bars[L::VF + s]);
                }
            }
#pragma unroll 1
            for (int i = max(0, it - L::NS); i < it; ++i) {
                lt::wait(&bars[L::KF + i % L::NS], (i / L::NS) & 1, &never, nullptr, 0);
                lt::wait(&bars[L::VF + i % L::NS], (i / L::NS) & 1, &never, nullptr, 0);
            }
        }
    } else if (warp >= lt::kSumB0) {
        const int wb = warp - lt::kSumB0;
        const int row = 32 * q4 + lane, c0 = (wb >> 2) * kC;  // row of the tile, first chunk of it
        const uint32_t ta = tmem + ((uint32_t)(32 * q4) << 16) + (wb >> 2) * kCols;
        const bool poller = wb == 0 && lane == 0;
        auto meet = [&]() {  // after the poller's waits
            __syncwarp();
            tc::named_bar(kNbAll, kBThreads);
        };
#pragma unroll
        for (int j = 0; j < kCols; ++j) sum[j] = 0.f;
        // tile it's products are done (so its pieces' buffers are free): the sums go to registers, the
        // region is released
        auto drain = [&](int it) {
            if (poller) lt::wait(&bars[L::AD + (it & 1)], (it >> 1) & 1, abort, status, 357);
            meet();
            tc::fence_after_sync();
#pragma unroll
            for (int cb = 0; cb < kCols; cb += 16) {
                uint32_t d[16];
                tc::tmem_ld16(ta + (it & 1) * D + cb, d);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[cb + j] += __uint_as_float(d[j]);
            }
            tc::fence_before_sync();
            if (it + 2 < total) tc::named_arrive(kNbDR + (it & 1), kBThreads + 32);
        };
#pragma unroll 1
        for (int it = 0, r = 0, ci = 0; it <= total; ++it, ci += ++r == items, r = r == items ? 0 : r) {
            if (L::NP == 1 && it > 0) drain(it - 1);
            if (it < total) {
                const int s = it % L::NS;
                const int r0 = (rev ? w.c1 - 1 - ci : w.c0 + ci) * kW, Wc = min(kW, w.len - r0);
                const bool padded = Wc < min(kW, a.n - r0);  // padding rows of the values may hold anything
                if (poller) {
                    lt::wait(&bars[L::KF + s], (it / L::NS) & 1, abort, status, 354);
                    if (padded) lt::wait(&bars[L::VF + s], (it / L::NS) & 1, abort, status, 356);
                }
                // g^(distance): of the tile's near end, and within the tile
                const int first = r0 - w.c0 * kW;  // the tile's first row in the segment
                const float near = pow_decay(log2g, (float)(rev ? first : seg_rows - first - Wc));
                const float wt = row < Wc ? a.s_state * near * gp[rev ? row : Wc - 1 - row] : 0.f;
                unsigned char *kt = sm + L::oK + s * L::kTile, *mt = sm + L::oM + (it % L::NP) * L::kTile,
                              *lo = sm + L::oL + (it % L::NP) * L::kTile;
                meet();
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    uint4 x[P];
#pragma unroll
                    for (int p = 0; p < P; ++p) x[p] = make_uint4(0, 0, 0, 0);
                    const uint32_t at = la_off((c0 + c) >> 3, row, (c0 + c) & 7);
                    if (row < Wc) lt::pieces8<P>(*reinterpret_cast<const uint4*>(kt + at), wt, x);
                    *reinterpret_cast<uint4*>(kt + at) = x[0];
                    *reinterpret_cast<uint4*>(mt + at) = x[1];
                    if (P == 3) *reinterpret_cast<uint4*>(lo + at) = x[P - 1];
                    if (padded && row >= Wc)
                        *reinterpret_cast<uint4*>(sm + L::oV + s * L::kTile + at) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async();
                tc::named_arrive(kNbKT + (it & 1), kBThreads + 32);
            }
            if (L::NP == 2 && it > 0) drain(it - 1);
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp >= lt::kSumB0) {
        const int row = 32 * q4 + lane, col = ((warp - lt::kSumB0) >> 2) * kCols;
        float* ex = reinterpret_cast<float*>(sm);  // D = 64: the middle pieces' rows, [64][65]
        if (D == 64) {
            if (row >= 64)
#pragma unroll
                for (int j = 0; j < kCols; ++j) ex[(row - 64) * 65 + col + j] = sum[j];
            tc::named_bar(kNbAll, kBThreads);
            if (row < 64)
#pragma unroll
                for (int j = 0; j < kCols; ++j) sum[j] += ex[row * 65 + col + j];
        }
        if (row < a.dx) {
#pragma unroll
            for (int j = 0; j < kCols; j += 4)  // dy is a multiple of 16
                if (col + j < a.dy)
                    *reinterpret_cast<float4*>(dst + row * a.dy + col + j) = make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 2 * D);
}

// [B][heads][n][Dreal] bf16 view, box of 128 rows x 64 columns (128-byte swizzle); columns past
// Dreal and rows past n read as zero and are not written.
bool lin_map(CUtensorMap* m, const hla2_view& w, int B, int heads, int n, int Dreal) {
    auto fn = la_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)Dreal, (cuuint64_t)n, (cuuint64_t)heads, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)w.sn * 2, (cuuint64_t)w.sh * 2, (cuuint64_t)w.sb * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)lt::kW, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(w.p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int P>
int launch_sum(const lt::Maps& m, const LinPass& a, cudaStream_t st) {
    if (raise_smem(lin_sum_tc_kernel<D, P>, lt::Sum<D, P>::kBytes) != cudaSuccess) return -1;
    return launch_pdl(lin_sum_tc_kernel<D, P>, dim3(a.B * a.Hs, a.nseg), dim3(lt::kSumThreads), lt::Sum<D, P>::kBytes, st, m,
                      a) == cudaSuccess
               ? 0
               : -1;
}

template <int D>
int launch_tc(const LinPass& a, bool summary, cudaStream_t st) {
    lt::Maps m;
    const int xh = a.Hs * a.rx, kh = a.Hs * a.rk;
    if (!lin_map(&m.k, a.k, a.B, kh, a.n, a.dx) || !lin_map(&m.v, a.v, a.B, kh, a.n, a.dy)) return -1;
    if (summary) {
        m.x = m.y = m.k;
        return a.exact_sums ? launch_sum<D, 3>(m, a, st) : launch_sum<D, 2>(m, a, st);
    }
    if (!lin_map(&m.x, a.x, a.B, xh, a.n, a.dx) || !lin_map(&m.y, a.y, a.B, xh, a.n, a.dy)) return -1;
    if (raise_smem(lin_out_tc_kernel<D>, lt::Out<D>::kBytes) != cudaSuccess) return -1;
    return launch_pdl(lin_out_tc_kernel<D>, dim3(a.B * a.Hs, a.nseg), dim3(lt::threads(D)), lt::Out<D>::kBytes, st, m, a) ==
                   cudaSuccess
               ? 0
               : -1;
}

}  // namespace

int launch_lin_tc(const LinPass& a, bool summary, cudaStream_t st) {
    if (a.B * a.Hs == 0 || a.nseg == 0) return 0;
    return a.dx > 64 || a.dy > 64 ? launch_tc<128>(a, summary, st) : launch_tc<64>(a, summary, st);
}

}  // namespace hla2
