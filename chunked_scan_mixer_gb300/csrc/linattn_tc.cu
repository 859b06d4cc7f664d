// First-order linear attention with a decay for each head on the 5th-generation tensor cores:
// bf16 rows, chunks of 128 rows, float32 sums.  The mathematics of a pass is in linattn_pass.h.
//
// Tiles are [128 rows][D] bf16 with D = 64 or 128, loaded and stored by TMA straight from and to
// the caller's strided tensors; a smaller dx or dy is filled with zeros by the copy, so one kernel
// covers every pair of sizes.  Per chunk, with Sig the state at its entry (forward; reverse
// mirrors the decays):
//   MMA-G   G = X K^T                                   128 x 128 float32 in tensor memory
//   EPI-1   G~ = mask(G) s_intra g^(i-j) -> bf16, over G's own columns: A operand of MMA-Y
//   MMA-C   Y = X Sig~ (Sig~ = bf16 of Sig);   EPI-C   Y <- s_carry g^(i+1) Y, in tensor memory
//   MMA-Y   Y += G~ V
//   EPI-Y   Y -> bf16 tile -> TMA store
//   KT      K~ = s_state g^(Wc-1-j) K in pieces of bf16, in shared memory
//   MMA-S   dSig = K~^T V;   EPI-S   Sig <- g^Wc Sig + dSig  (float32 registers), publish Sig~
//
// Roundings to bf16.  G~ and Sig~ are operands of one product each and are rounded once, which
// adds to the output about its own rounding (measured against 64 bits: 2.3e-3 relative where
// a float32 form rounded at the end has 1.65e-3).  The decayed keys are cut into two pieces (16
// bits, 2^-17) here, where they only feed Sig~, and into three (24 bits, exact to float32) in the
// summary kernel, whose sums become the states that are returned.  Decays stay float32 and out of
// the operands everywhere else.
//
// Work items.  A state head has rx x / y heads (queries that share a key head) or rk key / value
// heads (their gradients); item (chunk, r) is one product chain.  With rx > 1 the keys, values
// and the state are loaded and formed once per chunk for all its items; with rk > 1 X, Y and the state
// are, and Y and dSig accumulate over the items in tensor memory.
//
// Roles (512 threads, one CTA per SM): warp 0 allocates tensor memory and one thread issues every
// MMA; warp 1 issues the loads, warp 2 the stores; warps 4..7 (A: one row per thread) run EPI-1, EPI-C and
// EPI-Y; warps 8..15 (B) run KT and EPI-S.  The chains A and B only meet in Sig~.  Every wait is
// bounded; one that gives up records its site in the status word, and every role drains.
//
// D = 64 stacks the two key pieces as one 128-row A operand (rows 0..63 the high piece's
// features, 64..127 the low one's), so MMA-S has full height; the two halves of the state stay
// apart and MMA-C takes both (K = 128), which costs nothing there.
#include "fo_common.cuh"
#include "linattn_pass.h"

namespace hla2 {

namespace {

namespace lt {

constexpr int kW = 128;
constexpr int kThreads = 512;
constexpr int kA0 = 4, kAWarps = 4, kB0 = 8, kBWarps = 8;
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

// Wait for the phase of the given parity.  The waiting warp is suspended in hardware between
// polls (it has others to leave the issue slots to); after about two seconds it gives up.
constexpr long long kWaitClocks = 4LL * 1000 * 1000 * 1000;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int where) {
    if (tc::mbar_try_wait(bar, parity)) return true;
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

template <int D>
struct Out {  // shared memory of the output kernel
    static constexpr uint32_t kTile = (uint32_t)(D / 64) * kBlk;
    static constexpr int NX = D == 64 ? 3 : 2, NK = D == 64 ? 3 : 2, NV = D == 64 ? 3 : 1;
    static constexpr uint32_t oX = 0, oK = oX + NX * kTile, oV = oK + NK * kTile, oM = oV + NV * kTile, oS = oM + kTile;
    static constexpr uint32_t oGp = oS + kTile;          // g^0 .. g^128
    static constexpr uint32_t oT = oGp + 528;            // g^(31 - j) (reverse g^j), j = 0 .. 31
    static constexpr uint32_t oBar = oT + 128;
    enum {
        XF = 0, XE = XF + NX, OS = XE + NX, KF = OS + NX, KE = KF + NK, VF = KE + NK, VE = VF + NV, VZ = VE + NV,
        BG = VZ + NV, BGK = BG + 2, GT = BGK + 2, KT = GT + 2, BC, YD, YR, SD, SP, ME, kBars
    };
    static constexpr uint32_t oMisc = oBar + kBars * 8;
    static constexpr uint32_t kBytes = oMisc + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

// Tensor memory columns of the output kernel: two Gram regions, Y, dSig.
template <int D>
struct Cols {
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
__global__ void __launch_bounds__(lt::kThreads, 1) lin_out_tc_kernel(const __grid_constant__ lt::Maps maps, const LinPass a) {
    using L = lt::Out<D>;
    using C = lt::Cols<D>;
    constexpr int kW = lt::kW;
    constexpr int kBlocks = D / 64;
    constexpr int kSC = D / 2;  // state columns per B thread
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* gp = reinterpret_cast<float*>(sm + L::oGp);
    float* tt = reinterpret_cast<float*>(sm + L::oT);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::oMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::oMisc + 4);
    int* status = a.status;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const lt::Where w = lt::locate(a);
    const bool rev = a.rev != 0, mode_a = a.rx > 1, mode_b = a.rk > 1;
    const int items = mode_a ? a.rx : a.rk, total = w.nit * items;
    const float log2g = log2f(lin_decay(a, w.s));

    // rows of the segment past the sequence: zeros
    {
        const int z0 = max(w.c0, w.c1) * kW, z1 = min((w.c0 + a.seg_chunks) * kW, a.n);
        const int per = a.dy / 8, count = max(0, z1 - z0) * per;
        for (int h = 0; h < a.rx; ++h) {
            bf16* y = static_cast<bf16*>(const_cast<void*>(a.y.p)) + w.b * a.y.sb + (long long)(w.s * a.rx + h) * a.y.sh;
            for (int e = tid; e < count; e += lt::kThreads)
                *reinterpret_cast<uint4*>(y + (long long)(z0 + e / per) * a.y.sn + (e % per) * 8) = make_uint4(0, 0, 0, 0);
        }
    }
    if (w.nit == 0) return;

    for (int i = tid; i <= kW; i += lt::kThreads) gp[i] = pow_decay(log2g, (float)i);
    if (tid < 32) tt[tid] = pow_decay(log2g, (float)(rev ? tid : 31 - tid));
    if (tid == 0) {
        for (int i = 0; i < L::kBars; ++i) {
            const bool by_a = (i >= L::OS && i < L::OS + L::NX) || i == L::GT || i == L::GT + 1 || i == L::YR;
            const bool by_b = (i >= L::VZ && i < L::VZ + L::NV) || i == L::KT || i == L::SP;
            tc::mbar_init(&bars[i], by_a ? lt::kAWarps : by_b ? lt::kBWarps : 1);
        }
        *abort = 0;
        tc::mbar_fence_init();
    }
    if (warp == 0) tc::tmem_alloc(tmem_holder, 512);

    // B thread: state row sr, columns sc0 .. sc0 + kSC - 1.  D = 64: rows 64.. hold the low pieces' sums.
    const int q4 = warp & 3, half = (warp - lt::kB0) >> 2;
    const int sr = 32 * q4 + lane, sc0 = half * kSC;
    float sig[kSC];
    auto publish = [&]() {
#pragma unroll
        for (int j = 0; j < kSC / 8; ++j)
            *reinterpret_cast<uint4*>(sm + L::oS + la_off(sc0 / 64, sr, (sc0 % 64) / 8 + j)) = la_pack8(&sig[8 * j]);
    };
    if (warp >= lt::kB0) {
#pragma unroll
        for (int j = 0; j < kSC; ++j) sig[j] = 0.f;
        if (a.carry && sr < a.dx) {  // D = 64: dx <= 64, so only the high half takes it
            const float* src = a.carry + ((size_t)w.bs * a.nseg + blockIdx.y) * a.dx * a.dy;
#pragma unroll
            for (int j = 0; j < kSC; ++j)
                if (sc0 + j < a.dy)
                    sig[j] = a.carry_t ? src[(size_t)(sc0 + j) * a.dx + sr] : src[(size_t)sr * a.dy + sc0 + j];
        }
        publish();
        tc::fence_proxy_async();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    auto chunk_of = [&](int ci) { return rev ? w.c1 - 1 - ci : w.c0 + ci; };
    auto valid_of = [&](int ci) { return min(kW, w.len - chunk_of(ci) * kW); };
    volatile int never = 0;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------------------- MMA issue
            constexpr uint32_t I_G = tc::idesc_bf16(128, 128, 0, 0), I_C = tc::idesc_bf16(128, D, 0, 1),
                               I_Y = tc::idesc_bf16(128, D, 0, 1), I_S = tc::idesc_bf16(128, D, 1, 1);
            const uint32_t sX = smem_u32(sm + L::oX), sK = smem_u32(sm + L::oK), sV = smem_u32(sm + L::oV),
                           sM = smem_u32(sm + L::oM), sS = smem_u32(sm + L::oS);
            auto x_of = [&](int it) { return mode_b ? it / items : it; };
            auto kv_of = [&](int it) { return mode_b ? it : it / items; };
            auto issue_g = [&](int it) {
                const int r = it % items, xi = x_of(it), ki = kv_of(it), xs = xi % L::NX, ks_ = ki % L::NK;
                if (!mode_b || r == 0) lt::wait(&bars[L::XF + xs], (xi / L::NX) & 1, abort, status, 301);
                if (!mode_a || r == 0) lt::wait(&bars[L::KF + ks_], (ki / L::NK) & 1, abort, status, 302);
                tc::fence_after_sync();
                for (int ks = 0; ks < D / 16; ++ks)
                    tc::mma_ss(tmem + C::G(it), lt::kdesc(sX + xs * L::kTile, ks), lt::kdesc(sK + ks_ * L::kTile, ks), I_G,
                               ks > 0);
                tc::mma_commit(&bars[L::BG + (it & 1)]);
                if (!mode_a || r == items - 1) tc::mma_commit(&bars[L::BGK + (ki & 1)]);
            };
            issue_g(0);
            int groups = 0;  // Y regions begun
            for (int it = 0; it < total; ++it) {
                const int r = it % items, ci = it / items, xi = x_of(it), ki = kv_of(it);
                const int vs = ki % L::NV, ks_ = ki % L::NK;
                const bool first = r == 0, last = r == items - 1;
                const bool new_y = !mode_b || first, end_y = !mode_b || last;
                const bool state_now = (!mode_a || last) && ci + 1 < w.nit;
                if (new_y) {
                    if (first && ci > 0) lt::wait(&bars[L::SP], (ci - 1) & 1, abort, status, 303);
                    if (groups > 0) lt::wait(&bars[L::YR], (groups - 1) & 1, abort, status, 304);
                    tc::fence_after_sync();
                    ++groups;
                    const uint32_t x = sX + (xi % L::NX) * L::kTile;
                    for (int ks = 0; ks < 8; ++ks)  // D = 64: the two halves of the state in turn
                        tc::mma_ss(tmem + C::Y, lt::kdesc(x, D == 64 ? ks & 3 : ks), lt::mdesc(sS, ks), I_C, ks > 0);
                    tc::mma_commit(&bars[L::BC]);
                }
                // The next Gram overwrites the region that MMA-Y of the item before this one read: done with
                // the wait for YR above, else (the later items of a chunk) by that item's own commit.
                if (mode_b && !first)
                    lt::wait(&bars[L::KE + (it - 1) % L::NK], ((it - 1) / L::NK) & 1, abort, status, 308);
                if (it + 1 < total) issue_g(it + 1);
                if (!mode_a || first) {
                    lt::wait(&bars[L::VF + vs], (ki / L::NV) & 1, abort, status, 305);
                    if (a.lengths) lt::wait(&bars[L::VZ + vs], (ki / L::NV) & 1, abort, status, 306);
                }
                bool y_done = false, s_done = !state_now;
                const uint32_t v = sV + vs * L::kTile;
                const long long t0 = clock64();
                while (!y_done || !s_done) {
                    if (!y_done && tc::mbar_test_wait(&bars[L::GT + (it & 1)], (it >> 1) & 1)) {
                        tc::fence_after_sync();
                        for (int ks = 0; ks < 8; ++ks)
                            tc::mma_ts(tmem + C::Y, tmem + C::G(it) + 8 * ks, lt::mdesc(v, ks), I_Y, 1);
                        if (end_y) tc::mma_commit(&bars[L::YD]);
                        y_done = true;
                    }
                    if (!s_done && tc::mbar_test_wait(&bars[L::KT], ki & 1)) {
                        tc::fence_after_sync();
                        const uint32_t k = sK + ks_ * L::kTile, acc = mode_b && !first;
                        if (D == 64) {
                            for (int ks = 0; ks < 8; ++ks)
                                tc::mma_ss(tmem + C::S, lt::mdesc(k, ks, sM - k), lt::mdesc(v, ks), I_S, acc || ks > 0);
                        } else {
                            for (int ks = 0; ks < 8; ++ks)
                                tc::mma_ss(tmem + C::S, lt::mdesc(k, ks), lt::mdesc(v, ks), I_S, acc || ks > 0);
                            for (int ks = 0; ks < 8; ++ks)
                                tc::mma_ss(tmem + C::S, lt::mdesc(sM, ks), lt::mdesc(v, ks), I_S, 1);
                        }
                        tc::mma_commit(&bars[L::ME]);
                        if (last) tc::mma_commit(&bars[L::SD]);
                        s_done = true;
                    }
                    if (*abort) break;
                    if (clock64() - t0 > lt::kWaitClocks) {
                        *abort = 1;
                        if (status) atomicCAS(status, 0, 307);
                        break;
                    }
                }
                if (!mode_a || last) {  // the keys and values have been read
                    tc::mma_commit(&bars[L::KE + ks_]);
                    tc::mma_commit(&bars[L::VE + vs]);
                }
            }
            // drain: the last commit covers every MMA before it
            const int kl = kv_of(total - 1);
            lt::wait(&bars[L::VE + kl % L::NV], (kl / L::NV) & 1, &never, nullptr, 0);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ----------------------------------------------------------------------- loads
            int nx = 0, nkv = 0;
            auto load = [&](uint32_t slot, const CUtensorMap* m, int row, int h, uint64_t* bar) {
                tc::mbar_arrive_expect_tx(bar, L::kTile);
                for (int i = 0; i < kBlocks; ++i) lt::load_4d(sm + slot + i * lt::kBlk, m, 64 * i, row, h, w.b, bar);
            };
            for (int it = 0; it < total && !*abort; ++it) {
                const int r = it % items, row = chunk_of(it / items) * kW;
                const bool lx = !mode_b || r == 0, lkv = !mode_a || r == 0;
                const int xs = nx % L::NX, ks_ = nkv % L::NK, vs = nkv % L::NV;
                if (lx) {
                    if (nx >= L::NX && !lt::wait(&bars[L::XE + xs], (nx / L::NX - 1) & 1, abort, status, 311)) break;
                    load(L::oX + xs * L::kTile, &maps.x, row, w.s * a.rx + (mode_a ? r : 0), &bars[L::XF + xs]);
                    ++nx;
                }
                if (lkv) {
                    const int h = w.s * a.rk + (mode_b ? r : 0);
                    if (nkv >= L::NK && !lt::wait(&bars[L::KE + ks_], (nkv / L::NK - 1) & 1, abort, status, 312)) break;
                    load(L::oK + ks_ * L::kTile, &maps.k, row, h, &bars[L::KF + ks_]);
                    if (nkv >= L::NV && !lt::wait(&bars[L::VE + vs], (nkv / L::NV - 1) & 1, abort, status, 313)) {
                        ++nkv;  // the K load is in flight; its V is not
                        break;
                    }
                    load(L::oV + vs * L::kTile, &maps.v, row, h, &bars[L::VF + vs]);
                    ++nkv;
                }
            }
            // drain: every load has landed.  A wait for a load that was not issued (after an abort)
            // runs out; the others return at once.
            for (int i = max(0, nx - L::NX); i < nx; ++i)
                lt::wait(&bars[L::XF + i % L::NX], (i / L::NX) & 1, &never, nullptr, 0);
            for (int i = max(0, nkv - L::NK); i < nkv; ++i)
                lt::wait(&bars[L::KF + i % L::NK], (i / L::NK) & 1, &never, nullptr, 0);
            for (int i = max(0, nkv - L::NV); i < nkv; ++i)
                lt::wait(&bars[L::VF + i % L::NV], (i / L::NV) & 1, &never, nullptr, 0);
        }
    } else if (warp == 2) {
        if (lane == 0) {
            // ---------------------------------------------------------------------- stores
            const int groups = mode_b ? w.nit : total;
            for (int g = 0; g < groups; ++g) {
                const int slot = g % L::NX;
                if (!lt::wait(&bars[L::OS + slot], (g / L::NX) & 1, abort, status, 321)) break;
                const int row = chunk_of(mode_a ? g / items : g) * kW, h = w.s * a.rx + (mode_a ? g % items : 0);
                for (int i = 0; i < kBlocks; ++i)
                    if (64 * i < a.dy)
                        lt::store_4d(&maps.y, sm + L::oX + slot * L::kTile + i * lt::kBlk, 64 * i, row, h, w.b);
                tc::bulk_commit();
                tc::bulk_wait_read_all();
                tc::mbar_arrive(&bars[L::XE + slot]);
            }
            tc::bulk_wait_all();
        }
    } else if (warp >= lt::kA0 && warp < lt::kB0) {
        // ---------------------------------------------------- A: row i of the chunk per thread
        const int i = 32 * q4 + lane, row0 = 32 * q4;
        const uint32_t lanes = (uint32_t)row0 << 16;
        int groups = 0;
        for (int it = 0; it < total && !*abort; ++it) {
            const int r = it % items, ci = it / items, Wc = valid_of(ci);
            const bool new_y = !mode_b || r == 0, end_y = !mode_b || r == items - 1;
            const uint32_t tg = tmem + lanes + C::G(it);
            lt::wait(&bars[L::BG + (it & 1)], (it >> 1) & 1, abort, status, 331);
            tc::fence_after_sync();
            // EPI-1: 32 columns at a time.  A block is entirely kept (factor g^(i-cb-31) g^(31-j)),
            // entirely dropped, or the diagonal one (a factor per element).
#pragma unroll 1
            for (int cb = 0; cb < kW; cb += 32) {
                uint32_t pk[16];
                if (rev ? cb < row0 : cb > row0) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) pk[j] = 0u;
                } else {
                    uint32_t g[32];
                    tc::tmem_ld32(tg + cb, g);
                    tc::tmem_wait_ld();
                    if (cb == row0) {
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float f[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int dist = rev ? cb + j + e - i : i - cb - j - e;
                                const bool keep = dist >= 0 && (!rev || cb + j + e < Wc);
                                f[e] = keep ? __uint_as_float(g[j + e]) * (a.s_intra * gp[max(dist, 0)]) : 0.f;
                            }
                            pk[j / 2] = pack_bf16x2(f[0], f[1]);
                        }
                    } else {
                        const float base = a.s_intra * gp[rev ? cb - i : i - cb - 31];
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 t = *reinterpret_cast<const float4*>(tt + j);
                            float f0 = __uint_as_float(g[j]) * (base * t.x), f1 = __uint_as_float(g[j + 1]) * (base * t.y),
                                  f2 = __uint_as_float(g[j + 2]) * (base * t.z), f3 = __uint_as_float(g[j + 3]) * (base * t.w);
                            if (rev && Wc < kW) {  // columns past the sequence hold anything
                                f0 = cb + j < Wc ? f0 : 0.f;
                                f1 = cb + j + 1 < Wc ? f1 : 0.f;
                                f2 = cb + j + 2 < Wc ? f2 : 0.f;
                                f3 = cb + j + 3 < Wc ? f3 : 0.f;
                            }
                            pk[j / 2] = pack_bf16x2(f0, f1);
                            pk[j / 2 + 1] = pack_bf16x2(f2, f3);
                        }
                    }
                }
                tc::tmem_st16(tg + cb / 2, pk);  // columns that this thread has read
            }
            if (new_y) {  // EPI-C
                lt::wait(&bars[L::BC], groups & 1, abort, status, 332);
                tc::fence_after_sync();
                const float f = a.s_carry * gp[rev ? max(Wc - i, 0) : i + 1];
#pragma unroll 1
                for (int cb = 0; cb < D; cb += 16) {
                    uint32_t y[16];
                    tc::tmem_ld16(tmem + lanes + C::Y + cb, y);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(f * __uint_as_float(y[j]));
                    tc::tmem_st16(tmem + lanes + C::Y + cb, y);
                }
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[L::GT + (it & 1)]);
            if (!end_y) continue;
            // EPI-Y, into the X tile, which the products have read
            lt::wait(&bars[L::YD], groups & 1, abort, status, 333);
            tc::fence_after_sync();
            unsigned char* st = sm + L::oX + (groups % L::NX) * L::kTile;
            const bool live = i < Wc;
#pragma unroll 1
            for (int cb = 0; cb < D; cb += 32) {
                uint32_t y[32];
                tc::tmem_ld32(tmem + lanes + C::Y + cb, y);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    uint4 o = make_uint4(0, 0, 0, 0);
                    if (live) {
                        o.x = pack_bf16x2(__uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                        o.y = pack_bf16x2(__uint_as_float(y[j + 2]), __uint_as_float(y[j + 3]));
                        o.z = pack_bf16x2(__uint_as_float(y[j + 4]), __uint_as_float(y[j + 5]));
                        o.w = pack_bf16x2(__uint_as_float(y[j + 6]), __uint_as_float(y[j + 7]));
                    }
                    *reinterpret_cast<uint4*>(st + la_off((cb + j) / 64, i, ((cb + j) % 64) / 8)) = o;
                }
            }
            tc::fence_before_sync();
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&bars[L::YR]);
                tc::mbar_arrive(&bars[L::OS + groups % L::NX]);
            }
            ++groups;
        }
    } else if (warp >= lt::kB0) {
        // -------------------------------------------- B: keys' pieces, the values' padding, the state
        const int row = 32 * q4 + lane;             // KT: row of the chunk; 16-byte chunks of it below
        constexpr int kC = D / 16;                  // 16-byte chunks per thread
        const int c0 = half * kC;                   // chunk index over the whole row: block c / 8, chunk c % 8
        const uint32_t lanes = (uint32_t)(32 * q4) << 16;
        int nk = 0;  // key / value tiles seen
        for (int it = 0; it < total && !*abort; ++it) {
            const int r = it % items, ci = it / items, Wc = valid_of(ci);
            if (mode_a && r > 0 && r < items - 1) continue;
            const int vs = nk % L::NV, ks_ = nk % L::NK;
            if (a.lengths && (!mode_a || r == 0)) {
                lt::wait(&bars[L::VF + vs], (nk / L::NV) & 1, abort, status, 341);
                if (Wc < min(kW, a.n - chunk_of(ci) * kW) && row >= Wc) {
#pragma unroll
                    for (int c = c0; c < c0 + kC; ++c)
                        *reinterpret_cast<uint4*>(sm + L::oV + vs * L::kTile + la_off(c >> 3, row, c & 7)) =
                            make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[L::VZ + vs]);
            }
            if (mode_a && r < items - 1) continue;
            if (ci + 1 < w.nit) {
                lt::wait(&bars[L::KF + ks_], (nk / L::NK) & 1, abort, status, 342);
                lt::wait(&bars[L::BGK + (nk & 1)], (nk >> 1) & 1, abort, status, 343);  // the Gram products have read K
                if (nk > 0) lt::wait(&bars[L::ME], (nk - 1) & 1, abort, status, 344);   // the low piece has been read
                const float wt = row < Wc ? a.s_state * gp[rev ? row : Wc - 1 - row] : 0.f;
                unsigned char *kt = sm + L::oK + ks_ * L::kTile, *mt = sm + L::oM;
#pragma unroll
                for (int c = c0; c < c0 + kC; ++c) {
                    const uint32_t at = la_off(c >> 3, row, c & 7);
                    uint4 p[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                    if (row < Wc) lt::pieces8<2>(*reinterpret_cast<const uint4*>(kt + at), wt, p);
                    *reinterpret_cast<uint4*>(kt + at) = p[0];
                    *reinterpret_cast<uint4*>(mt + at) = p[1];
                }
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[L::KT]);
                if (r == items - 1) {  // EPI-S
                    lt::wait(&bars[L::SD], ci & 1, abort, status, 345);
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
                    publish();
                    tc::fence_before_sync();
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars[L::SP]);
                }
            }
            ++nk;
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
// segment's rows (all key / value heads of the state), weights relative to the segment, so the
// products accumulate in tensor memory from the first tile to the last.
// ----------------------------------------------------------------------------------------
namespace lt {
template <int D>
struct Sum {
    static constexpr uint32_t kTile = (uint32_t)(D / 64) * kBlk;
    static constexpr int NS = D == 64 ? 3 : 2;   // key / value slots
    static constexpr int NP = D == 64 ? 2 : 1;   // buffers of the two lower pieces
    static constexpr uint32_t oK = 0, oV = oK + NS * kTile, oM = oV + NS * kTile, oL = oM + NP * kTile,
                              oZ = oL + NP * kTile;  // D = 64: a tile of zeros beside the third piece
    static constexpr uint32_t oBar = oZ + (D == 64 ? kTile : 0);
    enum { KF = 0, VF = KF + NS, E = VF + NS, KT = E + NS, PE = KT + NP, kBars = PE + NP };
    static constexpr uint32_t oMisc = oBar + kBars * 8;
    static constexpr uint32_t kBytes = oMisc + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};
constexpr int kSumThreads = 384;  // warp 0 MMA, warp 1 loads, warps 4..11 pieces
}  // namespace lt

template <int D>
__global__ void __launch_bounds__(lt::kSumThreads, 1) lin_sum_tc_kernel(const __grid_constant__ lt::Maps maps, const LinPass a) {
    using L = lt::Sum<D>;
    constexpr int kW = lt::kW, kBlocks = D / 64, kC = D / 16;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::oBar);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::oMisc);
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::oMisc + 4);
    int* status = a.status;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q4 = warp & 3;
    const lt::Where w = lt::locate(a);
    const bool rev = a.rev != 0;
    const int items = a.rk, total = w.nit * items;
    float* dst = a.sums + ((size_t)w.bs * a.nseg + blockIdx.y) * a.dx * a.dy;
    if (w.nit == 0) {
        for (int e = tid; e < a.dx * a.dy; e += lt::kSumThreads) dst[e] = 0.f;
        return;
    }
    const float log2g = log2f(lin_decay(a, w.s));
    if (tid == 0) {
        for (int i = 0; i < L::kBars; ++i) tc::mbar_init(&bars[i], i >= L::KT && i < L::KT + L::NP ? lt::kBWarps : 1);
        *abort = 0;
        tc::mbar_fence_init();
    }
    if (warp == 0) tc::tmem_alloc(tmem_holder, 128);
    if (D == 64) {
        for (int e = tid; e < (int)(L::kTile / 16); e += lt::kSumThreads)
            *reinterpret_cast<uint4*>(sm + L::oZ + 16 * e) = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_holder;
    volatile int never = 0;
    const int seg_rows = min(w.len, w.c1 * kW) - w.c0 * kW;  // valid rows of the segment

    if (warp == 0) {
        if (lane == 0) {
            constexpr uint32_t I_S = tc::idesc_bf16(128, D, 1, 1);
            const uint32_t sK = smem_u32(sm + L::oK), sV = smem_u32(sm + L::oV), sM = smem_u32(sm + L::oM),
                           sL = smem_u32(sm + L::oL), sZ = smem_u32(sm + L::oZ);
            for (int it = 0; it < total; ++it) {
                const int s = it % L::NS, p = it % L::NP;
                lt::wait(&bars[L::VF + s], (it / L::NS) & 1, abort, status, 351);
                lt::wait(&bars[L::KT + p], (it / L::NP) & 1, abort, status, 352);
                tc::fence_after_sync();
                const uint32_t k = sK + s * L::kTile, v = sV + s * L::kTile, m = sM + p * L::kTile, l = sL + p * L::kTile;
                for (int ks = 0; ks < 8; ++ks)
                    tc::mma_ss(tmem, D == 64 ? lt::mdesc(k, ks, m - k) : lt::mdesc(k, ks), lt::mdesc(v, ks), I_S,
                               it > 0 || ks > 0);
                if (D != 64)
                    for (int ks = 0; ks < 8; ++ks) tc::mma_ss(tmem, lt::mdesc(m, ks), lt::mdesc(v, ks), I_S, 1);
                for (int ks = 0; ks < 8; ++ks)
                    tc::mma_ss(tmem, D == 64 ? lt::mdesc(l, ks, sZ - l) : lt::mdesc(l, ks), lt::mdesc(v, ks), I_S, 1);
                tc::mma_commit(&bars[L::E + s]);
                tc::mma_commit(&bars[L::PE + p]);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0;
            for (; it < total && !*abort; ++it) {
                const int s = it % L::NS, ci = it / items, h = w.s * a.rk + it % items;
                const int row = (rev ? w.c1 - 1 - ci : w.c0 + ci) * kW;
                if (it >= L::NS && !lt::wait(&bars[L::E + s], (it / L::NS - 1) & 1, abort, status, 353)) break;
                tc::mbar_arrive_expect_tx(&bars[L::KF + s], L::kTile);
                tc::mbar_arrive_expect_tx(&bars[L::VF + s], L::kTile);
                for (int i = 0; i < kBlocks; ++i) {
                    lt::load_4d(sm + L::oK + s * L::kTile + i * lt::kBlk, &maps.k, 64 * i, row, h, w.b, &bars[L::KF + s]);
                    lt::load_4d(sm + L::oV + s * L::kTile + i * lt::kBlk, &maps.v, 64 * i, row, h, w.b, &bars[L::VF + s]);
                }
            }
            for (int i = max(0, it - L::NS); i < it; ++i) {
                lt::wait(&bars[L::KF + i % L::NS], (i / L::NS) & 1, &never, nullptr, 0);
                lt::wait(&bars[L::VF + i % L::NS], (i / L::NS) & 1, &never, nullptr, 0);
            }
        }
    } else if (warp >= 4) {
        const int half = (warp - 4) >> 2, row = 32 * q4 + lane, c0 = half * kC;
        for (int it = 0; it < total && !*abort; ++it) {
            const int s = it % L::NS, p = it % L::NP, ci = it / items;
            const int r0 = (rev ? w.c1 - 1 - ci : w.c0 + ci) * kW, Wc = min(kW, w.len - r0);
            lt::wait(&bars[L::KF + s], (it / L::NS) & 1, abort, status, 354);
            if (it >= L::NP) lt::wait(&bars[L::PE + p], (it / L::NP - 1) & 1, abort, status, 355);
            const int at_seg = r0 - w.c0 * kW + row;  // row within the segment
            const float wt = row < Wc ? a.s_state * pow_decay(log2g, (float)(rev ? at_seg : seg_rows - 1 - at_seg)) : 0.f;
            unsigned char *kt = sm + L::oK + s * L::kTile, *mt = sm + L::oM + p * L::kTile, *lo = sm + L::oL + p * L::kTile;
#pragma unroll
            for (int c = c0; c < c0 + kC; ++c) {
                const uint32_t at = la_off(c >> 3, row, c & 7);
                uint4 x[3] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (row < Wc) lt::pieces8<3>(*reinterpret_cast<const uint4*>(kt + at), wt, x);
                *reinterpret_cast<uint4*>(kt + at) = x[0];
                *reinterpret_cast<uint4*>(mt + at) = x[1];
                *reinterpret_cast<uint4*>(lo + at) = x[2];
            }
            if (Wc < min(kW, a.n - r0)) {  // padding rows of the values may hold anything
                lt::wait(&bars[L::VF + s], (it / L::NS) & 1, abort, status, 356);
                if (row >= Wc)
#pragma unroll
                    for (int c = c0; c < c0 + kC; ++c)
                        *reinterpret_cast<uint4*>(sm + L::oV + s * L::kTile + la_off(c >> 3, row, c & 7)) =
                            make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[L::KT + p]);
        }
    }
    __syncwarp();
    // the sums: every product is done once the last tile's commit is
    const int lt_ = total - 1;
    lt::wait(&bars[L::PE + lt_ % L::NP], (lt_ / L::NP) & 1, &never, status, 357);
    tc::fence_after_sync();
    __syncthreads();
    if (warp >= 4) {
        constexpr int kCols = D / 2;
        const int half = (warp - 4) >> 2, row = 32 * q4 + lane, col = half * kCols;
        float* ex = reinterpret_cast<float*>(sm);  // D = 64: the low pieces' rows, [64][65]
#pragma unroll
        for (int cb = 0; cb < kCols; cb += 16) {
            uint32_t d[16];
            tc::tmem_ld16(tmem + ((uint32_t)(32 * q4) << 16) + col + cb, d);
            tc::tmem_wait_ld();
            if (D == 64) {
                if (row >= 64)
#pragma unroll
                    for (int j = 0; j < 16; ++j) ex[(row - 64) * 65 + col + cb + j] = __uint_as_float(d[j]);
                tc::named_bar(1, 256);
                if (row < a.dx)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (col + cb + j < a.dy)
                            dst[row * a.dy + col + cb + j] = __uint_as_float(d[j]) + ex[row * 65 + col + cb + j];
            } else if (row < a.dx) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (col + cb + j < a.dy) dst[row * a.dy + col + cb + j] = __uint_as_float(d[j]);
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, 128);
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

template <int D>
int launch_tc(const LinPass& a, bool summary, cudaStream_t st) {
    lt::Maps m;
    const int xh = a.Hs * a.rx, kh = a.Hs * a.rk;
    if (!lin_map(&m.k, a.k, a.B, kh, a.n, a.dx) || !lin_map(&m.v, a.v, a.B, kh, a.n, a.dy)) return -1;
    const dim3 grid(a.B * a.Hs, a.nseg);
    if (summary) {
        m.x = m.y = m.k;
        if (cudaFuncSetAttribute(lin_sum_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, lt::Sum<D>::kBytes) !=
            cudaSuccess)
            return -1;
        lin_sum_tc_kernel<D><<<grid, lt::kSumThreads, lt::Sum<D>::kBytes, st>>>(m, a);
    } else {
        if (!lin_map(&m.x, a.x, a.B, xh, a.n, a.dx) || !lin_map(&m.y, a.y, a.B, xh, a.n, a.dy)) return -1;
        if (cudaFuncSetAttribute(lin_out_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, lt::Out<D>::kBytes) !=
            cudaSuccess)
            return -1;
        lin_out_tc_kernel<D><<<grid, lt::kThreads, lt::Out<D>::kBytes, st>>>(m, a);
    }
    return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_lin_tc(const LinPass& a, bool summary, cudaStream_t st) {
    if (a.B * a.Hs == 0 || a.nseg == 0) return 0;
    return a.dx > 64 || a.dy > 64 ? launch_tc<128>(a, summary, st) : launch_tc<64>(a, summary, st);
}

}  // namespace hla2
