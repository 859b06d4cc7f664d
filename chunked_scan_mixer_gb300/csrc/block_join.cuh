// Shared by the forward and the backward of the block norms (block_join.cu, block_join_bwd.cu):
// sums over a row's threads, the ring of rows copied ahead, and the launch shapes.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "packed.cuh"

namespace hla2 {
int set_last_error(int code, const char* fmt, ...);

namespace {

constexpr int kMaxD = 8192;
constexpr int kSmallThreads = 256;  // CTA size of the sub-warp mapping

// Sums of N values over the threads of a row: TPR lanes of a warp, or the CTA (TPR == 0, or > 32: of that
// many threads).
// `red` alternates between two halves, so one barrier a call is enough.  Two values share a warp's
// steps: after an exchange each half of the lanes sums one of them.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[16][N], int& turn) {
    const int lane = threadIdx.x & 31;
    constexpr bool halves = N == 2 && (TPR == 0 || TPR >= 32);
    if constexpr (halves) {
        const bool up = lane & 16;
        const float give = up ? v[0] : v[1];
        v[0] = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    } else {
#pragma unroll
        for (int o = (TPR && TPR < 32 ? TPR : 32) / 2; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if constexpr (TPR == 0 || TPR > 32) {
        const int warp = threadIdx.x >> 5, nw = (TPR ? TPR : blockDim.x) >> 5, mask = nw > 8 ? 15 : 7;  // at most 16 warps
        const int which = halves ? lane >> 4 : 0;
        if (lane == 16 * which) red[turn][warp][which] = v[0];
        __syncthreads();
        v[0] = (lane & mask) < nw ? red[turn][lane & mask][which] : 0.f;
#pragma unroll
        for (int o = 8; o; o >>= 1)
            if (o < 8 || nw > 8) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        turn ^= 1;
    }
    if constexpr (halves) {
        const float mine = v[0];
        v[0] = __shfl_sync(0xffffffffu, mine, 0);
        v[1] = __shfl_sync(0xffffffffu, mine, 16);
    }
}

// What a call has: no block output (the norm alone); a block output with a gate for each value, a
// scale and a next norm (and dr); or a block output with any of them, told at run time.
enum { kNormOnly = 0, kAll = 1, kAny = 2 };

// Single bf16 elements, which cp.async does not copy: they wait in registers while a row is worked on and
// go to the ring (put) before the next row's loads.  With more than four a thread they go there at once.
template <typename T, int VEC, int NV>
constexpr bool kHolds = VEC * sizeof(T) == 2 && NV <= 4;

// One thread's ring: slot (stage, tensor, j) holds its j-th vector of that tensor's row.
template <typename T, int VEC, int NV>
struct Ring {
    static constexpr int kBytes = VEC * (int)sizeof(T);
    char* base;       // this thread's first slot
    uint32_t step;    // bytes between slots: the CTA's threads side by side
    int tensors;
    __device__ __forceinline__ Ring(char* sm, int n) : base(sm + threadIdx.x * kBytes), step(blockDim.x * kBytes), tensors(n) {}
    __device__ __forceinline__ char* at(int stage, int tensor, int j) const {
        return base + (uint32_t)((stage * tensors + tensor) * NV + j) * step;
    }
    __device__ __forceinline__ void copy(int stage, int tensor, int j, const T* p) const {
        char* d = at(stage, tensor, j);
        if constexpr (kBytes == 16) {
            cp_async16(d, p);
        } else if constexpr (kBytes == 4) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem_u32(d)), "l"(p));
        } else {
            *reinterpret_cast<T*>(d) = *p;
        }
    }
    __device__ __forceinline__ void put(int stage, int tensor, int j, T v) const { *reinterpret_cast<T*>(at(stage, tensor, j)) = v; }
    template <typename P, int N>
    __device__ __forceinline__ void get(int stage, int tensor, int j, P (&f)[N]) const {
        unpack(*reinterpret_cast<const Vec<T, VEC>*>(at(stage, tensor, j)), f);
    }
};
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N)); }

// The newest `ahead` (0 .. 3) groups may still be in flight.
__device__ __forceinline__ void cp_async_wait_but(int ahead) {
    switch (ahead) {
        case 0: cp_async_wait<0>(); break;
        case 1: cp_async_wait<1>(); break;
        case 2: cp_async_wait<2>(); break;
        default: cp_async_wait<3>(); break;
    }
}

// ---- launch choice ------------------------------------------------------------------------

bool al(const void* p, size_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }

// Elements per vector: 16 bytes where every row and vector allows it; else pairs of bf16 in 4 bytes; else
// single elements.
int vec_of(const hla2_block_args* a, const void* const* more, int nmore) {
    auto fits = [&](int vec) {
        const size_t b = (size_t)vec * (a->dtype == HLA2_BF16 ? 2 : 4);
        if (a->D % vec || !al(a->x, b) || !al(a->next_weight, b) || a->x_stride % vec) return false;
        if (a->y && (!al(a->y, b) || !al(a->post_weight, b) || !al(a->scale, b) || a->y_stride % vec)) return false;
        if (a->y && a->gate && a->gate_cols != 1 && (!al(a->gate, b) || a->gate_stride % vec)) return false;
        for (int i = 0; i < nmore; ++i)
            if (!al(more[i], b)) return false;
        return true;
    };
    const int wide = a->dtype == HLA2_BF16 ? 8 : 4;
    if (fits(wide)) return wide;
    if (a->dtype == HLA2_BF16 && fits(2)) return 2;
    return 1;
}

struct Shape {
    int tpr;      // threads per row in a sub-warp mapping, 0: a CTA per row, 256: a CTA of 256 per row
    int threads;  // CTA size
    int nv;       // vectors per thread
};
// At most 256 threads and 8 values a thread up to D = 2048 (the registers of the backward, which
// keeps five inputs, three weight gradients and one intermediate per value), then 512 threads.
constexpr int kNarrowD = 2048;
Shape shape_of(int D, int vec) {
    const int nvec = (D + vec - 1) / vec;
    if (nvec <= 32) {
        return {nvec <= 8 ? 8 : 32, kSmallThreads, 1};
    }
    // Rows of single elements: a width that the compiler knows, for the offsets of a thread's 4 or 8 elements.  Ten million
    // values without and with it, us, at D = 513, 777, 999, 1281, 2047: norm forward and backward, float32 61/57/52/60/54
    // and 68/54/49/53/50, bf16 68/63/55/69/62 and 74/55/47/63/48; join backward, bf16 145/150/127/186/145 and 111/88/77/100/78.
    // (It loses where the last of the four or eight is mostly idle, up to 12 % just above 512, and up to 10 % in the float32
    // join's forward above 1024.)
    if (vec == 1 && D > 512 && D <= kNarrowD) return {256, 256, D <= 1024 ? 4 : 8};
    const int most = D <= kNarrowD ? 256 : 512;
    int nv = 1;
    while ((nvec + nv - 1) / nv > most) nv *= 2;
    return {0, ((nvec + nv - 1) / nv + 31) / 32 * 32, nv};
}

// f(NV, TPR, MAXT) as integral constants for the shape
template <int VEC, class F>
int with_shape(int D, const Shape& s, F&& f) {
    using std::integral_constant;
    auto go = [&](auto nv, auto tpr, auto maxt) { return f(integral_constant<int, VEC>{}, nv, tpr, maxt); };
    const integral_constant<int, 1> one{};
    const integral_constant<int, 0> cta{};
    const integral_constant<int, kSmallThreads> small{};
    const integral_constant<int, 512> large{};
    switch (s.tpr) {
        case 8: return go(one, integral_constant<int, 8>{}, small);
        case 32: return go(one, integral_constant<int, 32>{}, small);
        case 256:
            if constexpr (VEC == 1) {
                if (s.nv == 4) return go(integral_constant<int, 4>{}, integral_constant<int, 256>{}, small);
                return go(integral_constant<int, 8>{}, integral_constant<int, 256>{}, small);
            }
            return -1;
        default: break;
    }
    if (D <= kNarrowD) {
        if (s.nv == 1) return go(one, cta, small);
        if constexpr (VEC < 8) {
            if (s.nv == 2) return go(integral_constant<int, 2>{}, cta, small);
        }
        if constexpr (VEC == 2) {
            if (s.nv == 4) return go(integral_constant<int, 4>{}, cta, small);
        }
        return -1;
    }
    if (s.nv == 8 / VEC) return go(integral_constant<int, 8 / VEC>{}, cta, large);
    if (s.nv == 16 / VEC) return go(integral_constant<int, 16 / VEC>{}, cta, large);
    return -1;
}
template <class F>
int with_vec(int D, int vec, const Shape& s, F&& f) {
    switch (vec) {
        case 8: return with_shape<8>(D, s, f);
        case 4: return with_shape<4>(D, s, f);
        case 2: return with_shape<2>(D, s, f);
        default: return with_shape<1>(D, s, f);
    }
}

int join_ok() { return set_last_error(HLA2_OK, "%s", ""); }

// Whether the call has a block output; without rows there is no address to go by.
bool has_y(const hla2_block_args* a) { return a->rows > 0 ? a->y != nullptr : a->post_weight != nullptr; }

int check_join(const char* fn, const hla2_block_args* a) {
    if (!a) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: args must not be NULL", fn);
    if (a->dtype != HLA2_F32 && a->dtype != HLA2_BF16)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: dtype must be HLA2_F32 or HLA2_BF16", fn);
    if (a->D < 1 || a->D > kMaxD)
        return set_last_error(a->D < 1 ? HLA2_ERR_INVALID_ARG : HLA2_ERR_UNSUPPORTED, "%s: D must be 1 .. %d (got %d)",
                              fn, kMaxD, a->D);
    if (a->rows < 0 || a->rows > 0x7fffffffLL)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: rows must be 0 .. 2^31 - 1", fn);
    if (!has_y(a) && !a->next_weight)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: nothing to form without y and next_weight", fn);
    if (a->y && !a->post_weight) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: y needs post_weight", fn);
    if (!has_y(a) && (a->gate || a->scale || a->post_weight))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: gate, scale and post_weight need y", fn);
    if (a->gate && (a->gate_act != HLA2_GATE_SIGMOID && a->gate_act != HLA2_GATE_SILU))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: unknown gate_act %d", fn, a->gate_act);
    if (a->gate && a->gate_cols != 1 && a->gate_cols != a->D)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: gate_cols must be 1 or D", fn);
    const size_t es = a->dtype == HLA2_BF16 ? 2 : 4;
    if (!al(a->x, es) || !al(a->y, es) || !al(a->gate, es) || !al(a->post_weight, es) || !al(a->scale, es) ||
        !al(a->next_weight, es))
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: a pointer is not aligned to its type", fn);
    if (a->rows > 0) {
        if (!a->x) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: x must not be NULL", fn);
        if (a->rows > 1 && (a->x_stride < 0 || (a->y && a->y_stride < 0) || (a->gate && a->gate_stride < 0)))
            return set_last_error(HLA2_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
    }
    return HLA2_OK;
}

// Rows of cols elements, `stride` apart
struct RowsOf {
    const void* p;
    long long stride;
    int cols;
};
Extent rows_extent(const hla2_block_args* a, const RowsOf& t) {
    return extent_of(t.p, (size_t)((a->rows - 1) * t.stride + t.cols) * (a->dtype == HLA2_BF16 ? 2 : 4));
}
// Whether contiguous rows that are written overlap what the call reads in another way than as exactly the same rows: a
// row is read whole before it is written, but its neighbours may be read earlier or later.
bool spoils(const hla2_block_args* a, const RowsOf& out, const RowsOf* more, int nmore) {
    const Extent eo = rows_extent(a, out);
    auto hits = [&](const RowsOf& t) {
        return t.p && meet(eo, rows_extent(a, t)) &&
               !(t.p == out.p && t.cols == out.cols && (t.stride == out.cols || a->rows == 1));
    };
    const RowsOf in[6] = {{a->x, a->x_stride, a->D}, {a->y, a->y_stride, a->D}, {a->gate, a->gate_stride, a->gate_cols},
                          {a->post_weight, 0, a->D}, {a->scale, 0, a->D}, {a->next_weight, 0, a->D}};
    for (int i = 0; i < 6; ++i)
        if (i < 3 ? hits(in[i]) : in[i].p && meet(eo, rows_extent(a, in[i]))) return true;
    for (int i = 0; i < nmore; ++i)
        if (hits(more[i])) return true;
    return false;
}

// Persistent CTAs and their ring.  Stages: as many rows ahead as fit in the SM's shared memory beside
// the CTAs that the registers allow (1024 threads of the forward, 512 of the backward, 768 where there
// is no block output), at most four, and no more than a CTA has rounds; one stage copies and waits.
// The backward with a block output at 768 threads spills: 272 us against 223 for 32768 rows of 2048.
struct Work {
    int ctas, stages;
    size_t smem;
};
Work work_of(const hla2_block_args* a, const Shape& s, int vec, int tensors, int threads_per_sm, size_t least,
             int sms) {
    const size_t slot = (size_t)vec * (a->dtype == HLA2_BF16 ? 2 : 4);
    const size_t stage = slot * s.threads * s.nv * tensors, room = 220 * 1024;
    int each = threads_per_sm / s.threads;
    if (each < 1) each = 1;
    if (each > 16) each = 16;
    Work w;
    w.stages = slot == 2 && s.nv > 4 ? 1 : 4;  // copied at once (kHolds): no use in a ring, which would leave the L1 little
    while (w.stages > 1 && (w.stages * stage + 2048) * each > room && !(each == 1 && w.stages * stage <= room)) --w.stages;
    while (each > 1 && (w.stages * stage + 2048) * each > room) --each;
    const int per = s.tpr ? kSmallThreads / s.tpr : 1;
    const long long need = (a->rows + per - 1) / per, most = (long long)each * sms;
    w.ctas = (int)(need < most ? need : most);
    if (w.ctas > 0 && need < (long long)w.stages * w.ctas) w.stages = (int)((need + w.ctas - 1) / w.ctas);
    w.smem = w.stages * stage > least ? w.stages * stage : least;
    return w;
}
constexpr int kFwdThreadsPerSm = 1024, kBwdThreadsPerSm = 512, kNormBwdThreadsPerSm = 768;

template <class K>
bool set_smem(K kernel, size_t bytes) {
    return bytes <= 40 * 1024 /* 48 KB with the static part */ || raise_smem(kernel, bytes) == cudaSuccess;
}

// Which kernel serves the call.
int mode_of(const hla2_block_args* a, const void* dr_or_h) {
    if (!a->y) return kNormOnly;
    return a->gate && a->gate_cols != 1 && a->scale && a->next_weight && dr_or_h ? kAll : kAny;
}

// f(VEC, NV, TPR, MAXT, MODE, zero of the type) as integral constants
template <class F>
int dispatch(const hla2_block_args* a, int mode, int vec, const Shape& s, F&& f) {
    return with_vec(a->D, vec, s, [&](auto v, auto nv, auto tpr, auto maxt) {
        auto typed = [&](auto zero) {
            using std::integral_constant;
            switch (mode) {
                case kNormOnly: return f(v, nv, tpr, maxt, integral_constant<int, kNormOnly>{}, zero);
                case kAll: return f(v, nv, tpr, maxt, integral_constant<int, kAll>{}, zero);
                default: return f(v, nv, tpr, maxt, integral_constant<int, kAny>{}, zero);
            }
        };
        constexpr int VEC = decltype(v)::value;
        if constexpr (VEC == 8 || VEC == 2) return typed(bf16{});
        else if constexpr (VEC == 4) return typed(float{});
        else return a->dtype == HLA2_BF16 ? typed(bf16{}) : typed(float{});
    });
}

}  // namespace
}  // namespace hla2
