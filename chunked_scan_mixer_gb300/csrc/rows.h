// Host side of the entry points that take rows of tokens (ssm_api.cu, short_conv.cu, layer_norm.cu): their tensors, and what
// is checked of them.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <numeric>

#include "common.cuh"

namespace hla2 {
int set_last_error(int code, const char* fmt, ...);

namespace {

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
bool al(const void* p, size_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) == 0; }
int elem_size(int dtype) { return dtype == HLA2_BF16 ? 2 : 4; }

// A tensor of the call with its strides of batch, group and token; those of dimensions of one element become packed ones.
struct Tensor {
    const char* name;
    const void* p;
    long long sb, sh, sn;
    int B, H, n, cols;

    Extent extent(int es) const {
        return extent_of(p, (size_t)((B - 1) * sb + (H - 1) * sh + (n - 1) * sn + cols) * es);
    }
    bool vec(int v, int es) const {
        return al(p, (size_t)v * es) && cols % v == 0 && sb % v == 0 && sh % v == 0 && sn % v == 0;
    }
    struct Dim { long long stride; int size; };
    // the dimensions but the columns, shorter strides first
    void dims(Dim (&d)[3]) const {
        d[0] = {sn, n}, d[1] = {sh, H}, d[2] = {sb, B};
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (d[j].stride > d[j + 1].stride) { const Dim t = d[j]; d[j] = d[j + 1], d[j + 1] = t; }
    }
    // whether no element has two places
    bool apart() const {
        Dim d[3];
        dims(d);
        long long span = cols;
        for (const Dim& x : d) {
            if (x.size > 1 && x.stride < span) return false;
            if (x.size > 1) span += (x.size - 1) * x.stride;
        }
        return true;
    }
    // elements that lie side by side at each of its rows, and the strides' greatest common divisor (0: one such block)
    void blocks(long long* block, long long* divisor) const {
        Dim d[3];
        dims(d);
        *block = cols, *divisor = 0;
        for (const Dim& x : d) {
            if (x.size <= 1) continue;
            if (*divisor == 0 && x.stride == *block) *block *= x.size;
            else *divisor = std::gcd(*divisor, x.stride);
        }
    }
};
// Whether two tensors of elements of es bytes share one.  Tensors whose address ranges meet may still lie side by side, as parts of the
// rows of one buffer: modulo a common divisor of all strides an element's place is its column's alone, so that they are apart
// where their columns are.  Tensors that interleave in another way count as sharing.
bool meet(const Tensor& a, const Tensor& b, int es) {
    if (!meet(a.extent(es), b.extent(es))) return false;
    long long na, nb, ga, gb;
    a.blocks(&na, &ga), b.blocks(&nb, &gb);
    const long long g = std::gcd(ga, gb);
    if (g == 0 || na > g || nb > g) return true;
    const long long by = (static_cast<const char*>(b.p) - static_cast<const char*>(a.p)) / es % g, at = by < 0 ? by + g : by;
    return at < na || at + nb > g;
}
// What a call reads, or writes
struct Places {
    int es;
    Extent flat[8];
    Tensor t[8];
    int flats = 0, tensors = 0;
    explicit Places(int es) : es(es) {}
    void add(const Extent& e) { flat[flats++] = e; }
    void add(const Tensor& e) { t[tensors++] = e; }
    bool meets(const Extent& e) const {
        for (int i = 0; i < flats; ++i)
            if (meet(e, flat[i])) return true;
        for (int i = 0; i < tensors; ++i)
            if (meet(e, t[i].extent(es))) return true;
        return false;
    }
    bool meets(const Tensor& e) const {
        for (int i = 0; i < flats; ++i)
            if (meet(e.extent(es), flat[i])) return true;
        for (int i = 0; i < tensors; ++i)
            if (meet(e, t[i], es)) return true;
        return false;
    }
};
Tensor rows(const char* name, const hla2_rows& r, int B, int n, int cols) {
    Tensor t{name, r.p, B > 1 ? r.sb : 0, 0, n > 1 ? r.sn : 0, B, 1, n, cols};
    return t;
}
Tensor view(const char* name, const hla2_view& r, int B, int H, int n, int cols) {
    Tensor t{name, r.p, B > 1 ? r.sb : 0, H > 1 ? r.sh : 0, n > 1 ? r.sn : 0, B, H, n, cols};
    return t;
}

int check_tensor(const char* fn, const Tensor& t, int es, bool written) {
    if (!t.p) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: %s must not be NULL", fn, t.name);
    if (!al(t.p, es)) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: %s is not aligned to its type", fn, t.name);
    if (t.sb < 0 || t.sh < 0 || t.sn < 0)
        return set_last_error(HLA2_ERR_INVALID_ARG, "%s: the strides of %s must not be negative", fn, t.name);
    if (written && !t.apart()) return set_last_error(HLA2_ERR_INVALID_ARG, "%s: rows of %s overlap", fn, t.name);
    return HLA2_OK;
}

}  // namespace
}  // namespace hla2
