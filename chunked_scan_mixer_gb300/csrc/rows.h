// Host side of the entry points that take rows of tokens (ssm_api.cu, short_conv.cu, layer_norm.cu): their tensors, and what
// is checked of them.
#pragma once

#include <nvtx3/nvToolsExt.h>

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
    // whether no element has two places
    bool apart() const {
        struct Dim { long long stride; int size; } d[3] = {{sn, n}, {sh, H}, {sb, B}};
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (d[j].stride > d[j + 1].stride) { const Dim t = d[j]; d[j] = d[j + 1], d[j + 1] = t; }
        long long span = cols;
        for (const Dim& x : d) {
            if (x.size > 1 && x.stride < span) return false;
            if (x.size > 1) span += (x.size - 1) * x.stride;
        }
        return true;
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
