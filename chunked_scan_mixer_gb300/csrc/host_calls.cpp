// The host side of the short calls around a layer, for Python (module _hla2_host).  These calls take a few
// microseconds on the GPU, less than their checks and allocations take in the interpreter: a step of one sequence
// takes 12 to 15 us a call there and 4.7 to 8.2 us here, four rows of a join 15 to 18 us and 6.0 to 9.6 us.
//
// Each function takes the tensors as the binding (hla2.py) does and covers the ordinary call: tensors of
// the current device and a supported type, contiguous or with strides that the kernels read in place, nothing
// to convert.  It returns None for any other, and where the library refuses the call, before anything has been
// launched; the binding then takes its own way, which converts, or says what is wrong.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "hla2.h"

namespace {

using at::Tensor;

// The library's entry points, from the library that the binding has loaded.
struct Entries {
    decltype(&hla2_linattn_forward) linattn_forward;
    decltype(&hla2_linattn_backward) linattn_backward;
    decltype(&hla2_linattn_decode_step) linattn_decode_step;
    decltype(&hla2_block_join) block_join;
    decltype(&hla2_block_join_backward) block_join_backward;
    decltype(&hla2_w4_matvec) w4_matvec;
    decltype(&hla2_ssm_forward) ssm_forward;
    decltype(&hla2_ssm_backward) ssm_backward;
    decltype(&hla2_ssm_decode_step) ssm_decode_step;
    decltype(&hla2_short_conv_forward) short_conv_forward;
    decltype(&hla2_short_conv_backward) short_conv_backward;
    decltype(&hla2_short_conv_decode_step) short_conv_decode_step;
    decltype(&hla2_layer_norm) layer_norm;
    decltype(&hla2_layer_norm_backward) layer_norm_backward;
} lib{};

constexpr size_t kStatusBytes = 256;  // at a workspace's start, for the calls with bounded waits

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }
bool none(PyObject* o) { return o == Py_None; }

// What the call's tensors share
struct Common {
    c10::DeviceIndex device;
    at::ScalarType type;
    int dtype;
    bool of(const Tensor& t) {
        device = t.is_cuda() ? t.get_device() : -1;
        type = t.scalar_type();
        dtype = type == at::kBFloat16 ? HLA2_BF16 : HLA2_F32;
        // the library launches on the current device
        return device >= 0 && device == c10::cuda::current_device() && (type == at::kBFloat16 || type == at::kFloat);
    }
    bool has(const Tensor& t) const { return has(t, type); }
    bool has(const Tensor& t, at::ScalarType s) const { return t.is_cuda() && t.get_device() == device && t.scalar_type() == s; }
    hla2_stream_t stream() const { return reinterpret_cast<hla2_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream()); }
};

bool aligned(const Tensor& t) { return (reinterpret_cast<uintptr_t>(t.data_ptr()) & 15u) == 0; }
bool is(const Tensor& t, std::initializer_list<int64_t> sizes) { return t.sizes() == at::IntArrayRef(sizes); }
bool fits(int64_t x) { return x >= 0 && x <= 0x7fffffff; }

// Optional contiguous tensor of a type and sizes: its address (NULL for None) into p
bool optional(const Common& c, PyObject* o, at::ScalarType s, std::initializer_list<int64_t> sizes, const void** p) {
    *p = nullptr;
    if (none(o)) return true;
    const Tensor* t = tensor(o);
    if (!t || !c.has(*t, s) || !is(*t, sizes) || !t->is_contiguous()) return false;
    *p = t->data_ptr();
    return true;
}

// Rows of D values: contiguous, or two dimensions with a row stride
bool rows_of(const Tensor& t, int64_t D, int64_t* stride) {
    if (t.dim() == 2) {
        if (t.size(1) != D || (t.stride(1) != 1 && D > 1) || t.stride(0) < 0) return false;
        *stride = t.stride(0);
        return true;
    }
    *stride = D;
    return t.dim() > 2 && t.size(-1) == D && t.is_contiguous();
}

// [B, heads, n, D] that the kernels read in place
bool view_of(const Tensor& t, hla2_view* v) {
    const int64_t per16 = 16 / t.element_size(), D = t.size(3);
    if (!aligned(t) || (t.stride(3) != 1 && D > 1)) return false;
    for (int i = 0; i < 3; ++i)
        if (t.size(i) > 1 && (t.stride(i) % per16 || t.stride(i) < D)) return false;
    *v = {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
    return true;
}
hla2_view out_view(const Tensor& t) { return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)}; }

// A new [B, heads, n, D] in the token / head order of `like`
Tensor like4(const Tensor& like, int64_t heads, int64_t D) {
    const int64_t B = like.size(0), n = like.size(2);
    if (like.stride(2) > like.stride(1)) return at::empty({B, n, heads, D}, like.options()).transpose(1, 2);
    return at::empty({B, heads, n, D}, like.options());
}

// Runs f, which returns a new reference or nullptr where the call is not its own.
template <class F>
PyObject* guarded(F&& f) {
    PyObject* r = nullptr;
    try {
        r = f();
    } catch (const std::exception&) {
        r = nullptr;
    }
    if (r) return r;
    PyErr_Clear();
    Py_RETURN_NONE;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap_all(std::initializer_list<const Tensor*> ts) {  // NULL: None
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    if (r)
        for (const Tensor* t : ts) PyTuple_SET_ITEM(r, i++, t ? wrap(*t) : Py_NewRef(Py_None));
    return r;
}

// ---- linear attention ------------------------------------------------------------------------

// q, k, v, gamma, scale, lengths, init_state, workspace -> checked sizes and arguments
struct Lin : Common {
    hla2_linattn_args a{};
    const Tensor *q, *k, *v;
    bool read(PyObject* const* p, PyObject* workspace) {
        q = tensor(p[0]), k = tensor(p[1]), v = tensor(p[2]);
        const Tensor* ws = tensor(workspace);
        if (!q || !k || !v || !ws || !of(*q) || !has(*k) || !has(*v) || q->dim() != 4 || k->dim() != 4 || v->dim() != 4)
            return false;
        const int64_t B = q->size(0), H = q->size(1), n = q->size(2), d = q->size(3), Hk = k->size(1), dv = v->size(3);
        if (B < 1 || H < 1 || n < 1 || Hk < 1 || H % Hk || !fits(B) || !fits(H) || !fits(n) || !is(*k, {B, Hk, n, d}) ||
            !is(*v, {B, Hk, n, dv}))
            return false;
        const void *gamma, *lengths, *init;
        if (!optional(*this, p[3], at::kFloat, {Hk}, &gamma) || !optional(*this, p[5], at::kInt, {B}, &lengths) ||
            !optional(*this, p[6], at::kFloat, {B, Hk, d, dv}, &init) || !has(*ws, at::kByte))
            return false;
        const double scale = PyFloat_AsDouble(p[4]);
        if (PyErr_Occurred()) return false;
        a.dtype = dtype, a.B = (int)B, a.H = (int)H, a.Hk = (int)Hk, a.n = (int)n, a.d = (int)d, a.dv = (int)dv;
        a.scale = (float)scale;
        a.gamma = static_cast<const float*>(gamma);
        a.lengths = static_cast<const int*>(lengths);
        a.init_state = static_cast<const float*>(init);
        a.workspace = ws->data_ptr();
        a.workspace_bytes = (size_t)ws->numel();
        return d <= 128 && dv <= 128 && view_of(*q, &a.q) && view_of(*k, &a.k) && view_of(*v, &a.v);
    }
    Tensor state() const { return at::empty({a.B, a.Hk, a.d, a.dv}, q->options().dtype(at::kFloat)); }
};

// (q, k, v, gamma, scale, lengths, init_state, want_final, workspace) -> out or (out, state)
PyObject* linattn_forward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Lin c;
        if (count != 9 || !c.read(p, p[8])) return nullptr;
        const bool want = p[7] == Py_True;
        const Tensor out = like4(*c.q, c.a.H, c.a.dv);
        Tensor fin;
        if (want) fin = c.state();
        if (lib.linattn_forward(&c.a, out_view(out), want ? fin.data_ptr<float>() : nullptr, c.stream())) return nullptr;
        return want ? wrap_all({&out, &fin}) : wrap(out);
    });
}

// (q, k, v, gamma, scale, lengths, init_state, dout, dfinal_state, workspace) -> (dq, dk, dv) or, with an init_state,
// its gradient too
PyObject* linattn_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Lin c;
        if (count != 10 || !c.read(p, p[9])) return nullptr;
        const Tensor* dout = tensor(p[7]);
        const void* dfin;
        hla2_view dov;
        if (!dout || !c.has(*dout) || !is(*dout, {c.a.B, c.a.H, c.a.n, c.a.dv}) || !view_of(*dout, &dov) ||
            !optional(c, p[8], at::kFloat, {c.a.B, c.a.Hk, c.a.d, c.a.dv}, &dfin))
            return nullptr;
        const Tensor dq = like4(*c.q, c.a.H, c.a.d), dk = like4(*c.k, c.a.Hk, c.a.d), dv = like4(*c.v, c.a.Hk, c.a.dv);
        Tensor dinit;
        if (c.a.init_state) dinit = c.state();
        if (lib.linattn_backward(&c.a, dov, out_view(dq), out_view(dk), out_view(dv), static_cast<const float*>(dfin),
                                 c.a.init_state ? dinit.data_ptr<float>() : nullptr, c.stream()))
            return nullptr;
        return c.a.init_state ? wrap_all({&dq, &dk, &dv, &dinit}) : wrap_all({&dq, &dk, &dv});
    });
}

// (state, q, k, v, gamma, scale) -> out
PyObject* linattn_decode_step(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        if (count != 6) return nullptr;
        const Tensor *st = tensor(p[0]), *q = tensor(p[1]), *k = tensor(p[2]), *v = tensor(p[3]);
        Common c;
        if (!st || !q || !k || !v || !c.of(*q) || !c.has(*k) || !c.has(*v) || !c.has(*st, at::kFloat) || q->dim() != 3 ||
            k->dim() != 3 || v->dim() != 3)
            return nullptr;
        const int64_t N = q->size(0), H = q->size(1), d = q->size(2), Hk = k->size(1), dv = v->size(2);
        const void* gamma;
        if (!is(*k, {N, Hk, d}) || !is(*v, {N, Hk, dv}) || !is(*st, {N, Hk, d, dv}) || !fits(N) || !fits(H) || !fits(d) ||
            !fits(dv) || !optional(c, p[4], at::kFloat, {Hk}, &gamma))
            return nullptr;
        for (const Tensor* t : {st, q, k, v})
            if (!t->is_contiguous() || !aligned(*t)) return nullptr;
        const double scale = PyFloat_AsDouble(p[5]);
        if (PyErr_Occurred()) return nullptr;
        const Tensor out = at::empty({N, H, dv}, q->options());
        if (lib.linattn_decode_step(st->data_ptr<float>(), q->data_ptr(), k->data_ptr(), v->data_ptr(), out.data_ptr(), (int)N,
                                    (int)H, (int)Hk, (int)d, (int)dv, static_cast<const float*>(gamma), (float)scale,
                                    c.dtype, c.stream()))
            return nullptr;
        return wrap(out);
    });
}

// ---- block norms -----------------------------------------------------------------------------

// x, y, post_weight, gate, act (0, 1), scale, next_weight, eps; y, gate, scale and next_weight may be None
struct Block : Common {
    hla2_block_args a{};
    const Tensor *x, *y = nullptr, *gate = nullptr;
    bool read(PyObject* const* p) {
        x = tensor(p[0]);
        if (!x || !of(*x) || x->dim() < 2 || x->numel() == 0) return false;
        const int64_t D = x->size(-1);
        int64_t xs, ys = 0, zs = 0;
        if (!fits(D) || !rows_of(*x, D, &xs)) return false;
        const void *pw, *sc, *nw;
        if (!optional(*this, p[2], type, {D}, &pw) || !optional(*this, p[5], type, {D}, &sc) ||
            !optional(*this, p[6], type, {D}, &nw))
            return false;
        if (!none(p[1])) {
            y = tensor(p[1]);
            if (!y || !has(*y) || y->sizes() != x->sizes() || !rows_of(*y, D, &ys)) return false;
        }
        if (!none(p[3])) {
            gate = tensor(p[3]);
            if (!y || !gate || !has(*gate) || gate->dim() != x->dim()) return false;
            const int64_t cols = gate->size(-1);
            if ((cols != 1 && cols != D) || gate->sizes().slice(0, gate->dim() - 1) != x->sizes().slice(0, x->dim() - 1) ||
                !rows_of(*gate, cols, &zs))
                return false;
            a.gate = gate->data_ptr();
            a.gate_cols = (int)cols;
        }
        const long act = PyLong_AsLong(p[4]);
        const double eps = PyFloat_AsDouble(p[7]);
        if (PyErr_Occurred()) return false;
        a.dtype = dtype, a.gate_act = (int)act, a.rows = x->numel() / D, a.D = (int)D, a.eps = (float)eps;
        a.x = x->data_ptr(), a.x_stride = xs;
        a.y = y ? y->data_ptr() : nullptr, a.y_stride = ys, a.gate_stride = zs;
        a.post_weight = pw, a.scale = sc, a.next_weight = nw;
        return true;
    }
    Tensor make(const Tensor& t) const { return at::empty(t.sizes(), t.options()); }
};

// (x, y, post_weight, gate, act, scale, next_weight, eps) -> (r, h), each None where it is not formed
PyObject* block_join(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Block c;
        if (count != 8 || !c.read(p)) return nullptr;
        Tensor r, h;
        if (c.y) r = c.make(*c.x);
        if (c.a.next_weight) h = c.make(*c.x);
        if (lib.block_join(&c.a, c.y ? r.data_ptr() : nullptr, c.a.next_weight ? h.data_ptr() : nullptr, c.stream()))
            return nullptr;
        return wrap_all({c.y ? &r : nullptr, c.a.next_weight ? &h : nullptr});
    });
}

// (x, y, post_weight, gate, act, scale, next_weight, eps, dr, dh, workspace) -> (dx, dy, dgate, dpost_weight, dscale,
// dnext_weight), each None where there is no such input
PyObject* block_join_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Block c;
        const Tensor* ws = count == 11 ? tensor(p[10]) : nullptr;
        if (!ws || !c.read(p) || !c.has(*ws, at::kByte) || (size_t)ws->numel() <= kStatusBytes) return nullptr;
        const void* d[2] = {nullptr, nullptr};
        for (int i = 0; i < 2; ++i) {
            if (none(p[8 + i])) continue;
            const Tensor* t = tensor(p[8 + i]);
            if (!t || !c.has(*t) || t->sizes() != c.x->sizes() || !t->is_contiguous()) return nullptr;
            d[i] = t->data_ptr();
        }
        const auto sums = c.x->options().dtype(at::kFloat);
        const Tensor dx = c.make(*c.x), dnw = c.a.next_weight ? at::empty({c.a.D}, sums) : Tensor();
        Tensor dy, dgate, dpw, dsc;
        if (c.y) dy = c.make(*c.y), dpw = at::empty({c.a.D}, sums);
        if (c.gate) dgate = c.make(*c.gate);
        if (c.a.scale) dsc = at::empty({c.a.D}, sums);
        auto at_ = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
        auto f32 = [](const Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; };
        if (lib.block_join_backward(&c.a, d[0], d[1], at_(dx), at_(dy), at_(dgate), f32(dpw), f32(dsc), f32(dnw),
                                    static_cast<char*>(ws->data_ptr()) + kStatusBytes, (size_t)ws->numel() - kStatusBytes,
                                    c.stream()))
            return nullptr;
        auto given = [](const Tensor& t) { return t.defined() ? &t : nullptr; };
        return wrap_all({&dx, given(dy), given(dgate), given(dpw), given(dsc), given(dnw)});
    });
}

// ---- 4-bit products --------------------------------------------------------------------------

// (x, qweight, scales, zeros, bias) -> y
PyObject* w4_matvec(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        if (count != 5) return nullptr;
        const Tensor *x = tensor(p[0]), *w = tensor(p[1]), *s = tensor(p[2]);
        Common c;
        if (!x || !w || !s || !c.of(*x) || !c.has(*s) || !c.has(*w, at::kByte) || x->dim() < 2 || w->dim() != 2 ||
            s->dim() != 2 || x->numel() == 0)
            return nullptr;
        const int64_t K = x->size(-1), N = w->size(0), groups = s->size(1), M = x->numel() / K;
        int64_t stride;
        const void *zeros, *bias;
        if (w->size(1) * 2 != K || s->size(0) != N || groups < 1 || K % groups || M > 16 || !fits(N) || !fits(K) ||
            !rows_of(*x, K, &stride) || !aligned(*x) || (stride * x->element_size()) % 16 || !w->is_contiguous() ||
            !aligned(*w) || !s->is_contiguous() || !optional(c, p[3], at::kByte, {N, groups}, &zeros) ||
            !optional(c, p[4], c.type, {N}, &bias))
            return nullptr;
        c10::SmallVector<int64_t, 4> sizes(x->sizes().begin(), x->sizes().end());
        sizes.back() = N;
        const Tensor y = at::empty(sizes, x->options());
        if (lib.w4_matvec(x->data_ptr(), stride, w->data_ptr(), s->data_ptr(), zeros, bias, y.data_ptr(), (int)M, (int)N,
                          (int)K, (int)(K / groups), c.dtype, c.stream()))
            return nullptr;
        return wrap(y);
    });
}

// ---- selective state space layer -------------------------------------------------------------

// [B, n, D] or, for single tokens, [B, D], with a contiguous last dimension
bool token_rows(const Tensor& t, hla2_rows* r) {
    const int64_t last = t.dim() - 1;
    if (t.stride(last) != 1 && t.size(last) > 1) return false;
    *r = {t.data_ptr(), t.stride(0), last == 2 ? t.stride(1) : 0};
    return true;
}
hla2_rows rows_out(const Tensor& t) { return {t.data_ptr(), t.stride(0), t.dim() == 3 ? t.stride(1) : 0}; }

// The scratch of a call behind its status word; None: none, which small calls do not need
bool scratch_of(const Common& c, PyObject* o, void** p, size_t* bytes) {
    *p = nullptr, *bytes = 0;
    if (none(o)) return true;
    const Tensor* ws = tensor(o);
    if (!ws || !c.has(*ws, at::kByte) || (size_t)ws->numel() <= kStatusBytes) return false;
    *p = static_cast<char*>(ws->data_ptr()) + kStatusBytes;
    *bytes = (size_t)ws->numel() - kStatusBytes;
    return true;
}
bool truth(PyObject* o, int* v) {
    if (o != Py_True && o != Py_False) return false;
    *v = o == Py_True;
    return true;
}
void* at_(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* f32_at(const Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; }
const Tensor* given(const Tensor& t) { return t.defined() ? &t : nullptr; }

// x, dt, a, b, c, skip, gate, dt_bias, dt_softplus, lengths, init_state; `tokens`: x is [B, n, D], else [B, D]
struct Ssm : Common {
    hla2_ssm_args a{};
    const Tensor *x, *b, *c, *gate = nullptr;
    // b or c: [B, n, N] or [B, n, G, N], without n for single tokens
    bool states(const Tensor& t, bool tokens, hla2_view* v) const {
        const int64_t last = t.dim() - 1, at = tokens ? 2 : 1;
        if (t.stride(last) != 1 && t.size(last) > 1) return false;
        *v = {t.data_ptr(), t.stride(0), last == at ? 0 : t.stride(at), tokens ? t.stride(1) : 0};
        return true;
    }
    bool read(PyObject* const* p, bool tokens) {
        const int64_t lead = tokens ? 2 : 1;
        x = tensor(p[0]), b = tensor(p[3]), c = tensor(p[4]);
        const Tensor *dt = tensor(p[1]), *A = tensor(p[2]);
        if (!x || !dt || !A || !b || !c || !of(*x) || !has(*dt) || !has(*b) || !has(*c) || !has(*A, at::kFloat) ||
            x->dim() != lead + 1 || dt->sizes() != x->sizes() || A->dim() != 2 || (b->dim() != lead + 1 && b->dim() != lead + 2) ||
            c->sizes() != b->sizes())
            return false;
        const int64_t B = x->size(0), n = tokens ? x->size(1) : 1, D = x->size(lead), N = A->size(1);
        const int64_t G = b->dim() == lead + 2 ? b->size(lead) : 1;
        if (B < 1 || n < 1 || D < 1 || G < 1 || !fits(B) || !fits(n) || !fits(D) || !fits(N) || A->size(0) != D || D % G ||
            b->size(0) != B || (tokens && b->size(1) != n) || b->size(b->dim() - 1) != N || !A->is_contiguous())
            return false;
        const void *skip, *bias, *lengths, *init;
        if (!optional(*this, p[5], at::kFloat, {D}, &skip) || !optional(*this, p[7], at::kFloat, {D}, &bias) ||
            !truth(p[8], &a.softplus) || !optional(*this, p[9], at::kInt, {B}, &lengths) ||
            !optional(*this, p[10], at::kFloat, {B, D, N}, &init))
            return false;
        if (!none(p[6])) {
            gate = tensor(p[6]);
            if (!gate || !has(*gate) || gate->sizes() != x->sizes() || !token_rows(*gate, &a.gate)) return false;
        }
        a.dtype = dtype, a.B = (int)B, a.n = (int)n, a.D = (int)D, a.N = (int)N, a.G = (int)G;
        a.a = A->data_ptr<float>();
        a.skip = static_cast<const float*>(skip), a.dt_bias = static_cast<const float*>(bias);
        a.lengths = static_cast<const int*>(lengths);
        a.init_state = static_cast<const float*>(init);
        return token_rows(*x, &a.x) && token_rows(*dt, &a.dt) && states(*b, tokens, &a.b) && states(*c, tokens, &a.c);
    }
    Tensor floats(std::initializer_list<int64_t> sizes) const { return at::empty(at::IntArrayRef(sizes), x->options().dtype(at::kFloat)); }
};

// (x, dt, a, b, c, skip, gate, dt_bias, dt_softplus, lengths, init_state, want_final, workspace) -> out or (out, state)
PyObject* ssm_forward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Ssm s;
        if (count != 13 || !s.read(p, true) || !scratch_of(s, p[12], &s.a.workspace, &s.a.workspace_bytes)) return nullptr;
        const bool want = p[11] == Py_True;
        const Tensor out = at::empty(s.x->sizes(), s.x->options());
        Tensor fin;
        if (want) fin = s.floats({s.a.B, s.a.D, s.a.N});
        if (lib.ssm_forward(&s.a, rows_out(out), f32_at(fin), s.stream())) return nullptr;
        return want ? wrap_all({&out, &fin}) : wrap(out);
    });
}

// (x, dt, a, b, c, skip, gate, dt_bias, dt_softplus, lengths, init_state, dout, dfinal_state, workspace) -> the gradients in
// SsmGrads' order, None where there is no such input
PyObject* ssm_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Ssm s;
        if (count != 14 || !s.read(p, true) || !scratch_of(s, p[13], &s.a.workspace, &s.a.workspace_bytes)) return nullptr;
        const Tensor* dout = tensor(p[11]);
        const void* dfin;
        hla2_rows dor;
        const int64_t B = s.a.B, n = s.a.n, D = s.a.D, N = s.a.N, G = s.a.G;
        if (!dout || !s.has(*dout) || dout->sizes() != s.x->sizes() || !token_rows(*dout, &dor) ||
            !optional(s, p[12], at::kFloat, {B, D, N}, &dfin))
            return nullptr;
        const auto like = s.x->options();
        const Tensor dx = at::empty({B, n, D}, like), ddt = at::empty({B, n, D}, like), da = s.floats({D, N});
        const Tensor db = at::empty(s.b->sizes(), like), dc = at::empty(s.b->sizes(), like);
        Tensor dskip, dgate, dbias, dinit;
        if (s.a.skip) dskip = s.floats({D});
        if (s.gate) dgate = at::empty({B, n, D}, like);
        if (s.a.dt_bias) dbias = s.floats({D});
        if (s.a.init_state) dinit = s.floats({B, D, N});
        hla2_ssm_grads g{};
        g.dx = rows_out(dx), g.ddt = rows_out(ddt);
        if (s.gate) g.dgate = rows_out(dgate);
        g.db = {db.data_ptr(), n * G * N, N, G * N}, g.dc = {dc.data_ptr(), n * G * N, N, G * N};
        g.da = f32_at(da), g.dskip = f32_at(dskip), g.ddt_bias = f32_at(dbias), g.dinit_state = f32_at(dinit);
        if (lib.ssm_backward(&s.a, dor, static_cast<const float*>(dfin), &g, s.stream())) return nullptr;
        return wrap_all({&dx, &ddt, &da, &db, &dc, given(dskip), given(dgate), given(dbias), given(dinit)});
    });
}

// (state, x, dt, a, b, c, skip, gate, dt_bias, dt_softplus) -> out
PyObject* ssm_decode_step(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        if (count != 10) return nullptr;
        PyObject* q[11] = {p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], Py_None, Py_None};
        const Tensor* st = tensor(p[0]);
        Ssm s;
        if (!st || !s.read(q, false) || !s.has(*st, at::kFloat) || !is(*st, {s.a.B, s.a.D, s.a.N}) || !st->is_contiguous()) return nullptr;
        const Tensor out = at::empty(s.x->sizes(), s.x->options());
        if (lib.ssm_decode_step(&s.a, st->data_ptr<float>(), rows_out(out), s.stream())) return nullptr;
        return wrap(out);
    });
}

// x, weight, bias, silu, lengths, init_state
struct Conv : Common {
    hla2_conv_args a{};
    const Tensor* x;
    bool read(PyObject* const* p, bool tokens) {
        x = tensor(p[0]);
        const Tensor* w = tensor(p[1]);
        if (!x || !w || !of(*x) || !has(*w) || x->dim() != (tokens ? 3 : 2) || w->dim() != 2 || !w->is_contiguous()) return false;
        const int64_t B = x->size(0), n = tokens ? x->size(1) : 1, D = x->size(x->dim() - 1), W = w->size(1);
        const void *lengths;
        if (B < 1 || n < 1 || D < 1 || !fits(B) || !fits(n) || !fits(D) || W < 2 || W > 4 || w->size(0) != D ||
            !optional(*this, p[2], type, {D}, &a.bias) || !truth(p[3], &a.silu) || !optional(*this, p[4], at::kInt, {B}, &lengths) ||
            !optional(*this, p[5], type, {B, W - 1, D}, &a.init_state))
            return false;
        a.dtype = dtype, a.B = (int)B, a.n = (int)n, a.D = (int)D, a.W = (int)W;
        a.weight = w->data_ptr();
        a.lengths = static_cast<const int*>(lengths);
        return token_rows(*x, &a.x);
    }
    Tensor state() const { return at::empty({a.B, a.W - 1, a.D}, x->options()); }
};

// (x, weight, bias, silu, lengths, init_state, want_final) -> out or (out, state)
PyObject* short_conv_forward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Conv s;
        if (count != 7 || !s.read(p, true)) return nullptr;
        const bool want = p[6] == Py_True;
        const Tensor out = at::empty(s.x->sizes(), s.x->options());
        Tensor fin;
        if (want) fin = s.state();
        if (lib.short_conv_forward(&s.a, rows_out(out), at_(fin), s.stream())) return nullptr;
        return want ? wrap_all({&out, &fin}) : wrap(out);
    });
}

// (x, weight, bias, silu, lengths, init_state, dout, dfinal_state, workspace) -> the gradients in ShortConvGrads' order
PyObject* short_conv_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Conv s;
        if (count != 9 || !s.read(p, true) || !scratch_of(s, p[8], &s.a.workspace, &s.a.workspace_bytes)) return nullptr;
        const Tensor* dout = tensor(p[6]);
        const void* dfin;
        hla2_rows dor;
        if (!dout || !s.has(*dout) || dout->sizes() != s.x->sizes() || !token_rows(*dout, &dor) ||
            !optional(s, p[7], s.type, {s.a.B, s.a.W - 1, s.a.D}, &dfin))
            return nullptr;
        const Tensor dx = at::empty(s.x->sizes(), s.x->options()), dw = at::empty({s.a.D, s.a.W}, s.x->options().dtype(at::kFloat));
        Tensor db, dinit;
        if (s.a.bias) db = at::empty({s.a.D}, s.x->options().dtype(at::kFloat));
        if (s.a.init_state) dinit = s.state();
        if (lib.short_conv_backward(&s.a, dor, dfin, rows_out(dx), f32_at(dw), f32_at(db), at_(dinit), s.stream())) return nullptr;
        return wrap_all({&dx, &dw, given(db), given(dinit)});
    });
}

// (state, x, weight, bias, silu) -> out
PyObject* short_conv_decode_step(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        if (count != 5) return nullptr;
        PyObject* q[6] = {p[1], p[2], p[3], p[4], Py_None, Py_None};
        const Tensor* st = tensor(p[0]);
        Conv s;
        if (!st || !s.read(q, false) || !s.has(*st) || !is(*st, {s.a.B, s.a.W - 1, s.a.D}) || !st->is_contiguous()) return nullptr;
        const Tensor out = at::empty(s.x->sizes(), s.x->options());
        if (lib.short_conv_decode_step(&s.a, st->data_ptr(), rows_out(out), s.stream())) return nullptr;
        return wrap(out);
    });
}

// x, weight, bias, eps
struct Norm : Common {
    hla2_norm_args a{};
    const Tensor* x;
    bool read(PyObject* const* p) {
        x = tensor(p[0]);
        if (!x || !of(*x) || x->dim() < 2 || x->numel() == 0) return false;
        const int64_t D = x->size(-1);
        int64_t stride;
        if (!fits(D) || !rows_of(*x, D, &stride) || none(p[1]) || !optional(*this, p[1], type, {D}, &a.weight) ||
            !optional(*this, p[2], type, {D}, &a.bias))
            return false;
        const double eps = PyFloat_AsDouble(p[3]);
        if (PyErr_Occurred()) return false;
        a.dtype = dtype, a.rows = x->numel() / D, a.D = (int)D, a.eps = (float)eps;
        a.x = x->data_ptr(), a.x_stride = stride;
        return true;
    }
};

// (x, weight, bias, eps) -> out
PyObject* layer_norm(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        Norm s;
        if (count != 4 || !s.read(p)) return nullptr;
        const Tensor out = at::empty(s.x->sizes(), s.x->options());
        if (lib.layer_norm(&s.a, out.data_ptr(), s.stream())) return nullptr;
        return wrap(out);
    });
}

// (x, weight, dout, eps, workspace) -> (dx, dweight, dbias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* p, Py_ssize_t count) {
    return guarded([&]() -> PyObject* {
        if (count != 5) return nullptr;
        PyObject* q[4] = {p[0], p[1], Py_None, p[3]};
        const Tensor* dout = tensor(p[2]);
        Norm s;
        void* ws;
        size_t bytes;
        if (!s.read(q) || !scratch_of(s, p[4], &ws, &bytes) || !dout || !s.has(*dout) || dout->sizes() != s.x->sizes() ||
            !dout->is_contiguous())
            return nullptr;
        const auto sums = s.x->options().dtype(at::kFloat);
        const Tensor dx = at::empty(s.x->sizes(), s.x->options()), dw = at::empty({s.a.D}, sums), db = at::empty({s.a.D}, sums);
        if (lib.layer_norm_backward(&s.a, dout->data_ptr(), dx.data_ptr(), f32_at(dw), f32_at(db), ws, bytes, s.stream())) return nullptr;
        return wrap_all({&dx, &dw, &db});
    });
}

// (address of each entry point, in the order of Entries)
PyObject* bind(PyObject*, PyObject* const* p, Py_ssize_t count) {
    constexpr Py_ssize_t kEntries = sizeof(Entries) / sizeof(void*);
    if (count != kEntries) {
        PyErr_SetString(PyExc_TypeError, "bind: one address for each entry point");
        return nullptr;
    }
    void* at[kEntries];
    for (Py_ssize_t i = 0; i < kEntries; ++i) at[i] = PyLong_AsVoidPtr(p[i]);
    if (PyErr_Occurred()) return nullptr;
    static_assert(sizeof(at) == sizeof(Entries));
    memcpy(&lib, at, sizeof(at));
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

}  // namespace

PyMODINIT_FUNC PyInit__hla2_host() {
    static PyMethodDef methods[] = {
        {"bind", fast(bind), METH_FASTCALL, nullptr},
        {"linattn_forward", fast(linattn_forward), METH_FASTCALL, nullptr},
        {"linattn_backward", fast(linattn_backward), METH_FASTCALL, nullptr},
        {"linattn_decode_step", fast(linattn_decode_step), METH_FASTCALL, nullptr},
        {"block_join", fast(block_join), METH_FASTCALL, nullptr},
        {"block_join_backward", fast(block_join_backward), METH_FASTCALL, nullptr},
        {"w4_matvec", fast(w4_matvec), METH_FASTCALL, nullptr},
        {"ssm_forward", fast(ssm_forward), METH_FASTCALL, nullptr},
        {"ssm_backward", fast(ssm_backward), METH_FASTCALL, nullptr},
        {"ssm_decode_step", fast(ssm_decode_step), METH_FASTCALL, nullptr},
        {"short_conv_forward", fast(short_conv_forward), METH_FASTCALL, nullptr},
        {"short_conv_backward", fast(short_conv_backward), METH_FASTCALL, nullptr},
        {"short_conv_decode_step", fast(short_conv_decode_step), METH_FASTCALL, nullptr},
        {"layer_norm", fast(layer_norm), METH_FASTCALL, nullptr},
        {"layer_norm_backward", fast(layer_norm_backward), METH_FASTCALL, nullptr},
        {nullptr, nullptr, 0, nullptr}};
    static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hla2_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};
    return PyModule_Create(&module);
}
