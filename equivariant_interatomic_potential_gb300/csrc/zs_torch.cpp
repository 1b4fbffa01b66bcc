// Short way from torch tensors to libzs for the calls of a training step.
//
// The Python binding checks, allocates and marshals in Python, which takes
// longer than the kernels of small calls run.  These functions do the same for
// the ordinary case (contiguous tensors of the current device, of the right types
// and shapes, its current stream) and give NotImplemented for everything else, which the
// binding then handles, refusals among it.  They call libzs through the
// addresses that `bind` is given.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "zs.h"

namespace {

decltype(&zs_grouped_matmul_ws) f_matmul;
decltype(&zs_grouped_matmul_dx_ws) f_dx;
decltype(&zs_grouped_matmul_workspace_bytes) f_matmul_bytes;
decltype(&zs_grouped_matmul_dw_workspace_bytes) f_dw_bytes;
decltype(&zs_grouped_matmul_dw_copy_bytes) f_dw_copy;
decltype(&zs_grouped_matmul_dw) f_dw;
decltype(&zs_norm_gate_residual) f_norm;
decltype(&zs_norm_gate_residual_backward_workspace_bytes) f_norm_bytes;
decltype(&zs_norm_gate_residual_backward) f_norm_backward;
decltype(&zs_build_csr_workspace_bytes) f_csr_bytes;
decltype(&zs_build_csr) f_csr;
decltype(&zs_embedding) f_embedding;
decltype(&zs_embedding_backward_workspace_bytes) f_embedding_bytes;
decltype(&zs_embedding_backward) f_embedding_backward;
decltype(&zs_route) f_route;
decltype(&zs_route_backward) f_route_backward;
decltype(&zs_dispatch) f_dispatch;
decltype(&zs_combine) f_combine;
decltype(&zs_combine_backward) f_combine_backward;
decltype(&zs_dropout) f_dropout;
PyObject* on_error;   // binding's check(function name, status): raises

const at::Tensor* plain(PyObject* o) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.get_device() == c10::cuda::current_device() && t.is_contiguous() ? &t : nullptr;
}
// -1: not a type of the training operators
int dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return ZS_F32;
        case at::kBFloat16: return ZS_BF16;
        case at::kHalf: return ZS_F16;
        default: return -1;
    }
}
bool is_array(const at::Tensor* t, at::ScalarType type, int64_t n) {
    return t && t->scalar_type() == type && t->dim() == 1 && t->size(0) == n;
}
bool is_matrix(const at::Tensor* t, at::ScalarType type, int64_t rows, int64_t cols) {
    return t && t->scalar_type() == type && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols;
}
at::Tensor make(at::IntArrayRef shape, const at::Tensor& like, at::ScalarType type) {
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));   // half the time of at::empty
}
zs_stream_t stream() { return reinterpret_cast<zs_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }
PyObject* not_here() { Py_RETURN_NOTIMPLEMENTED; }
PyObject* failed(const char* fn, int status) {
    PyObject* r = PyObject_CallFunction(on_error, "si", fn, status);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s -> %d", fn, status);
    return nullptr;
}
// C++ exceptions as the Python ones that torch makes of them (an allocation that fails: torch.OutOfMemoryError)
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const std::exception&) {
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

// Whether rows of K or of N elements are not whole 16-byte pieces.
bool odd(int d, int64_t K, int64_t N) { return (K | N) & (d == 0 ? 3 : 7); }

// (rows, w, row_ptr, perm, transposed) -> y or dx
PyObject* matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) return not_here();
        const at::Tensor *x = plain(args[0]), *w = plain(args[1]), *row_ptr = plain(args[2]);
        const at::Tensor* perm = args[3] == Py_None ? nullptr : plain(args[3]);
        const bool t = args[4] == Py_True;
        if (!x || !w || x->dim() != 2 || w->dim() != 3) return not_here();
        const int64_t M = x->size(0), G = w->size(0), N = w->size(1), K = w->size(2);
        const at::ScalarType type = w->scalar_type();
        const int d = dtype_of(*w);
        if (d < 0 || !is_matrix(x, type, M, t ? N : K) || !is_array(row_ptr, at::kInt, G + 1) ||
            (args[3] != Py_None && !is_array(perm, at::kInt, M)) || (K | N | G) >> 31)
            return not_here();
        at::Tensor out = make({M, t ? K : N}, *x, type), ws;
        const size_t bytes = perm || odd(d, K, N) ? f_matmul_bytes(d, M, (int32_t)K, (int32_t)N, (int32_t)G) : 0;
        if (bytes) ws = make({(int64_t)bytes}, *x, at::kByte);
        const int32_t* pp = perm ? static_cast<const int32_t*>(perm->const_data_ptr()) : nullptr;
        const int st = (t ? f_dx : f_matmul)(d, x->const_data_ptr(), t ? N : K, w->const_data_ptr(),
                                             static_cast<const int32_t*>(row_ptr->const_data_ptr()), pp, M, (int32_t)K, (int32_t)N,
                                             (int32_t)G, out.mutable_data_ptr(), t ? K : N, bytes ? ws.mutable_data_ptr() : nullptr, bytes,
                                             stream());
        if (st) return failed(t ? "zs_grouped_matmul_dx_ws" : "zs_grouped_matmul_ws", st);
        return THPVariable_Wrap(std::move(out));
    });
}

// (dy, x, row_ptr, perm) -> dw
PyObject* dw(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 4) return not_here();
        const at::Tensor *dy = plain(args[0]), *x = plain(args[1]), *row_ptr = plain(args[2]);
        const at::Tensor* perm = args[3] == Py_None ? nullptr : plain(args[3]);
        if (!dy || !x || !row_ptr || dy->dim() != 2 || x->dim() != 2) return not_here();
        const int64_t M = x->size(0), K = x->size(1), N = dy->size(1), G = row_ptr->numel() - 1;
        const at::ScalarType type = x->scalar_type();
        const int d = dtype_of(*x);
        if (d < 0 || G < 0 || !is_matrix(dy, type, M, N) || !is_array(row_ptr, at::kInt, G + 1) ||
            (args[3] != Py_None && !is_array(perm, at::kInt, M)) || (K | N | G) >> 31)
            return not_here();
        at::Tensor out = make({G, N, K}, *x, type), ws;
        const size_t bytes = f_dw_bytes(d, M, (int32_t)K, (int32_t)N, (int32_t)G) +
                             (perm || odd(d, K, N) ? f_dw_copy(d, M, (int32_t)K, (int32_t)N, (int32_t)G) : 0);
        if (bytes) ws = make({(int64_t)bytes}, *x, at::kByte);
        const int32_t* pp = perm ? static_cast<const int32_t*>(perm->const_data_ptr()) : nullptr;
        const int st = f_dw(d, dy->const_data_ptr(), N, x->const_data_ptr(), K,
                            static_cast<const int32_t*>(row_ptr->const_data_ptr()), pp, M, (int32_t)K, (int32_t)N, (int32_t)G,
                            out.mutable_data_ptr(), bytes ? ws.mutable_data_ptr() : nullptr, bytes, stream());
        if (st) return failed("zs_grouped_matmul_dw", st);
        return THPVariable_Wrap(std::move(out));
    });
}

// The operands of the residual norms, from args[0]: h, x, gate, w_post, scale, w_pre.
struct NormOperands {
    const at::Tensor *h, *x, *gate, *w_post, *scale, *w_pre;
    int64_t M, C, gate_cols;
    int d;
    bool read(PyObject* const* args) {
        h = plain(args[0]), x = plain(args[1]);
        gate = args[2] == Py_None ? nullptr : plain(args[2]);
        w_post = plain(args[3]), scale = plain(args[4]), w_pre = plain(args[5]);
        if (!h || h->dim() != 2 || (args[2] != Py_None && (!gate || gate->dim() != 2))) return false;
        M = h->size(0), C = h->size(1), gate_cols = gate ? gate->size(1) : 0;
        d = dtype_of(*h);
        return d >= 0 && C <= INT32_MAX && is_matrix(x, h->scalar_type(), M, C) &&
               (!gate || ((gate_cols == 1 || gate_cols == C) && is_matrix(gate, h->scalar_type(), M, gate_cols))) &&
               is_array(w_post, at::kFloat, C) && is_array(scale, at::kFloat, C) && is_array(w_pre, at::kFloat, C);
    }
    const void* gate_ptr() const { return gate ? gate->const_data_ptr() : nullptr; }
};
const float* floats(const at::Tensor* t) { return static_cast<const float*>(t->const_data_ptr()); }
float* floats(at::Tensor& t) { return static_cast<float*>(t.mutable_data_ptr()); }

// (h, x, gate, w_post, scale, w_pre, eps, kind, want_stats) -> (y, u, stats)
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        NormOperands o;
        if (n != 9 || !PyFloat_CheckExact(args[6]) || !o.read(args)) return not_here();
        at::Tensor y = make({o.M, o.C}, *o.h, o.h->scalar_type()), u = make({o.M, o.C}, *o.h, o.h->scalar_type()), stats;
        const int want = PyObject_IsTrue(args[8]);
        if (want < 0) return nullptr;
        if (want) stats = make({o.M, 4}, *o.h, at::kFloat);
        const int st = f_norm(o.d, (int)PyLong_AsLong(args[7]), o.h->const_data_ptr(), o.C, o.x->const_data_ptr(), o.C, o.gate_ptr(),
                              o.gate_cols, (int32_t)o.gate_cols, floats(o.w_post), floats(o.scale), floats(o.w_pre),
                              (float)PyFloat_AS_DOUBLE(args[6]), o.M, (int32_t)o.C, y.mutable_data_ptr(), u.mutable_data_ptr(),
                              want ? floats(stats) : nullptr, stream());
        if (st) return failed("zs_norm_gate_residual", st);
        PyObject* r = PyTuple_New(3);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(y)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(u)));
        PyTuple_SET_ITEM(r, 2, want ? THPVariable_Wrap(std::move(stats)) : Py_NewRef(Py_None));
        return r;
    });
}

// (dy, du, h, x, gate, w_post, scale, w_pre, stats, kind) -> (dh, dx, dgate, dw_post, dscale, dw_pre)
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        NormOperands o;
        if (n != 10 || !o.read(args + 2)) return not_here();
        const at::Tensor* dy = args[0] == Py_None ? nullptr : plain(args[0]);
        const at::Tensor* du = args[1] == Py_None ? nullptr : plain(args[1]);
        const at::ScalarType type = o.h->scalar_type();
        if ((args[0] != Py_None && !is_matrix(dy, type, o.M, o.C)) || (args[1] != Py_None && !is_matrix(du, type, o.M, o.C)) ||
            !is_matrix(plain(args[8]), at::kFloat, o.M, 4))
            return not_here();
        at::Tensor out[6] = {make({o.M, o.C}, *o.h, type), make({o.M, o.C}, *o.h, type), at::Tensor(), make({o.C}, *o.h, at::kFloat),
                             make({o.C}, *o.h, at::kFloat), make({o.C}, *o.h, at::kFloat)};
        if (o.gate) out[2] = make({o.M, o.gate_cols}, *o.h, type);
        const size_t bytes = f_norm_bytes(o.M, (int32_t)o.C);
        at::Tensor ws;
        if (bytes) ws = make({(int64_t)bytes}, *o.h, at::kByte);
        const int st = f_norm_backward(
            o.d, (int)PyLong_AsLong(args[9]), dy ? dy->const_data_ptr() : nullptr, o.C, du ? du->const_data_ptr() : nullptr, o.C,
            o.h->const_data_ptr(), o.C, o.x->const_data_ptr(), o.C, o.gate_ptr(), o.gate_cols, (int32_t)o.gate_cols, floats(o.w_post),
            floats(o.scale), floats(o.w_pre), floats(plain(args[8])), o.M, (int32_t)o.C, out[0].mutable_data_ptr(),
            out[1].mutable_data_ptr(), o.gate ? out[2].mutable_data_ptr() : nullptr, floats(out[3]), floats(out[4]), floats(out[5]),
            bytes ? ws.mutable_data_ptr() : nullptr, bytes, stream());
        if (st) return failed("zs_norm_gate_residual_backward", st);
        PyObject* r = PyTuple_New(6);
        if (!r) return nullptr;
        for (int i = 0; i < 6; ++i)
            PyTuple_SET_ITEM(r, i, i == 2 && !o.gate ? Py_NewRef(Py_None) : THPVariable_Wrap(std::move(out[i])));
        return r;
    });
}

// Numbers as they are ordinarily given; false for others and for those out of range.
bool number(PyObject* o, int64_t lo, int64_t hi, int64_t& v) {
    if (!PyLong_CheckExact(o)) return false;
    int over = 0;
    v = PyLong_AsLongLongAndOverflow(o, &over);
    return !over && v >= lo && v <= hi;
}
bool number(PyObject* o, double& v) {
    if (!PyFloat_CheckExact(o)) return false;
    v = PyFloat_AS_DOUBLE(o);
    return true;
}
const int32_t* ints(const at::Tensor* t) { return t ? static_cast<const int32_t*>(t->const_data_ptr()) : nullptr; }
int32_t* ints(at::Tensor& t) { return static_cast<int32_t*>(t.mutable_data_ptr()); }
PyObject* pair(at::Tensor&& a, at::Tensor&& b) {
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(a)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(b)));
    return r;
}

// (dst, N) -> (row_ptr, perm, bad_dst_count)
PyObject* csr(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        int64_t N;
        if (n != 2 || !number(args[1], 0, INT32_MAX, N)) return not_here();
        const at::Tensor* dst = plain(args[0]);
        if (!dst || dst->dim() != 1 || !is_array(dst, at::kInt, dst->size(0))) return not_here();
        const int64_t E = dst->size(0);
        at::Tensor row_ptr = make({N + 1}, *dst, at::kInt), perm = make({E}, *dst, at::kInt), bad = make({1}, *dst, at::kInt), ws;
        const size_t bytes = f_csr_bytes(E, (int32_t)N);
        if (bytes) ws = make({(int64_t)bytes}, *dst, at::kByte);
        const int st = f_csr(E ? ints(dst) : nullptr, E, (int32_t)N, ints(row_ptr), E ? ints(perm) : nullptr, ints(bad),
                             bytes ? ws.mutable_data_ptr() : nullptr, bytes, stream());
        if (st) return failed("zs_build_csr", st);
        PyObject* r = PyTuple_New(3);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(row_ptr)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(perm)));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(bad)));
        return r;
    });
}

// (w, ids, scale) -> y
PyObject* embedding(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        double scale;
        if (n != 3 || !number(args[2], scale)) return not_here();
        const at::Tensor *w = plain(args[0]), *ids = plain(args[1]);
        if (!w || !ids || w->dim() != 2 || ids->dim() != 1 || (w->size(0) | w->size(1)) >> 31) return not_here();
        const int64_t M = ids->size(0), V = w->size(0), C = w->size(1);
        const int d = dtype_of(*w);
        if (d < 0 || !is_array(ids, at::kInt, M)) return not_here();
        at::Tensor y = make({M, C}, *w, w->scalar_type());
        const int st = f_embedding(d, w->const_data_ptr(), C, ints(ids), M, (int32_t)V, (int32_t)C, (float)scale, y.mutable_data_ptr(), C,
                                   stream());
        return st ? failed("zs_embedding", st) : THPVariable_Wrap(std::move(y));
    });
}

// (dy, row_ptr, perm, scale) -> dw
PyObject* embedding_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        double scale;
        if (n != 4 || !number(args[3], scale)) return not_here();
        const at::Tensor *dy = plain(args[0]), *row_ptr = plain(args[1]), *perm = plain(args[2]);
        if (!dy || !row_ptr || dy->dim() != 2 || dy->size(1) >> 31) return not_here();
        const int64_t M = dy->size(0), C = dy->size(1), V = row_ptr->numel() - 1;
        const int d = dtype_of(*dy);
        if (d < 0 || V < 0 || V >> 31 || !is_array(row_ptr, at::kInt, V + 1) || !is_array(perm, at::kInt, M)) return not_here();
        at::Tensor dw = make({V, C}, *dy, dy->scalar_type()), ws;
        const size_t bytes = f_embedding_bytes(d, M, (int32_t)V, (int32_t)C);
        if (bytes) ws = make({(int64_t)bytes}, *dy, at::kByte);
        const int st = f_embedding_backward(d, dy->const_data_ptr(), C, ints(row_ptr), ints(perm), M, (int32_t)V, (int32_t)C, (float)scale,
                                            dw.mutable_data_ptr(), bytes ? ws.mutable_data_ptr() : nullptr, bytes, stream());
        return st ? failed("zs_embedding_backward", st) : THPVariable_Wrap(std::move(dw));
    });
}

// (logits, k, bias, score, groups, top_groups, group_top, renormalise, scale) -> (ids, weights)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        int64_t k, score, groups, top_groups, group_top;
        double scale;
        if (n != 9 || !number(args[1], 1, 1 << 20, k) || !number(args[3], 0, 1, score) || !number(args[4], 1, 1 << 20, groups) ||
            !number(args[5], 1, 1 << 20, top_groups) || !number(args[6], 1, 2, group_top) || !number(args[8], scale))
            return not_here();
        const at::Tensor *z = plain(args[0]), *bias = args[2] == Py_None ? nullptr : plain(args[2]);
        if (!z || z->dim() != 2 || z->size(1) >> 20) return not_here();
        const int64_t M = z->size(0), E = z->size(1);
        const int d = dtype_of(*z), renormalise = PyObject_IsTrue(args[7]);
        if (renormalise < 0) return nullptr;
        if (d < 0 || k > E || (args[2] != Py_None && !is_array(bias, at::kFloat, E))) return not_here();
        at::Tensor ids = make({M, k}, *z, at::kInt), weights = make({M, k}, *z, at::kFloat);
        const int st = f_route(d, (int32_t)score, z->const_data_ptr(), E, bias ? floats(bias) : nullptr, M, (int32_t)E, (int32_t)k,
                               (int32_t)groups, (int32_t)top_groups, (int32_t)group_top, renormalise, (float)scale, ints(ids),
                               floats(weights), stream());
        return st ? failed("zs_route", st) : pair(std::move(ids), std::move(weights));
    });
}

// (dweights, logits, ids, score, renormalise, scale) -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        int64_t score;
        double scale;
        if (n != 6 || !number(args[3], 0, 1, score) || !number(args[5], scale)) return not_here();
        const at::Tensor *g = plain(args[0]), *z = plain(args[1]), *ids = plain(args[2]);
        if (!g || !z || !ids || z->dim() != 2 || ids->dim() != 2 || z->size(1) >> 20) return not_here();
        const int64_t M = z->size(0), E = z->size(1), k = ids->size(1);
        const int d = dtype_of(*z), renormalise = PyObject_IsTrue(args[4]);
        if (renormalise < 0) return nullptr;
        if (d < 0 || k < 1 || k > E || !is_matrix(ids, at::kInt, M, k) || !is_matrix(g, at::kFloat, M, k)) return not_here();
        at::Tensor dz = make({M, E}, *z, z->scalar_type());
        const int st = f_route_backward(d, (int32_t)score, floats(g), z->const_data_ptr(), E, ints(ids), M, (int32_t)E, (int32_t)k,
                                        renormalise, (float)scale, dz.mutable_data_ptr(), stream());
        return st ? failed("zs_route_backward", st) : THPVariable_Wrap(std::move(dz));
    });
}

// (x, row_ptr, perm, k) -> (xs, slot)
PyObject* dispatch(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        int64_t k;
        if (n != 4 || !number(args[3], 1, INT32_MAX, k)) return not_here();
        const at::Tensor *x = plain(args[0]), *row_ptr = plain(args[1]), *perm = plain(args[2]);
        if (!x || !row_ptr || x->dim() != 2 || (x->size(0) | x->size(1)) >> 31) return not_here();
        const int64_t M = x->size(0), C = x->size(1), G = row_ptr->numel() - 1, R = M * k;
        const int d = dtype_of(*x);
        if (d < 0 || G < 0 || G >> 31 || R >> 31 || !is_array(row_ptr, at::kInt, G + 1) || !is_array(perm, at::kInt, R)) return not_here();
        at::Tensor xs = make({R, C}, *x, x->scalar_type()), slot = make({M, k}, *x, at::kInt);
        const int st = f_dispatch(d, x->const_data_ptr(), C, ints(row_ptr), ints(perm), M, (int32_t)k, (int32_t)G, (int32_t)C,
                                  xs.mutable_data_ptr(), ints(slot), stream());
        return st ? failed("zs_dispatch", st) : pair(std::move(xs), std::move(slot));
    });
}

// (h, slot, weights) -> y
PyObject* combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) return not_here();
        const at::Tensor *h = plain(args[0]), *slot = plain(args[1]), *weights = args[2] == Py_None ? nullptr : plain(args[2]);
        if (!h || !slot || h->dim() != 2 || slot->dim() != 2 || slot->scalar_type() != at::kInt || slot->size(1) < 1 ||
            (h->size(0) | h->size(1) | slot->size(1)) >> 31)
            return not_here();
        const int64_t M = slot->size(0), k = slot->size(1), R = h->size(0), C = h->size(1);
        const int d = dtype_of(*h);
        if (d < 0 || (args[2] != Py_None && !is_matrix(weights, at::kFloat, M, k))) return not_here();
        at::Tensor y = make({M, C}, *h, h->scalar_type());
        const int st = f_combine(d, h->const_data_ptr(), C, ints(slot), weights ? floats(weights) : nullptr, M, (int32_t)k, R, (int32_t)C,
                                 y.mutable_data_ptr(), C, stream());
        return st ? failed("zs_combine", st) : THPVariable_Wrap(std::move(y));
    });
}

// (dy, h, slot, weights, row_ptr) -> (dh, dweights)
PyObject* combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) return not_here();
        const at::Tensor *dy = plain(args[0]), *h = plain(args[1]), *slot = plain(args[2]), *weights = plain(args[3]), *row_ptr = plain(args[4]);
        if (!dy || !h || !slot || !row_ptr || h->dim() != 2 || slot->dim() != 2 || (slot->size(0) | slot->size(1) | h->size(1)) >> 31)
            return not_here();
        const int64_t M = slot->size(0), k = slot->size(1), R = M * k, C = h->size(1), G = row_ptr->numel() - 1;
        const at::ScalarType type = h->scalar_type();
        const int d = dtype_of(*h);
        if (d < 0 || k < 1 || G < 0 || G >> 31 || !is_matrix(h, type, R, C) || !is_matrix(dy, type, M, C) || !is_matrix(slot, at::kInt, M, k) ||
            !is_matrix(weights, at::kFloat, M, k) || !is_array(row_ptr, at::kInt, G + 1))
            return not_here();
        at::Tensor dh = make({R, C}, *h, type), dweights = make({M, k}, *h, at::kFloat);
        const int st = f_combine_backward(d, dy->const_data_ptr(), C, h->const_data_ptr(), C, ints(slot), floats(weights), ints(row_ptr), M,
                                          (int32_t)k, (int32_t)G, (int32_t)C, dh.mutable_data_ptr(), floats(dweights), stream());
        return st ? failed("zs_combine_backward", st) : pair(std::move(dh), std::move(dweights));
    });
}

// (h, p, seed, call, step, residual) -> y
PyObject* dropout(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        double p;
        int64_t seed, call, step = 0;
        if (n != 6 || !number(args[1], p) || !number(args[2], 0, INT64_MAX, seed) || !number(args[3], 0, UINT32_MAX, call)) return not_here();
        const at::Tensor *h = plain(args[0]), *r = args[5] == Py_None ? nullptr : plain(args[5]), *count = nullptr;
        if (!number(args[4], INT64_MIN, INT64_MAX, step)) {
            count = plain(args[4]);
            if (!count || count->scalar_type() != at::kLong || count->numel() != 1) return not_here();
        }
        if (!h || h->dim() != 2 || h->size(1) < 1 || (h->size(0) | h->size(1)) >> 31) return not_here();
        const int64_t M = h->size(0), C = h->size(1);
        const int d = dtype_of(*h);
        if (d < 0 || (args[5] != Py_None && !is_matrix(r, h->scalar_type(), M, C))) return not_here();
        at::Tensor y = make({M, C}, *h, h->scalar_type());
        const int st = f_dropout(d, h->const_data_ptr(), C, r ? r->const_data_ptr() : nullptr, C, M, (int32_t)C, p, (uint64_t)seed,
                                 (uint32_t)call, step, count ? static_cast<const int64_t*>(count->const_data_ptr()) : nullptr,
                                 y.mutable_data_ptr(), C, stream());
        return st ? failed("zs_dropout", st) : THPVariable_Wrap(std::move(y));
    });
}

// ({function name: address}, check)
PyObject* bind(PyObject*, PyObject* args) {
    PyObject *table, *check;
    if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &table, &check)) return nullptr;
    auto get = [&](const char* name) -> void* {
        PyObject* v = PyDict_GetItemString(table, name);
        if (!v) PyErr_Format(PyExc_KeyError, "%s", name);
        return v ? PyLong_AsVoidPtr(v) : nullptr;
    };
    f_matmul = reinterpret_cast<decltype(f_matmul)>(get("zs_grouped_matmul_ws"));
    f_dx = reinterpret_cast<decltype(f_dx)>(get("zs_grouped_matmul_dx_ws"));
    f_matmul_bytes = reinterpret_cast<decltype(f_matmul_bytes)>(get("zs_grouped_matmul_workspace_bytes"));
    f_dw_bytes = reinterpret_cast<decltype(f_dw_bytes)>(get("zs_grouped_matmul_dw_workspace_bytes"));
    f_dw_copy = reinterpret_cast<decltype(f_dw_copy)>(get("zs_grouped_matmul_dw_copy_bytes"));
    f_dw = reinterpret_cast<decltype(f_dw)>(get("zs_grouped_matmul_dw"));
    f_norm = reinterpret_cast<decltype(f_norm)>(get("zs_norm_gate_residual"));
    f_norm_bytes = reinterpret_cast<decltype(f_norm_bytes)>(get("zs_norm_gate_residual_backward_workspace_bytes"));
    f_norm_backward = reinterpret_cast<decltype(f_norm_backward)>(get("zs_norm_gate_residual_backward"));
    f_csr_bytes = reinterpret_cast<decltype(f_csr_bytes)>(get("zs_build_csr_workspace_bytes"));
    f_csr = reinterpret_cast<decltype(f_csr)>(get("zs_build_csr"));
    f_embedding = reinterpret_cast<decltype(f_embedding)>(get("zs_embedding"));
    f_embedding_bytes = reinterpret_cast<decltype(f_embedding_bytes)>(get("zs_embedding_backward_workspace_bytes"));
    f_embedding_backward = reinterpret_cast<decltype(f_embedding_backward)>(get("zs_embedding_backward"));
    f_route = reinterpret_cast<decltype(f_route)>(get("zs_route"));
    f_route_backward = reinterpret_cast<decltype(f_route_backward)>(get("zs_route_backward"));
    f_dispatch = reinterpret_cast<decltype(f_dispatch)>(get("zs_dispatch"));
    f_combine = reinterpret_cast<decltype(f_combine)>(get("zs_combine"));
    f_combine_backward = reinterpret_cast<decltype(f_combine_backward)>(get("zs_combine_backward"));
    f_dropout = reinterpret_cast<decltype(f_dropout)>(get("zs_dropout"));
    if (PyErr_Occurred()) return nullptr;
    Py_XSETREF(on_error, Py_NewRef(check));
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F)); }

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"matmul", fast<matmul>(), METH_FASTCALL, nullptr},
    {"dw", fast<dw>(), METH_FASTCALL, nullptr},
    {"norm", fast<norm>(), METH_FASTCALL, nullptr},
    {"norm_backward", fast<norm_backward>(), METH_FASTCALL, nullptr},
    {"csr", fast<csr>(), METH_FASTCALL, nullptr},
    {"embedding", fast<embedding>(), METH_FASTCALL, nullptr},
    {"embedding_backward", fast<embedding_backward>(), METH_FASTCALL, nullptr},
    {"route", fast<route>(), METH_FASTCALL, nullptr},
    {"route_backward", fast<route_backward>(), METH_FASTCALL, nullptr},
    {"dispatch", fast<dispatch>(), METH_FASTCALL, nullptr},
    {"combine", fast<combine>(), METH_FASTCALL, nullptr},
    {"combine_backward", fast<combine_backward>(), METH_FASTCALL, nullptr},
    {"dropout", fast<dropout>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "zs_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_zs_torch() { return PyModule_Create(&module); }
