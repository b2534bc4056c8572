// bind.cpp -- the Python binding of the calls around the 8-bit layers of an MLP block (block_api.cpp): argument checks and
// marshalling from torch tensors to the C ABI.  These calls are short (the norm of one token takes 3 us on the GPU), and the
// same checks in Python take longer than the launch (7.4 us a call, 4.2 here).
//
// Each function takes its tensors by position, None for one that is not given, and the stream (None: the device's current
// one) last; it raises TypeError or ValueError for tensors that the call does not take, and returns the library's status.
#include <Python.h>

#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../include/rtq.h"

namespace {

// The library, from the path that the package loads it from.
struct Library {
    decltype(&rtq_rmsnorm_forward) rmsnorm_forward;
    decltype(&rtq_rmsnorm_backward) rmsnorm_backward;
    decltype(&rtq_fp8_glu) fp8_glu;
    decltype(&rtq_glu_fp8_backward) glu_fp8_backward;
    decltype(&rtq_grad_norm) grad_norm;
    decltype(&rtq_grad_clip) grad_clip;
} lib;

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& message) {
    PyErr_SetString(type, message.c_str());
    throw Raised{};
}

std::string text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

using Shape = std::initializer_list<int64_t>;

enum Kind { kFloat, kCode, kE4M3, kScale };
int type_code(Kind kind, at::ScalarType t) {
    switch (kind) {
        case kFloat: return t == at::kFloat ? RTQ_F32 : (t == at::kBFloat16 ? RTQ_BF16 : -1);
        case kCode: return t == at::kFloat8_e4m3fn ? RTQ_E4M3 : (t == at::kFloat8_e5m2 ? RTQ_E5M2 : -1);
        case kE4M3: return t == at::kFloat8_e4m3fn ? RTQ_E4M3 : -1;
        default: return t == at::kFloat ? RTQ_F32 : (t == at::ScalarType::Float8_e8m0fnu ? RTQ_E8M0 : -1);
    }
}

// A tensor argument, checked: its type code and address; of None, no address.
struct Operand {
    const at::Tensor* t = nullptr;
    void* ptr = nullptr;
    rtq_dtype type = RTQ_F32;
    explicit operator bool() const { return t != nullptr; }
};

const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor, not " + Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}

// The call's device, taken from its first tensor.
struct Call {
    const at::Tensor* like;

    // shape: what it has to be.  same: a type it has to share (-1: any of the kind).
    Operand operand(PyObject* o, const char* name, Kind kind, Shape shape, bool optional = false, int same = -1) const {
        const at::Tensor* t = tensor(o, name, optional);
        if (t == nullptr) return {};
        const int code = type_code(kind, t->scalar_type());
        if (code < 0 || (same >= 0 && code != same))
            raise(PyExc_TypeError, std::string(name) + ": unsupported dtype " + c10::toString(t->scalar_type()));
        const at::IntArrayRef want(shape.begin(), shape.size());
        if (t->sizes() != want) raise(PyExc_ValueError, std::string(name) + ": shape " + text(t->sizes()) + ", expected " + text(want));
        place(*t, name);
        return {t, t->data_ptr(), static_cast<rtq_dtype>(code)};
    }
    void place(const at::Tensor& t, const char* name) const {
        if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
        if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a GPU tensor");
        if (t.device() != like->device())
            raise(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + like->device().str());
    }
    // f(stream) on the tensors' device: on the given stream, or the device's current one.
    template <typename F>
    PyObject* run(PyObject* stream, F f) const {
        const c10::DeviceIndex index = like->device().index();
        void* handle;
        if (stream == Py_None) {
            handle = c10::hip::getCurrentHIPStream(index).stream();
        } else {
            const auto attribute = [&](const char* name) {
                PyObject* v = PyObject_GetAttrString(stream, name);
                if (v == nullptr) throw Raised{};
                const long long n = PyLong_AsLongLong(v);
                Py_DECREF(v);
                if (n == -1 && PyErr_Occurred()) throw Raised{};
                return n;
            };
            if (attribute("device_index") != index)
                raise(PyExc_ValueError, "stream is on another device than the tensors (" + like->device().str() + ")");
            handle = reinterpret_cast<void*>(attribute("cuda_stream"));
        }
        rtq_status status;
        if (c10::hip::current_device() == index) {
            status = f(handle);
        } else {
            const c10::DeviceGuard guard(like->device());
            status = f(handle);
        }
        return PyLong_FromLong(status);
    }
};

// The first tensor of a call: of two dimensions.
Operand rows_of(PyObject* o, const char* name, Kind kind) {
    const at::Tensor* t = tensor(o, name);
    const int code = type_code(kind, t->scalar_type());
    if (code < 0) raise(PyExc_TypeError, std::string(name) + ": unsupported dtype " + c10::toString(t->scalar_type()));
    if (t->dim() != 2) raise(PyExc_ValueError, std::string(name) + ": shape " + text(t->sizes()) + ", expected two dimensions");
    if (t->size(1) > INT32_MAX || (kind == kE4M3 && t->size(0) / 2 > INT32_MAX))   // the library's lengths
        raise(PyExc_ValueError, std::string(name) + ": shape " + text(t->sizes()) + " is too large");
    Call{t}.place(*t, name);
    return {t, t->data_ptr(), static_cast<rtq_dtype>(code)};
}

struct Workspace {
    void* ptr = nullptr;
    size_t bytes = 0;
    Workspace(const Call& call, PyObject* o) {
        const at::Tensor* t = tensor(o, "workspace", true);
        if (t == nullptr) return;
        call.place(*t, "workspace");
        ptr = t->data_ptr();
        bytes = t->nbytes();
    }
};

void together(const Operand& a, const Operand& b, const char* names) {
    if (static_cast<bool>(a) != static_cast<bool>(b)) raise(PyExc_ValueError, std::string(names) + " are given together or not at all");
}

int64_t groups(int64_t d) { return (d + 127) / 128; }

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
// An activation's code; one that the library does not know stays one.
rtq_act act_of(PyObject* o) {
    const int64_t v = integer(o);
    return static_cast<rtq_act>(v < 0 || v > INT32_MAX ? INT32_MAX : v);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

// x, gamma, eps, residual, h, codes, scale, y, stream
PyObject* rmsnorm_forward(PyObject* const* a) {
    const Operand x = rows_of(a[0], "x", kFloat);
    const Call call{x.t};
    const int64_t rows = x.t->size(0), d = x.t->size(1);
    const Operand gamma = call.operand(a[1], "gamma", kFloat, {d});
    const float eps = number(a[2]);
    const Operand residual = call.operand(a[3], "residual", kFloat, {rows, d}, true);
    const Operand h = call.operand(a[4], "h", kFloat, {rows, d}, true, residual ? residual.type : -1);
    together(residual, h, "residual and h");
    const Operand codes = call.operand(a[5], "codes", kE4M3, {rows, d}, true);
    const Operand scale = call.operand(a[6], "scale", kScale, {groups(d), rows}, true);
    const Operand y = call.operand(a[7], "y", kFloat, {rows, d}, true, x.type);
    if (static_cast<bool>(codes) != static_cast<bool>(scale) || (!y && !codes)) raise(PyExc_ValueError, "give y, or codes and scale, or all of them");
    return call.run(a[8], [&](void* stream) {
        return lib.rmsnorm_forward(x.ptr, x.type, residual.ptr, residual ? residual.type : x.type, rows, static_cast<int32_t>(d), gamma.ptr,
                                   gamma.type, eps, h.ptr, y.ptr, codes.ptr, scale.ptr, scale.type, stream);
    });
}

// dn, h, gamma, eps, dh, dgamma, dresidual, accumulate, workspace, stream
PyObject* rmsnorm_backward(PyObject* const* a) {
    const Operand dn = rows_of(a[0], "dn", kFloat);
    const Call call{dn.t};
    const int64_t rows = dn.t->size(0), d = dn.t->size(1);
    const Operand h = call.operand(a[1], "h", kFloat, {rows, d});
    const Operand gamma = call.operand(a[2], "gamma", kFloat, {d});
    const float eps = number(a[3]);
    const Operand dh = call.operand(a[4], "dh", kFloat, {rows, d}, false, h.type);
    const Operand dgamma = call.operand(a[5], "dgamma", kFloat, {d}, true);
    const Operand dresidual = call.operand(a[6], "dresidual", kFloat, {rows, d}, true, h.type);
    const int accumulate = truth(a[7]) ? 1 : 0;
    const Workspace ws(call, a[8]);
    return call.run(a[9], [&](void* stream) {
        return lib.rmsnorm_backward(dn.ptr, dn.type, h.ptr, h.type, dresidual.ptr, rows, static_cast<int32_t>(d), gamma.ptr, gamma.type, eps,
                                    dh.ptr, dgamma.ptr, dgamma.type, accumulate, ws.ptr, ws.bytes, stream);
    });
}

// x_codes, x_scale, w_codes, w_scale, act, y, y_codes, y_scale, h_codes, h_scale, workspace, stream
PyObject* fp8_glu(PyObject* const* a) {
    const Operand x = rows_of(a[0], "x_codes", kE4M3);
    const Call call{x.t};
    const int64_t T = x.t->size(0), K = x.t->size(1);
    const Operand w = rows_of(a[2], "w_codes", kE4M3);
    const int64_t rows = w.t->size(0), N = rows / 2;
    call.operand(a[2], "w_codes", kE4M3, {rows, K});
    if (rows % 256 != 0)
        raise(PyExc_ValueError, "w_codes: " + std::to_string(rows) + " rows, expected two projections of a multiple of 128 each");
    const Operand w_scale = call.operand(a[3], "w_scale", kScale, {groups(rows), groups(K)});
    const Operand x_scale = call.operand(a[1], "x_scale", kScale, {groups(K), T}, false, w_scale.type);
    const rtq_act act = act_of(a[4]);
    const Operand y = call.operand(a[5], "y", kFloat, {T, N}, true);
    const Operand y_codes = call.operand(a[6], "y_codes", kE4M3, {T, N}, true);
    const Operand y_scale = call.operand(a[7], "y_scale", kScale, {groups(N), T}, true, w_scale.type);
    if (static_cast<bool>(y_codes) != static_cast<bool>(y_scale) || static_cast<bool>(y) == static_cast<bool>(y_codes))
        raise(PyExc_ValueError, "give either y, or y_codes and y_scale");
    const Operand h_codes = call.operand(a[8], "h_codes", kE4M3, {T, rows}, true);
    const Operand h_scale = call.operand(a[9], "h_scale", kScale, {groups(rows), T}, true, w_scale.type);
    together(h_codes, h_scale, "h_codes and h_scale");
    const Workspace ws(call, a[10]);
    return call.run(a[11], [&](void* stream) {
        return lib.fp8_glu(x.ptr, x_scale.ptr, T, w.ptr, w_scale.ptr, w_scale.type, static_cast<int32_t>(N), static_cast<int32_t>(K),
                           act, h_codes.ptr, h_scale.ptr, y.ptr, y.type, y_codes.ptr, y_scale.ptr, ws.ptr, ws.bytes, stream);
    });
}

// dy, h_codes, h_scale, act, dh, dh_codes, dh_scale, stream
PyObject* glu_fp8_backward(PyObject* const* a) {
    const Operand dy = rows_of(a[0], "dy", kFloat);
    const Call call{dy.t};
    const int64_t T = dy.t->size(0), N = dy.t->size(1);
    const Operand h = call.operand(a[1], "h_codes", kE4M3, {T, 2 * N});
    const Operand h_scale = call.operand(a[2], "h_scale", kScale, {groups(2 * N), T});
    const rtq_act act = act_of(a[3]);
    const Operand dh = call.operand(a[4], "dh", kFloat, {T, 2 * N}, true, dy.type);
    const Operand codes = call.operand(a[5], "dh_codes", kCode, {T, 2 * N}, true);
    const Operand scale = call.operand(a[6], "dh_scale", kScale, {groups(2 * N), T}, true, h_scale.type);
    if (static_cast<bool>(codes) != static_cast<bool>(scale) || (!dh && !codes))
        raise(PyExc_ValueError, "give dh, or dh_codes and dh_scale, or all of them");
    return call.run(a[7], [&](void* stream) {
        return lib.glu_fp8_backward(dy.ptr, dy.type, h.ptr, h_scale.ptr, h_scale.type, T, static_cast<int32_t>(N), act,
                                    dh.ptr, codes.ptr, codes ? codes.type : RTQ_E4M3, scale.ptr, stream);
    });
}

Operand norm_of(const Call& call, PyObject* o) {
    const at::Tensor* t = tensor(o, "norm");
    if (t->scalar_type() != at::kFloat) raise(PyExc_TypeError, std::string("norm: unsupported dtype ") + c10::toString(t->scalar_type()));
    if (t->dim() > 1 || t->numel() != 1) raise(PyExc_ValueError, "norm: shape " + text(t->sizes()) + ", expected (1,)");
    call.place(*t, "norm");
    return {t, t->data_ptr(), RTQ_F32};
}

// A list's tensors as they were when it was made: a tensor whose memory has been replaced since is refused.
struct List {
    const at::Tensor* first;
    const rtq_tensor* tensors;
    int32_t count;
    List(PyObject* tuple, PyObject* array)
        : tensors(reinterpret_cast<const rtq_tensor*>(integer(array))), count(static_cast<int32_t>(PyTuple_Size(tuple))) {
        if (count <= 0) throw Raised{};
        first = tensor(PyTuple_GET_ITEM(tuple, 0), "tensors");
        for (int32_t i = 0; i < count; ++i) check(PyTuple_GET_ITEM(tuple, i), tensors[i].data, tensors[i].n);
    }
    void outs(PyObject* tuple, void* const* at) const {
        for (int32_t i = 0; i < count; ++i) check(PyTuple_GET_ITEM(tuple, i), at[i], tensors[i].n);
    }
    static void check(PyObject* o, const void* data, int64_t n) {
        const at::Tensor* t = tensor(o, "tensors");
        if (t->data_ptr() != data || t->numel() != n) raise(PyExc_ValueError, "a tensor's memory has been replaced since the list was made");
    }
};

// tuple of tensors, address of their rtq_tensor array, norm, workspace, stream
PyObject* grad_norm(PyObject* const* a) {
    const List list(a[0], a[1]);
    const Call call{list.first};
    const Operand norm = norm_of(call, a[2]);
    const Workspace ws(call, a[3]);
    return call.run(a[4], [&](void* stream) { return lib.grad_norm(list.tensors, list.count, static_cast<float*>(norm.ptr), ws.ptr, ws.bytes, stream); });
}

// tuple of tensors, address of their rtq_tensor array, tuple of outs, address of their addresses, norm, most, stream
PyObject* grad_clip(PyObject* const* a) {
    const List list(a[0], a[1]);
    const Call call{list.first};
    const auto* outs = reinterpret_cast<void* const*>(integer(a[3]));
    if (a[2] != a[0]) list.outs(a[2], outs);
    const Operand norm = norm_of(call, a[4]);
    const float most = number(a[5]);
    return call.run(a[6], [&](void* stream) { return lib.grad_clip(list.tensors, outs, list.count, static_cast<const float*>(norm.ptr), most, stream); });
}

// No C++ exception goes into the interpreter.
template <PyObject* (*f)(PyObject* const*), Py_ssize_t kCount>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kCount) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", kCount, n);
        return nullptr;
    }
    if (lib.rmsnorm_forward == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, "the library has not been loaded");
        return nullptr;
    }
    try {
        return f(args);
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
        return nullptr;
    }
}

template <typename F>
bool find(void* handle, const char* name, F* f) {
    *f = reinterpret_cast<F>(dlsym(handle, name));
    if (*f == nullptr) PyErr_Format(PyExc_RuntimeError, "%s is missing in the library", name);
    return *f != nullptr;
}

// load(path): the library that the calls go to.
PyObject* load(PyObject*, PyObject* path) {
    const char* p = PyUnicode_AsUTF8(path);
    if (p == nullptr) return nullptr;
    void* handle = dlopen(p, RTLD_NOW | RTLD_LOCAL);
    if (handle == nullptr) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    if (!find(handle, "rtq_rmsnorm_backward", &lib.rmsnorm_backward) || !find(handle, "rtq_fp8_glu", &lib.fp8_glu) ||
        !find(handle, "rtq_glu_fp8_backward", &lib.glu_fp8_backward) || !find(handle, "rtq_grad_norm", &lib.grad_norm) ||
        !find(handle, "rtq_grad_clip", &lib.grad_clip) || !find(handle, "rtq_rmsnorm_forward", &lib.rmsnorm_forward))
        return nullptr;
    Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject* const*), Py_ssize_t kCount>
PyMethodDef entry(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(method<f, kCount>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"load", load, METH_O, nullptr},
    entry<rmsnorm_forward, 9>("rmsnorm_forward"),
    entry<rmsnorm_backward, 10>("rmsnorm_backward"),
    entry<fp8_glu, 12>("fp8_glu"),
    entry<glu_fp8_backward, 8>("glu_fp8_backward"),
    entry<grad_norm, 5>("grad_norm"),
    entry<grad_clip, 7>("grad_clip"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
