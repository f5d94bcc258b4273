// binding.h -- what the compiled front ends share: arguments' checks, marshalling of torch tensors, and the
// module's entries. Each front end includes it once, in its one source.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstring>
#include <string>

#include "mccb.h"

namespace {

using at::Tensor;
using Shape = at::IntArrayRef;

PyObject *error_class = nullptr;  // MccbError(status, where)

// A status that is not MCCB_OK, on its way to Python.
struct Status {
    int code;
    const char *where;
};
void ok(int code, const char *where) {
    if (code != MCCB_OK) throw Status{code, where};
}

// -- arguments ------------------------------------------------------------------------------------
Tensor tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) TORCH_CHECK_TYPE(false, name, " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}
Tensor maybe(PyObject *o, const char *name) { return o == Py_None ? Tensor() : tensor(o, name); }

std::string text(Shape s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

void check(const char *name, const Tensor &t, Shape shape, at::ScalarType type, at::Device device,
           bool contiguous) {
    TORCH_CHECK_VALUE(t.device() == device, name, " must live on ", device.str(), " (a HIP device)");
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", text(t.sizes()), ", expected ", text(shape));
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " has dtype ", toString(t.scalar_type()),
                      ", expected ", toString(type));
    if (contiguous) TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}
void check_if(const char *name, const Tensor &t, Shape shape, at::ScalarType type, at::Device device,
              bool contiguous = true) {
    if (t.defined()) check(name, t, shape, type, device, contiguous);
}

// The tensor that sets a call's type and device.
int32_t kind_of(const char *name, const Tensor &t, int64_t dims, const char *layout) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must live on a HIP device");
    TORCH_CHECK_VALUE(t.dim() == dims, name, " must be ", layout);
    if (t.scalar_type() == at::kBFloat16) return MCCB_BF16;
    TORCH_CHECK_VALUE(t.scalar_type() == at::kHalf, "dtype ", toString(t.scalar_type()),
                      " not supported (bfloat16, float16)");
    return MCCB_FP16;
}

void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
void strides3(const Tensor &t, int64_t (&s)[3], bool token) {
    if (!t.defined()) return;
    const auto v = t.strides();
    if (token) s[0] = 0, s[1] = v[0], s[2] = v[1];
    else s[0] = v[0], s[1] = v[1], s[2] = v[2];
}
// Strides along S, B, G, N of B or C, whose group axis may be left out.
void strides4(const Tensor &t, int64_t (&s)[4], bool token, bool grouped) {
    const auto v = t.strides();
    size_t i = 0;
    s[0] = token ? 0 : v[i++];
    s[1] = v[i++];
    s[2] = grouped ? v[i++] : 0;
    s[3] = v[i];
}

void *stream_of(const Tensor &t) { return (void *)c10::hip::getCurrentHIPStream(t.device().index()).stream(); }

Tensor make(Shape shape, const Tensor &like) { return at::empty(shape, like.options()); }
Tensor make(Shape shape, const Tensor &like, at::ScalarType type) {
    return at::empty(shape, like.options().dtype(type));
}
Tensor bytes(uint64_t n, const Tensor &like) {
    return n ? make({(int64_t)n}, like, at::kByte) : Tensor();
}

// Tensors of the caller's that a call wrote: their version moves on, as an in-place operation's does.
void wrote(std::initializer_list<Tensor> ts) {
    for (const Tensor &t : ts)
        if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

PyObject *out(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject *tuple(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor &t : ts) PyTuple_SET_ITEM(r, i++, out(t));
    return r;
}

// A [...,C] tensor as R evenly spaced, contiguous rows.
void rows_of(const char *name, const Tensor &t, int64_t &R, int64_t &ld) {
    const auto size = t.sizes(), stride = t.strides();
    const int64_t last = t.dim() - 1, C = size[last];
    TORCH_CHECK_VALUE(C <= 1 || stride[last] == 1, name, "'s last dimension must be contiguous");
    R = 1, ld = -1;
    for (int64_t i = last - 1; i >= 0; --i) {
        if (size[i] != 1) {
            if (ld < 0) ld = stride[i];
            else TORCH_CHECK_VALUE(size[i] == 0 || R == 0 || stride[i] == ld * R, name,
                                   "'s rows are not evenly spaced: make it contiguous");
        }
        R *= size[i];
    }
    if (ld < 0) ld = C;
}

// -- the module's entries --------------------------------------------------------------------------
// Every entry checks the argument count and turns what is thrown into a Python exception.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N || !error_class) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, N);
        return nullptr;
    }
    try {
        PyObject *r = F(v);
        if (PyErr_Occurred()) {
            Py_XDECREF(r);
            return nullptr;
        }
        return r;
    } catch (const Status &s) {
        PyObject *e = PyObject_CallFunction(error_class, "is", s.code, s.where);
        if (e) {
            PyErr_SetObject(error_class, e);
            Py_DECREF(e);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(error class, addresses): `lib` is a struct of pointers to functions, in the addresses' order.
template <typename Library>
PyObject *bind_to(Library &lib, PyObject *args) {
    constexpr Py_ssize_t kFunctions = sizeof(Library) / sizeof(void *);
    PyObject *cls, *addresses;
    if (!PyArg_ParseTuple(args, "OO!", &cls, &PyTuple_Type, &addresses)) return nullptr;
    if (PyTuple_GET_SIZE(addresses) != kFunctions) {
        PyErr_SetString(PyExc_ValueError, "wrong number of functions");
        return nullptr;
    }
    void *table[kFunctions];
    for (Py_ssize_t i = 0; i < kFunctions; ++i) {
        table[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
        if (!table[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function has no address");
            return nullptr;
        }
    }
    static_assert(sizeof(table) == sizeof(lib), "a table of function pointers");
    std::memcpy(&lib, table, sizeof(lib));
    Py_INCREF(cls);
    Py_XSETREF(error_class, cls);
    Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void *)&entry<name, n>, METH_FASTCALL, nullptr}

}  // namespace
