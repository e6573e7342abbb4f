// torch_args.h -- what the torch sides of the operators share (paged_torch.cpp,
// rows_torch.cpp): arguments as tensors and numbers, refusals as Python exceptions,
// the library's errors as ember.EmberError.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <string>

#include "ember.h"

namespace {

using at::Tensor;

decltype(&ember_last_error) f_error = nullptr;
PyObject* ember_error = nullptr;   // ember.EmberError

struct Bad {   // a Python exception to raise
    PyObject* type;
    std::string text;
};
[[noreturn]] void bad(const std::string& text) { throw Bad{PyExc_ValueError, text}; }

std::string describe(const Tensor& t) {
    std::string s = c10::toString(t.scalar_type());
    s += " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "] on " + t.device().str();
}

// A gradient would be lost without a word.  (The modes are thread-local and so asked
// for last: nearly no tensor here has either.)
void no_gradient(const Tensor& t, const char* what) {
    if (t.requires_grad() && c10::GradMode::is_enabled())
        bad(std::string(what) + " requires a gradient, which the operators here do not have (torch.no_grad() to go without)");
    if (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
        bad(std::string(what) + " has a forward-mode tangent, which the operators here do not carry on");
}
const Tensor& any_tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Bad{PyExc_TypeError, std::string(what) + " must be a tensor"};
    return THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* what) {
    const Tensor& t = any_tensor(o, what);
    no_gradient(t, what);
    return t;
}
bool given(PyObject* o) { return o != Py_None; }

// (c.device: the device that a call's tensors belong to)
template <class C>
void on_device(const C& c, const Tensor& t, const char* what) {
    if (!t.is_cuda() || t.device().index() != c.device)
        bad(std::string(what) + " must be on cuda:" + std::to_string(c.device) + ", not " + t.device().str());
}

// Contiguous, of one type and shape.
template <class C>
void* flat(const C& c, const Tensor& t, const char* what, at::ScalarType dtype, at::IntArrayRef shape) {
    on_device(c, t, what);
    if (t.scalar_type() != dtype || t.sizes() != shape || !t.is_contiguous()) {
        std::string s;
        for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
        bad(std::string(what) + " must be contiguous " + c10::toString(dtype) + " [" + s + "], not " + describe(t));
    }
    return t.data_ptr();
}
template <class C>
int32_t* ints(const C& c, PyObject* o, const char* what, int64_t n) {
    return static_cast<int32_t*>(flat(c, any_tensor(o, what), what, at::kInt, {n}));
}

template <class C>
Tensor make(const C& c, at::IntArrayRef shape, at::ScalarType dtype) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, c.device));
}

int32_t number(PyObject* o, const char* what) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v < INT_MIN || v > INT_MAX) bad(std::string(what) + " is beyond 32 bits");
    return (int32_t)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
int32_t count(int64_t n, const char* what) {
    if (n > INT_MAX) bad(std::string(what) + " has too many rows");
    return (int32_t)n;
}

void check(ember_status st, const char* where) {
    if (st == EMBER_OK) return;
    if (PyObject* e = PyObject_CallFunction(ember_error, "iss", (int)st, where, f_error())) {
        PyErr_SetObject(ember_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// A tensor of the caller's that a kernel writes: autograd notices if an earlier
// operation saved it.
void written(const Tensor& t) {
    if (t.defined() && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Runs f; nothing it throws leaves this module but as a Python exception.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    HANDLE_TH_ERRORS
    try {
        if (n != want) throw Bad{PyExc_TypeError, "wrong number of arguments"};
        return f();
    } catch (const Bad& b) {
        PyErr_SetString(b.type, b.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}

}  // namespace
