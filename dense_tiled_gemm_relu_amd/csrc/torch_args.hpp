// What the tensor front ends share: arguments, results and errors.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/util/StringUtil.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "gemm_relu.h"

namespace {

PyObject* status_error = nullptr;          // called with a status code, gives the exception to raise

// ---- arguments
template <class... A> [[noreturn]] void refuse(PyObject* type, const A&... words)
{
    PyErr_SetString(type, std::string(c10::str(words...)).c_str());
    throw python_error();
}
void expect_args(Py_ssize_t have, Py_ssize_t want)
{
    if (have != want) refuse(PyExc_TypeError, want, " arguments expected, not ", have);
}
const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, " must be a tensor, not ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
void* pointer(PyObject* o)
{
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw python_error();
    return p;
}
bool truth(PyObject* o)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw python_error();
    return t;
}

// the C-ABI's code of a type, or -1
int code_of(at::ScalarType t)
{
    return t == at::kHalf ? GEMM_RELU_F16 : t == at::kBFloat16 ? GEMM_RELU_BF16 : t == at::kFloat ? GEMM_RELU_F32 : -1;
}
const char* name_of(at::ScalarType t) { return c10::toString(t); }

// an activation tensor: rows of its last dimension
struct Rows {
    int64_t rows, cols, ld;      // elements from row to row
};
Rows rows_of(const at::Tensor& t, const char* name)
{
    const auto shape = t.sizes();
    if (shape.empty()) refuse(PyExc_ValueError, name, " must have at least one dimension");
    const int64_t cols = shape.back();
    if (t.is_contiguous()) {
        int64_t rows = 1;
        for (size_t k = 0; k + 1 < shape.size(); ++k) rows *= shape[k];
        return {rows, cols, cols};
    }
    if (shape.size() == 2 && t.stride(1) == 1 && t.stride(0) >= cols) return {shape[0], cols, t.stride(0)};
    refuse(PyExc_ValueError, name, " must be contiguous, or 2-D with contiguous rows");
}
Rows matrix_of(const at::Tensor& t, const char* name)
{
    if (t.dim() != 2) refuse(PyExc_ValueError, name, " must be 2-D");
    return rows_of(t, name);
}
void expect_vector(const at::Tensor& t, const char* name, int64_t n, at::ScalarType a, at::ScalarType b)
{
    const at::ScalarType s = t.scalar_type();
    if (s != a && s != b) {
        if (a == b) refuse(PyExc_TypeError, name, " must be ", name_of(a), ", not ", name_of(s));
        refuse(PyExc_TypeError, name, " must be ", name_of(a), " or ", name_of(b), ", not ", name_of(s));
    }
    if (t.numel() != n || !t.is_contiguous())
        refuse(PyExc_ValueError, name, " must be contiguous with ", n, " elements");
}
void expect_one_gpu(std::initializer_list<const at::Tensor*> all)
{
    const at::Tensor& first = **all.begin();
    for (const at::Tensor* t : all)
        if (t && (!t->is_cuda() || t->get_device() != first.get_device()))
            refuse(PyExc_ValueError, "all tensors must be on the same GPU");
}
// Results carry no autograd graph.  A caller who counts on one is told so: a result
// that needs no gradient would stop training without a word.  (Where the caller has
// switched gradients off, as torch.autograd.Function does, nothing is lost.)
void warn_of_lost_gradients(const char* name, std::initializer_list<const at::Tensor*> all)
{
    const bool recording = at::GradMode::is_enabled();
    for (const at::Tensor* t : all)
        if (t && ((recording && t->requires_grad()) || t->_fw_grad(/*level=*/0).defined())) {
            const std::string text = c10::str(name, ": an input requires a gradient, but the result carries no autograd graph; "
                                              "take the gradients from the *_backward functions, or call under torch.no_grad()");
            if (PyErr_WarnEx(PyExc_UserWarning, text.c_str(), 2) != 0) throw python_error();
            return;
        }
}
int float_code(const at::Tensor& x)
{
    const int c = code_of(x.scalar_type());
    if (c < 0) refuse(PyExc_TypeError, "x must be float16, bfloat16 or float32, not ", name_of(x.scalar_type()));
    return c;
}

// ---- results
at::Tensor make(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type)
{
    return at::empty(shape, at::TensorOptions().device(like.device()).dtype(type));
}
at::Tensor workspace(const at::Tensor& like, int64_t bytes) { return make(like, {bytes}, at::kByte); }
// like's shape with its last dimension dropped, or replaced by n
at::DimVector leading(const at::Tensor& like) { return at::DimVector(like.sizes().slice(0, size_t(like.dim() - 1))); }
at::DimVector with_last(const at::Tensor& like, int64_t n)
{
    at::DimVector shape = leading(like);
    shape.push_back(n);
    return shape;
}
void check(int status)
{
    if (status == GEMM_RELU_OK) return;
    PyObject* e = PyObject_CallFunction(status_error, "i", status);
    if (e) {
        PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
        Py_DECREF(e);
    }
    throw python_error();
}
PyObject* give(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* give(std::initializer_list<at::Tensor> all)
{
    PyObject* out = PyTuple_New(Py_ssize_t(all.size()));
    if (!out) throw python_error();
    Py_ssize_t k = 0;
    for (const at::Tensor& t : all) PyTuple_SET_ITEM(out, k++, THPVariable_Wrap(t));
    return out;
}
float* floats(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }

// Python's method table holds every calling convention as one pointer type
template <class F> constexpr PyCFunction method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

}  // namespace
