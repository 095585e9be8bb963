// Tensor front end of the feed-forward operators, as a CPython module
// (dense_tiled_gemm_relu_amd._ffn): argument checks, allocation of the results
// and the workspaces, and the call into the C-ABI of include/gemm_relu_ffn.h.
// It is C++ because a short kernel's call costs the host more than the device:
// one launch takes 2.9 us here, and the same checks and allocations took
// another 4 to 14 us a call in Python.
//
// The functions take their arguments by position, and last the raw stream of the
// current device that the call runs on; ffn.py holds the user's signatures.  The
// C functions' addresses come from the library that the package has loaded
// (bind), so there is one copy of it in the process.
#include "gemm_relu_ffn.h"
#include "torch_args.hpp"

namespace {

struct Api {
    decltype(&gemm_relu_layer_norm) layer_norm;
    decltype(&gemm_relu_layer_norm_backward_workspace) layer_norm_backward_workspace;
    decltype(&gemm_relu_layer_norm_backward) layer_norm_backward;
    decltype(&gemm_relu_gated) gated;
    decltype(&gemm_relu_gated_backward_workspace) gated_backward_workspace;
    decltype(&gemm_relu_gated_backward) gated_backward;
    decltype(&gemm_relu_quantize_rows) quantize_rows;
    decltype(&gemm_relu_i8) i8;
} api;

// ---- the operators
// x, weight, bias or None, eps, stats, stream
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 6);
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    const at::Tensor* b = a[2] == Py_None ? nullptr : &tensor(a[2], "bias");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    const bool stats = truth(a[4]);
    const int code = float_code(x);
    const Rows r = rows_of(x, "x");
    expect_vector(w, "weight", r.cols, x.scalar_type(), at::kFloat);
    if (b) expect_vector(*b, "bias", r.cols, w.scalar_type(), w.scalar_type());
    warn_of_lost_gradients("layer_norm", {&x, &w, b});
    expect_one_gpu({&x, &w, b});
    at::Tensor y = make(x, x.sizes(), x.scalar_type()), mean, rstd;
    if (stats) {
        mean = make(x, leading(x), at::kFloat);
        rstd = make(x, leading(x), at::kFloat);
    }
    check(api.layer_norm(x.data_ptr(), r.ld, w.data_ptr(), b ? b->data_ptr() : nullptr, y.data_ptr(),
                         stats ? floats(mean) : nullptr, stats ? floats(rstd) : nullptr, r.rows, r.cols, code,
                         code_of(w.scalar_type()), float(eps), pointer(a[5])));
    return stats ? give({y, mean, rstd}) : give(std::move(y));
    END_HANDLE_TH_ERRORS
}

// dy, x, weight, mean, rstd, stream
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 6);
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &w = tensor(a[2], "weight"),
                     &mean = tensor(a[3], "mean"), &rstd = tensor(a[4], "rstd");
    const int code = float_code(x);
    if (dy.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, "dy must have x's type");
    if (dy.sizes() != x.sizes()) refuse(PyExc_ValueError, "dy and x must have the same shape");
    const Rows r = rows_of(x, "x");
    const int64_t dy_ld = rows_of(dy, "dy").ld;
    expect_vector(w, "weight", r.cols, x.scalar_type(), at::kFloat);
    expect_vector(mean, "mean", r.rows, at::kFloat, at::kFloat);
    expect_vector(rstd, "rstd", r.rows, at::kFloat, at::kFloat);
    warn_of_lost_gradients("layer_norm_backward", {&x, &dy, &w, &mean, &rstd});
    expect_one_gpu({&x, &dy, &w, &mean, &rstd});
    at::Tensor dx = make(x, x.sizes(), x.scalar_type()), dw = make(w, w.sizes(), w.scalar_type()),
               db = make(w, w.sizes(), w.scalar_type());
    const int64_t bytes = api.layer_norm_backward_workspace(r.rows, r.cols);
    const at::Tensor ws = workspace(x, bytes < 0 ? 0 : bytes);
    check(api.layer_norm_backward(dy.data_ptr(), dy_ld, x.data_ptr(), r.ld, w.data_ptr(), floats(mean), floats(rstd),
                                  dx.data_ptr(), dw.data_ptr(), db.data_ptr(), r.rows, r.cols, code,
                                  code_of(w.scalar_type()), ws.data_ptr(), uint64_t(ws.numel()), pointer(a[5])));
    return give({dx, dw, db});
    END_HANDLE_TH_ERRORS
}

struct Gated {
    Rows x, w;
    int64_t hidden;
    int code;
};
Gated gated_args(const at::Tensor& x, const at::Tensor& w)
{
    Gated g;
    g.code = code_of(x.scalar_type());
    if (g.code < 0 || g.code == GEMM_RELU_F32 || w.scalar_type() != x.scalar_type())
        refuse(PyExc_TypeError, "x and weight must share dtype float16 or bfloat16");
    g.x = rows_of(x, "x");
    g.w = matrix_of(w, "weight");
    if (g.w.cols != g.x.cols || g.w.rows % 2)
        refuse(PyExc_ValueError, "weight must be (2 * hidden, ", g.x.cols, "), gate rows first");
    g.hidden = g.w.rows / 2;
    return g;
}
int activation_code(PyObject* o)
{
    const long c = PyLong_AsLong(o);
    if (c == -1 && PyErr_Occurred()) throw python_error();
    return int(c);
}

// x, weight, act (code), save, stream
PyObject* matmul_gated(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 5);
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    const int act = activation_code(a[2]);
    const bool save = truth(a[3]);
    const Gated g = gated_args(x, w);
    warn_of_lost_gradients("matmul_gated", {&x, &w});
    expect_one_gpu({&x, &w});
    at::Tensor h = make(x, with_last(x, g.hidden), x.scalar_type()), gu;
    if (save) gu = make(x, with_last(x, 2 * g.hidden), at::kFloat);
    check(api.gated(x.data_ptr(), g.x.ld, w.data_ptr(), g.w.ld, h.data_ptr(), save ? floats(gu) : nullptr, g.x.rows,
                    g.hidden, g.x.cols, g.code, act, pointer(a[4])));
    return save ? give({h, gu}) : give(std::move(h));
    END_HANDLE_TH_ERRORS
}

// dh, gu, x, weight, act (code), stream
PyObject* matmul_gated_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 6);
    const at::Tensor &dh = tensor(a[0], "dh"), &gu = tensor(a[1], "gu"), &x = tensor(a[2], "x"), &w = tensor(a[3], "weight");
    const int act = activation_code(a[4]);
    const Gated g = gated_args(x, w);
    if (dh.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, "dh must have x's type");
    if (dh.sizes() != at::IntArrayRef(with_last(x, g.hidden)))
        refuse(PyExc_ValueError, "dh must have matmul_gated's shape: x's, with ", g.hidden, " for the last dimension");
    const int64_t dh_ld = rows_of(dh, "dh").ld;
    expect_vector(gu, "gu", g.x.rows * 2 * g.hidden, at::kFloat, at::kFloat);
    warn_of_lost_gradients("matmul_gated_backward", {&x, &w, &dh, &gu});
    expect_one_gpu({&x, &w, &dh, &gu});
    at::Tensor dx = make(x, x.sizes(), x.scalar_type()), dw = make(w, w.sizes(), w.scalar_type());
    const int64_t bytes = api.gated_backward_workspace(g.x.rows, g.hidden, g.x.cols);
    const at::Tensor ws = workspace(x, bytes < 0 ? 0 : bytes);
    check(api.gated_backward(dh.data_ptr(), dh_ld, floats(gu), x.data_ptr(), g.x.ld, w.data_ptr(), g.w.ld, dx.data_ptr(),
                             dw.data_ptr(), g.x.rows, g.hidden, g.x.cols, g.code, act, ws.data_ptr(),
                             uint64_t(ws.numel()), pointer(a[5])));
    return give({dx, dw});
    END_HANDLE_TH_ERRORS
}

// x, stream
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 2);
    const at::Tensor& x = tensor(a[0], "x");
    const int code = float_code(x);
    const Rows r = rows_of(x, "x");
    warn_of_lost_gradients("quantize_rows", {&x});
    expect_one_gpu({&x});
    at::Tensor q = make(x, x.sizes(), at::kChar), scale = make(x, leading(x), at::kFloat);
    check(api.quantize_rows(x.data_ptr(), r.ld, q.data_ptr(), floats(scale), r.rows, r.cols, code, pointer(a[1])));
    return give({q, scale});
    END_HANDLE_TH_ERRORS
}

// x, x_scale, weight, weight_scale, out_dtype or None, stream
PyObject* matmul_i8(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 6);
    const at::Tensor &x = tensor(a[0], "x"), &xs = tensor(a[1], "x_scale"), &w = tensor(a[2], "weight"),
                     &ws = tensor(a[3], "weight_scale");
    if (x.scalar_type() != at::kChar || w.scalar_type() != at::kChar)
        refuse(PyExc_TypeError, "x and weight must be int8");
    at::ScalarType out = at::kBFloat16;
    if (a[4] != Py_None) {
        if (!THPDtype_Check(a[4])) refuse(PyExc_TypeError, "out_dtype must be a torch.dtype");
        out = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
    }
    const int code = code_of(out);
    if (code < 0) refuse(PyExc_TypeError, "out_dtype must be float16, bfloat16 or float32, not ", name_of(out));
    const Rows rx = rows_of(x, "x"), rw = matrix_of(w, "weight");
    if (rw.cols != rx.cols)
        refuse(PyExc_ValueError, "inner dimensions differ: ", rx.cols, " vs ", rw.cols);
    expect_vector(xs, "x_scale", rx.rows, at::kFloat, at::kFloat);
    expect_vector(ws, "weight_scale", rw.rows, at::kFloat, at::kFloat);
    warn_of_lost_gradients("matmul_i8", {&x, &xs, &w, &ws});
    expect_one_gpu({&x, &xs, &w, &ws});
    at::Tensor y = make(x, with_last(x, rw.rows), out);
    check(api.i8(x.data_ptr(), rx.ld, floats(xs), w.data_ptr(), rw.ld, floats(ws), y.data_ptr(), rx.rows, rw.rows, rx.cols,
                 code, pointer(a[5])));
    return give(std::move(y));
    END_HANDLE_TH_ERRORS
}

// the status error, then the C functions' addresses in the order of Api
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 9);
    Api b;
    auto set = [&](auto& fn, int k) { fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(pointer(a[k])); };
    set(b.layer_norm, 1);
    set(b.layer_norm_backward_workspace, 2);
    set(b.layer_norm_backward, 3);
    set(b.gated, 4);
    set(b.gated_backward_workspace, 5);
    set(b.gated_backward, 6);
    set(b.quantize_rows, 7);
    set(b.i8, 8);
    Py_INCREF(a[0]);
    Py_XDECREF(status_error);
    status_error = a[0];
    api = b;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"layer_norm", method(layer_norm), METH_FASTCALL, nullptr},
    {"layer_norm_backward", method(layer_norm_backward), METH_FASTCALL, nullptr},
    {"matmul_gated", method(matmul_gated), METH_FASTCALL, nullptr},
    {"matmul_gated_backward", method(matmul_gated_backward), METH_FASTCALL, nullptr},
    {"quantize_rows", method(quantize_rows), METH_FASTCALL, nullptr},
    {"matmul_i8", method(matmul_i8), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ffn", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ffn() { return PyModule_Create(&module); }
