// Tensor front end of the operators around the half layer, as a CPython module
// (dense_tiled_gemm_relu_amd._block): argument checks, allocation of the results and
// the workspaces, and the call into the C-ABI of include/gemm_relu_block.h.
//
// As in the feed-forward operators' module, the functions take their arguments by
// position, and last the raw stream of the current device that the call runs on;
// block.py holds the user's signatures.
#include "gemm_relu_block.h"
#include "torch_args.hpp"

namespace {

struct Api {
    decltype(&gemm_relu_act) act;
    decltype(&gemm_relu_act_backward_workspace) act_backward_workspace;
    decltype(&gemm_relu_act_backward) act_backward;
    decltype(&gemm_relu_add_norm) add_norm;
    decltype(&gemm_relu_add_norm_backward_workspace) add_norm_backward_workspace;
    decltype(&gemm_relu_add_norm_backward) add_norm_backward;
    decltype(&gemm_relu_orthogonalize_workspace) orthogonalize_workspace;
    decltype(&gemm_relu_orthogonalize) orthogonalize;
} api;

// ---- arguments that may be None
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
const void* data(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
PyObject* give_all(std::initializer_list<const at::Tensor*> all)
{
    PyObject* out = PyTuple_New(Py_ssize_t(all.size()));
    if (!out) throw python_error();
    Py_ssize_t k = 0;
    for (const at::Tensor* t : all) {
        PyObject* item = Py_None;
        if (t && t->defined())
            item = THPVariable_Wrap(*t);
        else
            Py_INCREF(item);
        PyTuple_SET_ITEM(out, k++, item);
    }
    return out;
}
int code_arg(PyObject* o)
{
    const long c = PyLong_AsLong(o);
    if (c == -1 && PyErr_Occurred()) throw python_error();
    return int(c);
}

// ---- product with bias, activation, residual
struct Act {
    Rows x, w;
    int code, bias_code;
};
Act act_args(const at::Tensor& x, const at::Tensor& w, const at::Tensor* bias)
{
    Act a;
    a.code = a.bias_code = code_of(x.scalar_type());
    if (a.code < 0 || a.code == GEMM_RELU_F32 || w.scalar_type() != x.scalar_type())
        refuse(PyExc_TypeError, "x and weight must share dtype float16 or bfloat16");
    a.x = rows_of(x, "x");
    a.w = matrix_of(w, "weight");
    if (a.w.cols != a.x.cols) refuse(PyExc_ValueError, "inner dimensions differ: ", a.x.cols, " vs ", a.w.cols);
    if (bias) {
        expect_vector(*bias, "bias", a.w.rows, x.scalar_type(), at::kFloat);
        a.bias_code = code_of(bias->scalar_type());
    }
    return a;
}
// dy, or the residual: of x's type, x's rows of n
Rows output_rows(const at::Tensor& t, const char* name, const at::Tensor& x, int64_t n)
{
    if (t.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, name, " must have x's type");
    if (t.sizes() != at::IntArrayRef(with_last(x, n)))
        refuse(PyExc_ValueError, name, " must have the result's shape: x's, with ", n, " for the last dimension");
    return rows_of(t, name);
}

// x, weight, bias or None, act (code), residual or None, save, stream
PyObject* matmul_act(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 7);
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
    const at::Tensor *bias = maybe(a[2], "bias"), *residual = maybe(a[4], "residual");
    const int act = code_arg(a[3]);
    const bool save = truth(a[5]);
    const Act s = act_args(x, w, bias);
    const Rows r = residual ? output_rows(*residual, "residual", x, s.w.rows) : Rows{};
    warn_of_lost_gradients("matmul_act", {&x, &w, bias, residual});
    expect_one_gpu({&x, &w, bias, residual});
    at::Tensor y = make(x, with_last(x, s.w.rows), x.scalar_type()), z;
    if (save && act != GEMM_RELU_ACT_NONE) z = make(x, with_last(x, s.w.rows), at::kFloat);
    check(api.act(x.data_ptr(), s.x.ld, w.data_ptr(), s.w.ld, data(bias), data(residual), r.ld, y.data_ptr(),
                  z.defined() ? floats(z) : nullptr, s.x.rows, s.w.rows, s.x.cols, s.code, s.bias_code, act, pointer(a[6])));
    return save ? give_all({&y, &z}) : give(std::move(y));
    END_HANDLE_TH_ERRORS
}

// dy, z or None, x, weight, act (code), bias or None, stream
PyObject* matmul_act_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 7);
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[2], "x"), &w = tensor(a[3], "weight");
    const int act = code_arg(a[4]);
    const at::Tensor *z = maybe(a[1], "z"), *bias = maybe(a[5], "bias");
    const Act s = act_args(x, w, bias);
    const Rows d = output_rows(dy, "dy", x, s.w.rows);
    if (act == GEMM_RELU_ACT_NONE)
        z = nullptr;
    else if (!z)
        refuse(PyExc_TypeError, "z must be a tensor, not NoneType: the gradient of an activation takes matmul_act's (save=True)");
    else
        expect_vector(*z, "z", s.x.rows * s.w.rows, at::kFloat, at::kFloat);
    warn_of_lost_gradients("matmul_act_backward", {&x, &w, &dy, z, bias});
    expect_one_gpu({&x, &w, &dy, z, bias});
    at::Tensor dx = make(x, x.sizes(), x.scalar_type()), dw = make(w, w.sizes(), w.scalar_type()), db;
    if (bias) db = make(*bias, bias->sizes(), bias->scalar_type());
    const int64_t bytes = api.act_backward_workspace(s.x.rows, s.w.rows, s.x.cols);
    const at::Tensor ws = workspace(x, bytes < 0 ? 0 : bytes);
    check(api.act_backward(dy.data_ptr(), d.ld, z ? floats(*z) : nullptr, x.data_ptr(), s.x.ld, w.data_ptr(), s.w.ld,
                           dx.data_ptr(), dw.data_ptr(), bias ? db.data_ptr() : nullptr, s.x.rows, s.w.rows, s.x.cols,
                           s.code, s.bias_code, act, ws.data_ptr(), uint64_t(ws.numel()), pointer(a[6])));
    return give_all({&dx, &dw, &db});
    END_HANDLE_TH_ERRORS
}

// ---- residual sum and norms
double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
// a matrix like x
Rows like_x(const at::Tensor& t, const char* name, const at::Tensor& x)
{
    if (t.scalar_type() != x.scalar_type()) refuse(PyExc_TypeError, name, " must have x's type");
    if (t.sizes() != x.sizes()) refuse(PyExc_ValueError, name, " and x must have the same shape");
    return rows_of(t, name);
}
struct AddNorm {
    Rows x, r;
    int code, wcode;
    int64_t gate_stride = 0;                    // 0: a gate of one row
    at::ScalarType wtype;
};
AddNorm add_norm_args(const at::Tensor& x, const at::Tensor& residual, const at::Tensor* w, const at::Tensor* bias,
                      const at::Tensor* gate, const at::Tensor* post)
{
    AddNorm a;
    a.code = float_code(x);
    a.x = rows_of(x, "x");
    a.r = like_x(residual, "residual", x);
    if (bias && !w) refuse(PyExc_ValueError, "bias needs a weight");
    const bool row_gate = gate && gate->dim() == 1;
    // weight, bias, post_weight and a gate of one row share a type: x's or float32
    const at::Tensor* const vectors[] = {w, bias, post, row_gate ? gate : nullptr};
    const char* const names[] = {"weight", "bias", "post_weight", "gate"};
    const at::Tensor* first = nullptr;
    for (int k = 0; k < 4; ++k)
        if (vectors[k]) {
            if (!first) {
                first = vectors[k];
                expect_vector(*first, names[k], a.x.cols, x.scalar_type(), at::kFloat);
            } else {
                expect_vector(*vectors[k], names[k], a.x.cols, first->scalar_type(), first->scalar_type());
            }
        }
    a.wtype = first ? first->scalar_type() : x.scalar_type();
    a.wcode = code_of(a.wtype);
    if (gate && !row_gate) a.gate_stride = like_x(*gate, "gate", x).ld;
    return a;
}

// x, residual, weight, bias, gate, scale, post_weight (tensors or None), norm (code), eps, stats, stream
PyObject* add_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 11);
    const at::Tensor &x = tensor(a[0], "x"), &residual = tensor(a[1], "residual");
    const at::Tensor *w = maybe(a[2], "weight"), *bias = maybe(a[3], "bias"), *gate = maybe(a[4], "gate"),
                     *post = maybe(a[6], "post_weight");
    const double scale = number(a[5]), eps = number(a[8]);
    const int norm = code_arg(a[7]);
    const bool keep = truth(a[9]);
    const AddNorm s = add_norm_args(x, residual, w, bias, gate, post);
    warn_of_lost_gradients("add_norm", {&x, &residual, w, bias, gate, post});
    expect_one_gpu({&x, &residual, w, bias, gate, post});
    at::Tensor sum = make(x, x.sizes(), x.scalar_type()), y, stats;
    if (w) y = make(x, x.sizes(), x.scalar_type());
    if (keep) stats = make(x, with_last(x, 4), at::kFloat);
    check(api.add_norm(x.data_ptr(), s.x.ld, residual.data_ptr(), s.r.ld, data(gate), s.gate_stride, data(post), data(w),
                       data(bias), sum.data_ptr(), w ? y.data_ptr() : nullptr, keep ? floats(stats) : nullptr, s.x.rows,
                       s.x.cols, s.code, s.wcode, norm, float(scale), float(eps), pointer(a[10])));
    return keep ? give_all({&sum, &y, &stats}) : give_all({&sum, &y});
    END_HANDLE_TH_ERRORS
}

// dy or None, ds or None, x, residual, stats, weight, bias, gate, scale, post_weight (tensors or None), norm (code), stream
PyObject* add_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 12);
    const at::Tensor *dy = maybe(a[0], "dy"), *ds = maybe(a[1], "ds"), *w = maybe(a[5], "weight"), *bias = maybe(a[6], "bias"),
                     *gate = maybe(a[7], "gate"), *post = maybe(a[9], "post_weight");
    const at::Tensor &x = tensor(a[2], "x"), &residual = tensor(a[3], "residual"), &stats = tensor(a[4], "stats");
    const double scale = number(a[8]);
    const int norm = code_arg(a[10]);
    const AddNorm s = add_norm_args(x, residual, w, bias, gate, post);
    if (bool(dy) != bool(w)) refuse(PyExc_ValueError, w ? "dy is missing: there is a weight" : "dy without a weight");
    if (!w && !ds) refuse(PyExc_ValueError, "ds is missing: without a weight no gradient reaches the sum otherwise");
    const int64_t dy_ld = dy ? like_x(*dy, "dy", x).ld : 0, ds_ld = ds ? like_x(*ds, "ds", x).ld : 0;
    expect_vector(stats, "stats", 4 * s.x.rows, at::kFloat, at::kFloat);
    warn_of_lost_gradients("add_norm_backward", {&x, &residual, dy, ds, &stats, w, bias, gate, post});
    expect_one_gpu({&x, &residual, dy, ds, &stats, w, bias, gate, post});
    // without gate and post_weight, and with scale 1, both gradients are the same
    const bool same = !gate && !post && float(scale) == 1.0f;
    at::Tensor dx, dr, dw, db, dg, dp;
    const auto like = [](const at::Tensor& t) { return make(t, t.sizes(), t.scalar_type()); };
    if (!same) dx = like(x);
    dr = w ? like(x) : *ds;
    if (w) dw = like(*w);
    if (bias) db = like(*bias);
    if (gate) dg = like(*gate);
    if (post) dp = like(*post);
    const auto out = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const int64_t bytes = api.add_norm_backward_workspace(s.x.rows, s.x.cols);
    const at::Tensor ws = workspace(x, bytes < 0 ? 0 : bytes);
    check(api.add_norm_backward(data(dy), dy_ld, data(ds), ds_ld, x.data_ptr(), s.x.ld, residual.data_ptr(), s.r.ld, data(gate),
                                s.gate_stride, data(post), data(w), floats(stats), out(dx), w ? out(dr) : nullptr, out(dg),
                                out(dp), out(dw), out(db), s.x.rows, s.x.cols, s.code, s.wcode, norm, float(scale),
                                ws.data_ptr(), uint64_t(ws.numel()), pointer(a[11])));
    return give_all({same ? &dr : &dx, &dr, &dw, &db, &dg, &dp});
    END_HANDLE_TH_ERRORS
}

// ---- orthogonalisation
// g, coefficients (a tuple of 3 numbers a step), eps, stream
PyObject* orthogonalize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 4);
    const at::Tensor& g = tensor(a[0], "g");
    const int code = code_of(g.scalar_type());
    if (code < 0) refuse(PyExc_TypeError, "g must be float16, bfloat16 or float32, not ", name_of(g.scalar_type()));
    if (g.dim() != 2 && g.dim() != 3) refuse(PyExc_ValueError, "g must be a matrix, or a batch of them (3-D)");
    const int64_t rows = g.size(-2), cols = g.size(-1), batch = g.dim() == 3 ? g.size(0) : 1;
    int64_t row_stride = cols, batch_stride = rows * cols;
    if (!g.is_contiguous()) {
        // (a dimension of one element may have any stride)
        row_stride = rows > 1 ? g.stride(-2) : cols;
        batch_stride = batch > 1 ? g.stride(0) : 0;
        if ((cols > 1 && g.stride(-1) != 1) || row_stride < cols) refuse(PyExc_ValueError, "g must have contiguous rows");
    }
    float coefficients[3 * 64];
    const Py_ssize_t count = PyTuple_Check(a[1]) ? PyTuple_GET_SIZE(a[1]) : -1;
    if (count < 0 || count % 3 || count > Py_ssize_t(sizeof coefficients / sizeof *coefficients))
        refuse(PyExc_ValueError, "at most 64 steps of three coefficients");
    for (Py_ssize_t k = 0; k < count; ++k) coefficients[k] = float(number(PyTuple_GET_ITEM(a[1], k)));
    const double eps = number(a[2]);
    warn_of_lost_gradients("orthogonalize", {&g});
    expect_one_gpu({&g});
    at::Tensor out = make(g, g.sizes(), at::kBFloat16);
    const int64_t bytes = api.orthogonalize_workspace(batch, rows, cols);
    const at::Tensor ws = workspace(g, bytes < 0 ? 0 : bytes);
    check(api.orthogonalize(g.data_ptr(), row_stride, batch_stride, out.data_ptr(), batch, rows, cols, code, coefficients,
                            int(count / 3), float(eps), ws.data_ptr(), uint64_t(ws.numel()), pointer(a[3])));
    return give(std::move(out));
    END_HANDLE_TH_ERRORS
}

// the status error, then the C functions' addresses in the order of Api
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 9);
    Api b;
    auto set = [&](auto& fn, int k) { fn = reinterpret_cast<std::remove_reference_t<decltype(fn)>>(pointer(a[k])); };
    set(b.act, 1);
    set(b.act_backward_workspace, 2);
    set(b.act_backward, 3);
    set(b.add_norm, 4);
    set(b.add_norm_backward_workspace, 5);
    set(b.add_norm_backward, 6);
    set(b.orthogonalize_workspace, 7);
    set(b.orthogonalize, 8);
    Py_INCREF(a[0]);
    Py_XDECREF(status_error);
    status_error = a[0];
    api = b;
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"matmul_act", method(matmul_act), METH_FASTCALL, nullptr},
    {"matmul_act_backward", method(matmul_act_backward), METH_FASTCALL, nullptr},
    {"add_norm", method(add_norm), METH_FASTCALL, nullptr},
    {"add_norm_backward", method(add_norm_backward), METH_FASTCALL, nullptr},
    {"orthogonalize", method(orthogonalize), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
