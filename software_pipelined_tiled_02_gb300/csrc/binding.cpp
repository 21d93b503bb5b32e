// binding.cpp -- the Python side of the feed-forward operators on torch tensors:
// argument checks, outputs, workspaces and the calls of the C ABI.
//
// A small operator takes the GPU a few microseconds, and as many checks and
// allocations made from Python take ten to thirty; made here, about one each.
// The operators' signatures and documentation are in operators.py, which hands
// its arguments on by position.
//
// The C ABI's functions come as addresses from the library that the package has
// loaded (bind), so the release and the debug-check build work alike.  Failures
// raise TypeError, ValueError or the package's TgemmError; a C++ exception
// (an allocation that fails) becomes torch's Python exception.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <string>

#include "tgemm.h"

namespace {

// The C ABI as loaded.
struct Api {
    decltype(&tgemm_layer_norm) layer_norm;
    decltype(&tgemm_layer_norm_workspace) layer_norm_workspace;
    decltype(&tgemm_layer_norm_backward) layer_norm_backward;
    decltype(&tgemm_dropout) dropout;
    decltype(&tgemm_ffn_forward) ffn_forward;
    decltype(&tgemm_ffn_backward) ffn_backward;
} api;
PyObject *tgemm_error;  // the package's exception class: TgemmError(code, what)

// A check that failed: the Python exception is set.
struct Failed {};

[[noreturn]] void fail(PyObject *kind, const char *format, ...)
{
    va_list args;
    va_start(args, format);
    PyErr_FormatV(kind, format, args);
    va_end(args);
    throw Failed{};
}

std::string shape_of(const at::Tensor &t)
{
    std::string s = "(";
    for (int64_t d = 0; d < t.dim(); ++d) s += (d ? ", " : "") + std::to_string(t.size(d));
    return s + (t.dim() == 1 ? ",)" : ")");
}

const char *name_of(at::ScalarType t)
{
    return t == at::kHalf ? "torch.float16" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat ? "torch.float32" : c10::toString(t);
}

std::string device_of(c10::Device d) { return d.str(); }

void check_status(int rc, const char *what, int64_t a, int64_t b)
{
    if (rc == TGEMM_OK) return;
    PyObject *text = PyUnicode_FromFormat("%s(%lld, %lld)", what, (long long)a, (long long)b);
    PyObject *e = text ? PyObject_CallFunction(tgemm_error, "iO", rc, text) : nullptr;
    if (e) PyErr_SetObject(tgemm_error, e);
    Py_XDECREF(e);
    Py_XDECREF(text);
    throw Failed{};
}

const at::Tensor &tensor(const char *name, PyObject *o)
{
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

// A tensor on the current CUDA device.
const at::Tensor &cuda_tensor(const char *name, PyObject *o)
{
    const at::Tensor &t = tensor(name, o);
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
    if (t.get_device() != c10::cuda::current_device())
        fail(PyExc_ValueError, "%s must be on the current CUDA device", name);
    return t;
}

void on_device_of(const char *name, const at::Tensor &t, const at::Tensor &x)
{
    if (t.device() != x.device())
        fail(PyExc_ValueError, "%s must be on %s, got %s", name, device_of(x.device()).c_str(), device_of(t.device()).c_str());
}

int dtype_code(const char *name, const at::Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kHalf: return TGEMM_F16;
    case at::kBFloat16: return TGEMM_BF16;
    case at::kFloat: return TGEMM_F32;
    default: fail(PyExc_TypeError, "%s must be fp16, bf16 or fp32, got %s", name, name_of(t.scalar_type()));
    }
}

// `t` has to have x's device, type and shape.
void like(const char *name, const at::Tensor &t, const at::Tensor &x)
{
    on_device_of(name, t, x);
    if (t.scalar_type() != x.scalar_type())
        fail(PyExc_TypeError, "%s must be %s, got %s", name, name_of(x.scalar_type()), name_of(t.scalar_type()));
    if (t.sizes() != x.sizes())
        fail(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_of(x).c_str(), shape_of(t).c_str());
}

// Rows of the last dimension's `width` elements, and the distance between them.
struct Rows {
    int64_t count, ld;
};

int64_t row_width(const at::Tensor &x)
{
    if (x.dim() < 1 || x.size(-1) < 1)
        fail(PyExc_ValueError, "x must have a last dimension of at least 1, got %s", shape_of(x).c_str());
    return x.size(-1);
}

Rows rows_of(const char *name, const at::Tensor &t, int64_t width)
{
    if (t.is_contiguous()) return {t.numel() / width, width};
    if (t.dim() != 2 || (t.stride(1) != 1 && width > 1))
        fail(PyExc_ValueError, "%s must be contiguous, or a matrix with contiguous rows", name);
    if (t.size(0) <= 1) return {t.size(0), width};
    if (t.stride(0) < width) fail(PyExc_ValueError, "the rows of %s must not overlap", name);
    return {t.size(0), t.stride(0)};
}

// A weight vector: x's type or fp32.
const at::Tensor &vector_of(const char *name, PyObject *o, int64_t width, const at::Tensor &x)
{
    const at::Tensor &t = tensor(name, o);
    on_device_of(name, t, x);
    if (t.dim() != 1 || t.size(0) != width || !t.is_contiguous())
        fail(PyExc_ValueError, "%s must be contiguous of shape (%lld,), got %s", name, (long long)width, shape_of(t).c_str());
    if (t.scalar_type() != x.scalar_type() && t.scalar_type() != at::kFloat)
        fail(PyExc_TypeError, "%s must be %s or torch.float32, got %s", name, name_of(x.scalar_type()), name_of(t.scalar_type()));
    return t;
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &x)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(x.device()));
}

tgemm_stream_t stream_of(const at::Tensor &x)
{
    return c10::cuda::getCurrentCUDAStream(x.get_device()).stream();
}

void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject *tuple_of(std::initializer_list<at::Tensor> list)
{
    PyObject *r = PyTuple_New(Py_ssize_t(list.size()));
    if (!r) throw Failed{};
    Py_ssize_t i = 0;
    for (const at::Tensor &t : list) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Failed{};
    return v;
}

bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Failed{};
    return v != 0;
}

// An integer modulo 2^64.
uint64_t word(PyObject *o)
{
    PyObject *i = PyNumber_Index(o);
    if (!i) throw Failed{};
    const uint64_t v = PyLong_AsUnsignedLongLongMask(i);
    Py_DECREF(i);
    if (v == uint64_t(-1) && PyErr_Occurred()) throw Failed{};
    return v;
}

// layer_norm(x, weight, bias, eps, stats)
PyObject *layer_norm(PyObject *const *a)
{
    const at::Tensor &x = cuda_tensor("x", a[0]);
    const int code = dtype_code("x", x);
    const int64_t width = row_width(x);
    const Rows r = rows_of("x", x, width);
    at::Tensor weight, bias;
    int wcode = code;
    if (a[1] != Py_None) wcode = dtype_code("weight", weight = vector_of("weight", a[1], width, x));
    if (a[2] != Py_None) {
        bias = vector_of("bias", a[2], width, x);
        if (weight.defined() && bias.scalar_type() != weight.scalar_type())
            fail(PyExc_TypeError, "weight and bias must have the same type, got %s and %s", name_of(weight.scalar_type()),
                 name_of(bias.scalar_type()));
        wcode = dtype_code("bias", bias);
    }
    const double eps = number(a[3]);
    const bool stats = truth(a[4]);
    at::Tensor y = empty(x.sizes(), x.scalar_type(), x), mean, rstd;
    if (stats) {
        mean = empty({r.count}, at::kFloat, x);
        rstd = empty({r.count}, at::kFloat, x);
    }
    check_status(api.layer_norm(r.count, width, code, wcode, ptr(x), r.ld, ptr(weight), ptr(bias), float(eps), ptr(y), width,
                                static_cast<float *>(ptr(mean)), static_cast<float *>(ptr(rstd)), stream_of(x)),
                 "layer_norm", r.count, width);
    return stats ? tuple_of({y, mean, rstd}) : THPVariable_Wrap(y);
}

// layer_norm_backward(dy, x, mean, rstd, weight)
PyObject *layer_norm_backward(PyObject *const *a)
{
    const at::Tensor &x = cuda_tensor("x", a[1]), &dy = tensor("dy", a[0]);
    const int code = dtype_code("x", x);
    const int64_t width = row_width(x);
    like("dy", dy, x);
    const Rows rx = rows_of("x", x, width), rdy = rows_of("dy", dy, width);
    const at::Tensor *stats[2];
    for (int i = 0; i < 2; ++i) {
        const char *name = i ? "rstd" : "mean";
        const at::Tensor &t = tensor(name, a[2 + i]);
        if (t.scalar_type() != at::kFloat)
            fail(PyExc_TypeError, "%s must be torch.float32, got %s", name, name_of(t.scalar_type()));
        on_device_of(name, t, x);
        if (t.numel() != rx.count || !t.is_contiguous())
            fail(PyExc_ValueError, "%s must be contiguous with one value a row (%lld), got %s", name, (long long)rx.count,
                 shape_of(t).c_str());
        stats[i] = &t;
    }
    at::Tensor weight;
    if (a[4] != Py_None) weight = vector_of("weight", a[4], width, x);
    const at::ScalarType wtype = weight.defined() ? weight.scalar_type() : x.scalar_type();
    const int wcode = weight.defined() ? dtype_code("weight", weight) : code;
    const int64_t need = api.layer_norm_workspace(rx.count, width);
    if (need < 0) check_status(int(-need), "layer_norm_backward", rx.count, width);
    const at::Tensor dx = empty(x.sizes(), x.scalar_type(), x), dw = empty({width}, wtype, x), db = empty({width}, wtype, x);
    const at::Tensor work = empty({need}, at::kByte, x);
    check_status(api.layer_norm_backward(rx.count, width, code, wcode, ptr(dy), rdy.ld, ptr(x), rx.ld,
                                         static_cast<float *>(ptr(*stats[0])), static_cast<float *>(ptr(*stats[1])),
                                         ptr(weight), ptr(dx), width, ptr(dw), ptr(db), ptr(work), need, stream_of(x)),
                 "layer_norm_backward", rx.count, width);
    return tuple_of({dx, dw, db});
}

// dropout(x, p, seed, offset, residual)
PyObject *dropout(PyObject *const *a)
{
    const at::Tensor &x = cuda_tensor("x", a[0]);
    const int code = dtype_code("x", x);
    if (!x.is_contiguous()) fail(PyExc_ValueError, "x must be contiguous");
    const double p = number(a[1]);
    if (!(p >= 0.0 && p <= 1.0)) fail(PyExc_ValueError, "p must lie between 0 and 1, got %S", a[1]);
    const uint64_t seed = word(a[2]), offset = word(a[3]);
    at::Tensor residual;
    if (a[4] != Py_None) {
        residual = tensor("residual", a[4]);
        like("residual", residual, x);
        if (!residual.is_contiguous()) fail(PyExc_ValueError, "residual must be contiguous");
    }
    const at::Tensor y = empty(x.sizes(), x.scalar_type(), x);
    check_status(api.dropout(x.numel(), code, ptr(x), ptr(residual), ptr(y), p, seed, offset, stream_of(x)), "dropout",
                 x.numel(), 1);
    return THPVariable_Wrap(y);
}

// A feed-forward plan as the Python side passes it: (handle, width, hidden,
// type code, device index).
struct Plan {
    tgemm_ffn_t handle;
    int64_t width, hidden;
    at::ScalarType type;
    int device;

    explicit Plan(PyObject *o)
    {
        unsigned long long h;
        long long w, f;
        int code;
        if (!PyArg_ParseTuple(o, "KLLii", &h, &w, &f, &code, &device)) throw Failed{};
        if (c10::cuda::current_device() != device)
            fail(PyExc_ValueError, "the plan is for cuda:%d, which is not the current device", device);
        handle = reinterpret_cast<tgemm_ffn_t>(uintptr_t(h));
        width = w;
        hidden = f;
        type = code == TGEMM_F16 ? at::kHalf : at::kBFloat16;
    }
};

// Elements from row to row of a matrix argument of a plan.
int64_t matrix(const Plan &p, const char *name, const at::Tensor &t, int64_t rows, int64_t cols)
{
    if (t.scalar_type() != p.type)
        fail(PyExc_TypeError, "%s must be %s, got %s", name, name_of(p.type), name_of(t.scalar_type()));
    if (!t.is_cuda() || t.get_device() != p.device)
        fail(PyExc_ValueError, "%s must be on cuda:%d, got %s", name, p.device, device_of(t.device()).c_str());
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        fail(PyExc_ValueError, "%s must have shape (%lld, %lld), got %s", name, (long long)rows, (long long)cols,
             shape_of(t).c_str());
    if (t.is_contiguous()) return cols;
    const int64_t ld = rows > 1 ? t.stride(0) : cols;
    if (t.stride(1) != 1 || ld < cols)
        fail(PyExc_ValueError, "the rows of %s must be contiguous and must not overlap", name);
    return ld;
}

int64_t tokens_of(const at::Tensor &x)
{
    if (x.dim() != 2) fail(PyExc_ValueError, "x must be a matrix, got %s", shape_of(x).c_str());
    return x.size(0);
}

// ffn_forward(plan, x, w_gate, w_up, w_down, save)
PyObject *ffn_forward(PyObject *const *a)
{
    const Plan p(a[0]);
    const at::Tensor &x = tensor("x", a[1]), &wg = tensor("w_gate", a[2]), &wu = tensor("w_up", a[3]);
    const at::Tensor &wd = tensor("w_down", a[4]);
    const int64_t tokens = tokens_of(x), D = p.width, F = p.hidden;
    const int64_t ldx = matrix(p, "x", x, tokens, D), ldg = matrix(p, "w_gate", wg, F, D);
    const int64_t ldu = matrix(p, "w_up", wu, F, D), ldd = matrix(p, "w_down", wd, D, F);
    const bool save = truth(a[5]);
    const at::Tensor y = empty({tokens, D}, p.type, x), h = empty({tokens, F}, p.type, x);
    at::Tensor g, u;
    if (save) {
        g = empty({tokens, F}, p.type, x);
        u = empty({tokens, F}, p.type, x);
    }
    check_status(api.ffn_forward(p.handle, tokens, ptr(x), ldx, ptr(wg), ldg, ptr(wu), ldu, ptr(wd), ldd, ptr(y), D, ptr(g),
                                 ptr(u), ptr(h), stream_of(x)),
                 "tgemm_ffn_forward", tokens, F);
    if (!save) return THPVariable_Wrap(y);
    PyObject *saved = tuple_of({g, u, h});
    PyObject *r = PyTuple_Pack(2, Py_None, saved);
    Py_DECREF(saved);
    if (!r) throw Failed{};
    Py_DECREF(Py_None);  // the place held for y
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(y));
    return r;
}

// ffn_backward(plan, dy, x, w_gate, w_up, w_down, saved)
PyObject *ffn_backward(PyObject *const *a)
{
    const Plan p(a[0]);
    const at::Tensor &dy = tensor("dy", a[1]), &x = tensor("x", a[2]), &wg = tensor("w_gate", a[3]);
    const at::Tensor &wu = tensor("w_up", a[4]), &wd = tensor("w_down", a[5]);
    const int64_t tokens = tokens_of(x), D = p.width, F = p.hidden;
    const int64_t lddy = matrix(p, "dy", dy, tokens, D), ldx = matrix(p, "x", x, tokens, D);
    const int64_t ldg = matrix(p, "w_gate", wg, F, D), ldu = matrix(p, "w_up", wu, F, D), ldd = matrix(p, "w_down", wd, D, F);
    if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 3)
        fail(PyExc_TypeError, "saved must be the tuple of three that the forward pass returned");
    const at::Tensor *saved[3];
    const char *names[3] = {"saved g", "saved u", "saved h"};
    for (int i = 0; i < 3; ++i) {
        saved[i] = &tensor(names[i], PyTuple_GET_ITEM(a[6], i));
        if (matrix(p, names[i], *saved[i], tokens, F) != F) fail(PyExc_ValueError, "%s must be contiguous", names[i]);
    }
    const at::Tensor dx = empty({tokens, D}, p.type, x), dwg = empty({F, D}, p.type, x), dwu = empty({F, D}, p.type, x);
    const at::Tensor dwd = empty({D, F}, p.type, x), work = empty({2, tokens, F}, p.type, x);  // dg and du
    char *dg = static_cast<char *>(ptr(work));
    check_status(api.ffn_backward(p.handle, tokens, ptr(dy), lddy, ptr(x), ldx, ptr(wg), ldg, ptr(wu), ldu, ptr(wd), ldd,
                                  ptr(*saved[0]), ptr(*saved[1]), ptr(*saved[2]), ptr(dx), D, ptr(dwg), ptr(dwu), ptr(dwd), dg,
                                  dg + tokens * F * 2, stream_of(x)),
                 "tgemm_ffn_backward", tokens, F);
    return tuple_of({dx, dwg, dwu, dwd});
}

// bind(addresses of the C ABI's functions in Api's order, TgemmError)
PyObject *bind(PyObject *const *a)
{
    void **slots[] = {reinterpret_cast<void **>(&api.layer_norm),          reinterpret_cast<void **>(&api.layer_norm_workspace),
                      reinterpret_cast<void **>(&api.layer_norm_backward), reinterpret_cast<void **>(&api.dropout),
                      reinterpret_cast<void **>(&api.ffn_forward),         reinterpret_cast<void **>(&api.ffn_backward)};
    if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 6) fail(PyExc_TypeError, "bind takes six addresses");
    for (int i = 0; i < 6; ++i) *slots[i] = reinterpret_cast<void *>(uintptr_t(word(PyTuple_GET_ITEM(a[0], i))));
    Py_INCREF(a[1]);
    Py_XDECREF(tgemm_error);
    tgemm_error = a[1];
    Py_RETURN_NONE;
}

// One Python-callable function: its argument count, and every way it can fail.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        if (n != N) fail(PyExc_TypeError, "%d arguments are wanted, got %zd", N, n);
        return F(args);
    } catch (const Failed &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 2>("bind"),
                         method<layer_norm, 5>("layer_norm"),
                         method<layer_norm_backward, 5>("layer_norm_backward"),
                         method<dropout, 5>("dropout"),
                         method<ffn_forward, 6>("ffn_forward"),
                         method<ffn_backward, 7>("ffn_backward"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module_def); }
