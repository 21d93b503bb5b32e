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
    decltype(&tgemm_route) route;
    decltype(&tgemm_route_backward) route_backward;
    decltype(&tgemm_gemm_fourbit) gemm_w4;
    decltype(&tgemm_experts_workspace) experts_workspace;
    decltype(&tgemm_experts_forward) experts_forward;
    decltype(&tgemm_experts_backward) experts_backward;
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

int integer(const char *name, PyObject *o)
{
    PyObject *i = PyNumber_Index(o);
    if (!i) throw Failed{};
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, "%s is out of range: %lld", name, v);
    return int(v);
}

// A contiguous tensor of the given type and shape (dimensions of -1 are any) on x's device.
const at::Tensor &block(const char *name, PyObject *o, at::ScalarType type, at::IntArrayRef sizes, const at::Tensor &x)
{
    const at::Tensor &t = tensor(name, o);
    on_device_of(name, t, x);
    if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be %s, got %s", name, name_of(type), name_of(t.scalar_type()));
    bool fits = t.dim() == int64_t(sizes.size()) && t.is_contiguous();
    std::string want;
    for (size_t d = 0; d < sizes.size(); ++d) {
        fits = fits && (sizes[d] < 0 || t.size(int64_t(d)) == sizes[d]);
        want += (d ? ", " : "") + (sizes[d] < 0 ? std::string("any") : std::to_string(sizes[d]));
    }
    if (!fits) fail(PyExc_ValueError, "%s must be contiguous of shape (%s), got %s", name, want.c_str(), shape_of(t).c_str());
    return t;
}

int scoring_of(PyObject *o)
{
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "softmax") == 0) return TGEMM_SOFTMAX;
        if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0) return TGEMM_SIGMOID;
    }
    fail(PyExc_ValueError, "scoring must be softmax or sigmoid, got %R", o);
}

// A matrix of logits, one row a token.
Rows logits_of(const at::Tensor &x)
{
    if (x.dim() != 2 || x.size(1) < 1) fail(PyExc_ValueError, "logits must be a matrix [tokens, experts], got %s", shape_of(x).c_str());
    return rows_of("logits", x, x.size(1));
}

// route(logits, top_k, scoring, bias, groups, top_groups, group_scores, renormalize, scale)
PyObject *route(PyObject *const *a)
{
    const at::Tensor &x = cuda_tensor("logits", a[0]);
    const int code = dtype_code("logits", x);
    const Rows r = logits_of(x);
    const int64_t experts = x.size(1);
    const int top = integer("top_k", a[1]), scoring = scoring_of(a[2]), groups = integer("groups", a[4]);
    if (top < 1 || top > experts || top > 32)
        fail(PyExc_ValueError, "top_k must lie between 1 and %lld, got %d", (long long)(experts < 32 ? experts : 32), top);
    if (experts > 1024) fail(PyExc_ValueError, "logits may have up to 1024 experts, got %lld", (long long)experts);
    if (groups < 1 || groups > 32 || experts % groups)
        fail(PyExc_ValueError, "groups must be 1 to 32 and divide %lld experts, got %d", (long long)experts, groups);
    const int top_groups = a[5] == Py_None ? groups : integer("top_groups", a[5]), group_scores = integer("group_scores", a[6]);
    if (top_groups < 1 || top_groups > groups || top > experts / groups * top_groups)
        fail(PyExc_ValueError, "top_groups must be 1 to %d and hold top_k experts, got %d", groups, top_groups);
    if (group_scores < 1 || group_scores > 2) fail(PyExc_ValueError, "group_scores must be 1 or 2, got %d", group_scores);
    at::Tensor bias;
    if (a[3] != Py_None) bias = block("bias", a[3], at::kFloat, {experts}, x);
    const bool renormalize = truth(a[7]);
    const double scale = number(a[8]);
    const at::Tensor weights = empty({r.count, top}, at::kFloat, x), chosen = empty({r.count, top}, at::kInt, x);
    check_status(api.route(r.count, experts, top, code, ptr(x), r.ld, static_cast<float *>(ptr(bias)), scoring, groups,
                           top_groups, group_scores, renormalize, float(scale), static_cast<float *>(ptr(weights)),
                           static_cast<int *>(ptr(chosen)), stream_of(x)),
                 "route", r.count, experts);
    return tuple_of({weights, chosen});
}

// route_backward(dweights, logits, experts, scoring, renormalize, scale)
PyObject *route_backward(PyObject *const *a)
{
    const at::Tensor &x = cuda_tensor("logits", a[1]);
    const int code = dtype_code("logits", x);
    const Rows r = logits_of(x);
    if (x.size(1) > 1024) fail(PyExc_ValueError, "logits may have up to 1024 experts, got %lld", (long long)x.size(1));
    const at::Tensor &chosen = block("experts", a[2], at::kInt, {r.count, -1}, x);
    const int64_t top = chosen.size(1);
    if (top < 1 || top > 32 || top > x.size(1))
        fail(PyExc_ValueError, "experts must hold 1 to 32 experts a token and no more than there are, got %s", shape_of(chosen).c_str());
    const at::Tensor &dw = block("dweights", a[0], at::kFloat, {r.count, top}, x);
    const int scoring = scoring_of(a[3]);
    const bool renormalize = truth(a[4]);
    const double scale = number(a[5]);
    const at::Tensor dl = empty(x.sizes(), x.scalar_type(), x);
    check_status(api.route_backward(r.count, x.size(1), int(top), code, static_cast<float *>(ptr(dw)), ptr(x), r.ld,
                                    static_cast<int *>(ptr(chosen)), scoring, renormalize, float(scale), ptr(dl), stream_of(x)),
                 "route_backward", r.count, x.size(1));
    return THPVariable_Wrap(dl);
}

// gemm_w4(x, packed, scales, zeros, experts, fp32 result)
PyObject *gemm_w4(PyObject *const *a)
{
    const at::Tensor &x = cuda_tensor("x", a[0]);
    const int code = dtype_code("x", x);
    if (code == TGEMM_F32) fail(PyExc_TypeError, "x must be fp16 or bf16, got %s", name_of(x.scalar_type()));
    const bool routed = a[4] != Py_None, f32 = truth(a[5]);
    const at::Tensor &packed = tensor("packed", a[1]);
    const int lead = routed ? 1 : 0;
    if (packed.dim() != 2 + lead)
        fail(PyExc_ValueError, routed ? "packed must be [experts, rows, width / 2], got %s" : "packed must be [rows, width / 2], got %s",
             shape_of(packed).c_str());
    const int64_t E = routed ? packed.size(0) : 1, n = packed.size(lead), k = 2 * packed.size(lead + 1);
    const at::Tensor &scales = tensor("scales", a[2]);
    if (scales.scalar_type() != x.scalar_type() && scales.scalar_type() != at::kFloat)
        fail(PyExc_TypeError, "scales must be %s or torch.float32, got %s", name_of(x.scalar_type()), name_of(scales.scalar_type()));
    const int64_t groups = scales.dim() == 2 + lead ? scales.size(lead + 1) : 0;
    if (E < 1 || n < 1 || groups < 1 || k % groups || k / groups % 32)
        fail(PyExc_ValueError, "packed %s and scales %s must make groups of a multiple of 32 weights", shape_of(packed).c_str(),
             shape_of(scales).c_str());
    at::DimVector wsize, ssize;
    if (routed) wsize.push_back(E), ssize.push_back(E);
    wsize.push_back(n), ssize.push_back(n);
    wsize.push_back(k / 2), ssize.push_back(groups);
    block("packed", a[1], at::kByte, wsize, x);
    block("scales", a[2], scales.scalar_type(), ssize, x);
    at::Tensor zeros, experts;
    if (a[3] != Py_None) zeros = block("zeros", a[3], at::kByte, ssize, x);
    if (x.dim() < 1 || x.size(-1) != k)
        fail(PyExc_ValueError, "x must have a last dimension of %lld, got %s", (long long)k, shape_of(x).c_str());
    const Rows r = rows_of("x", x, k);
    at::DimVector ysize(x.sizes().begin(), x.sizes().end() - 1);
    int64_t each = 1;
    if (routed) {
        experts = block("experts", a[4], at::kInt, {-1, -1}, x);
        const int64_t tokens = experts.size(0), top = experts.size(1);
        const bool per_pair = x.dim() == 3 && x.size(0) == tokens && x.size(1) == top;
        if (!per_pair && !(x.dim() == 2 && x.size(0) == tokens))
            fail(PyExc_ValueError, "x must be [tokens, width] or [tokens, top, width] for experts %s, got %s", shape_of(experts).c_str(),
                 shape_of(x).c_str());
        each = per_pair || top < 1 ? 1 : top;
        ysize = {tokens, top};
    }
    ysize.push_back(n);
    const at::Tensor y = empty(ysize, f32 ? at::kFloat : x.scalar_type(), x);
    check_status(api.gemm_w4(y.numel() / n, n, k, k / groups, code, ptr(x), r.ld, each, static_cast<uint8_t *>(ptr(packed)), ptr(scales),
                             scales.scalar_type() == at::kFloat ? int(TGEMM_F32) : code, static_cast<uint8_t *>(ptr(zeros)),
                             static_cast<int *>(ptr(experts)), E, ptr(y), f32 ? int(TGEMM_F32) : code, stream_of(x)),
                 "gemm_w4", y.numel() / n, n);
    return THPVariable_Wrap(y);
}

// A stack of an expert's matrices: elements from row to row and from expert to expert.
struct Strides {
    int64_t row, expert;
};
Strides stack(const Plan &p, const char *name, const at::Tensor &t, int64_t experts, int64_t rows, int64_t cols)
{
    if (t.scalar_type() != p.type)
        fail(PyExc_TypeError, "%s must be %s, got %s", name, name_of(p.type), name_of(t.scalar_type()));
    if (!t.is_cuda() || t.get_device() != p.device)
        fail(PyExc_ValueError, "%s must be on cuda:%d, got %s", name, p.device, device_of(t.device()).c_str());
    if (t.dim() != 3 || t.size(0) != experts || t.size(1) != rows || t.size(2) != cols)
        fail(PyExc_ValueError, "%s must have shape (%lld, %lld, %lld), got %s", name, (long long)experts, (long long)rows,
             (long long)cols, shape_of(t).c_str());
    if (t.is_contiguous()) return {cols, rows * cols};
    const int64_t row = rows > 1 ? t.stride(1) : cols, expert = experts > 1 ? t.stride(0) : rows * row;
    if (t.stride(2) != 1 || row < cols || expert < (rows - 1) * row + cols)
        fail(PyExc_ValueError, "the rows of %s must be contiguous, and neither they nor the experts may overlap", name);
    return {row, expert};
}

// The arguments that both passes share: x, experts, weights, w_gate, w_up and w_down from a[0] on.
struct Mixture {
    const at::Tensor &x, &wg, &wu, &wd;
    int64_t tokens, experts, top, ldx;
    const at::Tensor &chosen, &weights;
    Strides g, u, d;

    Mixture(const Plan &p, PyObject *const *a)
        : x(tensor("x", a[0])), wg(tensor("w_gate", a[3])), wu(tensor("w_up", a[4])), wd(tensor("w_down", a[5])),
          tokens(tokens_of(x)), experts(wg.dim() == 3 ? wg.size(0) : 1), top(0), ldx(matrix(p, "x", x, tokens, p.width)),
          chosen(block("experts", a[1], at::kInt, {tokens, -1}, x)), weights(block("weights", a[2], at::kFloat, {tokens, chosen.size(1)}, x))
    {
        top = chosen.size(1);
        if (top < 1 || top > 32) fail(PyExc_ValueError, "experts must hold 1 to 32 experts a token, got %s", shape_of(chosen).c_str());
        if (experts < 1) fail(PyExc_ValueError, "w_gate must be [experts, hidden, width], got %s", shape_of(wg).c_str());
        if (experts > 1024) fail(PyExc_ValueError, "w_gate may have up to 1024 experts, got %lld", (long long)experts);
        g = stack(p, "w_gate", wg, experts, p.hidden, p.width);
        u = stack(p, "w_up", wu, experts, p.hidden, p.width);
        d = stack(p, "w_down", wd, experts, p.width, p.hidden);
    }

    at::Tensor workspace(const Plan &p, int kind) const
    {
        const int64_t need = api.experts_workspace(p.handle, tokens, experts, int(top), kind);
        if (need < 0) check_status(int(-need), "tgemm_experts_workspace", tokens, experts);
        return empty({need}, at::kByte, x);
    }
};

// experts_forward(plan, x, experts, weights, w_gate, w_up, w_down, save)
PyObject *experts_forward(PyObject *const *a)
{
    const Plan p(a[0]);
    const Mixture m(p, a + 1);
    const bool save = truth(a[7]);
    const at::Tensor y = empty({m.tokens, p.width}, p.type, m.x);
    at::Tensor g, u, h;
    if (save) {
        g = empty({m.tokens * m.top, p.hidden}, p.type, m.x);
        u = empty({m.tokens * m.top, p.hidden}, p.type, m.x);
        h = empty({m.tokens * m.top, p.hidden}, p.type, m.x);
    }
    const at::Tensor work = m.workspace(p, save ? TGEMM_EXPERTS_TRAIN : TGEMM_EXPERTS_SERVE);
    check_status(api.experts_forward(p.handle, m.tokens, m.experts, int(m.top), ptr(m.x), m.ldx, static_cast<int *>(ptr(m.chosen)),
                                     static_cast<float *>(ptr(m.weights)), ptr(m.wg), m.g.row, m.g.expert, ptr(m.wu), m.u.row,
                                     m.u.expert, ptr(m.wd), m.d.row, m.d.expert, ptr(y), p.width, ptr(g), ptr(u), ptr(h), ptr(work),
                                     work.numel(), stream_of(m.x)),
                 "tgemm_experts_forward", m.tokens, m.experts);
    if (!save) return THPVariable_Wrap(y);
    PyObject *saved = tuple_of({g, u, h});
    PyObject *r = PyTuple_Pack(2, Py_None, saved);
    Py_DECREF(saved);
    if (!r) throw Failed{};
    Py_DECREF(Py_None);  // the place held for y
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(y));
    return r;
}

// experts_backward(plan, dy, x, experts, weights, w_gate, w_up, w_down, saved)
PyObject *experts_backward(PyObject *const *a)
{
    const Plan p(a[0]);
    const Mixture m(p, a + 2);
    const at::Tensor &dy = tensor("dy", a[1]);
    const int64_t D = p.width, F = p.hidden, E = m.experts, lddy = matrix(p, "dy", dy, m.tokens, D);
    if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 3)
        fail(PyExc_TypeError, "saved must be the tuple of three that the forward pass returned");
    const at::Tensor *saved[3];
    const char *names[3] = {"saved g", "saved u", "saved h"};
    for (int i = 0; i < 3; ++i) {
        saved[i] = &tensor(names[i], PyTuple_GET_ITEM(a[8], i));
        if (matrix(p, names[i], *saved[i], m.tokens * m.top, F) != F) fail(PyExc_ValueError, "%s must be contiguous", names[i]);
    }
    const at::Tensor dx = empty({m.tokens, D}, p.type, m.x), dweights = empty({m.tokens, m.top}, at::kFloat, m.x);
    const at::Tensor dwg = empty({E, F, D}, p.type, m.x), dwu = empty({E, F, D}, p.type, m.x), dwd = empty({E, D, F}, p.type, m.x);
    const at::Tensor work = m.workspace(p, TGEMM_EXPERTS_BACKWARD);
    check_status(api.experts_backward(p.handle, m.tokens, E, int(m.top), ptr(dy), lddy, ptr(m.x), m.ldx,
                                      static_cast<int *>(ptr(m.chosen)), static_cast<float *>(ptr(m.weights)), ptr(m.wg), m.g.row,
                                      m.g.expert, ptr(m.wu), m.u.row, m.u.expert, ptr(m.wd), m.d.row, m.d.expert, ptr(*saved[0]),
                                      ptr(*saved[1]), ptr(*saved[2]), ptr(dx), D, static_cast<float *>(ptr(dweights)), ptr(dwg),
                                      ptr(dwu), ptr(dwd), ptr(work), work.numel(), stream_of(m.x)),
                 "tgemm_experts_backward", m.tokens, E);
    return tuple_of({dx, dweights, dwg, dwu, dwd});
}

// bind(addresses of the C ABI's functions in Api's order, TgemmError)
PyObject *bind(PyObject *const *a)
{
    void **slots[] = {reinterpret_cast<void **>(&api.layer_norm),          reinterpret_cast<void **>(&api.layer_norm_workspace),
                      reinterpret_cast<void **>(&api.layer_norm_backward), reinterpret_cast<void **>(&api.dropout),
                      reinterpret_cast<void **>(&api.ffn_forward),         reinterpret_cast<void **>(&api.ffn_backward),
                      reinterpret_cast<void **>(&api.route),               reinterpret_cast<void **>(&api.route_backward),
                      reinterpret_cast<void **>(&api.gemm_w4),             reinterpret_cast<void **>(&api.experts_workspace),
                      reinterpret_cast<void **>(&api.experts_forward),     reinterpret_cast<void **>(&api.experts_backward)};
    constexpr int n = sizeof(slots) / sizeof(slots[0]);
    if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != n) fail(PyExc_TypeError, "bind takes %d addresses", n);
    for (int i = 0; i < n; ++i) *slots[i] = reinterpret_cast<void *>(uintptr_t(word(PyTuple_GET_ITEM(a[0], i))));
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
                         method<route, 9>("route"),
                         method<route_backward, 6>("route_backward"),
                         method<gemm_w4, 6>("gemm_w4"),
                         method<experts_forward, 8>("experts_forward"),
                         method<experts_backward, 9>("experts_backward"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module_def); }
