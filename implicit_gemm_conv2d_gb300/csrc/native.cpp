// native.cpp -- the allocating functions of train.py in C++: argument checks, outputs and
// workspace from torch's allocator, and the C ABI call (include/conv_train.h), without the
// interpreter in between.  A small call's time is the host's: about 1 us a tensor argument and
// output in Python and ctypes, about 0.1 here; a gradient list has hundreds.
#include <Python.h>

#include <array>
#include <cstdint>
#include <vector>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "conv_train.h"

namespace {

PyObject* g_error = nullptr;   // binding.ConvError
PyObject* g_memory = nullptr;  // torch.OutOfMemoryError

struct Raised {};  // a Python error is set

[[noreturn]] void value_error(const char* text)
{
    PyErr_SetString(PyExc_ValueError, text);
    throw Raised();
}

void check(int status, const char* where)
{
    if (status == CONV_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_ValueError, "%s: a tensor, got %s", name, Py_TYPE(o)->tp_name);
        throw Raised();
    }
    return THPVariable_Unpack(o);
}

const at::Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

void on_gpu(const at::Tensor& t)
{
    if (!t.is_cuda() || !t.is_contiguous()) value_error("tensors must be contiguous CUDA tensors");
}

// A call runs on the current device (include/conv_train.h): on another device's tensors its kernels
// would be given addresses that are not theirs.  Asked for one tensor of a call, before anything is
// allocated; the others are on that one's device.
void on_current(const at::Tensor& t)
{
    c10::DeviceIndex current = -1;
    if (c10::cuda::GetDevice(&current) == cudaSuccess && current == t.device().index()) return;
    PyErr_Format(PyExc_ValueError, "tensors on cuda:%d, which is not the current device: call under torch.cuda.device",
                 int(t.device().index()));
    throw Raised();
}

int dtype_code(const at::Tensor& t, const char* name)
{
    if (t.scalar_type() == at::kFloat) return CONV_F32;
    if (t.scalar_type() == at::kBFloat16) return CONV_BF16;
    PyErr_Format(PyExc_ValueError, "%s: float32 or bfloat16", name);
    throw Raised();
}

// t has the sizes, dtype and device given, and is a contiguous CUDA tensor.
const at::Tensor& same(const at::Tensor& t, const char* name, at::IntArrayRef sizes, at::ScalarType dtype,
                       const at::Device& device)
{
    if (t.sizes() != sizes || t.scalar_type() != dtype || t.device() != device) {
        PyErr_Format(PyExc_ValueError, "%s: another size, dtype or device than the call's other tensors give it", name);
        throw Raised();
    }
    on_gpu(t);
    return t;
}

int64_t integer(PyObject* o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

int32_t int32(PyObject* o)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) value_error("an integer beyond 32 bits");
    return int32_t(v);
}

int32_t size32(int64_t v)
{
    if (v > INT32_MAX) value_error("a size beyond 2^31 - 1");
    return int32_t(v);
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}

conv_stream_t stream_of(const at::Tensor& t)
{
    return reinterpret_cast<conv_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
}

at::Tensor workspace(size_t bytes, const at::Tensor& like)
{
    return bytes ? at::empty({int64_t(bytes)}, like.options().dtype(at::kByte)) : at::Tensor();
}
void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
const void* address(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

PyObject* wrap(const at::Tensor& t)
{
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject* wrap(const at::Tensor& a, const at::Tensor& b, const at::Tensor& c)
{
    PyObject* t = PyTuple_New(3);
    if (!t) throw Raised();
    PyTuple_SET_ITEM(t, 0, wrap(a));
    PyTuple_SET_ITEM(t, 1, wrap(b));
    PyTuple_SET_ITEM(t, 2, wrap(c));
    return t;
}

conv_gn_desc_t gn_desc(const at::Tensor& x, PyObject* groups, double eps, PyObject* act, PyObject* layout)
{
    conv_gn_desc_t d;
    d.dtype = dtype_code(x, "x");
    d.layout = int32(layout);
    d.act = int32(act);
    d.G = int32(groups);
    d.eps = float(eps);
    if (x.dim() < 2) value_error("x: at least (batch, channels)");
    on_gpu(x);
    on_current(x);
    const bool nhwc = d.layout == CONV_LAYOUT_NHWC;
    d.B = size32(x.size(0));
    d.C = size32(x.size(nhwc ? -1 : 1));
    int64_t p = 1;
    for (int64_t i = nhwc ? 1 : 2; i < x.dim() - (nhwc ? 1 : 0); ++i) p *= x.size(i);
    d.P = size32(p);
    return d;
}

const at::Tensor* channels(PyObject* o, const char* name, const at::Tensor& x, int64_t C)
{
    const at::Tensor* t = optional(o, name);
    if (t) same(*t, name, {C}, x.scalar_type(), x.device());
    return t;
}

// x, groups, gamma, beta, eps, act, layout, stats
PyObject* group_norm(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[0], "x");
    const conv_gn_desc_t d = gn_desc(x, a[1], number(a[4]), a[5], a[6]);
    const at::Tensor* gamma = channels(a[2], "gamma", x, d.C);
    const at::Tensor* beta = channels(a[3], "beta", x, d.C);
    at::Tensor y = at::empty(x.sizes(), x.options()), mean, rstd;
    if (PyObject_IsTrue(a[7])) {
        mean = at::empty({d.B, d.G}, x.options().dtype(at::kFloat));
        rstd = at::empty({d.B, d.G}, x.options().dtype(at::kFloat));
    }
    const size_t bytes = conv_gn_fwd_workspace_size(&d);
    const at::Tensor ws = workspace(bytes, x);
    check(conv_gn_fwd(&d, x.data_ptr(), address(gamma), address(beta), y.data_ptr(),
                      static_cast<float*>(address(mean)), static_cast<float*>(address(rstd)), address(ws), bytes,
                      stream_of(x)),
          "conv_gn_fwd");
    return wrap(y, mean, rstd);
}

// x, dy, groups, gamma, beta, mean, rstd, act, layout, param_grads
PyObject* group_norm_bwd(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[0], "x");
    const conv_gn_desc_t d = gn_desc(x, a[2], 0.0, a[7], a[8]);
    const at::Tensor& dy = same(tensor(a[1], "dy"), "dy", x.sizes(), x.scalar_type(), x.device());
    const at::Tensor* gamma = channels(a[3], "gamma", x, d.C);
    const at::Tensor* beta = channels(a[4], "beta", x, d.C);
    const std::array<int64_t, 2> stat = {d.B, d.G};
    const at::Tensor& mean = same(tensor(a[5], "mean"), "mean", stat, at::kFloat, x.device());
    const at::Tensor& rstd = same(tensor(a[6], "rstd"), "rstd", stat, at::kFloat, x.device());
    at::Tensor dx = at::empty(x.sizes(), x.options()), dgamma, dbeta;
    if (PyObject_IsTrue(a[9])) {
        dgamma = at::empty({d.C}, x.options());
        dbeta = at::empty({d.C}, x.options());
    }
    const size_t bytes = conv_gn_bwd_workspace_size(&d);
    const at::Tensor ws = workspace(bytes, x);
    check(conv_gn_bwd(&d, x.data_ptr(), dy.data_ptr(), address(gamma), address(beta),
                      static_cast<const float*>(mean.data_ptr()), static_cast<const float*>(rstd.data_ptr()),
                      dx.data_ptr(), address(dgamma), address(dbeta), address(ws), bytes, stream_of(x)),
          "conv_gn_bwd");
    return wrap(dx, dgamma, dbeta);
}

conv_embed_desc_t embed_desc(const at::Tensor& idx, const at::Tensor& t, const char* name, int64_t V, int64_t D,
                             PyObject* scale, PyObject* padding)
{
    conv_embed_desc_t d;
    if (idx.scalar_type() == at::kInt) d.index_dtype = CONV_INDEX_I32;
    else if (idx.scalar_type() == at::kLong) d.index_dtype = CONV_INDEX_I64;
    else value_error("idx: int32 or int64");
    d.dtype = dtype_code(t, name);
    if (idx.device() != t.device()) value_error("idx and its values are on different devices");
    on_gpu(idx);
    on_gpu(t);
    on_current(t);
    d.T = idx.numel();
    d.V = size32(V);
    d.D = size32(D);
    d.padding_idx = int32(padding);
    d.scale = float(number(scale));
    return d;
}

// idx, table, scale, padding_idx
PyObject* embed(PyObject* const* a)
{
    const at::Tensor &idx = tensor(a[0], "idx"), &table = tensor(a[1], "table");
    if (table.dim() != 2) value_error("table: (rows, values)");
    const conv_embed_desc_t d = embed_desc(idx, table, "table", table.size(0), table.size(1), a[2], a[3]);
    c10::SmallVector<int64_t, 6> sizes(idx.sizes().begin(), idx.sizes().end());
    sizes.push_back(d.D);
    at::Tensor y = at::empty(sizes, table.options());
    check(conv_embed_fwd(&d, idx.data_ptr(), table.data_ptr(), y.data_ptr(), stream_of(table)), "conv_embed_fwd");
    return wrap(y);
}

// idx, dy, V, scale, padding_idx
PyObject* embed_bwd(PyObject* const* a)
{
    const at::Tensor &idx = tensor(a[0], "idx"), &dy = tensor(a[1], "dy");
    if (dy.dim() != idx.dim() + 1 || dy.sizes().slice(0, idx.dim()) != idx.sizes())
        value_error("dy: idx's sizes and the values'");
    const conv_embed_desc_t d = embed_desc(idx, dy, "dy", integer(a[2]), dy.size(-1), a[3], a[4]);
    at::Tensor dtable = at::empty({d.V, d.D}, dy.options());
    const size_t bytes = conv_embed_bwd_workspace_size(&d);
    const at::Tensor ws = workspace(bytes, dy);
    check(conv_embed_bwd(&d, idx.data_ptr(), dy.data_ptr(), dtable.data_ptr(), address(ws), bytes, stream_of(dy)),
          "conv_embed_bwd");
    return wrap(dtable);
}

// grads, out (None: in place), max_norm (None: the norm only).  The sequences are tuples or lists.
PyObject* grads_call(PyObject* const* a)
{
    const bool clip = a[2] != Py_None;
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(a[0]);
    if (n == 0) value_error("an empty list of gradients");
    if (a[1] != Py_None && PySequence_Fast_GET_SIZE(a[1]) != n) value_error("out: a tensor for each gradient");
    if (n > INT32_MAX) value_error("a list beyond 2^31 - 1 gradients");
    PyObject** in = PySequence_Fast_ITEMS(a[0]);
    PyObject** out = a[1] != Py_None ? PySequence_Fast_ITEMS(a[1]) : in;
    std::vector<conv_grad_t> list(static_cast<size_t>(n));
    const at::Tensor& first = tensor(in[0], "a gradient");
    on_gpu(first);
    on_current(first);
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& g = tensor(in[i], "a gradient");
        on_gpu(g);
        if (g.device() != first.device()) value_error("gradients on different devices");
        list[size_t(i)] = {g.data_ptr(), g.data_ptr(), g.numel(), dtype_code(g, "a gradient")};
        if (out != in) {
            const at::Tensor& o = tensor(out[i], "out");
            if (o.numel() != g.numel() || o.scalar_type() != g.scalar_type() || o.device() != g.device())
                value_error("out: each tensor with its gradient's size, dtype and device");
            on_gpu(o);
            list[size_t(i)].out = o.data_ptr();
        }
    }
    at::Tensor norm = at::empty({}, first.options().dtype(at::kFloat));
    float* pn = static_cast<float*>(norm.data_ptr());
    const size_t bytes = conv_grad_norm_workspace_size(list.data(), int32_t(n));
    const at::Tensor ws = workspace(bytes, first);
    if (clip)
        check(conv_grad_clip(list.data(), int32_t(n), float(number(a[2])), pn, address(ws), bytes, stream_of(first)),
              "conv_grad_clip");
    else
        check(conv_grad_norm(list.data(), int32_t(n), pn, address(ws), bytes, stream_of(first)), "conv_grad_norm");
    return wrap(norm);
}

// The functions by position; nothing thrown leaves them.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    if (count != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_memory, e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The exception classes: a status code's, an allocation's.
PyObject* set_errors(PyObject* const* a)
{
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_INCREF(a[1]);
    Py_XSETREF(g_memory, a[1]);
    Py_RETURN_NONE;
}

#define ENTRY(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("group_norm", group_norm, 8),
                         ENTRY("group_norm_bwd", group_norm_bwd, 10),
                         ENTRY("embed", embed, 4),
                         ENTRY("embed_bwd", embed_bwd, 5),
                         ENTRY("grads", grads_call, 3),
                         ENTRY("set_errors", set_errors, 2),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_igconv_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__igconv_native(void) { return PyModule_Create(&module); }
