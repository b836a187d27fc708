// CPython binding of include/kda_layer.h for torch tensors: descriptors, output allocation and the
// call, nothing else.  Single-token steps run kernels of a few microseconds, less than the Python
// statements it takes to describe a dozen tensors; here that costs well under one.
//
// The library's functions come as addresses (attach), so that this module and the ctypes binding
// always call the same loaded library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "../../include/kda_layer.h"

namespace {

struct Api {
    decltype(&kda_conv) conv;
    decltype(&kda_conv_decode) conv_decode;
    decltype(&kda_qk_norm) qk_norm;
    decltype(&kda_ssm_workspace_size) ssm_size;
    decltype(&kda_ssm_prefill_ws) ssm_prefill;
    decltype(&kda_ssm_decode) ssm_decode;
    decltype(&kda_last_error) last_error;
} api{};
PyObject *kda_error = nullptr;      // the package's exception class
PyObject *raw_stream = nullptr;     // torch._C._cuda_getCurrentRawStream

struct Refused {                    // a Python exception is set
};

// The tensors of a call by position, described; the first one says where the call runs.
template <size_t N>
struct Call {
    kda_tensor_t d[N];
    at::Tensor t[N];
    c10::Device device;
    c10::OptionalDeviceGuard guard;

    explicit Call(PyObject *first) : device(place(first)), guard(device) {}

    static c10::Device place(PyObject *first)
    {
        if (!THPVariable_Check(first)) {
            PyErr_SetString(PyExc_TypeError, "tensors expected");
            throw Refused();
        }
        const c10::Device dev = THPVariable_Unpack(first).device();
        if (!dev.is_cuda()) {
            PyErr_SetString(PyExc_ValueError, "all tensors must be on one GPU");
            throw Refused();
        }
        return dev;
    }
    void put(size_t i, const at::Tensor &x)
    {
        if (x.device() != device) {
            PyErr_SetString(PyExc_ValueError, "all tensors must be on one GPU");
            throw Refused();
        }
        if (x.dim() > 4) {
            PyErr_SetString(PyExc_ValueError, "at most 4 dimensions");
            throw Refused();
        }
        kda_tensor_t &o = d[i];
        o.data = x.numel() ? x.data_ptr() : nullptr;
        const auto ty = x.scalar_type();
        o.dtype = ty == at::kBFloat16 ? KDA_BF16 : ty == at::kFloat ? KDA_F32 : ty == at::kInt ? KDA_I32 : -1;
        o.ndim = (int32_t)x.dim();
        for (int k = 0; k < o.ndim; ++k) {
            o.shape[k] = x.size(k);
            o.stride[k] = x.stride(k);
        }
        t[i] = x;
    }
    void put(size_t i, PyObject *x)         // None: no tensor
    {
        if (x == Py_None) return;
        if (!THPVariable_Check(x)) {
            PyErr_SetString(PyExc_TypeError, "tensors expected");
            throw Refused();
        }
        put(i, THPVariable_Unpack(x));
    }
    bool has(size_t i) const { return t[i].defined(); }
    kda_tensor_t *at(size_t i) { return has(i) ? &d[i] : nullptr; }
    void make(size_t i, at::IntArrayRef shape, at::ScalarType type)
    {
        put(i, at::empty(shape, at::TensorOptions().dtype(type).device(device)));
    }
    PyObject *object(size_t i) const
    {
        if (has(i)) return THPVariable_Wrap(t[i]);
        Py_RETURN_NONE;
    }
    void *stream() const
    {
        PyObject *index = PyLong_FromLong(device.index());
        PyObject *r = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
        Py_XDECREF(index);
        if (!r) throw Refused();
        void *s = PyLong_AsVoidPtr(r);
        Py_DECREF(r);
        return s;
    }
};

template <typename F>
void run(F &&f)
{
    kda_status_t st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    if (st == KDA_OK) return;
    PyObject *e = PyObject_CallFunction(kda_error, "is", (int)st, api.last_error());
    if (e) PyErr_SetObject(kda_error, e);
    Py_XDECREF(e);
    throw Refused();
}

int64_t extent(const at::Tensor &t, int64_t d)      // negative d: from the end; 0 where there is none
{
    if (d < 0) d += t.dim();
    return d >= 0 && d < t.dim() ? t.size(d) : 0;
}

// Sequences of a batch whose dense layout has `dims` dimensions (0 where the call will be refused).
int64_t sequences(const at::Tensor &cu, const at::Tensor &x, int64_t dims)
{
    return cu.defined() ? (cu.numel() > 0 ? cu.numel() - 1 : 0) : x.dim() == dims ? x.size(0) : 0;
}

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&f)
{
    HANDLE_TH_ERRORS
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *pair(PyObject *a, PyObject *b)
{
    PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

// (x, weight, bias, initial_state, cu_seqlens, out, final_state, want_final, activation)
PyObject *conv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject * {
        Call<7> c(a[0]);
        for (size_t i = 0; i < 7; ++i) c.put(i, a[i]);
        if (!c.has(5)) c.make(5, c.t[0].sizes(), c.t[0].scalar_type());
        if (!c.has(6) && PyObject_IsTrue(a[7]) && c.has(1))
            c.make(6, {sequences(c.t[4], c.t[0], 3), std::max<int64_t>(0, extent(c.t[1], -1) - 1), extent(c.t[0], -1)},
                   (c.has(3) ? c.t[3] : c.t[0]).scalar_type());
        const int act = (int)PyLong_AsLong(a[8]);
        void *s = c.stream();
        run([&] { return api.conv(c.at(0), c.at(1), c.at(2), c.at(3), c.at(4), c.at(5), c.at(6), act, s); });
        return pair(c.object(5), c.object(6));
    });
}

// (x, weight, bias, state_pool, state_indices, num_tokens, out, write_out, update, activation)
PyObject *conv_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        Call<7> c(a[0]);
        for (size_t i = 0; i < 7; ++i) c.put(i, a[i]);
        if (!c.has(6) && PyObject_IsTrue(a[7])) c.make(6, c.t[0].sizes(), c.t[0].scalar_type());
        const int update = PyObject_IsTrue(a[8]), act = (int)PyLong_AsLong(a[9]);
        void *s = c.stream();
        run([&] { return api.conv_decode(c.at(0), c.at(1), c.at(2), c.at(3), c.at(4), c.at(5), c.at(6), update, act, s); });
        return c.object(6);
    });
}

// (q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, norm, eps, layout, offset, scale)
PyObject *qk_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 13, [&]() -> PyObject * {
        Call<8> c(a[0]);
        for (size_t i = 0; i < 8; ++i) c.put(i, a[i]);
        if (!c.has(6)) c.make(6, c.t[0].sizes(), c.t[0].scalar_type());
        if (!c.has(7) && c.has(1)) c.make(7, c.t[1].sizes(), c.t[1].scalar_type());
        kda_qk_norm_options_t o{};
        o.norm = (int32_t)PyLong_AsLong(a[8]);
        o.norm_eps = (float)PyFloat_AsDouble(a[9]);
        o.rotary_layout = (int32_t)PyLong_AsLong(a[10]);
        o.rotary_offset = (int32_t)PyLong_AsLong(a[11]);
        o.rotary_scale = (float)PyFloat_AsDouble(a[12]);
        if (PyErr_Occurred()) throw Refused();
        void *s = c.stream();
        run([&] { return api.qk_norm(c.at(0), c.at(1), c.at(2), c.at(3), c.at(4), c.at(5), c.at(6), c.at(7), &o, s); });
        return pair(c.object(6), c.object(7));
    });
}

kda_ssm_options_t ssm_options(const kda_tensor_t *D, const kda_tensor_t *bias, const kda_tensor_t *z, PyObject *softplus,
                              PyObject *segment)
{
    kda_ssm_options_t o{};
    o.D = D;
    o.dt_bias = bias;
    o.z = z;
    o.dt_softplus = PyObject_IsTrue(softplus);
    if (segment) o.segment = (int32_t)PyLong_AsLong(segment);
    if (PyErr_Occurred()) throw Refused();
    return o;
}

// (x, dt, A, B, C, initial_state, cu_seqlens, out, final_state, D, dt_bias, z, workspace, want_final, softplus, segment)
PyObject *ssm_prefill(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 16, [&]() -> PyObject * {
        Call<13> c(a[0]);
        for (size_t i = 0; i < 12; ++i) c.put(i, a[i]);
        if (!c.has(7)) c.make(7, c.t[0].sizes(), c.t[0].scalar_type());
        if (!c.has(8) && PyObject_IsTrue(a[13]) && c.has(3))
            c.make(8, {sequences(c.t[6], c.t[0], 4), extent(c.t[0], -2), extent(c.t[3], -1), extent(c.t[0], -1)}, at::kFloat);
        const kda_ssm_options_t o = ssm_options(c.at(9), c.at(10), c.at(11), a[14], a[15]);
        size_t need = 0;
        run([&] { return api.ssm_size(c.at(0), c.at(1), c.at(2), c.at(3), c.at(4), c.at(5), c.at(6), c.at(7), c.at(8), &o, &need); });
        uintptr_t base = 0;
        size_t size = 0;
        if (need) {
            at::Tensor w;
            if (a[12] == Py_None) {
                w = at::empty({(int64_t)need + 256}, at::TensorOptions().dtype(at::kByte).device(c.device));
            } else {
                if (THPVariable_Check(a[12])) w = THPVariable_Unpack(a[12]);
                if (!w.defined() || w.device() != c.device || !w.is_contiguous()) {
                    PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous tensor on the operands' GPU");
                    throw Refused();
                }
            }
            const uintptr_t start = (uintptr_t)w.data_ptr();
            const size_t bytes = (size_t)w.numel() * w.element_size();
            base = (start + 255) / 256 * 256;
            size = base - start <= bytes ? bytes - (base - start) : 0;
            c.t[12] = w;
        }
        void *s = c.stream();
        run([&] {
            return api.ssm_prefill(c.at(0), c.at(1), c.at(2), c.at(3), c.at(4), c.at(5), c.at(6), c.at(7), c.at(8), &o,
                                   (void *)base, size, s);
        });
        return pair(c.object(7), c.object(8));
    });
}

// (x, dt, A, B, C, initial_state, cu_seqlens, segment)
PyObject *ssm_workspace_size(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 8, [&]() -> PyObject * {
        Call<8> c(a[0]);
        for (size_t i = 0; i < 7; ++i) c.put(i, a[i]);
        kda_tensor_t out = c.d[0];      // validated only: any address that overlaps nothing
        out.data = (void *)~(uintptr_t)0xffffffffffffffull;
        int64_t acc = 1;
        for (int k = out.ndim - 1; k >= 0; --k) {
            out.stride[k] = acc;
            acc *= out.shape[k];
        }
        const kda_ssm_options_t o = ssm_options(nullptr, nullptr, nullptr, Py_False, a[7]);
        size_t need = 0;
        run([&] { return api.ssm_size(c.at(0), c.at(1), c.at(2), c.at(3), c.at(4), c.at(5), c.at(6), &out, nullptr, &o, &need); });
        return PyLong_FromSize_t(need);
    });
}

// (x, dt, A, B, C, state_pool, state_indices, num_tokens, out, D, dt_bias, z, write_out, update, softplus)
PyObject *ssm_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 15, [&]() -> PyObject * {
        Call<12> c(a[0]);
        for (size_t i = 0; i < 12; ++i) c.put(i, a[i]);
        if (!c.has(8) && PyObject_IsTrue(a[12])) c.make(8, c.t[0].sizes(), c.t[0].scalar_type());
        const kda_ssm_options_t o = ssm_options(c.at(9), c.at(10), c.at(11), a[14], nullptr);
        const int update = PyObject_IsTrue(a[13]);
        void *s = c.stream();
        run([&] {
            return api.ssm_decode(c.at(0), c.at(1), c.at(2), c.at(3), c.at(4), c.at(5), c.at(6), c.at(7), c.at(8), update, &o, s);
        });
        return c.object(8);
    });
}

// (exception class, raw stream function, addresses of the seven library functions)
PyObject *attach(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    void *f[7];
    for (int i = 0; i < 7; ++i) f[i] = PyLong_AsVoidPtr(a[2 + i]);
    if (PyErr_Occurred()) return nullptr;
    Py_INCREF(a[0]);
    Py_INCREF(a[1]);
    kda_error = a[0];
    raw_stream = a[1];
    api.conv = (decltype(api.conv))f[0];
    api.conv_decode = (decltype(api.conv_decode))f[1];
    api.qk_norm = (decltype(api.qk_norm))f[2];
    api.ssm_size = (decltype(api.ssm_size))f[3];
    api.ssm_prefill = (decltype(api.ssm_prefill))f[4];
    api.ssm_decode = (decltype(api.ssm_decode))f[5];
    api.last_error = (decltype(api.last_error))f[6];
    Py_RETURN_NONE;
}

#define KDA_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KDA_METHOD(attach),  KDA_METHOD(conv),        KDA_METHOD(conv_decode),        KDA_METHOD(qk_norm),
                         KDA_METHOD(ssm_prefill), KDA_METHOD(ssm_workspace_size), KDA_METHOD(ssm_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_binding(void) { return PyModule_Create(&module); }
