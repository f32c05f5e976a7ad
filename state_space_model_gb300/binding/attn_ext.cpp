// The Python side of the attention entry points (include/ssd.h): torch
// tensors become ssd_tensor descriptors, missing outputs are allocated, and
// the C ABI is called on the current torch stream.  Marshalling only; the
// checks and the computation are the library's.
//
// It is compiled because these calls run once for each layer and token: a kv_append
// of 12 tensors takes 4.1 us of host time, checks and launch included; with the
// descriptors packed in Python and the call made through ctypes it took 24.5.
//
// The library's functions come as addresses (bind), so the one that _native
// loaded is the one that runs.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "ssd.h"

namespace {

decltype(&ssd_kv_append) g_append = nullptr;
decltype(&ssd_kv_read) g_read = nullptr;
decltype(&ssd_paged_attention) g_attention = nullptr;
decltype(&ssd_paged_attention_workspace_size) g_ws_size = nullptr;

int code_of(at::ScalarType t) {
    switch (t) {
    case at::kFloat: return SSD_F32;
    case at::kBFloat16: return SSD_BF16;
    case at::kInt: return SSD_I32;
    case at::kFloat8_e4m3fn: return SSD_F8E4M3;
    default: return 99;      // the library names it
    }
}

// The descriptors of one call and the device that its tensors share.
struct Call {
    ssd_tensor room[16];
    int n = 0, device = -1;
    bool bad = false;        // a Python exception is set

    ssd_tensor *add(const at::Tensor &t) {
        if (!t.is_cuda()) {
            PyErr_SetString(PyExc_ValueError, "all tensors must be CUDA tensors (the library "
                                              "takes device pointers)");
            bad = true;
            return nullptr;
        }
        const int dev = t.get_device();
        if (device < 0) device = dev;
        if (dev != device) {
            PyErr_Format(PyExc_ValueError, "tensors on different devices: cuda:%d and cuda:%d",
                         device, dev);
            bad = true;
            return nullptr;
        }
        if (t.dim() > 5) {
            PyErr_SetString(PyExc_ValueError, "tensors of more than 5 dimensions are not supported");
            bad = true;
            return nullptr;
        }
        ssd_tensor *d = &room[n++];
        d->data = t.numel() > 0 ? t.data_ptr() : nullptr;
        d->dtype = code_of(t.scalar_type());
        d->ndim = int32_t(t.dim());
        for (int i = 0; i < 5; ++i) {
            d->shape[i] = i < t.dim() ? t.size(i) : 0;
            d->stride[i] = i < t.dim() ? t.stride(i) : 0;
        }
        return d;
    }
    // None -> null
    ssd_tensor *add(PyObject *o) {
        if (bad || o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %s", Py_TYPE(o)->tp_name);
            bad = true;
            return nullptr;
        }
        return add(THPVariable_Unpack(o));
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream(int8_t(device)).stream(); }
};

const at::Tensor *tensor(PyObject *o) {
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    PyErr_Format(PyExc_TypeError, "expected a torch.Tensor, got %s", Py_TYPE(o)->tp_name);
    return nullptr;
}

// A new packed tensor beside `like` (at::empty without its dispatch: a call that makes
// its output, its log sums and its workspace spends half its host time there).
at::Tensor make(const at::Tensor &like, at::IntArrayRef shape, at::ScalarType dtype) {
    TORCH_CHECK_VALUE(like.is_cuda(), "all tensors must be CUDA tensors (the library takes device pointers)");
    return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
}

// Every function: C++ exceptions (torch's allocator) become Python's, and a
// status of the library is returned as an int for the caller to raise.
template <typename F>
PyObject *guarded(F &&f) {
    try {
        return f();
    } catch (const c10::ValueError &e) {
        PyErr_SetString(PyExc_ValueError, e.what_without_backtrace());
        return nullptr;
    } catch (const std::exception &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

bool count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
    return n == want;
}

// (q, k, v, slots, positions, cos, sin, q_weight, k_weight, eps, interleaved,
//  k_cache, v_cache, k_scale, v_scale, out) -> out, or a status
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (!count(n, 16)) return nullptr;
        const double eps = PyFloat_AsDouble(a[9]);
        const int inter = PyObject_IsTrue(a[10]);
        if (PyErr_Occurred()) return nullptr;
        const at::Tensor *q = tensor(a[0]);
        if (!q) return nullptr;
        at::Tensor out;
        if (a[15] == Py_None) {
            out = make(*q, q->sizes(), q->scalar_type());
        } else {
            const at::Tensor *o = tensor(a[15]);
            if (!o) return nullptr;
            out = *o;
        }
        Call c;
        ssd_tensor *in[9], *pool[4];
        for (int i = 0; i < 9; ++i) in[i] = c.add(a[i]);
        for (int i = 0; i < 4; ++i) pool[i] = c.add(a[11 + i]);
        ssd_tensor *o = c.bad ? nullptr : c.add(out);
        if (c.bad) return nullptr;
        void *stream = c.stream();
        ssd_status st;
        Py_BEGIN_ALLOW_THREADS
        st = g_append(in[0], in[1], in[2], in[3], in[4], in[5], in[6], in[7], in[8], float(eps),
                      inter, pool[0], pool[1], pool[2], pool[3], o, stream);
        Py_END_ALLOW_THREADS
        return st ? PyLong_FromLong(st) : THPVariable_Wrap(out);
    });
}

// (k_cache, v_cache, k_scale, v_scale, page_table, cu_lens, starts, tokens, f32 out,
//  k, v) -> (k, v), or a status.  f32 out: the dtype of rows read from codes.
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (!count(n, 11)) return nullptr;
        const int64_t tokens = PyLong_AsLongLong(a[7]);
        const int f32 = PyObject_IsTrue(a[8]);
        if (PyErr_Occurred()) return nullptr;
        at::Tensor kv[2];
        for (int i = 0; i < 2; ++i) {
            if (a[9 + i] != Py_None) {
                const at::Tensor *t = tensor(a[9 + i]);
                if (!t) return nullptr;
                kv[i] = *t;
                continue;
            }
            const at::Tensor *pool = tensor(a[0]);
            if (!pool) return nullptr;
            if (pool->dim() != 4) {
                PyErr_Format(PyExc_ValueError, "k_cache: %lld dimensions, expected 4",
                             (long long)pool->dim());
                return nullptr;
            }
            at::ScalarType dt = pool->scalar_type();
            if (dt == at::kFloat8_e4m3fn) dt = f32 ? at::kFloat : at::kBFloat16;
            kv[i] = make(*pool, {tokens, pool->size(1), pool->size(3)}, dt);
        }
        Call c;
        ssd_tensor *in[7];
        for (int i = 0; i < 7; ++i) in[i] = c.add(a[i]);
        ssd_tensor *k = c.bad ? nullptr : c.add(kv[0]);
        ssd_tensor *v = c.bad ? nullptr : c.add(kv[1]);
        if (c.bad) return nullptr;
        void *stream = c.stream();
        ssd_status st;
        Py_BEGIN_ALLOW_THREADS
        st = g_read(in[0], in[1], in[2], in[3], in[4], in[5], in[6], k, v, stream);
        Py_END_ALLOW_THREADS
        if (st) return PyLong_FromLong(st);
        PyObject *pk = THPVariable_Wrap(kv[0]), *pv = THPVariable_Wrap(kv[1]);
        PyObject *pair = PyTuple_Pack(2, pk, pv);
        Py_XDECREF(pk);
        Py_XDECREF(pv);
        return pair;
    });
}

// (q, k_cache, v_cache, k_scale, v_scale, page_table, lens, scale or None, window, want lse,
//  out, workspace) -> out or (out, lse), or a status
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        if (!count(n, 12)) return nullptr;
        const int64_t window = PyLong_AsLongLong(a[8]);
        const int want_lse = PyObject_IsTrue(a[9]);
        double scale = a[7] == Py_None ? 0.0 : PyFloat_AsDouble(a[7]);
        if (PyErr_Occurred()) return nullptr;
        const at::Tensor *q = tensor(a[0]), *pool = q ? tensor(a[1]) : nullptr;
        if (!pool) return nullptr;
        if (q->dim() != 4 || pool->dim() != 4) {
            PyErr_Format(PyExc_ValueError, "q and k_cache have 4 dimensions, got %lld and %lld",
                         (long long)q->dim(), (long long)pool->dim());
            return nullptr;
        }
        const int64_t B = q->size(0), T = q->size(1), H = q->size(2), D = q->size(3);
        if (a[7] == Py_None) scale = 1.0 / std::sqrt(double(D));
        Call c;
        ssd_tensor *in[7];
        for (int i = 0; i < 7; ++i) in[i] = c.add(a[i]);
        if (c.bad) return nullptr;
        at::Tensor out, lse;
        c10::DataPtr own;          // a workspace of this call: back to the cache when it returns
        void *room = nullptr;
        size_t bytes = 0;
        if (a[10] == Py_None) {
            out = make(*q, {B, T, H, D}, q->scalar_type());
        } else {
            const at::Tensor *t = tensor(a[10]);
            if (!t) return nullptr;
            out = *t;
        }
        if (want_lse) lse = make(*q, {B, T, H}, at::kFloat);
        ssd_tensor *o = c.add(out), *l = !c.bad && want_lse ? c.add(lse) : nullptr;
        if (c.bad) return nullptr;
        if (a[11] == Py_None) {
            const ssd_status st = g_ws_size(B, T, H, pool->size(1), D, code_of(pool->scalar_type()),
                                            &bytes);
            if (st) return PyLong_FromLong(st);
            if (bytes) own = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
            room = own.get();
        } else {
            const at::Tensor *t = tensor(a[11]);
            if (!t) return nullptr;
            if (!t->is_cuda() || t->get_device() != c.device) {
                PyErr_SetString(PyExc_ValueError, "workspace: not on the device of the tensors");
                return nullptr;
            }
            if (!t->is_contiguous()) {
                PyErr_SetString(PyExc_ValueError, "workspace: must be contiguous");
                return nullptr;
            }
            bytes = t->nbytes();
            room = bytes ? t->data_ptr() : nullptr;
        }
        void *stream = c.stream();
        ssd_status st;
        Py_BEGIN_ALLOW_THREADS
        st = g_attention(in[0], in[1], in[2], in[3], in[4], in[5], in[6], float(scale), window, o,
                         l, room, bytes, stream);
        Py_END_ALLOW_THREADS
        if (st) return PyLong_FromLong(st);
        PyObject *po = THPVariable_Wrap(out);
        if (!want_lse || !po) return po;
        PyObject *pl = THPVariable_Wrap(lse), *pair = PyTuple_Pack(2, po, pl);
        Py_DECREF(po);
        Py_XDECREF(pl);
        return pair;
    });
}

// Addresses of ssd_kv_append, ssd_kv_read, ssd_paged_attention and
// ssd_paged_attention_workspace_size
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count(n, 4)) return nullptr;
    void *p[4];
    for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    g_append = reinterpret_cast<decltype(g_append)>(p[0]);
    g_read = reinterpret_cast<decltype(g_read)>(p[1]);
    g_attention = reinterpret_cast<decltype(g_attention)>(p[2]);
    g_ws_size = reinterpret_cast<decltype(g_ws_size)>(p[3]);
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(bind), FAST(kv_append), FAST(kv_read), FAST(paged_attention),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attn_ext", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_ext() { return PyModule_Create(&g_module); }
