// calls.cpp -- the attention and page calls as a Python extension module:
// tensors to descriptors, the device and stream of the call, outputs and
// workspace, then the C ABI of include/kvq.h.
//
// These calls run once per layer and step next to kernels of a few
// microseconds; describing a dozen tensors through ctypes took longer than
// the kernels.  Argument rules beyond that are the library's own.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <string>
#include <vector>

#include "kvq.h"

namespace {

int type_code(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return KVQ_BF16;
        case at::kHalf: return KVQ_F16;
        case at::kFloat: return KVQ_F32;
        case at::kInt: return KVQ_I32;
        case at::kLong: return KVQ_I64;
        case at::kChar: return KVQ_I8;
        case at::kByte: return KVQ_U8;
        case at::kFloat8_e4m3fn: return KVQ_F8E4M3;
        case at::kFloat8_e5m2: return KVQ_F8E5M2;
        case at::kFloat8_e8m0fnu: return KVQ_E8M0;
        default: return -1;
    }
}

// The tensors of one call, and the CUDA device that all non-empty ones are on.
struct Call {
    const char* op;
    int device = -1;
    bool failed = false;

    explicit Call(const char* name) : op(name) {}

    bool add(const at::Tensor& t, kvq_tensor* d) {
        const int code = type_code(t.scalar_type());
        if (code < 0) {
            PyErr_Format(PyExc_TypeError, "%s: dtype %s has no kvq equivalent", op, c10::toString(t.scalar_type()));
            return false;
        }
        if (t.dim() > KVQ_MAX_DIMS) {
            PyErr_Format(PyExc_ValueError, "%s: too many dimensions", op);
            return false;
        }
        *d = kvq_tensor{};
        d->dtype = code;
        d->ndim = (int32_t)t.dim();
        for (int i = 0; i < d->ndim; ++i) {
            d->shape[i] = t.size(i);
            d->stride[i] = t.stride(i);
        }
        if (t.numel() == 0) return true;
        if (!t.is_cuda()) {
            PyErr_Format(PyExc_ValueError, "%s: tensors must be on a CUDA device, got one on %s", op,
                         t.device().str().c_str());
            return false;
        }
        if (device < 0) device = t.get_device();
        if (t.get_device() != device) {
            PyErr_Format(PyExc_ValueError, "%s: tensors on cuda:%d and %s; all must be on one device", op, device,
                         t.device().str().c_str());
            return false;
        }
        d->data = const_cast<void*>(t.const_data_ptr());
        return true;
    }

    // a Python tensor, or None (null)
    kvq_tensor* get(PyObject* o, kvq_tensor* d) {
        if (failed || o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", op, Py_TYPE(o)->tp_name);
            failed = true;
            return nullptr;
        }
        if (!add(THPVariable_Unpack(o), d)) {
            failed = true;
            return nullptr;
        }
        return d;
    }

    bool list(PyObject* o, std::vector<kvq_tensor>* d) {
        PyObject* seq = PySequence_Fast(o, "expected a sequence of tensors");
        if (!seq) return false;
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
        d->resize((size_t)n);
        bool ok = true;
        for (Py_ssize_t i = 0; i < n && ok; ++i) {
            PyObject* e = PySequence_Fast_GET_ITEM(seq, i);
            if (e == Py_None || !get(e, &(*d)[(size_t)i])) {
                if (!failed) PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got None", op);
                ok = false;
            }
        }
        Py_DECREF(seq);
        return ok;
    }

    // Run `f(stream)` with the device current; None: the device's current
    // stream (the legacy default one where every tensor is empty).  Returns
    // (status, stream, device or -1, result).
    template <typename F>
    PyObject* run(PyObject* stream, PyObject* result, F f) {
        void* s = nullptr;
        c10::cuda::OptionalCUDAGuard guard;
        if (device >= 0) guard.set_index(device);
        if (stream != Py_None) {
            s = PyLong_AsVoidPtr(stream);
            if (PyErr_Occurred()) return nullptr;
        } else if (device >= 0) {
            s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        }
        kvq_status st;
        Py_BEGIN_ALLOW_THREADS
        st = f(reinterpret_cast<kvq_stream>(s));
        Py_END_ALLOW_THREADS
        PyObject* stream_int = PyLong_FromVoidPtr(s);
        return Py_BuildValue("(iNiO)", (int)st, stream_int, device, result);
    }
};

bool count_is(const char* op, Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, %zd wanted", op, n, want);
    return false;
}

// C++ exceptions (an allocation that fails) become Python errors here
template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

struct Ref {
    PyObject* p;
    explicit Ref(PyObject* o) : p(o) {}
    ~Ref() { Py_XDECREF(p); }
};

// o itself, or for None a new tensor like `like` (nullptr with an error set)
PyObject* output(PyObject* o, PyObject* like) {
    if (o != Py_None || !THPVariable_Check(like)) {
        Py_INCREF(o);
        return o;
    }
    const at::Tensor& t = THPVariable_Unpack(like);
    return THPVariable_Wrap(at::empty(t.sizes(), t.options()));
}

PyObject* new_i32(PyObject* o, PyObject* like) {
    if (o != Py_None || !THPVariable_Check(like)) {
        Py_INCREF(o);
        return o;
    }
    const at::Tensor& t = THPVariable_Unpack(like);
    return THPVariable_Wrap(at::empty(t.sizes(), t.options().dtype(at::kInt)));
}

// softmax_scale: a number, or None for D ** -0.5
bool scale_of(PyObject* o, const kvq_tensor* q, float* scale) {
    if (o != Py_None) {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) return false;
        *scale = (float)v;
        return true;
    }
    const int64_t d = q && q->ndim > 0 ? q->shape[q->ndim - 1] : 0;
    *scale = d > 0 ? (float)(1.0 / std::sqrt((double)d)) : 1.0f;
    return true;
}

// q, k, v, cu_seqlens_q, cu_seqlens_k, out, lse, causal, softmax_scale, stream
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c("prompt_attention");
        if (!count_is(c.op, n, 10)) return nullptr;
        kvq_tensor d[7];
        Ref out(output(a[5], a[0]));
        if (!out.p) return nullptr;
        kvq_tensor *q = c.get(a[0], d), *k = c.get(a[1], d + 1), *v = c.get(a[2], d + 2), *cq = c.get(a[3], d + 3),
                   *ck = c.get(a[4], d + 4), *o = c.get(out.p, d + 5), *l = c.get(a[6], d + 6);
        if (c.failed) return nullptr;
        const int causal = PyObject_IsTrue(a[7]);
        float scale;
        if (causal < 0 || !scale_of(a[8], q, &scale)) return nullptr;
        return c.run(a[9], out.p, [&](kvq_stream s) { return kvq_prompt_attention(q, k, v, cq, ck, o, l, causal, scale, s); });
    });
}

// q, k_cache, v_cache, block_table, seq_lens, prefix_table, prefix_len, scale_k, scale_v, offset_k, offset_v, out,
// lse, softmax_scale, workspace, stream
PyObject* shared_prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c("shared_prefix_attention");
        if (!count_is(c.op, n, 16)) return nullptr;
        kvq_tensor d[13];
        Ref out(output(a[11], a[0]));
        if (!out.p) return nullptr;
        kvq_tensor *q = c.get(a[0], d), *k = c.get(a[1], d + 1), *v = c.get(a[2], d + 2), *t = c.get(a[3], d + 3),
                   *sl = c.get(a[4], d + 4), *pt = c.get(a[5], d + 5), *sk = c.get(a[7], d + 6), *sv = c.get(a[8], d + 7),
                   *ok = c.get(a[9], d + 8), *ov = c.get(a[10], d + 9), *o = c.get(out.p, d + 10), *l = c.get(a[12], d + 11),
                   *w = c.get(a[14], d + 12);
        if (c.failed) return nullptr;
        const long long prefix_len = PyLong_AsLongLong(a[6]);
        if (prefix_len == -1 && PyErr_Occurred()) return nullptr;
        float scale;
        if (!scale_of(a[13], q, &scale)) return nullptr;
        at::Tensor workspace;                     // lives to the end of the call: the allocator orders its next use
        if (!w && q && k && t && q->ndim == 3 && k->ndim == 4 && t->ndim == 2) {
            const int64_t need = kvq_shared_prefix_attention_workspace(q->shape[0], q->shape[1], k->shape[2], q->shape[2],
                                                                       prefix_len, t->shape[1] * k->shape[1]);
            if (need > 0) {
                workspace = at::empty({need}, THPVariable_Unpack(a[0]).options().dtype(at::kByte));
                if (!c.add(workspace, d + 12)) return nullptr;
                w = d + 12;
            }
        }
        return c.run(a[15], out.p, [&](kvq_stream s) {
            return kvq_shared_prefix_attention(q, k, v, t, sl, pt, prefix_len, sk, sv, ok, ov, o, l, scale, w, s);
        });
    });
}

// caches, src, dst, stream
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c("copy_pages");
        if (!count_is(c.op, n, 4)) return nullptr;
        std::vector<kvq_tensor> caches;
        kvq_tensor d[2];
        if (!c.list(a[0], &caches)) return nullptr;
        kvq_tensor *src = c.get(a[1], d), *dst = c.get(a[2], d + 1);
        if (c.failed) return nullptr;
        return c.run(a[3], Py_None, [&](kvq_stream s) {
            return kvq_copy_pages(caches.data(), (int32_t)caches.size(), src, dst, s);
        });
    });
}

// block_table, seq_lens, ref_count, rows, block_size, stream
PyObject* free_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c("free_pages");
        if (!count_is(c.op, n, 6)) return nullptr;
        kvq_tensor d[4];
        kvq_tensor *t = c.get(a[0], d), *l = c.get(a[1], d + 1), *r = c.get(a[2], d + 2), *rows = c.get(a[3], d + 3);
        if (c.failed) return nullptr;
        const long long block = PyLong_AsLongLong(a[4]);
        if (block == -1 && PyErr_Occurred()) return nullptr;
        return c.run(a[5], Py_None, [&](kvq_stream s) { return kvq_free_pages(t, l, r, rows, block, s); });
    });
}

// caches, block_table, seq_lens, ref_count, parents, children, block_size, fresh, stream
PyObject* fork_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c("fork_pages");
        if (!count_is(c.op, n, 9)) return nullptr;
        std::vector<kvq_tensor> caches;
        kvq_tensor d[6];
        Ref fresh(new_i32(a[7], a[5]));
        if (!fresh.p || !c.list(a[0], &caches)) return nullptr;
        kvq_tensor *t = c.get(a[1], d), *l = c.get(a[2], d + 1), *r = c.get(a[3], d + 2), *p = c.get(a[4], d + 3),
                   *ch = c.get(a[5], d + 4), *f = c.get(fresh.p, d + 5);
        if (c.failed) return nullptr;
        const long long block = PyLong_AsLongLong(a[6]);
        if (block == -1 && PyErr_Occurred()) return nullptr;
        return c.run(a[8], fresh.p, [&](kvq_stream s) {
            return kvq_fork_pages(caches.data(), (int32_t)caches.size(), t, l, r, p, ch, block, f, s);
        });
    });
}

// caches, block_table, ref_count, new_table, new_ref_count, page_map, stream
PyObject* compact_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c("compact_pages");
        if (!count_is(c.op, n, 7)) return nullptr;
        std::vector<kvq_tensor> caches;
        kvq_tensor d[5];
        Ref nt(new_i32(a[3], a[1])), nr(new_i32(a[4], a[2])), pm(new_i32(a[5], a[2]));
        if (!nt.p || !nr.p || !pm.p || !c.list(a[0], &caches)) return nullptr;
        kvq_tensor *t = c.get(a[1], d), *r = c.get(a[2], d + 1), *t2 = c.get(nt.p, d + 2), *r2 = c.get(nr.p, d + 3),
                   *m = c.get(pm.p, d + 4);
        if (c.failed) return nullptr;
        Ref result(PyTuple_Pack(3, nt.p, nr.p, pm.p));
        if (!result.p) return nullptr;
        return c.run(a[6], result.p, [&](kvq_stream s) {
            return kvq_compact_pages(caches.data(), (int32_t)caches.size(), t, r, t2, r2, m, s);
        });
    });
}

// the descriptor of a tensor as bytes (for tests)
PyObject* descriptor(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c("descriptor");
        if (!count_is(c.op, n, 1)) return nullptr;
        kvq_tensor d;
        if (!c.get(a[0], &d)) {
            if (!c.failed) PyErr_SetString(PyExc_TypeError, "descriptor: expected a tensor, got None");
            return nullptr;
        }
        return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&d), sizeof(d));
    });
}

#define KVQ_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KVQ_METHOD(prompt_attention), KVQ_METHOD(shared_prefix_attention), KVQ_METHOD(copy_pages),
                         KVQ_METHOD(free_pages), KVQ_METHOD(fork_pages), KVQ_METHOD(compact_pages),
                         KVQ_METHOD(descriptor), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "Attention and page calls of libkvq.so on torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
