// Native binding of the paged-cache calls: checks the tensors and passes their addresses to the C ABI
// on the tensors' current stream. A serving step makes these calls a few times per layer while their
// kernels run for microseconds: host time per call, launches included, against ctypes on one machine: tables
// 8.5 -> 4.8 us, append 6.9 -> 4.3 us, attention 11.9 -> 9.5 us (on a faster one 3.5, 3.1 and 5.9 us). Arguments and errors are those of block_sparse_long_summary_b200/cobs.py, which wraps it.
#include <ATen/core/Tensor.h>
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/cobs.h"

namespace {

// A refused argument: the Python error has been set.
struct Refused {};

[[noreturn]] void refuse(const char* fmt, const char* name, long long x = 0, long long y = 0, long long z = 0) {
    PyErr_Format(PyExc_ValueError, fmt, name, x, y, z);
    throw Refused();
}

const char* type_name(at::ScalarType t) {
    return t == at::kInt ? "torch.int32" : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kFloat ? "torch.float32" : "torch.uint8";
}

const at::Tensor& tensor_of(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Refused();
    }
    return THPVariable_Unpack(o);
}

struct Call {
    cobs_paged_params p;
    int dev;

    Call(PyObject* params, PyObject* anchor, const char* name) {
        const void* at = PyLong_AsVoidPtr(params);
        if (at == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "params");
            throw Refused();
        }
        p = *static_cast<const cobs_paged_params*>(at);
        const at::Tensor& t = tensor_of(anchor, name);
        if (!t.is_cuda()) refuse("%s must live on a CUDA device", name);
        dev = t.get_device();
    }
    at::ScalarType elem() const { return p.dtype == COBS_BF16 ? at::kBFloat16 : at::kFloat; }

    void place(const at::Tensor& t, const char* name, at::ScalarType type) const {
        if (!t.is_cuda() || t.get_device() != dev) refuse("%s must live on CUDA device %lld", name, dev);
        if (t.scalar_type() != type) {
            PyErr_Format(PyExc_ValueError, "%s must be %s", name, type_name(type));
            throw Refused();
        }
    }
    // a contiguous tensor of n elements
    template <typename T = void>
    T* flat(PyObject* o, const char* name, at::ScalarType type, long long n) const {
        const at::Tensor& t = tensor_of(o, name);
        place(t, name, type);
        if (t.numel() != n || !t.is_contiguous()) refuse("%s must be contiguous with %lld elements, not %lld", name, n, t.numel());
        return n ? static_cast<T*>(t.data_ptr()) : nullptr;
    }
    int32_t* ints(PyObject* o, const char* name, long long n) const { return flat<int32_t>(o, name, at::kInt, n); }
    void* cache(PyObject* o, const char* name) const { return flat(o, name, elem(), (long long)p.n_pages * p.Hkv * p.page * p.d); }
    // [n_tokens, heads, d] rows, each token's heads contiguous; the distance between tokens into stride
    void* rows(PyObject* o, const char* name, int heads, int64_t& stride) const {
        const at::Tensor& t = tensor_of(o, name);
        place(t, name, elem());
        if (t.dim() != 3 || t.size(0) != p.n_tokens || t.size(1) != heads || t.size(2) != p.d)
            refuse("%s must be [%lld, %lld, %lld]", name, p.n_tokens, heads, p.d);
        stride = 0;
        if (p.n_tokens == 0) return nullptr;
        if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != p.d)) refuse("%s: the heads of a token must be contiguous", name);
        if (p.n_tokens > 1 && t.stride(0) != (int64_t)heads * p.d) {
            if (t.stride(0) < (int64_t)heads * p.d) refuse("%s: token rows overlap", name);
            stride = t.stride(0);
        }
        return t.data_ptr();
    }
    cobs_stream_t stream(PyObject* o) const {
        if (o == Py_None) return reinterpret_cast<cobs_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
        PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
        if (v == nullptr) throw Refused();
        void* s = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (s == nullptr && PyErr_Occurred()) throw Refused();
        return static_cast<cobs_stream_t>(s);
    }
};

// Other Python threads go on while this one is in the library: a launch waits when the device's queue is full,
// maybe for a function of the host in some stream that itself needs the interpreter.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs f, which returns a status; C++ exceptions become Python errors.
template <typename F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, F&& f) {
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, nargs);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// params, cached_len, new_len, free_pages, free_count, block_table, cu_new, kv_len, slot_map, counts, stream
PyObject* tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Call c(a[0], a[1], "cached_len");
        const long long n_free = tensor_of(a[3], "free_pages").numel();
        if (n_free > INT32_MAX) refuse("%s: more than 2^31 - 1 entries", "free_pages");
        const auto *cached = c.ints(a[1], "cached_len", c.p.R), *fresh = c.ints(a[2], "new_len", c.p.R),
                   *pages = c.ints(a[3], "free_pages", n_free), *count = c.ints(a[4], "free_count", 1);
        int32_t *table = c.ints(a[5], "block_table", (long long)c.p.R * c.p.max_pages), *cu = c.ints(a[6], "cu_new", c.p.R + 1ll),
                *kv = c.ints(a[7], "kv_len", c.p.R), *slots = c.ints(a[8], "slot_map", c.p.n_tokens), *counts = c.ints(a[9], "counts", 4);
        const cobs_stream_t s = c.stream(a[10]);
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.dev));
        const Unlocked unlocked;
        return cobs_paged_tables(&c.p, cached, fresh, pages, (int32_t)n_free, count, table, cu, kv, slots, counts, s);
    });
}

// params, K, V, slot_map, k_cache, v_cache, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        Call c(a[0], a[4], "k_cache");
        int64_t ks, vs;
        const void *k = c.rows(a[1], "K", c.p.Hkv, ks), *v = c.rows(a[2], "V", c.p.Hkv, vs);
        if (ks != vs) refuse("%s must have the same token stride", "K and V");
        c.p.kv_stride = ks;
        const int32_t* slots = c.ints(a[3], "slot_map", c.p.n_tokens);
        void *kc = c.cache(a[4], "k_cache"), *vc = c.cache(a[5], "v_cache");
        const cobs_stream_t s = c.stream(a[6]);
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.dev));
        const Unlocked unlocked;
        return cobs_paged_append(&c.p, k, v, slots, kc, vc, s);
    });
}

// params, Q, k_cache, v_cache, block_table, cu_new, kv_len, O, lse or None, workspace, stream
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        Call c(a[0], a[2], "k_cache");
        int64_t qs;
        const void* q = c.rows(a[1], "Q", c.p.Hq, qs);
        c.p.q_stride = qs;
        const void *kc = c.cache(a[2], "k_cache"), *vc = c.cache(a[3], "v_cache");
        const int32_t *table = c.ints(a[4], "block_table", (long long)c.p.R * c.p.max_pages), *cu = c.ints(a[5], "cu_new", c.p.R + 1ll),
                      *kv = c.ints(a[6], "kv_len", c.p.R);
        void* o = c.flat(a[7], "O", c.elem(), (long long)c.p.n_tokens * c.p.Hq * c.p.d);
        float* lse = a[8] == Py_None ? nullptr : c.flat<float>(a[8], "lse", at::kFloat, (long long)c.p.n_tokens * c.p.Hq);
        const long long bytes = tensor_of(a[9], "workspace").numel();
        void* ws = c.flat(a[9], "workspace", at::kByte, bytes);
        const cobs_stream_t s = c.stream(a[10]);
        const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.dev));
        const Unlocked unlocked;
        return cobs_paged_attn(&c.p, q, kc, vc, table, cu, kv, o, lse, ws, (size_t)bytes, s);
    });
}

PyMethodDef methods[] = {{"tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(tables)), METH_FASTCALL, nullptr},
                         {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
                         {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attn)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module_def); }
