// torch_binding.cpp -- torch tensors into the paged-cache entry points of
// libfa.so: the work behind kv_append(), forward_paged() and
// forward_shared_prefix() of the Python package.
//
// A generation step is a few microseconds of GPU time, and the same checks,
// allocations and argument passing took 15 to 19 us per call in Python (4 to 9
// here).  The
// functions here read shapes, strides and pointers straight from the tensors,
// allocate what the caller did not give, and call the C ABI on torch's current
// stream.  They return a status code (int) where the C ABI refused, which the
// package raises as FAError.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

#include <cmath>
#include <mutex>

namespace {

using KvAppend = decltype(&fa_kv_append);
using FwdSharedPrefix = decltype(&fa_fwd_shared_prefix);
using WorkspaceBytes = decltype(&fa_fwd_shared_prefix_workspace_bytes);

// The entry points of the libfa.so that the package has loaded.
KvAppend g_kv_append = nullptr;
FwdSharedPrefix g_fwd = nullptr;
WorkspaceBytes g_workspace_bytes = nullptr;

// Calls on the default stream run one after another and share a workspace up
// to this size; another stream's calls, or a graph captured on one, may run
// beside them and get their own.
constexpr size_t kKeptWorkspace = (size_t)32 << 20;

struct Cache {
    fa_paged_kv c;
    int64_t B;
    at::ScalarType dtype;
    c10::DeviceIndex device;
    at::Tensor k, v, table, seq_len;       // what c points to
    std::mutex mutex;        // keeps the launches of two host threads' calls apart
    at::Tensor workspace;

    // Whether the tensors still have the memory that c points to (resize_() and
    // assignments to .data give a tensor another).
    bool in_place() const
    {
        return k.const_data_ptr() == c.k && v.const_data_ptr() == c.v && table.const_data_ptr() == c.table &&
               seq_len.const_data_ptr() == c.seq_len;
    }
};

constexpr const char *kCapsule = "fa_torch.cache";

void free_cache(PyObject *capsule) { delete static_cast<Cache *>(PyCapsule_GetPointer(capsule, kCapsule)); }

bool value_error(const char *text)
{
    PyErr_SetString(PyExc_ValueError, text);
    return false;
}

// Strides and base that the kernels' 16-byte accesses can follow.
bool followable(const at::Tensor &x)
{
    const auto s = x.strides();
    return s[3] == 1 && ((s[0] | s[1] | s[2]) & 7) == 0 && (reinterpret_cast<uintptr_t>(x.data_ptr()) & 15) == 0;
}

fa_rows rows_of(const at::Tensor &x)
{
    const auto s = x.strides();
    return fa_rows{x.data_ptr(), s[0], s[1], s[2]};
}

// `object` as a tensor [B, heads, T, D] of the cache (heads, T < 0: any), with
// strides that can be followed (a copy where the caller's cannot).
bool input(PyObject *object, const char *what, const Cache &cache, int64_t heads, int64_t T, at::Tensor &x)
{
    if (!THPVariable_Check(object)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        return false;
    }
    x = THPVariable_Unpack(object);
    if (x.dim() != 4 || x.size(0) != cache.B || (heads >= 0 && x.size(1) != heads) || (T >= 0 && x.size(2) != T) ||
        x.size(3) != cache.c.D) {
        PyErr_Format(PyExc_ValueError, "%s must have shape [B, heads, T, D] to match the cache: [%lld, %s, %s, %d]", what,
                     (long long)cache.B, heads >= 0 ? std::to_string(heads).c_str() : "Hq",
                     T >= 0 ? std::to_string(T).c_str() : "T", cache.c.D);
        return false;
    }
    if (x.scalar_type() != cache.dtype || !x.is_cuda() || x.get_device() != cache.device) {
        PyErr_Format(PyExc_ValueError, "%s must have the cache's dtype and device", what);
        return false;
    }
    if (!followable(x)) x = x.clone(at::MemoryFormat::Contiguous);
    return true;
}

// The caller's output like `like`, or a new one.
bool output(PyObject *object, const char *what, const at::Tensor &like, at::Tensor &x)
{
    if (object == Py_None) {
        x = at::empty(like.sizes(), at::TensorOptions().dtype(like.scalar_type()).device(like.device()));
        return true;
    }
    if (!THPVariable_Check(object)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        return false;
    }
    x = THPVariable_Unpack(object);
    if (x.sizes() != like.sizes() || x.scalar_type() != like.scalar_type() || x.device() != like.device()) {
        PyErr_Format(PyExc_ValueError, "%s must be a tensor like q", what);
        return false;
    }
    if (!followable(x)) {
        PyErr_Format(PyExc_ValueError,
                     "%s must have a contiguous last dimension, strides that are multiples of 8 and 16-byte alignment", what);
        return false;
    }
    return true;
}

// An optional one-dimensional tensor of the cache's device, made contiguous.
bool vector(PyObject *object, const char *text, at::ScalarType type, const Cache &cache, at::Tensor &x)
{
    if (!THPVariable_Check(object)) return value_error(text);
    x = THPVariable_Unpack(object);
    if (x.scalar_type() != type || x.dim() != 1 || !x.is_cuda() || x.get_device() != cache.device) return value_error(text);
    x = x.contiguous();
    return true;
}

Cache *cache_of(PyObject *capsule)
{
    Cache *cache = static_cast<Cache *>(PyCapsule_GetPointer(capsule, kCapsule));
    if (cache && !cache->in_place()) {
        value_error("a tensor of the cache has other memory than when the PagedKV was made: make a new one");
        return nullptr;
    }
    return cache;
}

// cache(address of an fa_paged_kv, k, v, table, seq_len), the four tensors that
// it points to -> capsule, which keeps them
PyObject *new_cache(PyObject *, PyObject *args)
{
    HANDLE_TH_ERRORS
    unsigned long long address;
    PyObject *x[4];
    if (!PyArg_ParseTuple(args, "KOOOO", &address, &x[0], &x[1], &x[2], &x[3])) return nullptr;
    for (PyObject *o : x)
        if (!THPVariable_Check(o)) {
            PyErr_SetString(PyExc_TypeError, "the caches, block_table and seq_len must be tensors");
            return nullptr;
        }
    const at::Tensor &k = THPVariable_Unpack(x[0]), &seq_len = THPVariable_Unpack(x[3]);
    Cache *cache = new Cache{*reinterpret_cast<const fa_paged_kv *>(address), seq_len.numel(), k.scalar_type(),
                             k.get_device(), k, THPVariable_Unpack(x[1]), THPVariable_Unpack(x[2]), seq_len, {}, {}};
    PyObject *capsule = PyCapsule_New(cache, kCapsule, free_cache);
    if (!capsule) delete cache;
    return capsule;
    END_HANDLE_TH_ERRORS
}

// kv_append(cache, k, v, q, inv_freq, interleaved, position_offset, q_out) ->
// q_out (None without q), or a status
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "kv_append takes 8 arguments");
        return nullptr;
    }
    Cache *cache = cache_of(a[0]);
    if (!cache) return nullptr;
    const c10::cuda::CUDAGuard guard(cache->device);
    at::Tensor k, v, q, q_out, freq;
    if (!input(a[1], "k", *cache, cache->c.Hkv, -1, k)) return nullptr;
    const int64_t T = k.size(2);
    if (!input(a[2], "v", *cache, cache->c.Hkv, T, v)) return nullptr;
    const bool queries = a[3] != Py_None;
    if (queries && (!input(a[3], "q", *cache, -1, T, q) || !output(a[7], "q_out", q, q_out))) return nullptr;
    if (!queries && a[7] != Py_None) {
        value_error("q_out needs q");
        return nullptr;
    }
    if (a[4] != Py_None &&
        !vector(a[4], "inv_freq must be a float32 tensor of one dimension on the cache's device", at::kFloat, *cache, freq))
        return nullptr;
    const int interleaved = PyObject_IsTrue(a[5]);
    const long long offset = PyLong_AsLongLong(a[6]);
    if (interleaved < 0 || (offset == -1 && PyErr_Occurred())) return nullptr;
    if (T > INT32_MAX || (queries && q.size(1) > INT32_MAX) || (freq.defined() && freq.numel() > INT32_MAX / 2)) {
        value_error("sizes must fit 32 bits");
        return nullptr;
    }
    const fa_rows rk = rows_of(k), rv = rows_of(v);
    fa_rows rq{}, ro{};
    if (queries) {
        rq = rows_of(q);
        ro = rows_of(q_out);
    }
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    fa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_kv_append(&cache->c, &rk, &rv, queries ? &rq : nullptr, queries ? &ro : nullptr, (int)cache->B,
                     queries ? (int)q.size(1) : 0, (int)T, freq.defined() ? freq.const_data_ptr<float>() : nullptr,
                     freq.defined() ? 2 * (int)freq.numel() : 0, interleaved, offset, cache->dtype == at::kHalf, stream);
    Py_END_ALLOW_THREADS
    if (st != FA_OK) return PyLong_FromLong(st);
    if (!queries) Py_RETURN_NONE;
    return THPVariable_Wrap(q_out);
    END_HANDLE_TH_ERRORS
}

// forward(cache, q, prefix_table, prefix_len, causal, scale, out, lse,
// return_lse, workspace) -> out or (out, lse), or a status
PyObject *forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "forward takes 10 arguments");
        return nullptr;
    }
    Cache *cache = cache_of(a[0]);
    if (!cache) return nullptr;
    const c10::cuda::CUDAGuard guard(cache->device);
    at::Tensor q, pages, out, lse, workspace;
    if (!input(a[1], "q", *cache, -1, -1, q)) return nullptr;
    const int64_t B = cache->B, Hq = q.size(1), T = q.size(2);
    if (Hq % cache->c.Hkv != 0) {
        value_error("the query heads must be a multiple of the cache's key heads");
        return nullptr;
    }
    if (Hq > INT32_MAX || T > INT32_MAX) {
        value_error("sizes must fit 32 bits");
        return nullptr;
    }
    if (a[2] != Py_None &&
        !vector(a[2], "prefix_table must be an int32 tensor of one dimension on the cache's device", at::kInt, *cache, pages))
        return nullptr;
    const long long prefix = PyLong_AsLongLong(a[3]);
    if (prefix == -1 && PyErr_Occurred()) return nullptr;
    if (prefix < 0 || prefix > (pages.defined() ? pages.numel() * cache->c.page_size : 0) || prefix > INT32_MAX) {
        value_error("prefix_len must lie in [0, what prefix_table's pages hold]");
        return nullptr;
    }
    const int causal = PyObject_IsTrue(a[4]), return_lse = PyObject_IsTrue(a[8]);
    const double scale = a[5] == Py_None ? NAN : PyFloat_AsDouble(a[5]);
    if (causal < 0 || return_lse < 0 || PyErr_Occurred()) return nullptr;
    if (!output(a[6], "out", q, out)) return nullptr;
    if (a[7] != Py_None) {
        if (!THPVariable_Check(a[7])) {
            PyErr_SetString(PyExc_TypeError, "lse must be a tensor");
            return nullptr;
        }
        lse = THPVariable_Unpack(a[7]);
        if (lse.sizes() != at::IntArrayRef({B, Hq, T}) || lse.scalar_type() != at::kFloat || lse.device() != q.device() ||
            !lse.is_contiguous()) {
            value_error("lse must be a contiguous float32 tensor [B, Hq, T] on the cache's device");
            return nullptr;
        }
    } else if (return_lse) {
        lse = at::empty({B, Hq, T}, at::TensorOptions().dtype(at::kFloat).device(q.device()));
    }
    bool kept = false;
    size_t size;
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    const auto bytes = [&](size_t count) {
        return at::empty({(int64_t)count}, at::TensorOptions().dtype(at::kByte).device(q.device()));
    };
    if (a[9] != Py_None) {
        if (!THPVariable_Check(a[9])) {
            PyErr_SetString(PyExc_TypeError, "workspace must be a tensor");
            return nullptr;
        }
        workspace = THPVariable_Unpack(a[9]);
        if (workspace.device() != q.device() || !workspace.is_contiguous()) {
            value_error("workspace must be a contiguous tensor on the cache's device");
            return nullptr;
        }
        size = workspace.nbytes();
    } else {
        size = g_workspace_bytes(&cache->c, (int)prefix, (int)B, (int)Hq, (int)T);
        kept = stream == nullptr && size <= kKeptWorkspace;
        if (!kept) workspace = bytes(size);
    }
    const fa_rows rq = rows_of(q), ro = rows_of(out);
    float *lse_ptr = lse.defined() ? lse.mutable_data_ptr<float>() : nullptr;
    const int32_t *table = pages.defined() ? pages.const_data_ptr<int32_t>() : nullptr;
    fa_status st;
    {
        // (the interpreter's lock is never waited for with the mutex held)
        struct Released {
            PyThreadState *state = PyEval_SaveThread();
            ~Released() { PyEval_RestoreThread(state); }
        } released;
        std::unique_lock<std::mutex> lock(cache->mutex, std::defer_lock);
        if (kept) {
            lock.lock();
            if (!cache->workspace.defined() || (size_t)cache->workspace.numel() < size) cache->workspace = bytes(size);
            workspace = cache->workspace;
        }
        st = g_fwd(&rq, &cache->c, table, (int)prefix, &ro, lse_ptr, (int)B, (int)Hq, (int)T, causal, (float)scale,
                   cache->dtype == at::kHalf, workspace.data_ptr(), size, stream);
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    if (!return_lse) return THPVariable_Wrap(out);
    PyObject *pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(out));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(lse));
    return pair;
    END_HANDLE_TH_ERRORS
}

// init(addresses of fa_kv_append, fa_fwd_shared_prefix and
// fa_fwd_shared_prefix_workspace_bytes)
PyObject *init(PyObject *, PyObject *args)
{
    unsigned long long x, y, z;
    if (!PyArg_ParseTuple(args, "KKK", &x, &y, &z)) return nullptr;
    g_kv_append = reinterpret_cast<KvAppend>(x);
    g_fwd = reinterpret_cast<FwdSharedPrefix>(y);
    g_workspace_bytes = reinterpret_cast<WorkspaceBytes>(z);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"cache", new_cache, METH_VARARGS, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(forward)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_torch() { return PyModule_Create(&g_module); }
