// torch_binding.cpp -- torch tensors into the paged-cache entry points of
// libfa.so: the work behind kv_append(), forward_paged(), forward_shared_prefix(),
// kv_read(), rotary() and the page operators of the Python package.
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
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

#include <array>
#include <cmath>
#include <mutex>
#include <optional>
#include <tuple>
#include <vector>

namespace {

// The entry points of the libfa.so that the package has loaded.
decltype(&fa_kv_append_at) g_kv_append = nullptr;
decltype(&fa_kv_append_q4) g_kv_append_q4 = nullptr;
decltype(&fa_fwd_shared_prefix) g_fwd = nullptr;
decltype(&fa_fwd_shared_prefix_workspace_bytes) g_workspace_bytes = nullptr;
decltype(&fa_fwd_paged_q4) g_fwd_q4 = nullptr;
decltype(&fa_fwd_paged_q4_workspace_bytes) g_workspace_bytes_q4 = nullptr;
decltype(&fa_kv_read) g_kv_read = nullptr;
decltype(&fa_kv_read_q4) g_kv_read_q4 = nullptr;
decltype(&fa_rotary) g_rotary = nullptr;
decltype(&fa_pages_workspace_bytes) g_pages_bytes = nullptr;
decltype(&fa_kv_grow) g_grow = nullptr;
decltype(&fa_kv_free) g_free = nullptr;
decltype(&fa_kv_fork) g_fork = nullptr;
decltype(&fa_kv_compact) g_compact = nullptr;
decltype(&fa_copy_pages) g_copy = nullptr;
decltype(&fa_copy_pages_q4) g_copy_q4 = nullptr;

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
    bool four = false;                     // a 4-bit cache: c4, and c's sizes and table
    fa_paged_kv4 c4{};
    at::Tensor ks, vs;
    std::mutex mutex;        // keeps the launches of two host threads' calls apart
    at::Tensor workspace;

    // Whether the tensors still have the memory that c points to (resize_() and
    // assignments to .data give a tensor another).
    bool in_place() const
    {
        return k.const_data_ptr() == c.k && v.const_data_ptr() == c.v && table.const_data_ptr() == c.table &&
               seq_len.const_data_ptr() == c.seq_len &&
               (!four || (ks.const_data_ptr() == c4.k_scales && vs.const_data_ptr() == c4.v_scales));
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
                             k.get_device(), k, THPVariable_Unpack(x[1]), THPVariable_Unpack(x[2]), seq_len};
    PyObject *capsule = PyCapsule_New(cache, kCapsule, free_cache);
    if (!capsule) delete cache;
    return capsule;
    END_HANDLE_TH_ERRORS
}

// cache4(address of an fa_paged_kv4, k, v, k_scales, v_scales, table, seq_len, whether
// queries are fp16) -> capsule
PyObject *new_cache4(PyObject *, PyObject *args)
{
    HANDLE_TH_ERRORS
    unsigned long long address;
    PyObject *x[6];
    int f16;
    if (!PyArg_ParseTuple(args, "KOOOOOOp", &address, &x[0], &x[1], &x[2], &x[3], &x[4], &x[5], &f16)) return nullptr;
    for (PyObject *o : x)
        if (!THPVariable_Check(o)) {
            PyErr_SetString(PyExc_TypeError, "the caches, scales, block_table and seq_len must be tensors");
            return nullptr;
        }
    const fa_paged_kv4 &c4 = *reinterpret_cast<const fa_paged_kv4 *>(address);
    fa_paged_kv c{};
    c.k = c4.k;
    c.v = c4.v;
    c.num_pages = c4.num_pages;
    c.page_size = c4.page_size;
    c.Hkv = c4.Hkv;
    c.D = c4.D;
    c.table = c4.table;
    c.table_stride = c4.table_stride;
    c.table_width = c4.table_width;
    c.seq_len = c4.seq_len;
    const at::Tensor &k = THPVariable_Unpack(x[0]), &seq_len = THPVariable_Unpack(x[5]);
    Cache *cache = new Cache{c, seq_len.numel(), f16 ? at::kHalf : at::kBFloat16, k.get_device(), k, THPVariable_Unpack(x[1]),
                             THPVariable_Unpack(x[4]), seq_len, true, c4, THPVariable_Unpack(x[2]), THPVariable_Unpack(x[3])};
    PyObject *capsule = PyCapsule_New(cache, kCapsule, free_cache);
    if (!capsule) delete cache;
    return capsule;
    END_HANDLE_TH_ERRORS
}

// Positions and the axes of the pairs (either may be None) of tokens [B, T] on a device.
struct Positions {
    at::Tensor n, pair_axis;
    fa_positions p{};
    const fa_positions *get() const { return n.defined() ? &p : nullptr; }
};

bool positions_of(PyObject *object, PyObject *axes, int64_t B, int64_t T, int64_t pairs, const at::Device &device, Positions &x)
{
    if (object == Py_None) return axes == Py_None || value_error("pair_axis needs positions");
    if (!THPVariable_Check(object)) {
        PyErr_SetString(PyExc_TypeError, "positions must be a tensor");
        return false;
    }
    x.n = THPVariable_Unpack(object);
    const int64_t d = x.n.dim();
    if (x.n.scalar_type() != at::kInt || x.n.device() != device || (d != 2 && d != 3) || x.n.size(d - 2) != B ||
        x.n.size(d - 1) != T || (d == 3 && (x.n.size(0) < 1 || x.n.size(0) > INT32_MAX)))
        return value_error("positions must be an int32 tensor [B, T] or [axes, B, T] on the same device");
    x.p.n = x.n.const_data_ptr<int32_t>();
    x.p.axes = d == 3 ? (int)x.n.size(0) : 1;
    x.p.stride_axis = d == 3 ? x.n.stride(0) : 0;
    x.p.stride_b = x.n.stride(d - 2);
    x.p.stride_t = x.n.stride(d - 1);
    if (axes == Py_None) return x.p.axes == 1 || value_error("positions of several axes need pair_axis");
    if (!THPVariable_Check(axes)) {
        PyErr_SetString(PyExc_TypeError, "pair_axis must be a tensor");
        return false;
    }
    x.pair_axis = THPVariable_Unpack(axes);
    if (x.pair_axis.scalar_type() != at::kInt || x.pair_axis.dim() != 1 || x.pair_axis.numel() != pairs || x.pair_axis.device() != device)
        return value_error("pair_axis must be an int32 tensor with an entry for each of inv_freq's, on the same device");
    x.pair_axis = x.pair_axis.contiguous();
    x.p.pair_axis = x.pair_axis.const_data_ptr<int32_t>();
    return true;
}

// kv_append(cache, k, v, q, inv_freq, interleaved, position_offset, q_out, positions,
// pair_axis) -> q_out (None without q), or a status
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "kv_append takes 10 arguments");
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
    Positions positions;
    if (!positions_of(a[8], a[9], cache->B, T, freq.defined() ? freq.numel() : 0, k.device(), positions)) return nullptr;
    const fa_rows rk = rows_of(k), rv = rows_of(v);
    fa_rows rq{}, ro{};
    if (queries) {
        rq = rows_of(q);
        ro = rows_of(q_out);
    }
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    fa_status st;
    Py_BEGIN_ALLOW_THREADS
    const auto run = [&](auto call, auto *c) {
        return call(c, &rk, &rv, queries ? &rq : nullptr, queries ? &ro : nullptr, (int)cache->B, queries ? (int)q.size(1) : 0,
                    (int)T, freq.defined() ? freq.const_data_ptr<float>() : nullptr, freq.defined() ? 2 * (int)freq.numel() : 0,
                    interleaved, positions.get(), offset, cache->dtype == at::kHalf, stream);
    };
    st = cache->four ? run(g_kv_append_q4, &cache->c4) : run(g_kv_append, &cache->c);
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
    if (cache->four && pages.defined()) {
        value_error("a 4-bit cache takes no prefix_table: the sequences' tables may share a prefix's pages");
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
        size = cache->four ? g_workspace_bytes_q4(&cache->c4, (int)B, (int)Hq, (int)T)
                           : g_workspace_bytes(&cache->c, (int)prefix, (int)B, (int)Hq, (int)T);
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
        const int f16 = cache->dtype == at::kHalf;
        st = cache->four ? g_fwd_q4(&rq, &cache->c4, &ro, lse_ptr, (int)B, (int)Hq, (int)T, causal, (float)scale, f16,
                                    workspace.data_ptr(), size, stream)
                         : g_fwd(&rq, &cache->c, table, (int)prefix, &ro, lse_ptr, (int)B, (int)Hq, (int)T, causal,
                                 (float)scale, f16, workspace.data_ptr(), size, stream);
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

// kv_read(cache, T) -> (k, v), or a status
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "kv_read takes 2 arguments");
        return nullptr;
    }
    Cache *cache = cache_of(a[0]);
    if (!cache) return nullptr;
    const long long T = PyLong_AsLongLong(a[1]);
    if (T == -1 && PyErr_Occurred()) return nullptr;
    if (T < 0 || T > INT32_MAX) {
        value_error("T must lie in [0, 2^31)");
        return nullptr;
    }
    const c10::cuda::CUDAGuard guard(cache->device);
    const auto like = at::TensorOptions().dtype(cache->dtype).device(cache->k.device());
    at::Tensor k = at::empty({cache->B, cache->c.Hkv, T, cache->c.D}, like), v = at::empty_like(k);
    const fa_rows rk = rows_of(k), rv = rows_of(v);
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    fa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = cache->four ? g_kv_read_q4(&cache->c4, &rk, &rv, (int)cache->B, (int)T, cache->dtype == at::kHalf, stream)
                     : g_kv_read(&cache->c, &rk, &rv, (int)cache->B, (int)T, stream);
    Py_END_ALLOW_THREADS
    if (st != FA_OK) return PyLong_FromLong(st);
    PyObject *pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(v));
    return pair;
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- rotation
// What the C ABI refused.
struct Refused {
    fa_status status;
};

// q and k (either may be undefined) turned; the arguments have been checked.
struct Turn {
    at::Tensor freq, n, pair_axis;
    bool interleaved, inverse;
    int64_t offset;

    std::array<at::Tensor, 2> operator()(std::array<at::Tensor, 2> x) const
    {
        std::array<at::Tensor, 2> y;
        fa_rows in[2]{}, out[2]{};
        int heads[2]{};
        const at::Tensor &first = x[0].defined() ? x[0] : x[1];
        const c10::cuda::CUDAGuard guard(first.device());
        for (int i = 0; i < 2; ++i) {
            if (!x[i].defined()) continue;
            // (a tangent of zeros may have no memory)
            if (x[i]._is_zerotensor() || !followable(x[i])) x[i] = x[i].clone(at::MemoryFormat::Contiguous);
            y[i] = at::empty(x[i].sizes(), at::TensorOptions().dtype(x[i].scalar_type()).device(x[i].device()));
            in[i] = rows_of(x[i]);
            out[i] = rows_of(y[i]);
            heads[i] = (int)x[i].size(1);
        }
        fa_positions p{};
        if (n.defined()) {
            const int64_t d = n.dim();
            p = fa_positions{n.const_data_ptr<int32_t>(), d == 3 ? n.stride(0) : 0, n.stride(d - 2), n.stride(d - 1),
                             d == 3 ? (int)n.size(0) : 1, pair_axis.defined() ? pair_axis.const_data_ptr<int32_t>() : nullptr};
        }
        const at::Tensor &like = x[0].defined() ? x[0] : x[1];
        const fa_status st = g_rotary(&in[0], &out[0], &in[1], &out[1], (int)like.size(0), heads[0], heads[1], (int)like.size(2),
                                      (int)like.size(3), freq.const_data_ptr<float>(), 2 * (int)freq.numel(), interleaved,
                                      n.defined() ? &p : nullptr, offset, inverse, like.scalar_type() == at::kHalf,
                                      c10::cuda::getCurrentCUDAStream(like.get_device()).stream());
        if (st != FA_OK) throw Refused{st};
        return y;
    }
};

std::array<at::Tensor, 2> turned(const std::array<at::Tensor, 2> &x, const Turn &turn);

// The same as an operation whose gradient turns back.  (The first tensor is defined.)
struct Rotary : torch::autograd::Function<Rotary> {
    static torch::autograd::variable_list forward(torch::autograd::AutogradContext *ctx, const at::Tensor &a,
                                                  const std::optional<at::Tensor> &b, const Turn &turn)
    {
        ctx->set_materialize_grads(false);
        torch::autograd::variable_list saved{turn.freq};
        if (turn.n.defined()) saved.push_back(turn.n);
        if (turn.pair_axis.defined()) saved.push_back(turn.pair_axis);
        ctx->save_for_backward(saved);
        ctx->saved_data["how"] = (int64_t)turn.interleaved | (int64_t)turn.inverse << 1;
        ctx->saved_data["offset"] = turn.offset;
        const auto y = turn({a, b.value_or(at::Tensor())});
        torch::autograd::variable_list out{y[0]};
        if (b.has_value()) out.push_back(y[1]);
        return out;
    }

    static torch::autograd::variable_list backward(torch::autograd::AutogradContext *ctx, torch::autograd::variable_list d)
    {
        torch::autograd::variable_list grads(3);
        std::vector<int> which;
        for (int i = 0; i < (int)d.size(); ++i)
            if (d[i].defined()) which.push_back(i);
        if (which.empty()) return grads;
        const auto saved = ctx->get_saved_variables();
        const int64_t how = ctx->saved_data["how"].toInt();
        const Turn back{saved[0], saved.size() > 1 ? saved[1] : at::Tensor(), saved.size() > 2 ? saved[2] : at::Tensor(),
                        (how & 1) != 0, (how & 2) == 0, ctx->saved_data["offset"].toInt()};
        try {
            const auto y = turned({d[which[0]], which.size() > 1 ? d[which[1]] : at::Tensor()}, back);
            for (size_t i = 0; i < which.size(); ++i) grads[which[i]] = y[i];
        } catch (const Refused &r) {
            TORCH_CHECK(false, "the gradient of rotary: status ", (int)r.status);
        }
        return grads;
    }
};

// q and k (either may be undefined) turned, differentiable both ways: through Rotary
// where a gradient may be asked for, and a forward-mode tangent turns as its tensor
// does, since the operation is linear.
std::array<at::Tensor, 2> turned(const std::array<at::Tensor, 2> &x, const Turn &turn)
{
    const auto is_dual = [](const at::Tensor &t) { return t.defined() && t._fw_grad(0).defined(); };
    if (is_dual(x[0]) || is_dual(x[1])) {
        std::array<at::Tensor, 2> value = x, tangent;
        for (int i = 0; i < 2; ++i)
            if (is_dual(x[i])) std::tie(value[i], tangent[i]) = at::_unpack_dual(x[i], 0);
        auto y = turned(value, turn);
        const auto t = turned(tangent, turn);
        for (int i = 0; i < 2; ++i)
            if (t[i].defined()) y[i] = at::_make_dual(y[i], t[i], 0);
        return y;
    }
    const auto asks = [](const at::Tensor &t) { return t.defined() && t.requires_grad(); };
    if (!at::GradMode::is_enabled() || !(asks(x[0]) || asks(x[1]))) return turn(x);
    const int first = x[0].defined() ? 0 : 1;
    const bool both = first == 0 && x[1].defined();
    const auto r = Rotary::apply(x[first], both ? std::optional<at::Tensor>(x[1]) : std::nullopt, turn);
    std::array<at::Tensor, 2> y;
    y[first] = r[0];
    if (both) y[1] = r[1];
    return y;
}

// rotary(q, k or None, inv_freq, positions, pair_axis, interleaved, position_offset) ->
// (q, k or None) turned, or a status
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "rotary takes 7 arguments");
        return nullptr;
    }
    at::Tensor x[2];
    const at::Tensor *first = &x[0];
    for (int i = 0; i < 2; ++i) {
        if (i == 1 && a[i] == Py_None) continue;
        if (!THPVariable_Check(a[i])) {
            PyErr_SetString(PyExc_TypeError, "q and k must be tensors");
            return nullptr;
        }
        x[i] = THPVariable_Unpack(a[i]);
        if (!x[i].is_cuda() || x[i].dim() != 4 || (x[i].scalar_type() != at::kHalf && x[i].scalar_type() != at::kBFloat16)) {
            value_error("q and k must be bf16 or fp16 CUDA tensors [B, heads, T, D]");
            return nullptr;
        }
        if (x[i].scalar_type() != first->scalar_type() || x[i].device() != first->device() || x[i].size(0) != first->size(0) ||
            x[i].size(2) != first->size(2) || x[i].size(3) != first->size(3)) {
            value_error("q and k must share dtype, device, B, T and D");
            return nullptr;
        }
        for (int d = 0; d < 4; ++d)
            if (x[i].size(d) > INT32_MAX) {
                value_error("sizes must fit 32 bits");
                return nullptr;
            }
    }
    if (!THPVariable_Check(a[2])) {
        PyErr_SetString(PyExc_TypeError, "inv_freq must be a tensor");
        return nullptr;
    }
    at::Tensor freq = THPVariable_Unpack(a[2]);
    if (freq.scalar_type() != at::kFloat || freq.dim() != 1 || freq.device() != first->device() || freq.numel() > INT32_MAX / 2) {
        value_error("inv_freq must be a float32 tensor of one dimension on the device of q and k");
        return nullptr;
    }
    // (a gradient that is asked for must not be missed without a word)
    if ((at::GradMode::is_enabled() && freq.requires_grad()) || freq._fw_grad(0).defined()) {
        value_error("rotary gives inv_freq no gradient: pass inv_freq.detach()");
        return nullptr;
    }
    const c10::cuda::CUDAGuard guard(first->device());
    freq = freq.contiguous();
    Positions positions;
    if (!positions_of(a[3], a[4], first->size(0), first->size(2), freq.numel(), first->device(), positions)) return nullptr;
    const int interleaved = PyObject_IsTrue(a[5]);
    const long long offset = PyLong_AsLongLong(a[6]);
    if (interleaved < 0 || (offset == -1 && PyErr_Occurred())) return nullptr;
    std::array<at::Tensor, 2> y;
    fa_status st = FA_OK;
    {
        struct Released {
            PyThreadState *state = PyEval_SaveThread();
            ~Released() { PyEval_RestoreThread(state); }
        } released;
        try {
            const Turn turn{freq.detach(), positions.n, positions.pair_axis, interleaved != 0, false, offset};
            y = turned({x[0], x[1]}, turn);
        } catch (const Refused &r) {
            st = r.status;
        }
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    PyObject *pair = PyTuple_New(2);
    if (!pair) return nullptr;
    for (int i = 0; i < 2; ++i) PyTuple_SET_ITEM(pair, i, y[i].defined() ? THPVariable_Wrap(y[i]) : Py_NewRef(Py_None));
    return pair;
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- pages
// An int32 vector of the cache's device, of `count` entries (< 0: any), contiguous.
bool entries(PyObject *object, const char *what, int64_t count, const Cache &cache, bool written, at::Tensor &x)
{
    if (!THPVariable_Check(object)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        return false;
    }
    x = THPVariable_Unpack(object);
    if (x.scalar_type() != at::kInt || x.dim() != 1 || !x.is_cuda() || x.get_device() != cache.device ||
        (count >= 0 && x.numel() != count) || x.numel() > INT32_MAX || (written && !x.is_contiguous())) {
        if (count >= 0)
            PyErr_Format(PyExc_ValueError, "%s must be a%s int32 tensor with %lld entries on the cache's device", what,
                         written ? " contiguous" : "n", (long long)count);
        else
            PyErr_Format(PyExc_ValueError, "%s must be an int32 tensor of one dimension on the cache's device", what);
        return false;
    }
    x = x.contiguous();
    return true;
}

bool table_of(const Cache &cache, PyObject *refs, at::Tensor &counts, fa_page_table &t)
{
    if (!entries(refs, "refs", cache.c.num_pages, cache, true, counts)) return false;
    t = fa_page_table{const_cast<int32_t *>(cache.c.table), cache.c.table_stride, cache.c.table_width, (int)cache.B,
                      const_cast<int32_t *>(cache.c.seq_len), counts.mutable_data_ptr<int32_t>(), cache.c.num_pages, cache.c.page_size};
    return true;
}

at::Tensor numbers(const Cache &cache, int64_t n)
{
    return at::empty({n}, at::TensorOptions().dtype(at::kInt).device(cache.k.device()));
}

// run(workspace, bytes, more) with a workspace of a page operator and `extra` bytes
// more behind it, the interpreter's lock released: the cache's own on the default
// stream, else a new one.
template <typename Run>
fa_status with_workspace(Cache &cache, const fa_page_table &t, int n, size_t extra, void *stream, const Run &run)
{
    const size_t size = g_pages_bytes(&t, n);
    const auto bytes = [&] { return at::empty({(int64_t)(size + extra)}, at::TensorOptions().dtype(at::kByte).device(cache.k.device())); };
    const bool kept = stream == nullptr && size + extra <= kKeptWorkspace;
    at::Tensor workspace;
    if (!kept) workspace = bytes();
    struct Released {
        PyThreadState *state = PyEval_SaveThread();
        ~Released() { PyEval_RestoreThread(state); }
    } released;
    std::unique_lock<std::mutex> lock(cache.mutex, std::defer_lock);
    if (kept) {
        lock.lock();
        if (!cache.workspace.defined() || (size_t)cache.workspace.numel() < size + extra) cache.workspace = bytes();
        workspace = cache.workspace;
    }
    uint8_t *w = static_cast<uint8_t *>(workspace.data_ptr());
    return run(w, size, reinterpret_cast<int32_t *>(w + size));        // (size is a multiple of 256)
}

// The caches in a tuple (a model's layers, whose pools are of one size and whose table
// is the first's); false with an error set.
bool layers_of(PyObject *object, std::vector<Cache *> &all)
{
    if (!PyTuple_Check(object) || PyTuple_GET_SIZE(object) == 0) return value_error("at least one cache must be given");
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(object); ++i) {
        Cache *c = cache_of(PyTuple_GET_ITEM(object, i));
        if (!c) return false;
        all.push_back(c);
    }
    return true;
}

// Whether every cache's pages can be copied, known before the table changes (no pairs: the
// C ABI's checks alone).
fa_status check_copies(const std::vector<Cache *> &all)
{
    for (const Cache *c : all) {
        const fa_status st = c->four ? g_copy_q4(&c->c4, nullptr, nullptr, nullptr, 0, nullptr) : g_copy(&c->c, nullptr, nullptr, nullptr, 0, nullptr);
        if (st != FA_OK) return st;
    }
    return FA_OK;
}

// The pages that a call listed, in every cache.
fa_status copy_listed(const std::vector<Cache *> &all, const int32_t *src, const int32_t *dst, const int32_t *count, int n, void *stream)
{
    for (Cache *c : all) {
        const fa_status st = c->four ? g_copy_q4(&c->c4, src, dst, count, n, stream) : g_copy(&c->c, src, dst, count, n, stream);
        if (st != FA_OK) return st;
    }
    return FA_OK;
}

// grow(cache, refs, tokens) -> taken, or a status
PyObject *grow(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Cache *cache = n == 3 ? cache_of(a[0]) : nullptr;
    if (!cache) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_TypeError, "grow takes 3 arguments"), nullptr);
    const c10::cuda::CUDAGuard guard(cache->device);
    at::Tensor refs, tokens;
    fa_page_table t;
    if (!table_of(*cache, a[1], refs, t) || !entries(a[2], "tokens", cache->B, *cache, false, tokens)) return nullptr;
    at::Tensor taken = numbers(*cache, cache->B);
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    const fa_status st = with_workspace(*cache, t, 0, 0, stream, [&](void *w, size_t size, int32_t *) {
        return g_grow(&t, tokens.const_data_ptr<int32_t>(), taken.mutable_data_ptr<int32_t>(), w, size, stream);
    });
    return st != FA_OK ? PyLong_FromLong(st) : THPVariable_Wrap(taken);
    END_HANDLE_TH_ERRORS
}

// free(cache, refs, rows) -> status
PyObject *free_rows(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Cache *cache = n == 3 ? cache_of(a[0]) : nullptr;
    if (!cache) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_TypeError, "free takes 3 arguments"), nullptr);
    const c10::cuda::CUDAGuard guard(cache->device);
    at::Tensor refs, rows;
    fa_page_table t;
    if (!table_of(*cache, a[1], refs, t) || !entries(a[2], "rows", -1, *cache, false, rows)) return nullptr;
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    return PyLong_FromLong(g_free(&t, rows.const_data_ptr<int32_t>(), (int)rows.numel(), stream));
    END_HANDLE_TH_ERRORS
}

// fork(caches, refs, parent, child) -> the pages that were copied to, or a status
PyObject *fork_rows(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    std::vector<Cache *> all;
    if (n != 4) return PyErr_SetString(PyExc_TypeError, "fork takes 4 arguments"), nullptr;
    if (!layers_of(a[0], all)) return nullptr;
    Cache *cache = all[0];
    const c10::cuda::CUDAGuard guard(cache->device);
    at::Tensor refs, parent, child;
    fa_page_table t;
    if (!table_of(*cache, a[1], refs, t) || !entries(a[2], "parent", -1, *cache, false, parent) ||
        !entries(a[3], "child", parent.numel(), *cache, false, child))
        return nullptr;
    const fa_status copies = check_copies(all);
    if (copies != FA_OK) return PyLong_FromLong(copies);
    const int count = (int)parent.numel();
    at::Tensor dst = numbers(*cache, count);
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    const fa_status st = with_workspace(*cache, t, count, 4 * (size_t)count, stream, [&](void *w, size_t size, int32_t *src) {
        const fa_status s = g_fork(&t, parent.const_data_ptr<int32_t>(), child.const_data_ptr<int32_t>(), count, src,
                                   dst.mutable_data_ptr<int32_t>(), w, size, stream);
        return s != FA_OK ? s : copy_listed(all, src, dst.const_data_ptr<int32_t>(), nullptr, count, stream);
    });
    return st != FA_OK ? PyLong_FromLong(st) : THPVariable_Wrap(dst);
    END_HANDLE_TH_ERRORS
}

// compact(caches, refs) -> moved, or a status
PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    std::vector<Cache *> all;
    if (n != 2) return PyErr_SetString(PyExc_TypeError, "compact takes 2 arguments"), nullptr;
    if (!layers_of(a[0], all)) return nullptr;
    Cache *cache = all[0];
    const c10::cuda::CUDAGuard guard(cache->device);
    at::Tensor refs;
    fa_page_table t;
    if (!table_of(*cache, a[1], refs, t)) return nullptr;
    const fa_status copies = check_copies(all);
    if (copies != FA_OK) return PyLong_FromLong(copies);
    const int pages = cache->c.num_pages;
    at::Tensor moved = numbers(*cache, pages);
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    const fa_status st = with_workspace(*cache, t, 0, 8 * (size_t)pages + 4, stream, [&](void *w, size_t size, int32_t *src) {
        int32_t *dst = src + pages, *count = dst + pages;
        const fa_status s = g_compact(&t, moved.mutable_data_ptr<int32_t>(), src, dst, count, w, size, stream);
        return s != FA_OK ? s : copy_listed(all, src, dst, count, pages, stream);
    });
    return st != FA_OK ? PyLong_FromLong(st) : THPVariable_Wrap(moved);
    END_HANDLE_TH_ERRORS
}

// copy_pages(cache, src, dst, count) -> status
PyObject *copy_pages(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Cache *cache = n == 4 ? cache_of(a[0]) : nullptr;
    if (!cache) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_TypeError, "copy_pages takes 4 arguments"), nullptr);
    const c10::cuda::CUDAGuard guard(cache->device);
    at::Tensor src, dst, count;
    if (!entries(a[1], "src", -1, *cache, false, src) || !entries(a[2], "dst", src.numel(), *cache, false, dst)) return nullptr;
    if (a[3] != Py_None && !entries(a[3], "count", 1, *cache, false, count)) return nullptr;
    const int32_t *m = count.defined() ? count.const_data_ptr<int32_t>() : nullptr;
    void *stream = c10::cuda::getCurrentCUDAStream(cache->device).stream();
    const auto run = [&](auto call, auto *c) {
        return call(c, src.const_data_ptr<int32_t>(), dst.const_data_ptr<int32_t>(), m, (int)src.numel(), stream);
    };
    return PyLong_FromLong(cache->four ? run(g_copy_q4, &cache->c4) : run(g_copy, &cache->c));
    END_HANDLE_TH_ERRORS
}

// init(addresses of the entry points, in the order below)
PyObject *init(PyObject *, PyObject *args)
{
    unsigned long long x[16];
    if (!PyArg_ParseTuple(args, "KKKKKKKKKKKKKKKK", &x[0], &x[1], &x[2], &x[3], &x[4], &x[5], &x[6], &x[7], &x[8], &x[9],
                          &x[10], &x[11], &x[12], &x[13], &x[14], &x[15]))
        return nullptr;
    int i = 0;
    const auto put = [&](auto &f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(x[i++]); };
    put(g_kv_append);
    put(g_kv_append_q4);
    put(g_fwd);
    put(g_workspace_bytes);
    put(g_fwd_q4);
    put(g_workspace_bytes_q4);
    put(g_kv_read);
    put(g_kv_read_q4);
    put(g_rotary);
    put(g_pages_bytes);
    put(g_grow);
    put(g_free);
    put(g_fork);
    put(g_compact);
    put(g_copy);
    put(g_copy_q4);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"cache", new_cache, METH_VARARGS, nullptr},
    {"cache4", new_cache4, METH_VARARGS, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(forward)), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_read)), METH_FASTCALL, nullptr},
    {"rotary", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotary)), METH_FASTCALL, nullptr},
    {"grow", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grow)), METH_FASTCALL, nullptr},
    {"free", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(free_rows)), METH_FASTCALL, nullptr},
    {"fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fork_rows)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(compact)), METH_FASTCALL, nullptr},
    {"copy_pages", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(copy_pages)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fa_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_torch() { return PyModule_Create(&g_module); }
