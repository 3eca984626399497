// fa_cache_py.cpp -- the usual call of the paged caches', the page plan's and the
// rotary positions' Python functions, in C++: the same checks as cache.py, cache4.py,
// pages.py and rope.py of the package, the outputs' allocation and the call of the C
// ABI.  A call that is anything but usual (a stream of its own, another device than the
// current one, an argument that does not pass) is handed back, and the Python function
// goes through it, which also words the error.  What it saves is time on the host, which is most of a small call: a
// fa_decode_cache of one sequence of 500 keys takes 9.7 us in place of 26 (8.4 of
// them on the GPU), a fa_cache_write of one token 4.2 in place of 12, a choice of
// pages and the attention over them 22 in place of 55, a fa_rope of one token 5.1
// (2.1 on the GPU), a fa_cache4_write of a step 2.7.
//
// A CPython module without state but the addresses of the library's functions,
// which cache.py sets (bind), so that either build of the library can be used.
// It says which ABI and which torch it was compiled for; cache.py binds it only
// where both are those it runs with.
#include <Python.h>

#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

struct Library {
    decltype(&fa_cache_write) write;
    decltype(&fa_cache_read) read;
    decltype(&fa_decode_cache) decode;
    decltype(&fa_decode_cache_workspace_size) decode_workspace;
    decltype(&fa_cache_select) select;
    decltype(&fa_cache_select_workspace_size) select_workspace;
    decltype(&fa_cache4_write) write4;
    decltype(&fa_cache4_read) read4;
    decltype(&fa_decode_cache4) decode4;
    decltype(&fa_decode_cache4_workspace_size) decode4_workspace;
    decltype(&fa_cache_plan) plan;
    decltype(&fa_cache_trim) trim;
    decltype(&fa_rope) rope;
};
Library lib = {};

using at::ScalarType;
using at::Tensor;

// A plain tensor of the current device, or NULL.
const Tensor *plain(PyObject *o, int device)
{
    if (!THPVariable_CheckExact(o))
        return nullptr;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || t.get_device() != device || t.is_conj() || t.is_neg())
        return nullptr;
    return &t;
}

// ... contiguous, of a type and shape.
const Tensor *exact(PyObject *o, int device, ScalarType type, at::IntArrayRef shape)
{
    const Tensor *t = plain(o, device);
    return t && t->scalar_type() == type && t->sizes() == shape && t->is_contiguous() ? t : nullptr;
}

bool to_int(int64_t x, int &out)
{
    out = static_cast<int>(x);
    return x >= 0 && x <= 0x7fffffff;
}

bool describe(PyObject *cache, int device, fa_cache_t &c)
{
    if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 6)
        return false;
    const Tensor *k = plain(PyTuple_GET_ITEM(cache, 0), device);
    if (!k || k->dim() != 4 || !k->is_contiguous())
        return false;
    if (k->scalar_type() == at::kFloat8_e4m3fn)
        c.format = FA_E4M3;
    else if (k->scalar_type() == at::kChar)
        c.format = FA_INT8;
    else
        return false;
    const int64_t pair[2] = {k->size(0), k->size(1)}, mean[3] = {k->size(0), k->size(1), k->size(3)};
    const Tensor *v = exact(PyTuple_GET_ITEM(cache, 1), device, k->scalar_type(), k->sizes());
    const Tensor *ks = exact(PyTuple_GET_ITEM(cache, 2), device, at::kFloat, pair);
    const Tensor *vs = exact(PyTuple_GET_ITEM(cache, 3), device, at::kFloat, pair);
    if (!v || !ks || !vs || !to_int(k->size(0), c.num_pages) || !to_int(k->size(1), c.heads) ||
        !to_int(k->size(2), c.page) || !to_int(k->size(3), c.d))
        return false;
    c.k = k->data_ptr();
    c.v = v->data_ptr();
    c.k_scale = static_cast<float *>(ks->data_ptr());
    c.v_scale = static_cast<float *>(vs->data_ptr());
    c.k_mean = nullptr;
    c.k_mean_scale = nullptr;
    if (PyTuple_GET_ITEM(cache, 4) != Py_None || PyTuple_GET_ITEM(cache, 5) != Py_None) {
        const Tensor *m = exact(PyTuple_GET_ITEM(cache, 4), device, at::kChar, mean);
        const Tensor *ms = exact(PyTuple_GET_ITEM(cache, 5), device, at::kFloat, pair);
        if (!m || !ms)
            return false;
        c.k_mean = static_cast<signed char *>(m->data_ptr());
        c.k_mean_scale = static_cast<float *>(ms->data_ptr());
    }
    return true;
}

struct Batch {
    const int *lens, *table;
    long long stride;
    int pages, B;
};

bool describe_batch(PyObject *table, PyObject *lens, int device, Batch &b)
{
    const Tensor *t = plain(table, device), *n = plain(lens, device);
    if (!t || !n || t->dim() != 2 || n->dim() != 1 || t->scalar_type() != at::kInt || n->scalar_type() != at::kInt ||
        t->size(0) != n->size(0) || (t->size(1) > 1 && t->stride(1) != 1) || !n->is_contiguous() ||
        !to_int(t->size(0), b.B) || !to_int(t->size(1), b.pages))
        return false;
    b.lens = static_cast<const int *>(n->data_ptr());
    b.table = static_cast<const int *>(t->data_ptr());
    b.stride = b.B > 1 ? t->stride(0) : b.pages;
    return true;
}

// Rows of d contiguous 16-bit values.
const Tensor *rows(PyObject *o, int device, int dim, int d, fa_dtype_t &type)
{
    const Tensor *t = plain(o, device);
    if (!t || t->dim() != dim || t->size(dim - 1) != d || (t->stride(dim - 1) != 1 && t->numel() != 0))
        return nullptr;
    if (t->scalar_type() == at::kHalf)
        type = FA_FP16;
    else if (t->scalar_type() == at::kBFloat16)
        type = FA_BF16;
    else
        return nullptr;
    return t;
}

ScalarType scalar_of(fa_dtype_t type) { return type == FA_FP16 ? at::kHalf : at::kBFloat16; }

Tensor empty(at::IntArrayRef shape, ScalarType type, int device)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<int8_t>(device))));
}

// The caller's output or workspace if given, else a new one; false if it does not fit.
bool output(PyObject *given, at::IntArrayRef shape, ScalarType type, int device, Tensor &t)
{
    if (given == Py_None) {
        t = empty(shape, type, device);
        return true;
    }
    const Tensor *g = exact(given, device, type, shape);
    if (!g)
        return false;
    t = *g;
    return true;
}
// A contiguous tensor of its own at an element of a buffer's memory.  An allocation is 1.2 us
// of a small call; the outputs of one share theirs, up to kShared elements (two that are larger
// are worth having apart: either may be freed before the other).
constexpr int64_t kShared = 1 << 18;
Tensor part(const Tensor &buffer, int64_t at, at::IntArrayRef shape)
{
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(), buffer.dtype());
    impl->set_storage_offset(at);
    impl->set_sizes_contiguous(shape);
    return Tensor(std::move(impl));
}
int64_t up_to_128(int64_t n) { return (n + 127) / 128 * 128; }  // 256 bytes of the smallest type here

// Two outputs of one type, new ones or the caller's; false if one does not fit.
bool outputs(PyObject *const (&given)[2], at::IntArrayRef shape0, at::IntArrayRef shape1, ScalarType type, int device,
             Tensor (&t)[2])
{
    const at::IntArrayRef shapes[2] = {shape0, shape1};
    const int64_t n = c10::multiply_integers(shape0);
    if (given[0] == Py_None && given[1] == Py_None && n + c10::multiply_integers(shape1) <= kShared) {
        const Tensor both = empty({up_to_128(n) + c10::multiply_integers(shape1)}, type, device);
        t[0] = part(both, 0, shape0);
        t[1] = part(both, up_to_128(n), shape1);
        return true;
    }
    for (int i = 0; i < 2; ++i)
        if (!output(given[i], shapes[i], type, device, t[i]))
            return false;
    return true;
}

bool workspace_of(PyObject *given, size_t need, int device, Tensor &t)
{
    if (given == Py_None) {
        t = empty({static_cast<int64_t>(need < 16 ? 16 : need)}, at::kByte, device);
        return true;
    }
    const Tensor *g = plain(given, device);
    if (!g || !g->is_contiguous())
        return false;
    t = *g;
    return true;
}

void *stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

// What a call gives back: None where it is not the usual one, the status where
// the library refused, else the result.
PyObject *handed_back() { Py_RETURN_NONE; }

template <typename F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (...) {  // such as memory that cannot be had: cache.py will meet it, and say so
        return handed_back();
    }
}

// write(cache, k, v, page_table, seq_lens, cu_seqlens)
PyObject *py_write(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 6 || !lib.write)
            return handed_back();
        const int device = c10::cuda::current_device();
        fa_cache_t c;
        Batch b;
        fa_dtype_t type, vtype;
        int T;
        if (!describe(a[0], device, c) || !describe_batch(a[3], a[4], device, b))
            return handed_back();
        const Tensor *k = rows(a[1], device, 3, c.d, type), *v = rows(a[2], device, 3, c.d, vtype);
        if (!k || !v || type != vtype || k->sizes() != v->sizes() || k->size(1) != c.heads || !to_int(k->size(0), T))
            return handed_back();
        const int *cu = nullptr;
        if (a[5] != Py_None) {
            const Tensor *t = exact(a[5], device, at::kInt, {static_cast<int64_t>(b.B) + 1});
            if (!t)
                return handed_back();
            cu = static_cast<const int *>(t->data_ptr());
        }
        return PyLong_FromLong(lib.write(&c, k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1), v->stride(0),
                                         v->stride(1), cu, b.lens, b.table, b.stride, b.pages, b.B, T, type,
                                         stream_of(device)));
    });
}

// read(cache, page_table, seq_lens, N, fp16?, k, v)
PyObject *py_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 7 || !lib.read || !PyLong_Check(a[3]))
            return handed_back();
        const int device = c10::cuda::current_device();
        fa_cache_t c;
        Batch b;
        int N;
        if (!describe(a[0], device, c) || !describe_batch(a[1], a[2], device, b) || !to_int(PyLong_AsLongLong(a[3]), N)) {
            PyErr_Clear();
            return handed_back();
        }
        const fa_dtype_t type = a[4] == Py_True ? FA_FP16 : FA_BF16;
        const int64_t shape[4] = {b.B, c.heads, N, c.d};
        Tensor k, v;
        if (!output(a[5], shape, scalar_of(type), device, k) || !output(a[6], shape, scalar_of(type), device, v))
            return handed_back();
        const fa_status_t s = lib.read(&c, k.data_ptr(), v.data_ptr(), b.lens, b.table, b.stride, b.pages, b.B, N, type,
                                       stream_of(device));
        if (s != FA_OK)
            return PyLong_FromLong(s);
        PyObject *pk = a[5] == Py_None ? THPVariable_Wrap(k) : Py_NewRef(a[5]);
        PyObject *pv = a[6] == Py_None ? THPVariable_Wrap(v) : Py_NewRef(a[6]);
        return Py_BuildValue("(NN)", pk, pv);
    });
}

// decode(q, cache, page_table, seq_lens, pages, o, lse, scale, causal, return_lse, workspace)
PyObject *py_decode(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 11 || !lib.decode || (a[7] != Py_None && !PyFloat_Check(a[7])) || !PyBool_Check(a[8]) ||
            !PyBool_Check(a[9]))
            return handed_back();
        const int device = c10::cuda::current_device();
        fa_cache_t c;
        Batch b;
        fa_dtype_t type;
        int Hq, Nq, slots = 0;
        if (!describe(a[1], device, c) || !describe_batch(a[2], a[3], device, b))
            return handed_back();
        const Tensor *q = rows(a[0], device, 4, c.d, type);
        if (!q || q->size(0) != b.B || !to_int(q->size(1), Hq) || !to_int(q->size(2), Nq) || c.heads < 1 || Hq % c.heads)
            return handed_back();
        const int *listed = nullptr;
        if (a[4] != Py_None) {
            const Tensor *p = plain(a[4], device);
            if (!p || p->dim() != 4 || p->scalar_type() != at::kInt || !p->is_contiguous() || p->size(0) != b.B ||
                p->size(1) != c.heads || p->size(2) != Nq || !to_int(p->size(3), slots))
                return handed_back();
            listed = static_cast<const int *>(p->data_ptr());
        }
        const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.d)) : PyFloat_AS_DOUBLE(a[7]);
        const int64_t shape[4] = {b.B, Hq, Nq, c.d};
        Tensor o, lse, ws;
        if (!output(a[5], shape, q->scalar_type(), device, o))
            return handed_back();
        const bool with_lse = a[6] != Py_None || a[9] == Py_True;
        if (with_lse && !output(a[6], at::IntArrayRef(shape, 3), at::kFloat, device, lse))
            return handed_back();
        if (!workspace_of(a[10], lib.decode_workspace(b.B, Hq, c.heads, Nq, c.d), device, ws))
            return handed_back();
        const fa_status_t s =
            lib.decode(&c, q->data_ptr(), q->stride(0), q->stride(1), q->stride(2), o.data_ptr(),
                       with_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, b.lens, b.table, b.stride, b.pages, listed,
                       slots, ws.data_ptr(), ws.nbytes(), b.B, Hq, Nq, static_cast<float>(scale), a[8] == Py_True, type,
                       stream_of(device));
        if (s != FA_OK)
            return PyLong_FromLong(s);
        PyObject *po = a[5] == Py_None ? THPVariable_Wrap(o) : Py_NewRef(a[5]);
        PyObject *pl = !with_lse ? Py_NewRef(Py_None) : a[6] == Py_None ? THPVariable_Wrap(lse) : Py_NewRef(a[6]);
        return Py_BuildValue("(NN)", po, pl);
    });
}

// select(q, cache, page_table, seq_lens, slots, keep_first, keep_last, causal, pages, workspace)
PyObject *py_select(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 10 || !lib.select || !PyLong_Check(a[4]) || !PyLong_Check(a[5]) || !PyLong_Check(a[6]) ||
            !PyBool_Check(a[7]))
            return handed_back();
        const int device = c10::cuda::current_device();
        fa_cache_t c;
        Batch b;
        fa_dtype_t type;
        int Hq, Nq, slots, first, last;
        if (!describe(a[1], device, c) || !describe_batch(a[2], a[3], device, b) ||
            !to_int(PyLong_AsLongLong(a[4]), slots) || !to_int(PyLong_AsLongLong(a[5]), first) ||
            !to_int(PyLong_AsLongLong(a[6]), last) || slots < 1) {
            PyErr_Clear();
            return handed_back();
        }
        const Tensor *q = rows(a[0], device, 4, c.d, type);
        if (!q || q->size(0) != b.B || !to_int(q->size(1), Hq) || !to_int(q->size(2), Nq) || c.heads < 1 || Hq % c.heads ||
            (Hq == 0 && b.B > 0))
            return handed_back();
        const int64_t shape[4] = {b.B, c.heads, Nq, slots};
        Tensor pages, ws;
        if (!output(a[8], shape, at::kInt, device, pages) ||
            !workspace_of(a[9], lib.select_workspace(b.B, c.heads, Nq, b.pages), device, ws))
            return handed_back();
        const fa_status_t s = lib.select(&c, q->data_ptr(), q->stride(0), q->stride(1), q->stride(2), b.lens, b.table,
                                         b.stride, b.pages, static_cast<int *>(pages.data_ptr()), slots, first, last,
                                         ws.data_ptr(), ws.nbytes(), b.B, Hq, Nq, a[7] == Py_True, type, stream_of(device));
        if (s != FA_OK)
            return PyLong_FromLong(s);
        return a[8] == Py_None ? THPVariable_Wrap(pages) : Py_NewRef(a[8]);
    });
}

bool describe4(PyObject *cache, int device, fa_cache4_t &c)
{
    if (!PyTuple_Check(cache) || PyTuple_GET_SIZE(cache) != 1)
        return false;
    const Tensor *t = plain(PyTuple_GET_ITEM(cache, 0), device);
    if (!t || t->dim() != 4 || t->scalar_type() != at::kByte || !t->is_contiguous() || t->size(3) % 36 != 0 ||
        !to_int(t->size(0), c.num_pages) || !to_int(t->size(1), c.heads) || !to_int(t->size(2), c.page) ||
        !to_int(t->size(3) / 9 * 8, c.d))
        return false;
    c.data = t->data_ptr();
    return true;
}

// write4(cache, k, v, slots)
PyObject *py_write4(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 4 || !lib.write4)
            return handed_back();
        const int device = c10::cuda::current_device();
        fa_cache4_t c;
        fa_dtype_t type, vtype;
        int T;
        if (!describe4(a[0], device, c))
            return handed_back();
        const Tensor *k = rows(a[1], device, 3, c.d, type), *v = rows(a[2], device, 3, c.d, vtype);
        if (!k || !v || type != vtype || k->sizes() != v->sizes() || k->size(1) != c.heads || !to_int(k->size(0), T))
            return handed_back();
        const Tensor *slots = exact(a[3], device, at::kInt, {k->size(0)});
        if (!slots)
            return handed_back();
        return PyLong_FromLong(lib.write4(&c, k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1), v->stride(0),
                                          v->stride(1), static_cast<const int *>(slots->data_ptr()), T, type,
                                          stream_of(device)));
    });
}

// read4(cache, page_table, seq_lens, N, fp16?, k, v)
PyObject *py_read4(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 7 || !lib.read4 || !PyLong_Check(a[3]))
            return handed_back();
        const int device = c10::cuda::current_device();
        fa_cache4_t c;
        Batch b;
        int N;
        if (!describe4(a[0], device, c) || !describe_batch(a[1], a[2], device, b) || !to_int(PyLong_AsLongLong(a[3]), N)) {
            PyErr_Clear();
            return handed_back();
        }
        const fa_dtype_t type = a[4] == Py_True ? FA_FP16 : FA_BF16;
        const int64_t shape[4] = {b.B, c.heads, N, c.d};
        Tensor out[2];
        if (!outputs({a[5], a[6]}, shape, shape, scalar_of(type), device, out))
            return handed_back();
        const Tensor &k = out[0], &v = out[1];
        const fa_status_t s = lib.read4(&c, k.data_ptr(), v.data_ptr(), b.lens, b.table, b.stride, b.pages, b.B, N, type,
                                        stream_of(device));
        if (s != FA_OK)
            return PyLong_FromLong(s);
        PyObject *pk = a[5] == Py_None ? THPVariable_Wrap(k) : Py_NewRef(a[5]);
        PyObject *pv = a[6] == Py_None ? THPVariable_Wrap(v) : Py_NewRef(a[6]);
        return Py_BuildValue("(NN)", pk, pv);
    });
}

// decode4(q, cache, page_table, seq_lens, o, lse, scale, causal, return_lse, workspace)
PyObject *py_decode4(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 10 || !lib.decode4 || (a[6] != Py_None && !PyFloat_Check(a[6])) || !PyBool_Check(a[7]) ||
            !PyBool_Check(a[8]))
            return handed_back();
        const int device = c10::cuda::current_device();
        fa_cache4_t c;
        Batch b;
        fa_dtype_t type;
        int Hq, Nq;
        if (!describe4(a[1], device, c) || !describe_batch(a[2], a[3], device, b))
            return handed_back();
        const Tensor *q = rows(a[0], device, 4, c.d, type);
        if (!q || q->size(0) != b.B || !to_int(q->size(1), Hq) || !to_int(q->size(2), Nq) || c.heads < 1 || Hq % c.heads)
            return handed_back();
        const double scale = a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.d)) : PyFloat_AS_DOUBLE(a[6]);
        const int64_t shape[4] = {b.B, Hq, Nq, c.d};
        Tensor o, lse, ws;
        if (!output(a[4], shape, q->scalar_type(), device, o))
            return handed_back();
        const bool with_lse = a[5] != Py_None || a[8] == Py_True;
        if (with_lse && !output(a[5], at::IntArrayRef(shape, 3), at::kFloat, device, lse))
            return handed_back();
        if (!workspace_of(a[9], lib.decode4_workspace(b.B, Hq, c.heads, Nq, c.d), device, ws))
            return handed_back();
        const fa_status_t s =
            lib.decode4(&c, q->data_ptr(), q->stride(0), q->stride(1), q->stride(2), o.data_ptr(),
                        with_lse ? static_cast<float *>(lse.data_ptr()) : nullptr, b.lens, b.table, b.stride, b.pages,
                        ws.data_ptr(), ws.nbytes(), b.B, Hq, Nq, static_cast<float>(scale), a[7] == Py_True, type,
                        stream_of(device));
        if (s != FA_OK)
            return PyLong_FromLong(s);
        PyObject *po = a[4] == Py_None ? THPVariable_Wrap(o) : Py_NewRef(a[4]);
        PyObject *pl = !with_lse ? Py_NewRef(Py_None) : a[5] == Py_None ? THPVariable_Wrap(lse) : Py_NewRef(a[5]);
        return Py_BuildValue("(NN)", po, pl);
    });
}

// The pool of a plan or a trim, their lengths, and where the counts go.
struct PoolArgs {
    Tensor ring, counts, out;
    Batch b;
    const Tensor *other;
    int num_pages, page;
};

bool describe_pool(PyObject *pool, PyObject *table, PyObject *lens, PyObject *other, PyObject *page, PyObject *out, int device,
                   PoolArgs &x)
{
    if (!PyTuple_Check(pool) || PyTuple_GET_SIZE(pool) != 2 || !PyLong_Check(page))
        return false;
    const Tensor *ring = plain(PyTuple_GET_ITEM(pool, 0), device);
    const Tensor *counts = exact(PyTuple_GET_ITEM(pool, 1), device, at::kLong, {2});
    const Tensor *to = out == Py_None ? counts : exact(out, device, at::kLong, {2});
    if (!ring || !counts || !to || ring->dim() != 1 || ring->scalar_type() != at::kInt || !ring->is_contiguous() ||
        !to_int(ring->size(0), x.num_pages) || !to_int(PyLong_AsLongLong(page), x.page) ||
        !describe_batch(table, lens, device, x.b))
        return false;
    x.other = exact(other, device, at::kInt, {x.b.B});
    if (!x.other)
        return false;
    x.ring = *ring;
    x.counts = *counts;
    x.out = *to;
    return true;
}

// plan(pool, page_table, seq_lens, new_lens, page, T, counts): the four tensors of a new plan
PyObject *py_plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 7 || !lib.plan || !PyLong_Check(a[5]))
            return handed_back();
        const int device = c10::cuda::current_device();
        PoolArgs x;
        int T;
        if (!describe_pool(a[0], a[1], a[2], a[3], a[4], a[6], device, x) || !to_int(PyLong_AsLongLong(a[5]), T) ||
            x.b.B == 0) {
            PyErr_Clear();
            return handed_back();
        }
        const int64_t B = x.b.B, rows = up_to_128(T), lens = up_to_128(B + 1);
        const Tensor all = empty({2 * rows + 2 * lens}, at::kInt, device);
        const Tensor positions = part(all, 0, {T}), slots = part(all, rows, {T});
        const Tensor cu = part(all, 2 * rows, {B + 1}), ends = part(all, 2 * rows + lens, {B});
        auto ints = [](const Tensor &t) { return static_cast<int *>(t.data_ptr()); };
        const fa_status_t s =
            lib.plan(ints(x.ring), x.num_pages, static_cast<const long long *>(x.counts.data_ptr()),
                     const_cast<int *>(x.b.table), x.b.stride, x.b.pages, x.b.lens, ints(*x.other), ints(cu), ints(ends),
                     ints(positions), ints(slots), static_cast<long long *>(x.out.data_ptr()), x.page, x.b.B, T,
                     stream_of(device));
        if (s != FA_OK)
            return PyLong_FromLong(s);
        return Py_BuildValue("(NNNN)", THPVariable_Wrap(cu), THPVariable_Wrap(ends), THPVariable_Wrap(positions),
                             THPVariable_Wrap(slots));
    });
}

// trim(pool, page_table, seq_lens, keep_lens, page, counts)
PyObject *py_trim(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 6 || !lib.trim)
            return handed_back();
        const int device = c10::cuda::current_device();
        PoolArgs x;
        if (!describe_pool(a[0], a[1], a[2], a[3], a[4], a[5], device, x) || x.b.B == 0) {
            PyErr_Clear();
            return handed_back();
        }
        return PyLong_FromLong(lib.trim(static_cast<int *>(x.ring.data_ptr()), x.num_pages,
                                        static_cast<const long long *>(x.counts.data_ptr()), x.b.table, x.b.stride,
                                        x.b.pages, x.b.lens, static_cast<const int *>(x.other->data_ptr()),
                                        static_cast<long long *>(x.out.data_ptr()), x.page, x.b.B, stream_of(device)));
    });
}

// rope(q, k, rope, positions, backward, q_out, k_out): (q, k) turned
PyObject *py_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&]() -> PyObject * {
        if (n != 7 || !lib.rope || !PyTuple_Check(a[2]) || PyTuple_GET_SIZE(a[2]) != 3 || !PyBool_Check(a[4]))
            return handed_back();
        const int device = c10::cuda::current_device();
        const Tensor *turns = plain(PyTuple_GET_ITEM(a[2], 0), device);
        PyObject *interleaved = PyTuple_GET_ITEM(a[2], 1), *factor = PyTuple_GET_ITEM(a[2], 2);
        fa_rope_t rope;
        if (!turns || turns->dim() != 1 || turns->scalar_type() != at::kLong || !turns->is_contiguous() ||
            !PyBool_Check(interleaved) || !PyFloat_Check(factor) || !to_int(turns->size(0), rope.pairs))
            return handed_back();
        rope.turns = static_cast<const unsigned long long *>(turns->data_ptr());
        rope.interleaved = interleaved == Py_True;
        rope.factor = static_cast<float>(PyFloat_AS_DOUBLE(factor));
        const Tensor *x[2] = {plain(a[0], device), a[1] == Py_None ? nullptr : plain(a[1], device)};
        if (!x[0] || (x[0]->dim() != 3 && x[0]->dim() != 4) || (a[1] == Py_None ? a[6] != Py_None : !x[1]))
            return handed_back();
        const int dim = static_cast<int>(x[0]->dim()), tokens = dim == 3 ? 0 : 2;
        const int64_t d = x[0]->size(dim - 1);
        int B = 1, N, width;
        if (!to_int(x[0]->size(tokens), N) || (dim == 4 && !to_int(x[0]->size(0), B)) || !to_int(d, width))
            return handed_back();
        fa_rope_rows_t r[2];
        Tensor y[2];
        fa_dtype_t type = FA_FP16;
        for (int i = 0; i < (x[1] ? 2 : 1); ++i) {
            fa_dtype_t own;
            const Tensor *t = rows(a[i], device, dim, width, own);
            if (!t || (i && (own != type || t->size(0) != x[0]->size(0) || t->size(tokens) != N)))
                return handed_back();
            type = own;
            PyObject *given = a[5 + i];
            if (given == Py_None && x[1] && a[5] == Py_None && a[6] == Py_None && x[0]->numel() + x[1]->numel() <= kShared) {
                if (i == 0) {  // both in one allocation
                    const int64_t n = up_to_128(t->numel());
                    y[1] = empty({n + x[1]->numel()}, t->scalar_type(), device);
                    y[0] = part(y[1], 0, t->sizes());
                } else {
                    y[1] = part(y[1], up_to_128(x[0]->numel()), t->sizes());
                }
            } else if (given == Py_None) {
                y[i] = empty(t->sizes(), t->scalar_type(), device);
            } else {
                fa_dtype_t as;
                const Tensor *o = rows(given, device, dim, width, as);
                if (!o || as != own || o->sizes() != t->sizes())
                    return handed_back();
                y[i] = *o;
            }
            r[i].x = t->data_ptr();
            r[i].y = y[i].data_ptr();
            r[i].x_batch = dim == 4 ? t->stride(0) : 0;
            r[i].y_batch = dim == 4 ? y[i].stride(0) : 0;
            r[i].x_head = t->stride(1);
            r[i].y_head = y[i].stride(1);
            r[i].x_row = t->stride(tokens);
            r[i].y_row = y[i].stride(tokens);
            if (!to_int(t->size(1), r[i].heads))
                return handed_back();
        }
        const int *positions = nullptr;
        int64_t stride = 0;
        if (a[3] != Py_None) {
            const Tensor *p = plain(a[3], device);
            if (!p || p->scalar_type() != at::kInt || p->dim() < 1 || p->dim() > dim - 2 || p->size(p->dim() - 1) != N ||
                (p->dim() == 2 && p->size(0) != B) || (p->stride(p->dim() - 1) != 1 && N > 1))
                return handed_back();
            positions = static_cast<const int *>(p->data_ptr());
            stride = p->dim() == 2 ? p->stride(0) : 0;
        }
        const fa_status_t s = lib.rope(&rope, &r[0], x[1] ? &r[1] : nullptr, positions, stride, B, N, width, a[4] == Py_True,
                                       type, stream_of(device));
        if (s != FA_OK)
            return PyLong_FromLong(s);
        PyObject *pq = a[5] == Py_None ? THPVariable_Wrap(y[0]) : Py_NewRef(a[5]);
        PyObject *pk = !x[1] ? Py_NewRef(Py_None) : a[6] == Py_None ? THPVariable_Wrap(y[1]) : Py_NewRef(a[6]);
        return Py_BuildValue("(NN)", pq, pk);
    });
}

// bind(the library's functions' addresses, in the order of Library)
constexpr int kFunctions = 13;
static_assert(sizeof(Library) == kFunctions * sizeof(void *), "an address each");
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[kFunctions];
    if (n != kFunctions) {
        PyErr_SetString(PyExc_TypeError, "an address for each function");
        return nullptr;
    }
    for (int i = 0; i < kFunctions; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "an address is zero");
            return nullptr;
        }
    lib = {reinterpret_cast<decltype(lib.write)>(p[0]),     reinterpret_cast<decltype(lib.read)>(p[1]),
           reinterpret_cast<decltype(lib.decode)>(p[2]),    reinterpret_cast<decltype(lib.decode_workspace)>(p[3]),
           reinterpret_cast<decltype(lib.select)>(p[4]),    reinterpret_cast<decltype(lib.select_workspace)>(p[5]),
           reinterpret_cast<decltype(lib.write4)>(p[6]),    reinterpret_cast<decltype(lib.read4)>(p[7]),
           reinterpret_cast<decltype(lib.decode4)>(p[8]),   reinterpret_cast<decltype(lib.decode4_workspace)>(p[9]),
           reinterpret_cast<decltype(lib.plan)>(p[10]),     reinterpret_cast<decltype(lib.trim)>(p[11]),
           reinterpret_cast<decltype(lib.rope)>(p[12])};
    Py_RETURN_NONE;
}

template <typename F>
constexpr PyMethodDef method(const char *name, F f)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method("bind", py_bind),       method("write", py_write),   method("read", py_read),
                         method("decode", py_decode),   method("select", py_select), method("write4", py_write4),
                         method("read4", py_read4),     method("decode4", py_decode4), method("plan", py_plan),
                         method("trim", py_trim),       method("rope", py_rope),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_cache_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_cache_py()
{
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddIntConstant(m, "abi", FA_ABI_VERSION) < 0 ||
              PyModule_AddStringConstant(m, "torch", FA_TORCH_VERSION) < 0)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
