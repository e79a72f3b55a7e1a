// binding.cpp -- argument marshalling of the decode-step operators for Python:
// checks of types and shapes, allocation of outputs, the stream, and the call
// of the C entry point of the same name.  No arithmetic.
//
// A call of these operators takes 2 to 10 us on the GPU for a few tokens; the
// same checks made in Python took 25 to 37 us a call on the host.  Here they
// read the tensors' fields directly: 2.3 to 2.7 us with the launch (4 to 5 with
// the two of the adapters or the verification, 7 with the four of the experts),
// 0.9 more for each tensor that the call makes, and 11 for an attention
// workspace, which has to be zeroed.
//
// Every function takes positional arguments from w4q.py and returns
// (status, results...); a wrong type or shape raises ValueError.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "w4q.h"

namespace {

using at::Tensor;

[[noreturn]] void fail(const char *name, const char *what)
{
    C10_THROW_ERROR(ValueError, c10::str(name, " ", what));
}

// A CUDA tensor; the call's device is the first one's.
struct Call {
    c10::Device device = c10::Device(c10::kCPU);
    bool any = false;

    const Tensor &cuda(PyObject *o, const char *name)
    {
        if (!THPVariable_Check(o))
            fail(name, "must be a CUDA tensor");
        const Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda())
            fail(name, "must be a CUDA tensor");
        if (!any) {
            device = t.device();
            any = true;
        } else if (t.device() != device) {
            fail(name, "must be on the same device as the other tensors");
        }
        return t;
    }
    // contiguous, of one type
    const Tensor &dense(PyObject *o, const char *name, at::ScalarType type)
    {
        const Tensor &t = cuda(o, name);
        if (t.scalar_type() != type)
            C10_THROW_ERROR(ValueError, c10::str(name, " must be ", type, ", got ", t.scalar_type()));
        if (!t.is_contiguous())
            fail(name, "must be contiguous");
        return t;
    }
    void *optional(PyObject *o, const char *name, at::ScalarType type, int64_t numel)
    {
        if (o == Py_None)
            return nullptr;
        const Tensor &t = dense(o, name, type);
        if (t.numel() != numel)
            C10_THROW_ERROR(ValueError, c10::str(name, " must have ", numel, " elements, got ", t.numel()));
        return t.data_ptr();
    }
};

// Head rows bf16 [tokens, heads, head_dim]: a token's heads one after the
// other, the tokens at any stride.
struct Heads {
    void *ptr = nullptr;
    int64_t tokens = 0, stride = 0;
    int heads = 0, dim = 0;
};
Heads heads_of(Call &c, PyObject *o, const char *name, int64_t tokens, int64_t heads, int64_t dim)
{
    const Tensor &t = c.cuda(o, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3)
        fail(name, "must be bfloat16 [tokens, heads, head_dim]");
    Heads h;
    h.tokens = t.size(0);
    const int64_t n = t.size(1), d = t.size(2);
    if ((tokens >= 0 && h.tokens != tokens) || (heads >= 0 && n != heads) || (dim >= 0 && d != dim) || n > INT32_MAX ||
        d > INT32_MAX)
        C10_THROW_ERROR(ValueError, c10::str(name, " must be [", tokens, ", ", heads, ", ", dim, "] (-1: any), got ", t.sizes()));
    if ((d > 1 && t.stride(2) != 1) || (n > 1 && t.stride(1) != d))
        fail(name, "must hold a token's heads one after the other");
    h.ptr = t.data_ptr();
    h.heads = (int)n;
    h.dim = (int)d;
    h.stride = h.tokens > 1 ? t.stride(0) : n * d;
    return h;
}

// The stream of a call: an integer, or None for the current one; the device
// and the stream are current while it lives, so what is allocated belongs to
// the stream.
struct OnStream {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard guard;
    void *stream;
    OnStream(const Call &c, PyObject *o) : device(c.device)
    {
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(c.device.index()).stream();
        } else {
            const unsigned long long v = PyLong_AsUnsignedLongLong(o);
            if (PyErr_Occurred())
                throw python_error();
            stream = reinterpret_cast<void *>(v);
            guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), c.device.index()));
        }
    }
};

// Whether a new tensor concerns the allocator alone: no dispatch mode or transform wants to see it, and
// memory that is not initialised need not be filled.
bool only_allocates()
{
    const at::Context &torch = at::globalContext();
    return (c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty() &&
           !(torch.deterministicAlgorithms() && torch.deterministicFillUninitializedMemory());
}

// (Straight from the allocator 0.9 us, 2.0 by at::empty.)
Tensor fresh(const Call &c, at::IntArrayRef shape, at::ScalarType type)
{
    if (!only_allocates())
        return at::empty(shape, at::TensorOptions().dtype(type).device(c.device));
    return Tensor(at::detail::empty_cuda(shape, type, c.device, std::nullopt));
}

// `o`, or a new tensor where it is None
Tensor out_or_new(Call &c, PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType type)
{
    if (o == Py_None)
        return fresh(c, shape, type);
    int64_t n = 1;
    for (const int64_t s : shape)
        n *= s;
    c.optional(o, name, type, n);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}
double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}
bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}

void count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        C10_THROW_ERROR(TypeError, c10::str(n, " arguments, ", want, " expected"));
}

struct Table {
    const float *ptr = nullptr;
    int64_t positions = 0;
    int rot = 0;
};
Table table_of(Call &c, PyObject *o)
{
    Table t;
    if (o != Py_None) {
        const Tensor &x = c.dense(o, "cos_sin", at::kFloat);
        if (x.dim() != 2 || x.size(1) > INT32_MAX)
            fail("cos_sin", "must be [positions, rot]");
        t.ptr = x.data_ptr<float>();
        t.positions = x.size(0);
        t.rot = (int)x.size(1);
    }
    return t;
}

// args[0..5]: k_cache, v_cache, k_scale, v_scale, block_table, seq_lens
w4q_kv8_cache cache_of(Call &c, PyObject *const *a)
{
    const Tensor &k = c.cuda(a[0], "k_cache");
    if (k.dim() != 4)
        fail("k_cache", "must be [blocks, kv_heads, page, head_dim]");
    if (k.scalar_type() != at::kChar && k.scalar_type() != at::kFloat8_e4m3fn)
        fail("k_cache", "must be int8 or float8_e4m3fn");
    c.dense(a[0], "k_cache", k.scalar_type());
    const Tensor &v = c.dense(a[1], "v_cache", k.scalar_type());
    if (v.sizes() != k.sizes())
        fail("v_cache", "must have the shape of k_cache");
    const Tensor &table = c.dense(a[4], "block_table", at::kInt), &lens = c.dense(a[5], "seq_lens", at::kInt);
    if (table.dim() != 2 || lens.dim() != 1 || table.size(0) != lens.size(0))
        fail("block_table", "must be [seqs, width], seq_lens [seqs]");
    w4q_kv8_cache s;
    s.k = k.data_ptr();
    s.v = v.data_ptr();
    s.k_scale = static_cast<float *>(c.optional(a[2], "k_scale", at::kFloat, k.size(0) * k.size(1)));
    s.v_scale = static_cast<float *>(c.optional(a[3], "v_scale", at::kFloat, k.size(0) * k.size(1)));
    s.block_table = table.data_ptr<int>();
    s.seq_lens = lens.data_ptr<int>();
    s.blocks = k.size(0);
    auto clip = [](int64_t x) { return (int32_t)std::min<int64_t>(x, INT32_MAX); };
    s.seqs = clip(table.size(0));
    s.width = clip(table.size(1));
    s.kv_heads = clip(k.size(1));
    s.page = clip(k.size(2));
    s.head_dim = clip(k.size(3));
    s.format = k.scalar_type() == at::kChar ? 0 : 1;
    return s;
}

PyObject *result(int status, const Tensor *a = nullptr, const Tensor *b = nullptr)
{
    PyObject *t = PyTuple_New(3);
    if (t == nullptr)
        return nullptr;
    PyTuple_SET_ITEM(t, 0, PyLong_FromLong(status));
    for (int i = 0; i < 2; ++i) {
        const Tensor *x = i == 0 ? a : b;
        if (x != nullptr && x->defined()) {
            PyTuple_SET_ITEM(t, 1 + i, THPVariable_Wrap(*x));
        } else {
            Py_INCREF(Py_None);
            PyTuple_SET_ITEM(t, 1 + i, Py_None);
        }
    }
    return t;
}

// q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, q_out, k_out, stream
PyObject *py_qk_norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 11);
    Call c;
    const Heads q = heads_of(c, a[0], "q", -1, -1, -1);
    const Heads k = a[1] == Py_None ? Heads() : heads_of(c, a[1], "k", q.tokens, -1, q.dim);
    const Table table = table_of(c, a[4]);
    void *qw = c.optional(a[2], "q_weight", at::kBFloat16, q.dim), *kw = c.optional(a[3], "k_weight", at::kBFloat16, q.dim);
    void *pos = c.optional(a[5], "positions", at::kInt, q.tokens);
    const OnStream on(c, a[10]);
    const Tensor qo = out_or_new(c, a[8], "q_out", {q.tokens, q.heads, q.dim}, at::kBFloat16);
    Tensor ko;
    if (a[1] != Py_None)
        ko = out_or_new(c, a[9], "k_out", {k.tokens, k.heads, k.dim}, at::kBFloat16);
    if (q.tokens == 0)  // a tensor without elements has no address
        return result(W4Q_OK, &qo, &ko);
    const int st = qk_norm_rope(q.ptr, k.ptr, q.tokens, q.heads, k.heads, q.dim, q.stride, k.stride, qw, kw,
                                (float)number(a[6]), table.ptr, table.positions, table.rot, truth(a[7]),
                                static_cast<const int32_t *>(pos), qo.data_ptr(), ko.defined() ? ko.data_ptr() : nullptr,
                                on.stream);
    return result(st, &qo, &ko);
    END_HANDLE_TH_ERRORS
}

// k, v, (cache: 6), cu_tokens, q, q_out, q_weight, k_weight, cos_sin, eps, interleaved, stream
PyObject *py_kv8_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 17);
    Call c;
    const w4q_kv8_cache cache = cache_of(c, a + 2);
    const Heads k = heads_of(c, a[0], "k", -1, cache.kv_heads, cache.head_dim);
    const Heads v = heads_of(c, a[1], "v", k.tokens, cache.kv_heads, cache.head_dim);
    const Heads q = a[9] == Py_None ? Heads() : heads_of(c, a[9], "q", k.tokens, -1, cache.head_dim);
    void *cu = c.optional(a[8], "cu_tokens", at::kInt, (int64_t)cache.seqs + 1);
    void *qw = c.optional(a[11], "q_weight", at::kBFloat16, cache.head_dim);
    void *kw = c.optional(a[12], "k_weight", at::kBFloat16, cache.head_dim);
    const Table table = table_of(c, a[13]);
    const OnStream on(c, a[16]);
    Tensor qo;
    if (a[9] != Py_None)
        qo = out_or_new(c, a[10], "q_out", {q.tokens, q.heads, q.dim}, at::kBFloat16);
    if (k.tokens == 0)
        return result(a[8] == Py_None ? W4Q_ERR_INVALID_ARG : W4Q_OK, &qo);
    const int st = kv8_append(&cache, k.ptr, v.ptr, k.stride, v.stride, k.tokens, static_cast<const int32_t *>(cu), q.ptr,
                              q.stride, q.heads, qo.defined() ? qo.data_ptr() : nullptr, qw, kw, (float)number(a[14]),
                              table.ptr, table.positions, table.rot, truth(a[15]), on.stream);
    return result(st, &qo);
    END_HANDLE_TH_ERRORS
}

// (cache: 6), cu_tokens, tokens, stream
PyObject *py_kv8_read(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 9);
    Call c;
    const w4q_kv8_cache cache = cache_of(c, a);
    void *cu = c.optional(a[6], "cu_tokens", at::kInt, (int64_t)cache.seqs + 1);
    if (a[7] == Py_None && a[6] != Py_None)
        fail("tokens", "must be given with cu_tokens");
    const int64_t tokens = a[7] == Py_None ? cache.seqs : integer(a[7]);
    if (tokens < 0)
        fail("tokens", "must not be negative");
    const OnStream on(c, a[8]);
    const Tensor k = fresh(c, {tokens, cache.kv_heads, cache.head_dim}, at::kBFloat16);
    const Tensor v = fresh(c, {tokens, cache.kv_heads, cache.head_dim}, at::kBFloat16);
    const int st = tokens == 0 ? W4Q_OK
                               : kv8_read(&cache, static_cast<const int32_t *>(cu), tokens, k.data_ptr(), v.data_ptr(), on.stream);
    return result(st, &k, &v);
    END_HANDLE_TH_ERRORS
}

// q, (cache: 6), scale, window, out, lse, workspace, stream
PyObject *py_kv8_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 13);
    Call c;
    const w4q_kv8_cache cache = cache_of(c, a + 1);
    const Tensor &q = c.cuda(a[0], "q");
    if (q.scalar_type() != at::kBFloat16 || q.dim() != 4 || q.size(0) != cache.seqs || q.size(3) != cache.head_dim)
        C10_THROW_ERROR(ValueError, c10::str("q must be bfloat16 [", cache.seqs, ", queries, heads, ", cache.head_dim, "]"));
    const int64_t s = q.size(0), m = q.size(1), h = q.size(2), d = q.size(3);
    if (q.stride(3) != 1 || (h > 1 && q.stride(2) != d))
        fail("q", "must hold a token's heads one after the other");
    if (s > 1 && m > 1 && q.stride(0) != m * q.stride(1))
        fail("q", "must hold its query tokens at one stride");
    if (m > INT32_MAX || h > INT32_MAX)
        fail("q", "is too large");
    const int64_t stride = m > 1 ? q.stride(1) : (s > 1 ? q.stride(0) : h * d);
    void *lse = c.optional(a[10], "lse", at::kFloat, s * m * h);
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt((double)d) : number(a[7]);
    const OnStream on(c, a[12]);
    const Tensor out = out_or_new(c, a[9], "out", {s, m, h, d}, at::kBFloat16);
    Tensor ws;
    if (a[11] == Py_None) {
        const size_t need = kv8_workspace_bytes(s, (int)m, (int)h, cache.kv_heads, cache.head_dim);
        ws = at::zeros({(int64_t)std::max<size_t>(need, 16)}, at::TensorOptions().dtype(at::kByte).device(c.device));
    } else {
        ws = c.cuda(a[11], "workspace");
        if (!ws.is_contiguous())
            fail("workspace", "must be contiguous");
    }
    const int st = kv8_attention(&cache, q.data_ptr(), stride, out.data_ptr(), static_cast<float *>(lse), (int)m, (int)h,
                                 (float)scale, integer(a[8]), ws.data_ptr(), ws.nbytes(), on.stream);
    return result(st, &out);
    END_HANDLE_TH_ERRORS
}

// x, router, w13, w2, inter, topk, bias, sigmoid, renormalize, scale, out, ids, weights, workspace, stream
PyObject *py_moe_w4a16(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 15);
    Call c;
    const Tensor &x = c.dense(a[0], "x", at::kBFloat16), &router = c.dense(a[1], "router", at::kBFloat16);
    if (x.dim() != 2 || router.dim() != 2 || router.size(1) != x.size(1))
        fail("x", "must be [tokens, hidden], router [experts, hidden]");
    const int64_t m = x.size(0), h = x.size(1), e = router.size(0), i = integer(a[4]), k = integer(a[5]);
    const Tensor &w13 = c.dense(a[2], "w13", at::kByte), &w2 = c.dense(a[3], "w2", at::kByte);
    if (i > 0 && ((size_t)w13.numel() != w4_packed_bytes(e * 2 * i, h, 32) || (size_t)w2.numel() != w4_packed_bytes(e * h, i, 32)))
        C10_THROW_ERROR(ValueError, c10::str("w13 and w2 must be packed from [", e * 2 * i, ", ", h, "] and [", e * h, ", ", i, "]"));
    if (k > INT32_MAX || k < 0)
        fail("topk", "is out of range");
    void *bias = c.optional(a[6], "bias", at::kFloat, e);
    void *ids = c.optional(a[11], "ids", at::kInt, m * k), *weights = c.optional(a[12], "weights", at::kFloat, m * k);
    const OnStream on(c, a[14]);
    const Tensor out = out_or_new(c, a[10], "out", {m, h}, at::kBFloat16);
    Tensor ws;
    if (a[13] == Py_None) {
        ws = fresh(c, {(int64_t)std::max<size_t>(moe_workspace_bytes(m, h, i, e, (int)k), 16)}, at::kByte);
    } else {
        ws = c.cuda(a[13], "workspace");
        if (!ws.is_contiguous())
            fail("workspace", "must be contiguous");
    }
    const int st = moe_w4a16(x.data_ptr(), router.data_ptr(), static_cast<const float *>(bias), w13.data_ptr(), w2.data_ptr(),
                             out.data_ptr(), m, h, i, e, (int)k, truth(a[7]), truth(a[8]), (float)number(a[9]),
                             static_cast<int32_t *>(ids), static_cast<float *>(weights), ws.data_ptr(), ws.nbytes(), on.stream);
    return result(st, &out);
    END_HANDLE_TH_ERRORS
}

// status and up to three tensors (None for an undefined one)
PyObject *result3(int status, const Tensor &a, const Tensor &b = Tensor(), const Tensor &c = Tensor())
{
    PyObject *t = PyTuple_New(4);
    if (t == nullptr)
        return nullptr;
    PyTuple_SET_ITEM(t, 0, PyLong_FromLong(status));
    const Tensor *x[3] = {&a, &b, &c};
    for (int i = 0; i < 3; ++i)
        if (x[i]->defined()) {
            PyTuple_SET_ITEM(t, 1 + i, THPVariable_Wrap(*x[i]));
        } else {
            Py_INCREF(Py_None);
            PyTuple_SET_ITEM(t, 1 + i, Py_None);
        }
    return t;
}

// bf16 rows [tokens, n] of contiguous elements at any stride
struct Rows {
    void *ptr = nullptr;
    int64_t tokens = 0, n = 0, stride = 0;
};
Rows rows_of(Call &c, PyObject *o, const char *name, int64_t tokens, int64_t n)
{
    const Tensor &t = c.cuda(o, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || (tokens >= 0 && t.size(0) != tokens) || (n >= 0 && t.size(1) != n))
        C10_THROW_ERROR(ValueError, c10::str(name, " must be bfloat16 [", tokens, ", ", n, "] (-1: any), got ", t.scalar_type(), " ",
                                             t.sizes()));
    if (t.size(1) > 1 && t.stride(1) != 1)
        fail(name, "must hold a row's elements one after the other");
    Rows r;
    r.ptr = t.data_ptr();
    r.tokens = t.size(0);
    r.n = t.size(1);
    r.stride = r.tokens > 1 ? t.stride(0) : r.n;
    if (r.stride < r.n)
        fail(name, "must have rows that do not overlap");
    return r;
}

// The given rows, or new ones
Rows rows_out(Call &c, PyObject *o, const char *name, int64_t tokens, int64_t n, Tensor *t)
{
    *t = o == Py_None ? fresh(c, {tokens, n}, at::kBFloat16) : THPVariable_Check(o) ? THPVariable_Unpack(o) : Tensor();
    if (o != Py_None)
        return rows_of(c, o, name, tokens, n);
    return {t->data_ptr(), tokens, n, n};
}

// The given workspace, or a new one
Tensor scratch(Call &c, PyObject *o, size_t need)
{
    if (o == Py_None)
        return fresh(c, {(int64_t)std::max<size_t>(need, 16)}, at::kByte);
    const Tensor &t = c.cuda(o, "workspace");
    if (!t.is_contiguous())
        fail("workspace", "must be contiguous");
    return t;
}

// x, residual, weight, eps, sum_out, out, stream
PyObject *py_add_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 7);
    Call c;
    const Rows x = rows_of(c, a[0], "x", -1, -1);
    const Rows r = a[1] == Py_None ? Rows() : rows_of(c, a[1], "residual", x.tokens, x.n);
    void *w = c.optional(a[2], "weight", at::kBFloat16, x.n);
    const float eps = (float)number(a[3]);
    if (a[1] == Py_None && a[4] != Py_None)
        fail("sum_out", "needs a residual");
    const OnStream on(c, a[6]);
    Tensor sum;
    const Rows s = a[1] == Py_None ? Rows() : rows_out(c, a[4], "sum_out", x.tokens, x.n, &sum);
    const Tensor out = out_or_new(c, a[5], "out", {x.tokens, x.n}, at::kBFloat16);
    const int st = x.tokens == 0 ? W4Q_OK
                                 : add_rms_norm(x.ptr, x.stride, r.ptr, r.stride, w, eps, x.tokens, x.n, s.ptr, s.stride,
                                                out.data_ptr(), on.stream);
    return result3(st, out, sum);
    END_HANDLE_TH_ERRORS
}

// x, residual, weight, eps, row, sum_out, codes, scales, out, stream
PyObject *py_add_rms_norm_a8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 10);
    Call c;
    const Rows x = rows_of(c, a[0], "x", -1, -1);
    const Rows r = a[1] == Py_None ? Rows() : rows_of(c, a[1], "residual", x.tokens, x.n);
    void *w = c.optional(a[2], "weight", at::kBFloat16, x.n);
    const float eps = (float)number(a[3]);
    const bool row = truth(a[4]);
    if (a[1] == Py_None && a[5] != Py_None)
        fail("sum_out", "needs a residual");
    void *out = c.optional(a[8], "out", at::kBFloat16, x.tokens * x.n);
    const OnStream on(c, a[9]);
    Tensor sum;
    const Rows s = a[1] == Py_None ? Rows() : rows_out(c, a[5], "sum_out", x.tokens, x.n, &sum);
    const Tensor codes = out_or_new(c, a[6], "codes", {x.tokens, x.n}, at::kChar);
    const Tensor scales = row ? out_or_new(c, a[7], "scales", {x.tokens}, at::kFloat)
                              : out_or_new(c, a[7], "scales", {x.tokens, x.n / 32}, at::kFloat);
    const int st = x.tokens == 0 ? W4Q_OK
                                 : add_rms_norm_a8(x.ptr, x.stride, r.ptr, r.stride, w, eps, x.tokens, x.n, row, s.ptr,
                                                   s.stride, static_cast<int8_t *>(codes.data_ptr()),
                                                   static_cast<float *>(scales.data_ptr()), out, on.stream);
    return result3(st, codes, scales, sum);
    END_HANDLE_TH_ERRORS
}

// xq, sx, packed, N, K, group, out, workspace, stream
PyObject *py_w4a8_gemm_codes(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 9);
    Call c;
    const Tensor &xq = c.dense(a[0], "xq", at::kChar), &sx = c.dense(a[1], "sx", at::kFloat);
    const Tensor &packed = c.dense(a[2], "packed", at::kByte);
    const int64_t N = integer(a[3]), K = integer(a[4]), group = integer(a[5]);
    if (xq.dim() != 2 || xq.size(1) != K)
        C10_THROW_ERROR(ValueError, c10::str("xq must be int8 [M, ", K, "]"));
    const int64_t m = xq.size(0);
    const bool row = sx.dim() == 1;
    if (row ? sx.size(0) != m : sx.dim() != 2 || sx.size(0) != m || sx.size(1) != K / 32)
        C10_THROW_ERROR(ValueError, c10::str("sx must be float32 [", m, "] or [", m, ", ", K / 32, "], got ", sx.sizes()));
    if (group != 32)
        return result3(W4Q_ERR_UNSUPPORTED, Tensor());
    if (m == 0 || N <= 0 || K <= 0)  // a tensor without elements has no address
        return result3(W4Q_ERR_INVALID_ARG, Tensor());
    const size_t bytes = w4_packed_bytes(N, K, 32);
    if (bytes != 0 && (size_t)packed.numel() < bytes)
        C10_THROW_ERROR(ValueError, c10::str("packed must have ", bytes, " bytes, got ", packed.numel()));
    const OnStream on(c, a[8]);
    const Tensor out = out_or_new(c, a[6], "out", {m, N}, at::kBFloat16);
    const size_t need = a[7] == Py_None ? w4_workspace_bytes(m, N, K, 32) : 0;
    const Tensor ws = scratch(c, a[7], need);
    const int st = w4a8_gemm_codes(static_cast<const int8_t *>(xq.data_ptr()), static_cast<const float *>(sx.data_ptr()), row,
                                   packed.data_ptr(), out.data_ptr(), m, N, K, 32, ws.data_ptr(), ws.nbytes(), on.stream);
    return result3(st, out);
    END_HANDLE_TH_ERRORS
}

// y, x, A, B, ids, scales, out, workspace, stream
PyObject *py_lora_add(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 9);
    Call c;
    const Rows y = rows_of(c, a[0], "y", -1, -1), x = rows_of(c, a[1], "x", y.tokens, -1);
    const Tensor &A = c.dense(a[2], "A", at::kBFloat16), &B = c.dense(a[3], "B", at::kBFloat16);
    if (A.dim() != 3 || B.dim() != 3 || B.size(0) != A.size(0) || B.size(2) != A.size(1) || A.size(2) != x.n || B.size(1) != y.n)
        C10_THROW_ERROR(ValueError, c10::str("A must be [adapters, rank, ", x.n, "], B [adapters, ", y.n, ", rank], got ", A.sizes(),
                                             " and ", B.sizes()));
    const int64_t adapters = A.size(0), rank = A.size(1);
    const int32_t *ids = static_cast<const int32_t *>(c.optional(a[4], "ids", at::kInt, y.tokens));
    if (a[4] == Py_None)
        fail("ids", "must be given");
    const float *scales = static_cast<const float *>(c.optional(a[5], "scales", at::kFloat, adapters));
    const OnStream on(c, a[8]);
    Tensor out;
    const Rows o = rows_out(c, a[6], "out", y.tokens, y.n, &out);
    const Tensor ws = scratch(c, a[7], lora_workspace_bytes(y.tokens, x.n, y.n, rank, adapters));
    const int st = lora_add(y.ptr, y.stride, x.ptr, x.stride, A.data_ptr(), B.data_ptr(), ids, scales, o.ptr, o.stride, y.tokens,
                            x.n, y.n, rank, adapters, ws.data_ptr(), ws.nbytes(), on.stream);
    return result3(st, out);
    END_HANDLE_TH_ERRORS
}

// logits, drafts, uniforms, noise, draft_probs, counts, temperature, tokens, accepted, logprobs, workspace, stream
PyObject *py_verify_drafts(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 12);
    Call c;
    const Tensor &l = c.cuda(a[0], "logits");
    if ((l.scalar_type() != at::kBFloat16 && l.scalar_type() != at::kFloat) || l.dim() != 3)
        fail("logits", "must be bfloat16 or float32 [seqs, drafts + 1, vocab]");
    const int64_t s = l.size(0), m = l.size(1), v = l.size(2);
    if (m < 1)
        fail("logits", "must have a row behind the last draft");
    if ((v > 1 && l.stride(2) != 1) || (s > 1 && m > 1 && l.stride(0) != m * l.stride(1)))
        fail("logits", "must hold a row's elements one after the other and its rows at one stride");
    const int64_t stride = m > 1 ? l.stride(1) : (s > 1 ? l.stride(0) : v), d = m - 1;
    const Tensor &ids = c.dense(a[1], "drafts", at::kInt);
    if (ids.numel() != s * d)
        C10_THROW_ERROR(ValueError, c10::str("drafts must be [", s, ", ", d, "], got ", ids.sizes()));
    void *u = c.optional(a[2], "uniforms", at::kFloat, s * d), *e = c.optional(a[3], "noise", at::kFloat, s * v);
    void *q = c.optional(a[4], "draft_probs", at::kFloat, s * d * v);
    void *counts = c.optional(a[5], "counts", at::kInt, s), *heat = c.optional(a[6], "temperature", at::kFloat, s);
    void *logprobs = c.optional(a[9], "logprobs", at::kFloat, s * m);
    const OnStream on(c, a[11]);
    const Tensor tokens = out_or_new(c, a[7], "tokens", {s, m}, at::kInt), accepted = out_or_new(c, a[8], "accepted", {s}, at::kInt);
    const Tensor ws = scratch(c, a[10], verify_workspace_bytes(s, d, v));
    const int st = verify_drafts(l.data_ptr(), stride, l.scalar_type() == at::kFloat, static_cast<const int32_t *>(ids.data_ptr()),
                                 static_cast<const float *>(q), static_cast<const int32_t *>(counts), static_cast<const float *>(heat),
                                 static_cast<const float *>(u), static_cast<const float *>(e), s, d, v,
                                 static_cast<int32_t *>(tokens.data_ptr()), static_cast<int32_t *>(accepted.data_ptr()),
                                 static_cast<float *>(logprobs), ws.data_ptr(), ws.nbytes(), on.stream);
    return result3(st, tokens, accepted);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"qk_norm_rope", (PyCFunction)(void (*)(void))py_qk_norm_rope, METH_FASTCALL, nullptr},
    {"kv8_append", (PyCFunction)(void (*)(void))py_kv8_append, METH_FASTCALL, nullptr},
    {"kv8_read", (PyCFunction)(void (*)(void))py_kv8_read, METH_FASTCALL, nullptr},
    {"kv8_attention", (PyCFunction)(void (*)(void))py_kv8_attention, METH_FASTCALL, nullptr},
    {"moe_w4a16", (PyCFunction)(void (*)(void))py_moe_w4a16, METH_FASTCALL, nullptr},
    {"add_rms_norm", (PyCFunction)(void (*)(void))py_add_rms_norm, METH_FASTCALL, nullptr},
    {"add_rms_norm_a8", (PyCFunction)(void (*)(void))py_add_rms_norm_a8, METH_FASTCALL, nullptr},
    {"w4a8_gemm_codes", (PyCFunction)(void (*)(void))py_w4a8_gemm_codes, METH_FASTCALL, nullptr},
    {"lora_add", (PyCFunction)(void (*)(void))py_lora_add, METH_FASTCALL, nullptr},
    {"verify_drafts", (PyCFunction)(void (*)(void))py_verify_drafts, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w4q_binding", "Argument marshalling of libw4q.so's decode-step operators.",
                      -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w4q_binding(void) { return PyModule_Create(&module); }
