// paged_tensors.cpp -- the tensor forms of the paged-cache entry points: reads addresses,
// shapes and strides off torch tensors, checks them, fills the descriptor and calls the
// library (module _paged of the package; device.py has the documented functions).
//
// A decode step is a few microseconds on the GPU, and a dozen tensors take as long to be
// asked for their shapes and strides from Python: paged_rows 7.7 us there, 1 us here.
//
// Each function takes its arguments by position and returns the library's status.  What
// the tensors get wrong is a ValueError that names the argument.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <string>

#include "gattn.h"

namespace {

struct Bad {};             // a Python error is set

[[noreturn]] void bad(const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(PyExc_ValueError, fmt, ap);
    va_end(ap);
    throw Bad();
}

std::string shape_of(const at::Tensor &t)
{
    std::string s = "got (";
    for (int64_t x : t.sizes())
        s += std::to_string(x) + ",";
    s += "), strides (";
    for (int64_t x : t.strides())
        s += std::to_string(x) + ",";
    return s + ")";
}

// The arguments of a call and the device of its first tensor.
struct Args {
    PyObject *const *v;
    int64_t dev = 0;

    bool none(int i) const { return v[i] == Py_None; }
    int64_t num(int i) const
    {
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred())
            throw Bad();
        return x;
    }
    int32_t i32(int i, const char *name) const
    {
        const int64_t x = num(i);
        if (x != (int32_t)x)
            bad("%s is out of range", name);
        return (int32_t)x;
    }
    float real(int i) const
    {
        const double x = PyFloat_AsDouble(v[i]);
        if (x == -1.0 && PyErr_Occurred())
            throw Bad();
        return (float)x;
    }
    const at::Tensor &any(int i, const char *name) const
    {
        if (!THPVariable_Check(v[i]))
            bad("%s must be a tensor", name);
        return THPVariable_Unpack(v[i]);
    }
    // a tensor beside the first one, of one of two types
    const at::Tensor &of(int i, const char *name, at::ScalarType a, at::ScalarType b) const
    {
        const at::Tensor &t = any(i, name);
        if (t.layout() != at::kStrided)
            bad("%s must be a dense tensor", name);
        if (t.get_device() != dev)
            bad("%s lies on device %d, not beside the first tensor (%d)", name, (int)t.get_device(), (int)dev);
        if (t.scalar_type() != a && t.scalar_type() != b)
            bad("%s has type %s, not %s%s%s", name, c10::toString(t.scalar_type()), c10::toString(a),
                a == b ? "" : " or ", a == b ? "" : c10::toString(b));
        return t;
    }
    const at::Tensor &of(int i, const char *name, at::ScalarType a) const { return of(i, name, a, a); }
};

constexpr auto kF32 = at::kFloat, kBF16 = at::kBFloat16, kI32 = at::kInt;

// A dimension of one or no entries may have any stride: a valid one stands in.

struct Rows {
    void *p;
    int64_t tok, head;
};

// [rows][heads][elements]; the sizes that are given (>= 0) have to be those
Rows rows(const at::Tensor &t, const char *name, int64_t T, int64_t H, int64_t d)
{
    if (t.dim() != 3 || (T >= 0 && (t.size(0) != T || t.size(1) != H || t.size(2) != d)))
        T < 0 ? bad("%s must have shape [rows][heads][elements] (%s)", name, shape_of(t).c_str())
              : bad("%s must have shape [%lld][%lld][%lld] (%s)", name, (long long)T, (long long)H, (long long)d,
                    shape_of(t).c_str());
    if (t.size(2) > 1 && t.stride(2) != 1)
        bad("%s needs contiguous elements: %s", name, shape_of(t).c_str());
    return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(8, t.size(1) * t.size(2)),
            t.size(1) > 1 ? t.stride(1) : std::max<int64_t>(8, t.size(2))};
}

// a contiguous vector of n entries; NULL for None
void *flat(const Args &a, int i, const char *name, at::ScalarType type, int64_t n)
{
    if (a.none(i))
        return nullptr;
    const at::Tensor &t = a.of(i, name, type);
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        bad("%s must have shape [%lld], contiguous (%s)", name, (long long)n, shape_of(t).c_str());
    return t.data_ptr();
}

// row offsets: sets the number of sequences
const int32_t *offsets(const Args &a, int i, int32_t &n)
{
    const at::Tensor &t = a.of(i, "cu_rows", kI32);
    if (t.dim() != 1 || t.size(0) < 1 || t.size(0) > INT32_MAX || !t.is_contiguous())
        bad("cu_rows must have shape [num_seqs + 1], contiguous (%s)", shape_of(t).c_str());
    n = (int32_t)t.size(0) - 1;
    return static_cast<const int32_t *>(t.data_ptr());
}

struct Table {
    const int32_t *p;
    int32_t width;
    int64_t stride;
};

Table page_table(const Args &a, int i, const char *name, int64_t n)
{
    const at::Tensor &t = a.of(i, name, kI32);
    if (t.dim() != 2 || t.size(0) != n || (t.size(1) > 1 && t.stride(1) != 1) || t.size(1) > INT32_MAX)
        bad("%s must have shape [%lld][width], contiguous rows (%s)", name, (long long)n, shape_of(t).c_str());
    return {static_cast<const int32_t *>(t.data_ptr()), (int32_t)t.size(1),
            n > 1 ? t.stride(0) : std::max<int64_t>(1, t.size(1))};
}

// Pools [pages][Hk][page_size][d] and their table; iv < 0: keys only.
gattn_pages pools(const Args &a, int ik, int iv, int it, int64_t n, int32_t &Hk, int32_t &d)
{
    gattn_pages g = {};
    for (int x = 0; x < (iv < 0 ? 1 : 2); ++x) {
        const char *name = x ? "v_pages" : "k_pages";
        const at::Tensor &t = a.of(x ? iv : ik, name, kBF16);
        if (t.dim() != 4 || (t.size(3) > 1 && t.stride(3) != 1))
            bad("%s must have shape [pages][heads][page_size][elements], contiguous elements (%s)", name, shape_of(t).c_str());
        if (x == 0) {
            if (t.numel() > 0 && (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || t.size(2) > INT32_MAX || t.size(3) > INT32_MAX))
                bad("k_pages is too large");
            g.num_pages = (int32_t)t.size(0);
            Hk = (int32_t)t.size(1);
            g.page_size = (int32_t)t.size(2);
            d = (int32_t)t.size(3);
        } else if (t.size(0) != g.num_pages || t.size(1) != Hk || t.size(2) != g.page_size || t.size(3) != d) {
            bad("v_pages must have k_pages's shape (%s)", shape_of(t).c_str());
        }
        const int64_t tok = g.page_size > 1 ? t.stride(2) : std::max(8, d);
        const int64_t head = Hk > 1 ? t.stride(1) : std::max<int64_t>(8, (int64_t)g.page_size * d);
        const int64_t page = g.num_pages > 1 ? t.stride(0) : std::max<int64_t>(8, (int64_t)Hk * g.page_size * d);
        if (x) {
            g.v_pages = t.data_ptr();
            g.v_stride_token = tok, g.v_stride_head = head, g.v_stride_page = page;
        } else {
            g.k_pages = t.data_ptr();
            g.k_stride_token = tok, g.k_stride_head = head, g.k_stride_page = page;
        }
    }
    const Table t = page_table(a, it, "table", n);
    g.table = t.p;
    g.table_width = t.width;
    g.table_stride = t.stride;
    return g;
}

struct Received {
    float *p;
    int32_t width;
    int64_t seq, head;
};

// weights [n][Hk][positions]
Received received(const Args &a, int i, const char *name, int64_t n, int32_t Hk)
{
    const at::Tensor &t = a.of(i, name, kF32);
    if (t.dim() != 3 || t.size(0) != n || t.size(1) != Hk || (t.size(2) > 1 && t.stride(2) != 1) || t.size(2) > INT32_MAX)
        bad("%s must have shape [%lld][%d][positions], contiguous positions (%s)", name, (long long)n, (int)Hk,
            shape_of(t).c_str());
    return {static_cast<float *>(t.data_ptr()), (int32_t)t.size(2), n > 1 ? t.stride(0) : Hk * t.size(2),
            Hk > 1 ? t.stride(1) : t.size(2)};
}

int32_t dtype_of(const at::Tensor &t) { return t.scalar_type() == kF32 ? GATTN_DTYPE_F32 : GATTN_DTYPE_BF16; }

// sizes of the row tensors: [rows][heads][elements] of the first one
void sizes(const at::Tensor &q, int32_t &T, int32_t &H)
{
    if (q.numel() > 0 && (q.size(0) > INT32_MAX || q.size(1) > INT32_MAX))
        bad("q is too large");
    T = (int32_t)q.size(0);
    H = (int32_t)q.size(1);
}

void on_gpu(const Args &a)
{
    if (a.dev < 0)
        bad("the tensors must be on a CUDA device");
}

template <class F>
PyObject *call(F f)
{
    gattn_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

gattn_stream stream_of(const Args &a, int i) { return reinterpret_cast<gattn_stream>((uintptr_t)a.num(i)); }

// Runs f(args), with what it throws as a Python error.
template <class F>
PyObject *guarded(PyObject *const *v, Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want)
        return PyErr_Format(PyExc_TypeError, "%zd arguments are needed (got %zd)", want, n);
    try {
        Args a{v};
        return f(a);
    } catch (const Bad &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// q k v k_pages v_pages table cu_rows cache_pos positions q_norm k_norm q_out status
// rotary_dims rope_pairs rope_scaling rope_theta rope_factor rope_original beta_fast
// beta_slow rope_size rms_eps stream
PyObject *paged_rows(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    return guarded(v, n, 24, [](Args &a) {
        gattn_paged_rows_desc p = {};
        a.dev = a.any(0, "q").get_device();
        const at::Tensor &q = a.of(0, "q", kF32, kBF16);
        const Rows qr = rows(q, "q", -1, 0, 0);
        const int64_t d = q.size(2);
        sizes(q, p.total_rows, p.num_heads);
        p.cu_rows = offsets(a, 6, p.num_seqs);
        p.pages = pools(a, 3, 4, 5, p.num_seqs, p.num_kv_heads, p.head_dim);
        if (p.head_dim != d)
            bad("k_pages must have q's head_dim %lld (got %d)", (long long)d, (int)p.head_dim);
        const at::Tensor &k = a.of(1, "k", q.scalar_type()), &w = a.of(2, "v", q.scalar_type());
        const Rows kr = rows(k, "k", p.total_rows, p.num_kv_heads, d), vr = rows(w, "v", p.total_rows, p.num_kv_heads, d);
        const Rows o = rows(a.of(11, "q_out", kBF16), "q_out", p.total_rows, p.num_heads, d);
        p.x_dtype = dtype_of(q);
        p.cache_pos = static_cast<const int32_t *>(flat(a, 7, "cache_pos", kI32, p.num_seqs));
        p.positions = static_cast<const int32_t *>(flat(a, 8, "positions", kI32, p.total_rows));
        p.q_norm = static_cast<const uint16_t *>(flat(a, 9, "q_norm", kBF16, d));
        p.k_norm = static_cast<const uint16_t *>(flat(a, 10, "k_norm", kBF16, d));
        p.status = static_cast<uint32_t *>(flat(a, 12, "status", kI32, 1));
        p.q = qr.p, p.q_stride_token = qr.tok, p.q_stride_head = qr.head;
        p.k = kr.p, p.k_stride_token = kr.tok, p.k_stride_head = kr.head;
        p.v = vr.p, p.v_stride_token = vr.tok, p.v_stride_head = vr.head;
        p.q_out = o.p, p.o_stride_token = o.tok, p.o_stride_head = o.head;
        p.rotary_dims = a.i32(13, "rotary_dims");
        p.rope_pairs = a.i32(14, "rope_pairs");
        p.rope_scaling = a.i32(15, "rope_scaling");
        p.rope_theta = a.real(16);
        p.rope_factor = a.real(17);
        p.rope_original = a.i32(18, "original");
        p.rope_beta_fast = a.real(19);
        p.rope_beta_slow = a.real(20);
        p.rope_size = a.real(21);
        p.rms_eps = a.real(22);
        const gattn_stream s = stream_of(a, 23);
        on_gpu(a);
        if (!p.num_seqs || !p.total_rows)
            return PyLong_FromLong(0);
        return call([&] { return gattn_paged_rows(&p, s); });
    });
}

// What attention and weights have in common, arguments 0 .. 6:
// q k_pages v_pages table cu_rows cache_pos lse, then scale
void attended(Args &a, bool values, gattn_paged_attention_desc &p)
{
    a.dev = a.any(0, "q").get_device();
    const at::Tensor &q = a.of(0, "q", kBF16);
    const Rows qr = rows(q, "q", -1, 0, 0);
    const int64_t d = q.size(2);
    sizes(q, p.total_rows, p.num_heads);
    p.cu_rows = offsets(a, 4, p.num_seqs);
    p.pages = pools(a, 1, values ? 2 : -1, 3, p.num_seqs, p.num_kv_heads, p.head_dim);
    if (p.head_dim != d)
        bad("k_pages must have q's head_dim %lld (got %d)", (long long)d, (int)p.head_dim);
    p.q = qr.p, p.q_stride_token = qr.tok, p.q_stride_head = qr.head;
    p.cache_pos = static_cast<const int32_t *>(flat(a, 5, "cache_pos", kI32, p.num_seqs));
    if (!a.none(6)) {
        const at::Tensor &l = a.of(6, "lse", kF32);
        if (l.dim() != 2 || l.size(0) != p.total_rows || l.size(1) != p.num_heads || !l.is_contiguous())
            bad("lse must have shape [%d][%d], contiguous (%s)", (int)p.total_rows, (int)p.num_heads, shape_of(l).c_str());
        p.lse = static_cast<float *>(l.data_ptr());
    }
    p.scale = a.none(7) ? (float)(1. / std::sqrt((double)d)) : a.real(7);
}

// .. scale gate out workspace status stream
PyObject *paged_attention(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    return guarded(v, n, 13, [](Args &a) {
        gattn_paged_attention_desc p = {};
        attended(a, true, p);
        p.gate_dtype = GATTN_DTYPE_BF16;
        p.g_stride_token = p.g_stride_head = 8;
        if (!a.none(8)) {
            const at::Tensor &t = a.of(8, "gate", kF32, kBF16);
            const Rows g = rows(t, "gate", p.total_rows, p.num_heads, p.head_dim);
            p.gate = g.p, p.g_stride_token = g.tok, p.g_stride_head = g.head;
            p.gate_dtype = dtype_of(t);
        }
        const Rows o = rows(a.of(9, "out", kBF16), "out", p.total_rows, p.num_heads, p.head_dim);
        p.out = o.p, p.o_stride_token = o.tok, p.o_stride_head = o.head;
        const at::Tensor &w = a.of(10, "workspace", at::kByte);
        if (!w.is_contiguous())
            bad("workspace must be contiguous (%s)", shape_of(w).c_str());
        p.workspace = w.data_ptr();
        p.workspace_bytes = w.numel();
        p.status = static_cast<uint32_t *>(flat(a, 11, "status", kI32, 1));
        const gattn_stream s = stream_of(a, 12);
        on_gpu(a);
        if (!p.num_seqs || !p.total_rows)
            return PyLong_FromLong(0);
        return call([&] { return gattn_paged_attention(&p, s); });
    });
}

// .. scale weights weights_out status stream
PyObject *paged_weights(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    return guarded(v, n, 12, [](Args &a) {
        gattn_paged_weights_desc p = {};
        attended(a, false, p.attention);
        const int32_t seqs = p.attention.num_seqs, Hk = p.attention.num_kv_heads;
        const Received o = received(a, 9, "weights_out", seqs, Hk);
        p.weights_out = o.p, p.weights_width = o.width, p.w_stride_seq = o.seq, p.w_stride_head = o.head;
        if (!a.none(8)) {
            const Received i = received(a, 8, "weights", seqs, Hk);
            if (i.width != o.width || i.seq != o.seq || i.head != o.head)
                bad("weights must have weights_out's shape and strides");
            p.weights = i.p;
        }
        p.attention.status = static_cast<uint32_t *>(flat(a, 10, "status", kI32, 1));
        const gattn_stream s = stream_of(a, 11);
        if (!p.attention.lse)
            bad("lse must be a tensor");
        on_gpu(a);
        if (!seqs || !p.attention.total_rows)
            return PyLong_FromLong(0);
        return call([&] { return gattn_paged_weights(&p, s); });
    });
}

// k_pages v_pages table lengths weights keep recent out_table weights_out kept lengths_out
// status stream
PyObject *paged_evict(PyObject *, PyObject *const *v, Py_ssize_t n)
{
    return guarded(v, n, 13, [](Args &a) {
        gattn_paged_evict_desc p = {};
        a.dev = a.any(0, "k_pages").get_device();
        const at::Tensor &len = a.of(3, "lengths", kI32);
        if (len.dim() != 1 || !len.is_contiguous() || len.size(0) > INT32_MAX)
            bad("lengths must have shape [num_seqs], contiguous (%s)", shape_of(len).c_str());
        p.num_seqs = (int32_t)len.size(0);
        p.lengths = static_cast<const int32_t *>(len.data_ptr());
        p.pages = pools(a, 0, 1, 2, p.num_seqs, p.num_kv_heads, p.head_dim);
        const Received w = received(a, 4, "weights", p.num_seqs, p.num_kv_heads);
        p.weights = w.p, p.weights_width = w.width, p.w_stride_seq = w.seq, p.w_stride_head = w.head;
        p.keep = a.i32(5, "keep");
        p.recent = a.i32(6, "recent");
        if (!a.none(7)) {
            const Table t = page_table(a, 7, "out_table", p.num_seqs);
            p.out_table = t.p, p.out_table_width = t.width;
            p.out_table_stride = t.stride;
            // one sequence's table and a view of it: neither has a stride of its own
            if (p.num_seqs == 1 && t.p == p.pages.table)
                p.pages.table_stride = p.out_table_stride = std::max(p.pages.table_stride, t.stride);
        }
        if (!a.none(8)) {
            const Received o = received(a, 8, "weights_out", p.num_seqs, p.num_kv_heads);
            p.weights_out = o.p, p.weights_out_width = o.width, p.wo_stride_seq = o.seq, p.wo_stride_head = o.head;
        }
        const at::Tensor &k = a.of(9, "kept", kI32);
        if (k.dim() != 3 || k.size(0) != p.num_seqs || k.size(1) != p.num_kv_heads || k.size(2) != p.keep || !k.is_contiguous())
            bad("kept must be contiguous, of shape [%d][%d][%d] (%s)", (int)p.num_seqs, (int)p.num_kv_heads, (int)p.keep,
                shape_of(k).c_str());
        p.kept = static_cast<int32_t *>(k.data_ptr());
        p.lengths_out = static_cast<int32_t *>(flat(a, 10, "lengths_out", kI32, p.num_seqs));
        p.status = static_cast<uint32_t *>(flat(a, 11, "status", kI32, 1));
        const gattn_stream s = stream_of(a, 12);
        on_gpu(a);
        if (!p.num_seqs)
            return PyLong_FromLong(0);
        return call([&] { return gattn_paged_evict(&p, s); });
    });
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(paged_rows), FAST(paged_attention), FAST(paged_weights), FAST(paged_evict), {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
