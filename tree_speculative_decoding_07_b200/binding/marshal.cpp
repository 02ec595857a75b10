// marshal.cpp -- argument marshalling of the calls on the paged cache, in C++.
//
// A small call's kernels take 5 to 10 us; checking a dozen tensors, filling the
// descriptors and allocating the outputs took about as long again in Python
// (15 us for one new token over 128 cached ones, 7 here).  This module does just
// that: it checks the tensors, fills tv_cache_desc and tv_rotary_desc, allocates
// what was not given and calls libtreeverify.  Nothing is computed or kept here.
//
// Errors: TypeError and ValueError for tensors that do not fit, the module's
// TreeVerifyError for a status that is not TV_OK, torch's own for an
// allocation that fails.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "treeverify.h"

namespace {

PyObject* g_error = nullptr;  // TreeVerifyError(status, what)

struct Raised {};  // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Raised();
}
[[noreturn]] void type_error(const std::string& what) { refuse(PyExc_TypeError, what); }
[[noreturn]] void value_error(const std::string& what) { refuse(PyExc_ValueError, what); }

void check(tv_status s, const char* what) {
    if (s == TV_OK) return;
    if (PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, what)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

std::string shape_of(c10::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument, or nullptr for None.  All of a call's have to lie on one GPU: Launch refuses
// host tensors, after the checks of types, shapes and strides, which therefore need no GPU.
struct Args {
    PyObject* const* v;
    int device = -1;
    bool on_host = false;

    const at::Tensor* tensor(int i, const char* name, bool optional = false) {
        if (v[i] == Py_None) {
            if (!optional) type_error(std::string(name) + " is required");
            return nullptr;
        }
        if (!THPVariable_Check(v[i])) type_error(std::string(name) + " must be a tensor");
        const at::Tensor& t = THPVariable_Unpack(v[i]);
        if (!t.is_cuda()) on_host = true;
        else if (device < 0) device = t.get_device();
        else if (t.get_device() != device)
            value_error("all tensors must be on one GPU: cuda:" + std::to_string(device) + " and cuda:" +
                        std::to_string(t.get_device()));
        return &t;
    }
    int64_t integer(int i, const char* name, int64_t lo = INT32_MIN, int64_t hi = INT32_MAX) const {
        PyObject* x = PyNumber_Index(v[i]);
        if (!x) throw Raised();
        int over = 0;
        const long long r = PyLong_AsLongLongAndOverflow(x, &over);
        Py_DECREF(x);
        if (over || r < lo || r > hi) value_error(std::string(name) + " is out of range");
        return r;
    }
    float real(int i) const {
        const double r = PyFloat_AsDouble(v[i]);
        if (r == -1.0 && PyErr_Occurred()) throw Raised();
        return (float)r;
    }
};

// The GPU and the stream of a call, made current for it, so that what is allocated
// belongs to the stream that the kernels run on.
struct Launch {
    std::optional<c10::cuda::CUDAStreamGuard> stream_guard;
    std::optional<c10::cuda::CUDAGuard> device_guard;
    void* stream = nullptr;

    Launch(PyObject* s, const Args& args) {
        if (args.on_host || args.device < 0) value_error("all tensors must be CUDA tensors");
        const int device = args.device;
        if (s == Py_None) {
            if (c10::cuda::current_device() != device) device_guard.emplace((c10::DeviceIndex)device);
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
            return;
        }
        uintptr_t raw = 0;
        if (PyLong_Check(s)) {
            raw = (uintptr_t)PyLong_AsSize_t(s);
        } else {
            PyObject* index = PyObject_GetAttrString(s, "device_index");
            if (!index) throw Raised();
            const long at = PyLong_AsLong(index);
            Py_DECREF(index);
            if (at != device && !PyErr_Occurred())
                value_error("the stream is on cuda:" + std::to_string(at) + ", the tensors on cuda:" +
                            std::to_string(device));
            PyObject* p = PyErr_Occurred() ? nullptr : PyObject_GetAttrString(s, "cuda_stream");
            if (!p) throw Raised();
            raw = (uintptr_t)PyLong_AsSize_t(p);
            Py_DECREF(p);
        }
        if (PyErr_Occurred()) throw Raised();
        stream = reinterpret_cast<void*>(raw);
        if (raw) stream_guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                                       (c10::DeviceIndex)device));
        else stream_guard.emplace(c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)device));
    }
};

// A contiguous tensor of the given type and shape.
void want(const char* name, const at::Tensor& t, at::ScalarType type, c10::IntArrayRef shape) {
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + c10::toString(type) + ", not " + c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
        value_error(std::string(name) + " must have the shape " + shape_of(shape) + ", not " + shape_of(t.sizes()));
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}

// An empty tensor has no address, which the C calls would take for "not given".
void want_status(const at::Tensor& t) {
    want("dev_status", t, at::kInt, t.sizes());
    if (t.numel() == 0) value_error("dev_status must have an element");
}

// Sums per cached token: [batch][heads][width]; the width.
int64_t want_sums(const char* name, const at::Tensor& t, int64_t batch, int64_t heads) {
    const int64_t width = t.dim() ? t.size(-1) : 0;
    want(name, t, at::kFloat, {batch, heads, width});
    if (width == 0) value_error(std::string(name) + " must have an entry for every cached token");
    return width;
}

at::Tensor make(c10::IntArrayRef shape, at::ScalarType type, int device) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(c10::DeviceType::CUDA, (c10::DeviceIndex)device));
}

template <typename T = void> T* ptr(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
template <typename T = void> T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

int32_t narrow(int64_t x, const char* name) {
    if (x > INT32_MAX) value_error(std::string(name) + " is too large");
    return (int32_t)x;
}

// Strides of the first three dimensions of a cache (those of dimensions of size 1 say nothing: the
// row's); the last has to be 1, and no two rows may share memory.
void row_strides(const char* name, const at::Tensor& c, int64_t (&s)[3]) {
    const int64_t d = c.size(3);
    if (c.stride(3) != 1 && d > 1) value_error(std::string(name) + ": the elements of a head's row must be contiguous");
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i) s[i] = c.size(i) > 1 ? c.stride(i) : d;
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[order[j]] < s[order[i]]) std::swap(order[i], order[j]);
    int64_t end = d;
    for (int i : order)
        if (c.size(i) > 1) {
            if (s[i] < end) value_error(std::string(name) + ": rows overlap");
            end = s[i] * (c.size(i) - 1) + end;
        }
}

tv_cache_desc describe(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, int64_t heads, float scale,
                         int64_t max_kv_len) {
    tv_cache_desc d = {};
    switch (k.scalar_type()) {
        case at::kBFloat16: d.dtype = TV_BF16; break;
        case at::kFloat: d.dtype = TV_F32; break;
        case at::kHalf: d.dtype = TV_F16; break;
        default: type_error(std::string("unsupported dtype ") + c10::toString(k.scalar_type()));
    }
    if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
        type_error("k_cache and v_cache must be [num_blocks][block_size][num_kv_heads][head_dim] of one type");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || !table.is_contiguous())
        type_error("block_table must be a contiguous int32 [batch][max_blocks]");
    d.batch = narrow(table.size(0), "batch");
    d.num_kv_heads = narrow(k.size(2), "num_kv_heads");
    d.num_q_heads = heads < 0 ? d.num_kv_heads : narrow(heads, "num_q_heads");
    d.head_dim = narrow(k.size(3), "head_dim");
    d.block_size = narrow(k.size(1), "block_size");
    d.max_blocks_per_seq = narrow(table.size(1), "max_blocks_per_seq");
    d.num_blocks = narrow(k.size(0), "num_blocks");
    d.softmax_scale = scale;
    d.max_kv_len = (int32_t)max_kv_len;
    if (!k.is_contiguous() || !v.is_contiguous()) {
        int64_t sk[3], sv[3];
        row_strides("k_cache", k, sk);
        row_strides("v_cache", v, sv);
        if (sk[0] != sv[0] || sk[1] != sv[1] || sk[2] != sv[2])
            value_error("k_cache and v_cache must have the same strides");
        d.block_stride = sk[0];
        d.token_stride = sk[1];
        d.head_stride = sk[2];
    }
    return d;
}

// A stride between rows, for a descriptor in which 0 means contiguous: an expanded tensor's 0 would be
// read as that, far past the one row that it has.
int64_t row_apart(const char* name, const char* of, int64_t stride, int64_t row) {
    if (stride < row)
        value_error(std::string(name) + ": the rows of one " + of + " must not overlap the next one's (stride " +
                    std::to_string(stride) + ", row " + std::to_string(row) + "; call contiguous() on an expanded tensor)");
    return stride;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* x = THPVariable_Wrap(a);
    PyObject* y = x ? THPVariable_Wrap(b) : nullptr;
    PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

// (k_cache, v_cache, block_table, num_q_heads or None, softmax_scale, max_kv_len) -> the descriptor's bytes; the
// tensors may lie anywhere
PyObject* cache_desc(Args a) {
    const at::Tensor &k = *a.tensor(0, "k_cache"), &v = *a.tensor(1, "v_cache"), &table = *a.tensor(2, "block_table");
    const int64_t heads = a.v[3] == Py_None ? -1 : a.integer(3, "num_q_heads", 0);
    const tv_cache_desc d = describe(k, v, table, heads, a.real(4), a.integer(5, "max_kv_len"));
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&d), sizeof d);
}

// (q, k_cache, v_cache, block_table, kv_lens, softmax_scale, attn_weights, out, lse, workspace, max_kv_len,
//  dev_status, stream) -> (out, lse)
PyObject* decode_attention(Args a) {
    const at::Tensor &q = *a.tensor(0, "q"), &k = *a.tensor(1, "k_cache"), &v = *a.tensor(2, "v_cache");
    const at::Tensor &table = *a.tensor(3, "block_table"), &lens = *a.tensor(4, "kv_lens");
    const at::Tensor *w = a.tensor(6, "attn_weights", true), *out_p = a.tensor(7, "out", true);
    const at::Tensor *lse_p = a.tensor(8, "lse", true), *ws_p = a.tensor(9, "workspace", true);
    const at::Tensor* status = a.tensor(11, "dev_status", true);
    if (q.dim() != 3 || q.scalar_type() != k.scalar_type())
        type_error("q must be [batch][heads][head_dim] of the caches' type");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    tv_cache_desc d = describe(k, v, table, Hq, a.real(5), a.integer(10, "max_kv_len"));
    if (d.batch != B || d.head_dim != D) value_error("q, block_table and the caches disagree on batch or head_dim");
    if (!q.is_contiguous()) {
        if ((D > 1 && q.stride(2) != 1) || (Hq > 1 && q.stride(1) != D))
            value_error("q: the heads of a sequence must be contiguous");
        if (B > 1) d.q_stride = row_apart("q", "sequence", q.stride(0), Hq * D);
    }
    want("kv_lens", lens, at::kInt, {B});
    if (w) d.weight_stride = want_sums("attn_weights", *w, B, d.num_kv_heads);
    if (status) want_status(*status);
    if (out_p) want("out", *out_p, q.scalar_type(), {B, Hq, D});
    if (lse_p) want("lse", *lse_p, at::kFloat, {B, Hq});
    Launch launch(a.v[12], a);
    tv_decode_plan plan;
    check(tv_decode_attention_plan(&d, w != nullptr, &plan), "tv_decode_attention_plan");
    at::Tensor out = out_p ? *out_p : make({B, Hq, D}, q.scalar_type(), a.device);
    at::Tensor lse = lse_p ? *lse_p : make({B, Hq}, at::kFloat, a.device);
    at::Tensor ws;
    size_t bytes = plan.workspace_bytes;
    if (ws_p) {
        if (!ws_p->is_contiguous()) value_error("workspace must be contiguous");
        ws = *ws_p;
        bytes = (size_t)ws.numel() * ws.element_size();
    } else if (bytes) {
        ws = make({(int64_t)bytes}, at::kByte, a.device);
    }
    check(tv_decode_attention(&d, ptr(q), ptr(k), ptr(v), ptr<int32_t>(table), ptr<int32_t>(lens), ptr(out),
                              ptr<float>(lse), ptr<float>(w), ws.defined() ? ptr(ws) : nullptr, bytes,
                              ptr<int32_t>(status), launch.stream),
          "tv_decode_attention");
    return pair(out, lse);
}

// (k_cache, v_cache, block_table, kv_lens, weights, budget, sink, recent, dst_block_table, weights_out, kept,
//  new_kv_lens, max_kv_len, dev_status, stream) -> (new_kv_lens, kept)
PyObject* evict_cache(Args a) {
    const at::Tensor &k = *a.tensor(0, "k_cache"), &v = *a.tensor(1, "v_cache"), &table = *a.tensor(2, "block_table");
    const at::Tensor &lens = *a.tensor(3, "kv_lens"), &w = *a.tensor(4, "weights");
    const at::Tensor *dst = a.tensor(8, "dst_block_table", true), *wo = a.tensor(9, "weights_out", true);
    const at::Tensor *kept_p = a.tensor(10, "kept", true), *new_p = a.tensor(11, "new_kv_lens", true);
    const at::Tensor* status = a.tensor(13, "dev_status", true);
    tv_cache_desc d = describe(k, v, table, -1, 0.f, a.integer(12, "max_kv_len"));
    const int64_t B = d.batch, H = d.num_kv_heads, budget = a.integer(5, "budget");
    const int64_t sink = a.integer(6, "sink"), recent = a.integer(7, "recent");
    want("kv_lens", lens, at::kInt, {B});
    const int64_t width = want_sums("weights", w, B, H);
    d.weight_stride = width;
    if (wo) want("weights_out", *wo, at::kFloat, {B, H, width});
    if (dst) want("dst_block_table", *dst, at::kInt, table.sizes());
    if (kept_p) want("kept", *kept_p, at::kInt, {B, H, budget});
    if (new_p) want("new_kv_lens", *new_p, at::kInt, {B});
    if (status) want_status(*status);
    Launch launch(a.v[14], a);
    at::Tensor kept = kept_p ? *kept_p : make({B, H, budget > 0 ? budget : 0}, at::kInt, a.device);
    at::Tensor lens_out = new_p ? *new_p : make({B}, at::kInt, a.device);
    check(tv_evict_cache(&d, (int32_t)budget, (int32_t)sink, (int32_t)recent, ptr(k), ptr(v), ptr<int32_t>(table),
                         ptr<int32_t>(lens), ptr<float>(w), ptr<int32_t>(dst), ptr<float>(wo), ptr<int32_t>(kept),
                         ptr<int32_t>(lens_out), ptr<int32_t>(status), launch.stream),
          "tv_evict_cache");
    return pair(lens_out, kept);
}

// Elements between consecutive nodes of [B][N][H][D]: heads contiguous, sequences N nodes apart.
int64_t node_stride(const char* name, const at::Tensor& t) {
    if (t.is_contiguous()) return 0;
    const int64_t B = t.size(0), N = t.size(1), H = t.size(2), D = t.size(3);
    if ((D > 1 && t.stride(3) != 1) || (H > 1 && t.stride(2) != D))
        value_error(std::string(name) + ": the heads of a node must be contiguous");
    if (N == 1) return B > 1 ? row_apart(name, "sequence", t.stride(0), H * D) : 0;
    if (B > 1 && t.stride(0) != N * t.stride(1))
        value_error(std::string(name) + ": sequences must lie num_nodes nodes apart");
    return row_apart(name, "node", t.stride(1), H * D);
}

// (k, v, inv_freq, k_cache, v_cache, block_table, prefix_lens, q, q_out, parent_idx, positions, position_base,
//  axis_of_pair (bytes), interleaved, node_counts, dev_status, stream) -> q_out
PyObject* rotary_write(Args a) {
    const at::Tensor &k = *a.tensor(0, "k"), &v = *a.tensor(1, "v"), &freq = *a.tensor(2, "inv_freq");
    const at::Tensor &ck = *a.tensor(3, "k_cache"), &cv = *a.tensor(4, "v_cache"), &table = *a.tensor(5, "block_table");
    const at::Tensor &prefix = *a.tensor(6, "prefix_lens"), *q = a.tensor(7, "q", true), *out_p = a.tensor(8, "q_out", true);
    const at::Tensor *parent = a.tensor(9, "parent_idx", true), *pos = a.tensor(10, "positions", true);
    const at::Tensor *base = a.tensor(11, "position_base", true), *counts = a.tensor(14, "node_counts", true);
    const at::Tensor* status = a.tensor(15, "dev_status", true);
    const at::ScalarType type = k.scalar_type();
    if (k.dim() != 4 || v.sizes() != k.sizes() || type != ck.scalar_type() || v.scalar_type() != type)
        type_error("k and v must be [batch][nodes][num_kv_heads][head_dim] of the caches' type");
    const int64_t B = k.size(0), N = k.size(1), H = k.size(2), D = k.size(3);
    int64_t Hq = H;
    tv_rotary_desc r = {};
    if (q) {
        if (q->dim() != 4 || q->scalar_type() != type || q->size(0) != B || q->size(1) != N || q->size(3) != D)
            type_error("q must be [batch][nodes][num_q_heads][head_dim] of k's type");
        Hq = q->size(2);
        r.q_stride = node_stride("q", *q);
    }
    tv_cache_desc d = describe(ck, cv, table, Hq, 0.f, 0);
    if (d.batch != B || d.num_kv_heads != H || d.head_dim != D)
        value_error("k, block_table and the caches disagree on batch, heads or head_dim");
    const int64_t pairs = freq.numel();
    if (pairs > 128) value_error("inv_freq must have at most 128 entries");
    want("inv_freq", freq, at::kFloat, {pairs});
    want("prefix_lens", prefix, at::kInt, {B});
    if (base) want("position_base", *base, at::kInt, {B});
    if (parent) want("parent_idx", *parent, at::kInt, {B, N});
    if (counts) want("node_counts", *counts, at::kInt, {B});
    if (status) want_status(*status);
    r.num_nodes = narrow(N, "num_nodes");
    r.rotary_dim = (int32_t)(2 * pairs);
    r.interleaved = PyObject_IsTrue(a.v[13]);
    if (r.interleaved < 0) throw Raised();
    r.num_axes = 1;
    r.k_stride = node_stride("k", k);
    r.v_stride = node_stride("v", v);
    r.node_counts = ptr<int32_t>(counts);
    if (a.v[12] != Py_None) {
        char* axes;
        Py_ssize_t n;
        if (PyBytes_AsStringAndSize(a.v[12], &axes, &n) < 0) throw Raised();
        if (n != pairs) value_error("axis_of_pair must have an entry for each of inv_freq");
        for (Py_ssize_t i = 0; i < n; ++i) {
            r.axis_of_pair[i] = (uint8_t)axes[i];
            if (r.axis_of_pair[i] >= r.num_axes) r.num_axes = r.axis_of_pair[i] + 1;
        }
    }
    if (pos) {
        const int64_t n = pos->dim() ? pos->size(0) : 0;
        if (n < r.num_axes) value_error("axis_of_pair names an axis that positions lacks");
        want("positions", *pos, at::kInt, {n, B, N});
        r.num_axes = narrow(n, "num_axes");
    }
    if (out_p) want("q_out", *out_p, type, {B, N, Hq, D});
    Launch launch(a.v[16], a);
    at::Tensor out;
    if (out_p) out = *out_p;
    else if (q) out = make({B, N, Hq, D}, type, a.device);
    check(tv_rotary_write(&d, &r, ptr(q), ptr(k), ptr(v), ptr<float>(freq), ptr<int32_t>(parent), ptr<int32_t>(pos),
                          ptr<int32_t>(base), ptr<int32_t>(prefix), ptr<int32_t>(table),
                          out.defined() ? ptr(out) : nullptr, ptr(ck), ptr(cv), ptr<int32_t>(status), launch.stream),
          "tv_rotary_write");
    if (!out.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(out);
}

template <PyObject* (*F)(Args), int COUNT> PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != COUNT) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return F(Args{args});
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

#define FAST(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FAST(decode_attention, 13), FAST(evict_cache, 15), FAST(rotary_write, 17), FAST(cache_desc, 6),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
