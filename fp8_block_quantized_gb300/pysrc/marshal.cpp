// Argument marshalling of the operators around the linear layer, for Python.
//
// These calls run once or more per layer and decoding step, where reading a
// tensor's type, shape and address attribute by attribute in Python costs more
// than the kernel takes (9 to 20 us a call against 2 to 4).  Each function here
// checks the tensors it is given as binding.py does, takes their addresses and
// calls the C entry point of its name, whose address binding.py passes to
// bind().  A status other than JET_OK is raised as JetError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>

#include "jet_fp8.h"

namespace {

decltype(&jet_add_rmsnorm_quant_1x128) f_norm;
decltype(&jet_add_rmsnorm_bwd) f_norm_bwd;
decltype(&jet_rope) f_rope;
decltype(&jet_rope_kv_cache_write) f_rope_kv;
decltype(&jet_kv_slot_map) f_slots;
decltype(&jet_sample_unaligned) f_sample;
decltype(&jet_workspace_bytes) f_workspace;
decltype(&jet_kv_attention) f_attention;
decltype(&jet_kv_attention_workspace) f_attention_workspace;
decltype(&jet_head_logp) f_head;
decltype(&jet_head_logp_bwd) f_head_bwd;
decltype(&jet_swiglu_bwd_quant_1x128) f_swiglu_bwd;
PyObject *jet_error;

// Thrown once a Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const char *format, const char *name, PyObject *what) {
    PyErr_Format(type, format, name, what);
    throw Raised();
}

const char *type_name(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return "another type";
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s: expected a tensor, got %R", name, o);
    return THPVariable_Unpack(o);
}

void need_type(PyObject *o, const at::Tensor &t, at::ScalarType type, const char *name) {
    if (t.scalar_type() == type) return;
    PyObject *got = PyObject_GetAttrString(o, "dtype");
    if (!got) throw Raised();
    PyErr_Format(PyExc_TypeError, "%s: expected %s, got %S", name, type_name(type), got);
    Py_DECREF(got);
    throw Raised();
}

void *address(const at::Tensor &t) { return t.numel() ? t.data_ptr() : nullptr; }

// The address of a contiguous CUDA tensor of this type and shape, or of None.
template <typename T>
T *arg(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    need_type(o, t, type, name);
    if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size())) {
        PyObject *want = PyTuple_New((Py_ssize_t)shape.size()), *got = PyObject_GetAttrString(o, "shape");
        for (size_t i = 0; want && i < shape.size(); ++i)
            PyTuple_SET_ITEM(want, (Py_ssize_t)i, PyLong_FromLongLong(shape.begin()[i]));
        if (want && got) PyErr_Format(PyExc_ValueError, "%s: expected shape %R, got %R", name, want, got);
        Py_XDECREF(want);
        Py_XDECREF(got);
        throw Raised();
    }
    if (t.numel() && (!t.is_cuda() || !t.is_contiguous())) {
        PyErr_Format(PyExc_ValueError, "%s: must be a contiguous CUDA tensor", name);
        throw Raised();
    }
    return static_cast<T *>(address(t));
}

void need_dims(const at::Tensor &t, int64_t n, const char *name) {
    if (t.dim() == n) return;
    PyErr_Format(PyExc_ValueError, "%s: expected %s dimensions, got %lld", name, n == 2 ? "two" : "three",
                 (long long)t.dim());
    throw Raised();
}

// A tensor of two dimensions; its sizes.
std::pair<int64_t, int64_t> matrix(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    need_dims(t, 2, name);
    return {t.size(0), t.size(1)};
}

struct Heads {
    uint16_t *p = nullptr;
    int64_t ld = 0, H = 0;
};

// [T, H, D] BF16 heads, dense within a token; None has none.
Heads heads(PyObject *o, const char *name, int64_t T, int64_t D) {
    Heads h;
    if (o == Py_None) return h;
    const at::Tensor &t = tensor(o, name);
    need_type(o, t, at::kBFloat16, name);
    if (t.dim() != 3 || t.size(0) != T || t.size(2) != D) {
        PyErr_Format(PyExc_ValueError, "%s: expected %lld tokens of heads of %lld channels", name,
                     (long long)T, (long long)D);
        throw Raised();
    }
    h.H = t.size(1);
    h.ld = h.H * D;
    if (!t.numel()) return h;
    if (!t.is_cuda() || (D > 1 && t.stride(2) != 1) || (h.H > 1 && t.stride(1) != D)) {
        PyErr_Format(PyExc_ValueError,
                     "%s: must be a CUDA tensor whose tokens hold contiguous heads", name);
        throw Raised();
    }
    h.p = static_cast<uint16_t *>(t.data_ptr());
    if (T > 1) h.ld = t.stride(0);
    return h;
}

int64_t numel(PyObject *o, const char *name) { return tensor(o, name).numel(); }

// None, or a tensor of the current device (whose stream the call runs on).
void on_this_device(PyObject *o) {
    if (o == Py_None) return;
    const at::Tensor &t = tensor(o, "argument");
    if (t.numel() && t.is_cuda() && t.get_device() != c10::cuda::current_device()) {
        PyErr_SetString(PyExc_ValueError, "the tensors must be on the current device");
        throw Raised();
    }
}

// The workspace given, or `need` bytes allocated beside `like` on the current stream.
at::Tensor workspace(PyObject *o, const at::Tensor &like, size_t need) {
    if (o != Py_None) {
        const at::Tensor &t = tensor(o, "ws");
        on_this_device(o);
        arg<void>(o, "ws", t.scalar_type(), {t.numel()});
        return t;
    }
    return need ? at::empty({(int64_t)need}, like.options().dtype(at::kByte)) : at::Tensor();
}

// The stream to run on: None is the current one; else a stream object or its handle.
void *stream_of(PyObject *o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
    if (!h) {
        PyErr_Clear();
        h = Py_NewRef(o);
    }
    void *s = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Raised();
    return s;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

// Calls the library without the interpreter's lock (a launch can wait for room in
// the stream's queue) and raises what it returns.
template <typename F>
void call(const char *fn, F f) {
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f();
    Py_END_ALLOW_THREADS;
    if (status == JET_OK) return;
    if (PyObject *args = Py_BuildValue("(si)", fn, status)) {
        PyErr_SetObject(jet_error, args);
        Py_DECREF(args);
    }
    throw Raised();
}

// ------------------------------------------------------------------ the calls

void norm(PyObject *const *a) {  // x, d, g, eps, h, q, s, rstd, stream
    const auto size = matrix(a[0], "x");
    const int64_t M = size.first, K = size.second;
    const auto *x = arg<uint16_t>(a[0], "x", at::kBFloat16, {M, K});
    const auto *d = arg<uint16_t>(a[1], "d", at::kBFloat16, {M, K});
    const auto *g = arg<uint16_t>(a[2], "g", at::kBFloat16, {K});
    const float eps = (float)number(a[3]);
    auto *h = arg<uint16_t>(a[4], "h", at::kBFloat16, {M, K});
    auto *q = arg<uint8_t>(a[5], "q", at::kByte, {M, K});
    auto *s = arg<float>(a[6], "s", at::kFloat, {K / 128, M});
    auto *rstd = arg<float>(a[7], "rstd", at::kFloat, {M});
    void *stream = stream_of(a[8]);
    call("jet_add_rmsnorm_quant_1x128",
         [&] { return f_norm(x, d, g, M, K, eps, h, q, s, rstd, stream); });
}

void norm_bwd(PyObject *const *a) {  // h, g, rstd, dys (a tuple), dres, dx, dg, ws, stream
    const auto size = matrix(a[0], "h");
    const int64_t M = size.first, K = size.second;
    const auto *h = arg<uint16_t>(a[0], "h", at::kBFloat16, {M, K});
    const auto *g = arg<uint16_t>(a[1], "g", at::kBFloat16, {K});
    const auto *rstd = arg<float>(a[2], "rstd", at::kFloat, {M});
    const Py_ssize_t n = PyTuple_Size(a[3]);
    if (n < 0) throw Raised();
    if (n < 1 || n > 3) {
        PyErr_Format(PyExc_ValueError, "dys: expected one to three gradients, got %zd", n);
        throw Raised();
    }
    const uint16_t *dy[3] = {};
    for (Py_ssize_t i = 0; i < n; ++i)
        dy[i] = arg<uint16_t>(PyTuple_GET_ITEM(a[3], i), "dys", at::kBFloat16, {M, K});
    const auto *dres = arg<uint16_t>(a[4], "dres", at::kBFloat16, {M, K});
    auto *dx = arg<uint16_t>(a[5], "dx", at::kBFloat16, {M, K});
    auto *dg = arg<float>(a[6], "dg", at::kFloat, {K});
    at::Tensor ws;  // given, or allocated on the current stream
    if (a[7] == Py_None) {
        const size_t need = f_workspace(JET_OP_ADD_RMSNORM_BWD, M, 0, K);
        if (need) ws = at::empty({(int64_t)need}, tensor(a[0], "h").options().dtype(at::kByte));
    } else {
        ws = tensor(a[7], "ws");
        arg<void>(a[7], "ws", ws.scalar_type(), {ws.numel()});
    }
    void *room = ws.defined() ? address(ws) : nullptr, *stream = stream_of(a[8]);
    const size_t bytes = ws.defined() ? ws.nbytes() : 0;
    call("jet_add_rmsnorm_bwd", [&] {
        return f_norm_bwd(h, g, rstd, dy[0], dy[1], dy[2], dres, M, K, dx, dg, room, bytes, stream);
    });
}

void rope(PyObject *const *a) {  // q, k, inv_freq, pos, q_out, k_out, layout, mscale, backward, stream
    const char *first = a[0] != Py_None ? "q" : "k";
    const at::Tensor &t = tensor(a[0] != Py_None ? a[0] : a[1], first);
    need_dims(t, 3, first);
    const int64_t T = t.size(0), D = t.size(2), R = 2 * numel(a[2], "inv_freq");
    const Heads q = heads(a[0], "q", T, D), k = heads(a[1], "k", T, D);
    const Heads qo = heads(a[4], "q_out", T, D), ko = heads(a[5], "k_out", T, D);
    if (qo.H != q.H || ko.H != k.H) {
        PyErr_SetString(PyExc_ValueError, "q_out and k_out must have the heads of q and k");
        throw Raised();
    }
    const auto *freq = arg<double>(a[2], "inv_freq", at::kDouble, {R / 2});
    const auto *pos = arg<int64_t>(a[3], "pos", at::kLong, {T});
    const int layout = (int)integer(a[6]), backward = (int)integer(a[8]);
    const float mscale = (float)number(a[7]);
    void *stream = stream_of(a[9]);
    call("jet_rope", [&] {
        return f_rope(q.p, q.ld, q.H, k.p, k.ld, k.H, T, D, R, freq, pos, layout, mscale, backward,
                      qo.p, qo.ld, ko.p, ko.ld, stream);
    });
}

void rope_kv(PyObject *const *a) {  // q, k, v, inv_freq, pos, k_scale, v_scale, slots, q_out,
                                    // k_cache, v_cache, layout, mscale, stream
    const at::Tensor &t = tensor(a[0], "q");
    need_dims(t, 3, "q");
    const int64_t T = t.size(0), D = t.size(2), R = 2 * numel(a[3], "inv_freq");
    const Heads q = heads(a[0], "q", T, D), k = heads(a[1], "k", T, D), v = heads(a[2], "v", T, D);
    const Heads qo = heads(a[8], "q_out", T, D);
    if (qo.H != q.H || v.H != k.H) {
        PyErr_SetString(PyExc_ValueError, "q_out must have the heads of q, and v those of k");
        throw Raised();
    }
    const at::Tensor &cache = tensor(a[9], "k_cache");
    const int64_t S = cache.dim() ? cache.size(0) : 0;
    const auto *freq = arg<double>(a[3], "inv_freq", at::kDouble, {R / 2});
    const auto *pos = arg<int64_t>(a[4], "pos", at::kLong, {T});
    const auto *ks = arg<float>(a[5], "k_scale", at::kFloat, {k.H});
    const auto *vs = arg<float>(a[6], "v_scale", at::kFloat, {k.H});
    const auto *slots = arg<int64_t>(a[7], "slots", at::kLong, {T});
    auto *kc = arg<uint8_t>(a[9], "k_cache", at::kByte, {S, k.H, D});
    auto *vc = arg<uint8_t>(a[10], "v_cache", at::kByte, {S, k.H, D});
    const int layout = (int)integer(a[11]);
    const float mscale = (float)number(a[12]);
    void *stream = stream_of(a[13]);
    call("jet_rope_kv_cache_write", [&] {
        return f_rope_kv(q.p, q.ld, q.H, k.p, k.ld, v.p, v.ld, k.H, T, D, R, freq, pos, layout,
                         mscale, ks, vs, slots, qo.p, qo.ld, kc, vc, S, stream);
    });
}

void slots(PyObject *const *a) {  // cached, added, block_size, table, free_blocks, free_next,
                                  // offsets, positions, slots, rows, counts, stream
    const int64_t B = numel(a[0], "cached"), width = matrix(a[3], "table").second;
    const int64_t n_free = numel(a[4], "free_blocks"), N = numel(a[8], "slots");
    const auto *cached = arg<int32_t>(a[0], "cached", at::kInt, {B});
    const auto *added = arg<int32_t>(a[1], "added", at::kInt, {B});
    auto *table = arg<int32_t>(a[3], "table", at::kInt, {B, width});
    const auto *free_blocks = arg<int32_t>(a[4], "free_blocks", at::kInt, {n_free});
    const auto *next = arg<int64_t>(a[5], "free_next", at::kLong, {1});
    auto *offsets = arg<int64_t>(a[6], "offsets", at::kLong, {B + 1});
    auto *positions = arg<int64_t>(a[7], "positions", at::kLong, {N});
    auto *out = arg<int64_t>(a[8], "slots", at::kLong, {N});
    auto *rows = arg<int32_t>(a[9], "rows", at::kInt, {N});
    auto *counts = arg<int64_t>(a[10], "counts", at::kLong, {2});
    const int64_t block_size = integer(a[2]);
    void *stream = stream_of(a[11]);
    call("jet_kv_slot_map", [&] {
        return f_slots(cached, added, B, block_size, table, width, free_blocks, n_free, next, N,
                       offsets, positions, out, rows, counts, stream);
    });
}

void sample(PyObject *const *a) {  // logits, u, temperature, top_k, top_p, min_p, token, logp,
                                   // logp_all, kept, stream
    const auto size = matrix(a[0], "logits");
    const int64_t B = size.first, V = size.second;
    const at::Tensor &x = tensor(a[0], "logits");
    if (x.scalar_type() != at::kBFloat16 && x.scalar_type() != at::kFloat) {
        PyErr_SetString(PyExc_TypeError, "logits: expected torch.bfloat16 or torch.float32");
        throw Raised();
    }
    if (x.numel() && (!x.is_cuda() || (V > 1 && x.stride(1) != 1))) {
        PyErr_SetString(PyExc_ValueError, "logits: must be a CUDA tensor with contiguous rows");
        throw Raised();
    }
    const auto *u = arg<float>(a[1], "u", at::kFloat, {B});
    const auto *temperature = arg<float>(a[2], "temperature", at::kFloat, {B});
    const auto *top_k = arg<int32_t>(a[3], "top_k", at::kInt, {B});
    const auto *top_p = arg<float>(a[4], "top_p", at::kFloat, {B});
    const auto *min_p = arg<float>(a[5], "min_p", at::kFloat, {B});
    auto *token = arg<int64_t>(a[6], "token", at::kLong, {B});
    auto *logp = arg<float>(a[7], "logp", at::kFloat, {B});
    auto *logp_all = arg<float>(a[8], "logp_all", at::kFloat, {B});
    auto *kept = arg<int32_t>(a[9], "kept", at::kInt, {B});
    const void *rows = address(x);
    const int dtype = x.scalar_type() == at::kFloat ? JET_FP32 : JET_BF16;
    const int64_t ld = B > 1 ? x.stride(0) : V;
    void *stream = stream_of(a[10]);
    call("jet_sample", [&] {
        return f_sample(rows, dtype, B, V, ld, u, temperature, top_k, top_p, min_p, token, logp,
                        logp_all, kept, stream);
    });
}

void attention(PyObject *const *a) {  // q, k_cache, v_cache, k_scale, v_scale, table, block_size,
                                      // offsets, lengths, out, lse, prefix_offsets,
                                      // prefix_lengths, scale, ws, stream
    const at::Tensor &t = tensor(a[0], "q"), &cache = tensor(a[1], "k_cache");
    need_dims(t, 3, "q");
    need_dims(cache, 3, "k_cache");
    const int64_t T = t.size(0), D = t.size(2), S = cache.size(0), Hk = cache.size(1);
    const Heads q = heads(a[0], "q", T, D), out = heads(a[9], "out", T, D);
    if (out.H != q.H) {
        PyErr_SetString(PyExc_ValueError, "out must have the heads of q");
        throw Raised();
    }
    for (int i = 0; i < 13; ++i)
        if (i != 6) on_this_device(a[i]);
    const auto *kc = arg<uint8_t>(a[1], "k_cache", at::kByte, {S, Hk, D});
    const auto *vc = arg<uint8_t>(a[2], "v_cache", at::kByte, {S, Hk, D});
    const auto *ks = arg<float>(a[3], "k_scale", at::kFloat, {Hk});
    const auto *vs = arg<float>(a[4], "v_scale", at::kFloat, {Hk});
    const int64_t B = numel(a[8], "lengths"), width = matrix(a[5], "table").second;
    const auto *table = arg<int32_t>(a[5], "table", at::kInt, {B, width});
    const int64_t block_size = integer(a[6]);
    const auto *offsets = arg<int64_t>(a[7], "offsets", at::kLong, {B + 1});
    const auto *lengths = arg<int32_t>(a[8], "lengths", at::kInt, {B});
    auto *lse = arg<float>(a[10], "lse", at::kFloat, {T, q.H});
    const int64_t Ng = a[12] == Py_None ? 0 : numel(a[12], "prefix_lengths");
    if ((a[11] == Py_None) != (a[12] == Py_None)) {
        PyErr_SetString(PyExc_ValueError, "prefix_offsets and prefix_lengths come together");
        throw Raised();
    }
    const auto *po = arg<int64_t>(a[11], "prefix_offsets", at::kLong, {Ng + 1});
    const auto *pl = arg<int32_t>(a[12], "prefix_lengths", at::kInt, {Ng});
    const float scale = a[13] == Py_None ? 1.0f / std::sqrt((float)(D > 0 ? D : 1)) : (float)number(a[13]);
    const at::Tensor ws = workspace(a[14], t, f_attention_workspace(T, q.H, Hk, D, B, Ng));
    void *room = ws.defined() ? address(ws) : nullptr, *stream = stream_of(a[15]);
    const size_t bytes = ws.defined() ? ws.nbytes() : 0;
    call("jet_kv_attention", [&] {
        return f_attention(q.p, q.ld, T, q.H, Hk, D, kc, vc, S, ks, vs, table, width, block_size,
                           offsets, lengths, B, po, pl, Ng, scale, out.p, out.ld, lse, room, bytes,
                           stream);
    });
}

void head(PyObject *const *a) {  // x, w, target, scale, logp, lse, ws, stream
    const auto size = matrix(a[0], "x");
    const int64_t T = size.first, K = size.second, V = matrix(a[1], "w").first;
    const auto *x = arg<uint16_t>(a[0], "x", at::kBFloat16, {T, K});
    const auto *w = arg<uint16_t>(a[1], "w", at::kBFloat16, {V, K});
    const auto *target = arg<int64_t>(a[2], "target", at::kLong, {T});
    const float scale = (float)number(a[3]);
    auto *logp = arg<float>(a[4], "logp", at::kFloat, {T});
    auto *lse = arg<float>(a[5], "lse", at::kFloat, {T});
    for (int i : {0, 1, 2, 4, 5}) on_this_device(a[i]);
    const at::Tensor ws = workspace(a[6], tensor(a[0], "x"), f_workspace(JET_OP_HEAD_LOGP, T, V, K));
    void *room = ws.defined() ? address(ws) : nullptr, *stream = stream_of(a[7]);
    const size_t bytes = ws.defined() ? ws.nbytes() : 0;
    call("jet_head_logp",
         [&] { return f_head(x, w, T, K, V, target, scale, logp, lse, room, bytes, stream); });
}

void head_bwd(PyObject *const *a) {  // x, w, target, lse, dlogp, scale, dx, dw, ws, stream
    const auto size = matrix(a[0], "x");
    const int64_t T = size.first, K = size.second, V = matrix(a[1], "w").first;
    const auto *x = arg<uint16_t>(a[0], "x", at::kBFloat16, {T, K});
    const auto *w = arg<uint16_t>(a[1], "w", at::kBFloat16, {V, K});
    const auto *target = arg<int64_t>(a[2], "target", at::kLong, {T});
    const auto *lse = arg<float>(a[3], "lse", at::kFloat, {T});
    const auto *dlogp = arg<float>(a[4], "dlogp", at::kFloat, {T});
    const float scale = (float)number(a[5]);
    auto *dx = arg<uint16_t>(a[6], "dx", at::kBFloat16, {T, K});
    auto *dw = arg<uint16_t>(a[7], "dw", at::kBFloat16, {V, K});
    for (int i : {0, 1, 2, 3, 4, 6, 7}) on_this_device(a[i]);
    const at::Tensor ws = workspace(a[8], tensor(a[0], "x"), f_workspace(JET_OP_HEAD_LOGP_BWD, T, V, K));
    void *room = ws.defined() ? address(ws) : nullptr, *stream = stream_of(a[9]);
    const size_t bytes = ws.defined() ? ws.nbytes() : 0;
    call("jet_head_logp_bwd", [&] {
        return f_head_bwd(x, w, T, K, V, target, lse, dlogp, scale, dx, dw, room, bytes, stream);
    });
}

// [M, F] BF16 rows, which may be strided; its row stride.
uint16_t *rows(PyObject *o, const char *name, int64_t M, int64_t F, int64_t &ld) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || t.size(0) != M || t.size(1) != F) {
        PyErr_Format(PyExc_ValueError, "%s: expected bfloat16 [%lld, %lld]", name, (long long)M, (long long)F);
        throw Raised();
    }
    if (t.numel() && (!t.is_cuda() || (F > 1 && t.stride(1) != 1))) {
        PyErr_Format(PyExc_ValueError, "%s: must be a CUDA tensor with contiguous rows", name);
        throw Raised();
    }
    ld = M > 1 ? t.stride(0) : F;
    return static_cast<uint16_t *>(address(t));
}

void swiglu_bwd(PyObject *const *a) {  // gate, up, dh, qg, sg, qu, su, stream
    const auto size = matrix(a[0], "gate");
    const int64_t M = size.first, F = size.second;
    int64_t ld = F, ldu = F;
    const uint16_t *gate = rows(a[0], "gate", M, F, ld), *up = rows(a[1], "up", M, F, ldu);
    if (ld != ldu) {
        PyErr_SetString(PyExc_ValueError, "gate and up must have the same row stride");
        throw Raised();
    }
    const auto *dh = arg<uint16_t>(a[2], "dh", at::kBFloat16, {M, F});
    auto *qg = arg<uint8_t>(a[3], "qg", at::kByte, {M, F});
    auto *sg = arg<float>(a[4], "sg", at::kFloat, {F / 128, M});
    auto *qu = arg<uint8_t>(a[5], "qu", at::kByte, {M, F});
    auto *su = arg<float>(a[6], "su", at::kFloat, {F / 128, M});
    for (int i = 0; i < 7; ++i) on_this_device(a[i]);
    void *stream = stream_of(a[7]);
    call("jet_swiglu_bwd_quant_1x128",
         [&] { return f_swiglu_bwd(gate, up, ld, dh, M, F, qg, sg, qu, su, stream); });
}

// ------------------------------------------------------------------ the module

template <void (*F)(PyObject *const *), int kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        F(args);
        Py_RETURN_NONE;
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// bind(JetError, the addresses of the twelve C functions in the order above)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 13) {
        PyErr_SetString(PyExc_TypeError, "bind: expected the error class and twelve addresses");
        return nullptr;
    }
    void *p[12];
    for (int i = 0; i < 12; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i + 1]);
        if (PyErr_Occurred()) return nullptr;
    }
    f_norm = reinterpret_cast<decltype(f_norm)>(p[0]);
    f_norm_bwd = reinterpret_cast<decltype(f_norm_bwd)>(p[1]);
    f_rope = reinterpret_cast<decltype(f_rope)>(p[2]);
    f_rope_kv = reinterpret_cast<decltype(f_rope_kv)>(p[3]);
    f_slots = reinterpret_cast<decltype(f_slots)>(p[4]);
    f_sample = reinterpret_cast<decltype(f_sample)>(p[5]);
    f_workspace = reinterpret_cast<decltype(f_workspace)>(p[6]);
    f_attention = reinterpret_cast<decltype(f_attention)>(p[7]);
    f_attention_workspace = reinterpret_cast<decltype(f_attention_workspace)>(p[8]);
    f_head = reinterpret_cast<decltype(f_head)>(p[9]);
    f_head_bwd = reinterpret_cast<decltype(f_head_bwd)>(p[10]);
    f_swiglu_bwd = reinterpret_cast<decltype(f_swiglu_bwd)>(p[11]);
    Py_XSETREF(jet_error, Py_NewRef(args[0]));
    Py_RETURN_NONE;
}

#define ENTRY(name, f, n) {name, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("add_rmsnorm_quant_1x128", norm, 9),
                         ENTRY("add_rmsnorm_bwd", norm_bwd, 9),
                         ENTRY("rope", rope, 10),
                         ENTRY("rope_kv_cache_write", rope_kv, 14),
                         ENTRY("kv_slot_map", slots, 12),
                         ENTRY("sample", sample, 11),
                         ENTRY("kv_attention", attention, 16),
                         ENTRY("head_logp", head, 8),
                         ENTRY("head_logp_bwd", head_bwd, 10),
                         ENTRY("swiglu_bwd_quant_1x128", swiglu_bwd, 8),
                         {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
