// Python entry of the decoder-layer operators (cache append, paged attention, block
// norm, rotation without a cache, prompt and chunk attention): checks the tensors, fills
// the argument struct of include/w4a4.h and calls the C ABI.  A call of one of them takes
// a dozen tensors, and reading their type, shape,
// strides, device and pointer through Python attributes takes twice as long as the
// launch (5 us beside 2 us on the Grace host), which a decode step's short kernels
// cannot hide; here it is 0.1 us.
//
// Arguments go by position or name, None stands for NULL; a call runs on its tensors'
// device, whichever is current.  One that is refused raises the package's W4A4Error
// (W4A4_ERR_INVALID_ARG for a tensor that does not fit).
#include <Python.h>

#include <cmath>
#include <memory>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w4a4.h"

namespace {

using at::ScalarType;

bool type_of(ScalarType t, int32_t& out) {
    switch (t) {
        case ScalarType::Half: out = W4A4_F16; return true;
        case ScalarType::BFloat16: out = W4A4_BF16; return true;
        case ScalarType::Float: out = W4A4_F32; return true;
        case ScalarType::Float8_e4m3fn: out = W4A4_E4M3; return true;
        default: return false;
    }
}

// A strided dense tensor on device `dev`, or nullptr.
const at::Tensor* tensor(PyObject* o, int dev) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    return t.defined() && t.is_cuda() && t.layout() == at::kStrided && t.get_device() == dev ? &t : nullptr;
}

// [rows, heads, dim] with a contiguous last dimension
bool heads_of(PyObject* o, int dev, ScalarType type, int64_t rows, int64_t heads, int64_t dim, const void*& p,
              int64_t& row_stride, int64_t& head_stride) {
    const at::Tensor* t = tensor(o, dev);
    if (!t || t->dim() != 3 || t->scalar_type() != type) return false;
    const auto s = t->sizes(), st = t->strides();
    if (s[0] != rows || s[1] != heads || s[2] != dim || st[2] != 1) return false;
    p = t->data_ptr(), row_stride = st[0], head_stride = st[1];
    return true;
}

// n contiguous elements, or None
template <class T>
bool vector_of(PyObject* o, int dev, ScalarType type, int64_t n, T*& p) {
    if (o == Py_None) {
        p = nullptr;
        return true;
    }
    const at::Tensor* t = tensor(o, dev);
    if (!t || t->scalar_type() != type || t->numel() != n || !t->is_contiguous()) return false;
    p = static_cast<T*>(t->data_ptr());
    return true;
}

// [rows, width] with a contiguous last dimension
bool matrix_of(PyObject* o, int dev, ScalarType type, int64_t rows, int64_t width, void*& p, int64_t& stride) {
    const at::Tensor* t = tensor(o, dev);
    if (!t || t->dim() != 2 || t->scalar_type() != type || t->size(0) != rows || t->size(1) != width || t->stride(1) != 1)
        return false;
    p = t->data_ptr(), stride = t->stride(0);
    return true;
}

bool fits(int64_t n) { return n >= 0 && n <= INT32_MAX; }

// A torch stream, a handle, or None: the device's current stream.
bool stream_of(PyObject* o, int dev, cudaStream_t& s) {
    if (o == Py_None) {
        s = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream();
        return true;
    }
    PyObject* handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!handle) return false;
    s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
    Py_DECREF(handle);
    return !PyErr_Occurred();
}

// Makes `dev` the current device, on which the C ABI works, for the length of a call.
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    explicit OnDevice(int dev) {
        if (c10::cuda::current_device() != dev) guard.set_device(c10::Device(c10::kCUDA, c10::DeviceIndex(dev)));
    }
};

// Interned names, filled in when the module is loaded.
PyObject *n_struct, *n_device, *n_ws, *n_workspace, *n_refuse, *n_stream_id;

// What a PagedKVCache keeps for its calls: the C struct and its device.
const w4a4_kv_cache* cache_of(PyObject* o, int& dev) {
    PyObject* bytes = PyObject_GetAttr(o, n_struct);
    if (!bytes) return nullptr;
    const w4a4_kv_cache* c = nullptr;  // the object holds the bytes for the length of the call
    if (PyBytes_Check(bytes) && PyBytes_GET_SIZE(bytes) == sizeof(w4a4_kv_cache))
        c = reinterpret_cast<const w4a4_kv_cache*>(PyBytes_AS_STRING(bytes));
    Py_DECREF(bytes);
    PyObject* device = PyObject_GetAttr(o, n_device);
    if (!device) return nullptr;
    dev = int(PyLong_AsLong(device));
    Py_DECREF(device);
    return c;
}

// The cache object's workspace for `heads` query heads and the stream that it was made on, as
// the object keeps them: a new reference to (tensor, handle).
PyObject* workspace_of(PyObject* cache, int64_t heads) {
    PyObject* key = PyLong_FromLongLong(heads);
    PyObject* kept = PyObject_GetAttr(cache, n_ws);
    PyObject* pair = nullptr;
    for (int tries = 0; tries < 2 && !pair && kept && PyDict_Check(kept); ++tries) {
        pair = Py_XNewRef(PyDict_GetItemWithError(kept, key));
        if (pair || PyErr_Occurred() || tries) break;
        PyObject* made = PyObject_CallMethodOneArg(cache, n_workspace, key);
        Py_XDECREF(made);
        if (!made) break;
    }
    Py_XDECREF(kept);
    Py_DECREF(key);
    if (pair && (!PyTuple_Check(pair) || PyTuple_GET_SIZE(pair) != 2)) Py_CLEAR(pair);
    return pair;
}

// Keeps the allocator from handing `ws` out again while `s` may still use it, if the cache
// object is dropped before then.  Only for streams that torch owns: at the memory's release
// the allocator records an event on each, and one that the caller has made (a handle, an
// external stream) may be gone by then.
void keep_for(const at::Tensor& ws, PyObject* o, int dev, cudaStream_t s) {
    if (PyLong_Check(o)) return;
    int64_t id = 0;
    if (o == Py_None) {
        id = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).id();
    } else {
        PyObject* number = PyObject_GetAttr(o, n_stream_id);
        if (number) id = PyLong_AsLongLong(number);
        Py_XDECREF(number);
        if (PyErr_Occurred()) return PyErr_Clear();  // no torch stream
    }
    if (id != 0 && id == int64_t(reinterpret_cast<intptr_t>(s))) return;  // an external stream's id is its handle
    c10::cuda::CUDACachingAllocator::recordStream(
        ws.storage().data_ptr(), c10::cuda::CUDAStream::unpack3(id, c10::DeviceIndex(dev), c10::DeviceType::CUDA));
}

// A rotation table, fp32 [rows, 2, rot_dim / 2], or None.
bool rope_of(PyObject* o, int dev, const float*& p, int32_t& rows, int32_t& rot_dim) {
    p = nullptr, rows = rot_dim = 0;
    if (o == Py_None) return true;
    const at::Tensor* rope = tensor(o, dev);
    if (!rope || rope->dim() != 3 || rope->size(1) != 2 || !fits(rope->size(0)) || !fits(2 * rope->size(2)) ||
        !vector_of(o, dev, ScalarType::Float, rope->numel(), p))
        return false;
    rows = int32_t(rope->size(0)), rot_dim = int32_t(2 * rope->size(2));
    return p != nullptr;  // not an empty table
}

// The workspace of an attention call over `cache`: the one given, or the cache object's own, held by `kept`.
bool attention_workspace(PyObject* given, PyObject* cache, PyObject* stream, int64_t heads, int dev, cudaStream_t s,
                         std::unique_ptr<PyObject, void (*)(PyObject*)>& kept, void*& p, uint64_t& bytes) {
    const bool own = given == Py_None;
    kept.reset(own ? workspace_of(cache, heads) : Py_NewRef(given));
    if (!kept) return false;  // its own error is set
    const at::Tensor* ws = tensor(own ? PyTuple_GET_ITEM(kept.get(), 0) : kept.get(), dev);
    if (!ws || !ws->is_contiguous()) return false;
    p = ws->data_ptr(), bytes = uint64_t(ws->nbytes());
    if (own && PyLong_AsVoidPtr(PyTuple_GET_ITEM(kept.get(), 1)) != s) keep_for(*ws, stream, dev, s);
    return true;
}

// A parameter's default: required, or one of these.
enum Default { kRequired, kNone, kZero, kOne, kOneF, kEps, kFalse, kTrue };
struct Param {
    const char* name;
    Default def;
};

constexpr Param kAppend[] = {{"q", kRequired},    {"k", kRequired},  {"v", kRequired},    {"positions", kRequired},
                             {"cache", kRequired}, {"q_out", kRequired}, {"seqs", kNone},  {"rope", kNone},
                             {"q_gain", kNone},   {"k_gain", kNone}, {"eps", kEps},       {"interleaved", kFalse},
                             {"stream", kNone}};
w4a4_status kv_append(PyObject* const* a) {
    int dev = -1;
    const w4a4_kv_cache* c = cache_of(a[4], dev);
    const at::Tensor* q = c ? tensor(a[0], dev) : nullptr;
    w4a4_kv_append_args x{};
    x.bytes = sizeof(x);
    if (!c || !q || q->dim() != 3 || !type_of(q->scalar_type(), x.dtype)) return W4A4_ERR_INVALID_ARG;
    const ScalarType type = q->scalar_type();
    const int64_t n = q->size(0), heads = q->size(1);
    const void* out = nullptr;
    if (!fits(n) || !fits(heads) ||
        !heads_of(a[0], dev, type, n, heads, c->head_dim, x.q, x.q_token_stride, x.q_head_stride) ||
        !heads_of(a[1], dev, type, n, c->kv_heads, c->head_dim, x.k, x.k_token_stride, x.k_head_stride) ||
        !heads_of(a[2], dev, type, n, c->kv_heads, c->head_dim, x.v, x.v_token_stride, x.v_head_stride) ||
        !vector_of(a[3], dev, ScalarType::Int, n, x.positions) ||
        !heads_of(a[5], dev, type, n, heads, c->head_dim, out, x.out_token_stride, x.out_head_stride) ||
        !vector_of(a[6], dev, ScalarType::Int, n, x.seqs) || !vector_of(a[8], dev, type, c->head_dim, x.q_gain) ||
        !vector_of(a[9], dev, type, c->head_dim, x.k_gain))
        return W4A4_ERR_INVALID_ARG;
    x.q_out = const_cast<void*>(out);
    if (!rope_of(a[7], dev, x.rope, x.rope_rows, x.rot_dim)) return W4A4_ERR_INVALID_ARG;
    x.tokens = int32_t(n), x.q_heads = int32_t(heads);
    x.eps = float(PyFloat_AsDouble(a[10]));
    x.interleaved = PyObject_IsTrue(a[11]);
    cudaStream_t stream;
    if (!stream_of(a[12], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    const OnDevice on(dev);
    return w4a4_kv_append(c, &x, stream);
}

constexpr Param kAttention[] = {{"q", kRequired}, {"cache", kRequired}, {"lengths", kRequired}, {"out", kRequired},
                                {"lse", kNone},   {"scale", kNone},     {"window", kZero},      {"workspace", kNone},
                                {"stream", kNone}};
w4a4_status paged_attention(PyObject* const* a) {
    int dev = -1;
    const w4a4_kv_cache* c = cache_of(a[1], dev);
    const at::Tensor* q = c ? tensor(a[0], dev) : nullptr;
    w4a4_paged_attention_args x{};
    x.bytes = sizeof(x);
    if (!q || q->dim() != 3 || !type_of(q->scalar_type(), x.dtype)) return W4A4_ERR_INVALID_ARG;
    const ScalarType type = q->scalar_type();
    const int64_t n = c->seqs, heads = q->size(1);
    const void* out = nullptr;
    if (!fits(heads) || !heads_of(a[0], dev, type, n, heads, c->head_dim, x.q, x.q_token_stride, x.q_head_stride) ||
        !vector_of(a[2], dev, ScalarType::Int, n, x.lengths) ||
        !heads_of(a[3], dev, type, n, heads, c->head_dim, out, x.out_token_stride, x.out_head_stride) ||
        !vector_of(a[4], dev, ScalarType::Float, n * heads, x.lse))
        return W4A4_ERR_INVALID_ARG;
    x.out = const_cast<void*>(out);
    x.scale = a[5] == Py_None ? 1.f / std::sqrt(float(c->head_dim)) : float(PyFloat_AsDouble(a[5]));
    const int64_t window = PyLong_AsLongLong(a[6]);
    x.window = int32_t(window < INT32_MAX ? window : INT32_MAX);
    x.q_heads = int32_t(heads);
    cudaStream_t stream;
    if (window < 0 || !stream_of(a[8], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    const OnDevice on(dev);
    std::unique_ptr<PyObject, void (*)(PyObject*)> kept(nullptr, Py_DecRef);
    if (!attention_workspace(a[7], a[1], a[8], heads, dev, stream, kept, x.workspace, x.workspace_bytes))
        return W4A4_ERR_INVALID_ARG;
    return w4a4_paged_attention(c, &x, stream);
}

constexpr Param kNorm[] = {{"y", kRequired},   {"r", kRequired},     {"x", kRequired},       {"r_out", kRequired},
                           {"gate", kNone},    {"rows_per_gate", kZero}, {"scale", kOneF},   {"post", kOne},
                           {"post_gain", kNone}, {"post_bias", kNone}, {"pre", kOne},        {"pre_gain", kNone},
                           {"pre_bias", kNone}, {"eps", kEps},         {"stream", kNone}};
w4a4_status block_norm(PyObject* const* a) {
    w4a4_block_norm_args x{};
    x.bytes = sizeof(x);
    if (!THPVariable_Check(a[0]) || !THPVariable_Check(a[1])) return W4A4_ERR_INVALID_ARG;
    const at::Tensor &y = THPVariable_Unpack(a[0]), &r = THPVariable_Unpack(a[1]);
    if (!y.defined() || !r.defined() || !y.is_cuda() || y.dim() != 2 || !type_of(y.scalar_type(), x.dtype) ||
        !type_of(r.scalar_type(), x.res_dtype))
        return W4A4_ERR_INVALID_ARG;
    const int dev = y.get_device();
    const ScalarType type = y.scalar_type(), res = r.scalar_type();
    const int64_t rows = y.size(0), width = y.size(1), per = PyLong_AsLongLong(a[5]);
    void *py = nullptr, *pr = nullptr;
    if (!fits(rows) || !fits(width) || !fits(per) || !matrix_of(a[0], dev, type, rows, width, py, x.y_stride) ||
        !matrix_of(a[1], dev, res, rows, width, pr, x.r_stride) ||
        (a[2] != Py_None && !matrix_of(a[2], dev, type, rows, width, x.x, x.x_stride)) ||
        !matrix_of(a[3], dev, res, rows, width, x.r_out, x.r_out_stride))
        return W4A4_ERR_INVALID_ARG;
    x.y = py, x.r = pr;
    if (a[4] != Py_None) {
        const at::Tensor* g = tensor(a[4], dev);
        const int64_t need = per > 0 ? (rows + per - 1) / per : 1;
        if (!g || g->scalar_type() != type || g->dim() < 1 || g->dim() > 2 || g->size(-1) != width ||
            g->stride(-1) != 1 || (g->dim() == 2 ? g->size(0) : 1) < need)
            return W4A4_ERR_INVALID_ARG;
        x.gate = g->data_ptr(), x.gate_stride = g->dim() == 2 ? g->stride(0) : width;
    }
    if (!vector_of(a[8], dev, type, width, x.post_gain) || !vector_of(a[9], dev, type, width, x.post_bias) ||
        !vector_of(a[11], dev, type, width, x.pre_gain) || !vector_of(a[12], dev, type, width, x.pre_bias))
        return W4A4_ERR_INVALID_ARG;
    x.rows = int32_t(rows), x.width = int32_t(width), x.rows_per_gate = int32_t(per);
    x.scale = float(PyFloat_AsDouble(a[6])), x.eps = float(PyFloat_AsDouble(a[13]));
    const int64_t post = PyLong_AsLongLong(a[7]), pre = PyLong_AsLongLong(a[10]);
    x.post = int32_t(post), x.pre = int32_t(pre);
    cudaStream_t stream;
    if (!fits(post) || !fits(pre) || !stream_of(a[14], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    const OnDevice on(dev);
    return w4a4_block_norm(&x, stream);
}

constexpr Param kRope[] = {{"q", kRequired},     {"k", kRequired}, {"positions", kRequired}, {"q_out", kRequired},
                           {"k_out", kRequired}, {"rope", kNone},  {"q_gain", kNone},        {"k_gain", kNone},
                           {"eps", kEps},        {"interleaved", kFalse}, {"stream", kNone}};
w4a4_status qk_rope(PyObject* const* a) {
    w4a4_qk_rope_args x{};
    x.bytes = sizeof(x);
    if (!THPVariable_Check(a[0]) || !THPVariable_Check(a[1])) return W4A4_ERR_INVALID_ARG;
    const at::Tensor &q = THPVariable_Unpack(a[0]), &k = THPVariable_Unpack(a[1]);
    if (!q.defined() || !k.defined() || !q.is_cuda() || q.dim() != 3 || k.dim() != 3 || !type_of(q.scalar_type(), x.dtype))
        return W4A4_ERR_INVALID_ARG;
    const int dev = q.get_device();
    const ScalarType type = q.scalar_type();
    const int64_t n = q.size(0), heads = q.size(1), kv = k.size(1), dim = q.size(2);
    const void *q_out = nullptr, *k_out = nullptr;
    if (!fits(n) || !fits(heads) || !fits(kv) || !fits(dim) ||
        !heads_of(a[0], dev, type, n, heads, dim, x.q, x.q_token_stride, x.q_head_stride) ||
        !heads_of(a[1], dev, type, n, kv, dim, x.k, x.k_token_stride, x.k_head_stride) ||
        !vector_of(a[2], dev, ScalarType::Int, n, x.positions) ||
        !heads_of(a[3], dev, type, n, heads, dim, q_out, x.q_out_token_stride, x.q_out_head_stride) ||
        !heads_of(a[4], dev, type, n, kv, dim, k_out, x.k_out_token_stride, x.k_out_head_stride) ||
        !rope_of(a[5], dev, x.rope, x.rope_rows, x.rot_dim) || !vector_of(a[6], dev, type, dim, x.q_gain) ||
        !vector_of(a[7], dev, type, dim, x.k_gain))
        return W4A4_ERR_INVALID_ARG;
    x.q_out = const_cast<void*>(q_out), x.k_out = const_cast<void*>(k_out);
    x.tokens = int32_t(n), x.q_heads = int32_t(heads), x.kv_heads = int32_t(kv), x.head_dim = int32_t(dim);
    x.eps = float(PyFloat_AsDouble(a[8]));
    x.interleaved = PyObject_IsTrue(a[9]);
    cudaStream_t stream;
    if (!stream_of(a[10], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    const OnDevice on(dev);
    return w4a4_qk_rope(&x, stream);
}

// scale, window and causal of an attention call
template <class X>
bool mask_of(PyObject* scale, PyObject* window, PyObject* causal, int dim, X& x) {
    x.scale = scale == Py_None ? 1.f / std::sqrt(float(dim)) : float(PyFloat_AsDouble(scale));
    const int64_t w = PyLong_AsLongLong(window);
    x.window = int32_t(w < INT32_MAX ? w : INT32_MAX);
    x.causal = PyObject_IsTrue(causal);
    return w >= 0 && !PyErr_Occurred();
}

constexpr Param kPrompt[] = {{"q", kRequired}, {"k", kRequired}, {"v", kRequired}, {"starts", kRequired}, {"out", kRequired},
                             {"lse", kNone},   {"scale", kNone}, {"window", kZero}, {"causal", kTrue}, {"stream", kNone}};
w4a4_status prompt_attention(PyObject* const* a) {
    w4a4_prompt_attention_args x{};
    x.bytes = sizeof(x);
    if (!THPVariable_Check(a[0]) || !THPVariable_Check(a[1]) || !THPVariable_Check(a[3])) return W4A4_ERR_INVALID_ARG;
    const at::Tensor &q = THPVariable_Unpack(a[0]), &k = THPVariable_Unpack(a[1]), &starts = THPVariable_Unpack(a[3]);
    if (!q.defined() || !k.defined() || !starts.defined() || !q.is_cuda() || q.dim() != 3 || k.dim() != 3 ||
        starts.numel() < 1 || !type_of(q.scalar_type(), x.dtype))
        return W4A4_ERR_INVALID_ARG;
    const int dev = q.get_device();
    const ScalarType type = q.scalar_type();
    const int64_t n = q.size(0), heads = q.size(1), kv = k.size(1), dim = q.size(2), seqs = starts.numel() - 1;
    const void* out = nullptr;
    if (!fits(n) || !fits(heads) || !fits(kv) || !fits(dim) || !fits(seqs) ||
        !heads_of(a[0], dev, type, n, heads, dim, x.q, x.q_token_stride, x.q_head_stride) ||
        !heads_of(a[1], dev, type, n, kv, dim, x.k, x.k_token_stride, x.k_head_stride) ||
        !heads_of(a[2], dev, type, n, kv, dim, x.v, x.v_token_stride, x.v_head_stride) ||
        !vector_of(a[3], dev, ScalarType::Int, seqs + 1, x.starts) ||
        !heads_of(a[4], dev, type, n, heads, dim, out, x.out_token_stride, x.out_head_stride) ||
        !vector_of(a[5], dev, ScalarType::Float, n * heads, x.lse) || !mask_of(a[6], a[7], a[8], int(dim), x))
        return W4A4_ERR_INVALID_ARG;
    x.out = const_cast<void*>(out);
    x.tokens = int32_t(n), x.seqs = int32_t(seqs), x.q_heads = int32_t(heads), x.kv_heads = int32_t(kv);
    x.head_dim = int32_t(dim);
    cudaStream_t stream;
    if (!stream_of(a[9], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    const OnDevice on(dev);
    return w4a4_prompt_attention(&x, stream);
}

constexpr Param kChunk[] = {{"q", kRequired}, {"cache", kRequired}, {"starts", kRequired}, {"lengths", kRequired},
                            {"out", kRequired}, {"lse", kNone},     {"scale", kNone},      {"window", kZero},
                            {"causal", kTrue},  {"workspace", kNone}, {"stream", kNone}};
w4a4_status chunk_attention(PyObject* const* a) {
    int dev = -1;
    const w4a4_kv_cache* c = cache_of(a[1], dev);
    const at::Tensor* q = c ? tensor(a[0], dev) : nullptr;
    w4a4_chunk_attention_args x{};
    x.bytes = sizeof(x);
    if (!q || q->dim() != 3 || !type_of(q->scalar_type(), x.dtype)) return W4A4_ERR_INVALID_ARG;
    const ScalarType type = q->scalar_type();
    const int64_t n = q->size(0), heads = q->size(1);
    const void* out = nullptr;
    if (!fits(n) || !fits(heads) || !heads_of(a[0], dev, type, n, heads, c->head_dim, x.q, x.q_token_stride, x.q_head_stride) ||
        !vector_of(a[2], dev, ScalarType::Int, int64_t(c->seqs) + 1, x.starts) ||
        !vector_of(a[3], dev, ScalarType::Int, c->seqs, x.lengths) ||
        !heads_of(a[4], dev, type, n, heads, c->head_dim, out, x.out_token_stride, x.out_head_stride) ||
        !vector_of(a[5], dev, ScalarType::Float, n * heads, x.lse) || !mask_of(a[6], a[7], a[8], c->head_dim, x))
        return W4A4_ERR_INVALID_ARG;
    x.out = const_cast<void*>(out);
    x.tokens = int32_t(n), x.q_heads = int32_t(heads);
    cudaStream_t stream;
    if (!stream_of(a[10], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    const OnDevice on(dev);
    std::unique_ptr<PyObject, void (*)(PyObject*)> kept(nullptr, Py_DecRef);
    if (!attention_workspace(a[9], a[1], a[10], heads, dev, stream, kept, x.workspace, x.workspace_bytes))
        return W4A4_ERR_INVALID_ARG;
    return w4a4_chunk_attention(c, &x, stream);
}

// The Python callable of F: fills in F's parameters, calls it, raises where it refuses.
template <w4a4_status (*F)(PyObject* const*), const Param* P, int N>
struct Function {
    static PyObject* names[N];
    static PyObject* defaults[N];
    static const char* title;

    static bool init(const char* name) {
        title = name;
        for (int i = 0; i < N; ++i) {
            if (!(names[i] = PyUnicode_InternFromString(P[i].name))) return false;
            switch (P[i].def) {
                case kRequired: defaults[i] = nullptr; break;
                case kNone: defaults[i] = Py_None; break;
                case kZero: defaults[i] = PyLong_FromLong(0); break;
                case kOne: defaults[i] = PyLong_FromLong(1); break;
                case kOneF: defaults[i] = PyFloat_FromDouble(1.0); break;
                case kEps: defaults[i] = PyFloat_FromDouble(1e-6); break;
                case kFalse: defaults[i] = Py_False; break;
                case kTrue: defaults[i] = Py_True; break;
            }
        }
        return true;
    }

    static PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* kwnames) {
        if (n > N) {
            PyErr_Format(PyExc_TypeError, "%s() takes %d arguments, %zd were given", title, N, n);
            return nullptr;
        }
        PyObject* a[N];
        for (int i = 0; i < N; ++i) a[i] = i < n ? args[i] : nullptr;
        const Py_ssize_t named = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t k = 0; k < named; ++k) {
            PyObject* name = PyTuple_GET_ITEM(kwnames, k);
            int i = 0;
            while (i < N && name != names[i]) ++i;
            if (i == N)  // not the interned string: compare the text
                for (i = 0; i < N && PyUnicode_Compare(name, names[i]) != 0;) ++i;
            if (i == N || a[i]) {
                PyErr_Format(PyExc_TypeError, i == N ? "%s() has no argument %R" : "%s() got %R twice", title, name);
                return nullptr;
            }
            a[i] = args[n + k];
        }
        for (int i = 0; i < N; ++i)
            if (!a[i] && !(a[i] = defaults[i])) {
                PyErr_Format(PyExc_TypeError, "%s() needs %R", title, names[i]);
                return nullptr;
            }
        w4a4_status st = W4A4_ERR_INVALID_ARG;
        try {
            st = F(a);
        } catch (const std::exception&) {  // torch refuses what it is asked about a tensor
        }
        if (st == W4A4_OK) Py_RETURN_NONE;
        // an argument that is no number, an object that is no cache: the same refusal
        if (PyErr_Occurred() && (PyErr_ExceptionMatches(PyExc_TypeError) || PyErr_ExceptionMatches(PyExc_AttributeError) ||
                                 PyErr_ExceptionMatches(PyExc_OverflowError) || PyErr_ExceptionMatches(PyExc_ValueError)))
            PyErr_Clear();
        if (!PyErr_Occurred()) {
            PyObject* package = PyImport_ImportModule("w4a4_quantized_gemm_gb300");
            PyObject* refuse = package ? PyObject_GetAttr(package, n_refuse) : nullptr;
            PyObject* done = refuse ? PyObject_CallFunction(refuse, "si", title, int(st)) : nullptr;
            Py_XDECREF(done);
            Py_XDECREF(refuse);
            Py_XDECREF(package);
            if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", title, int(st));
        }
        return nullptr;
    }
};
template <w4a4_status (*F)(PyObject* const*), const Param* P, int N>
PyObject* Function<F, P, N>::names[N];
template <w4a4_status (*F)(PyObject* const*), const Param* P, int N>
PyObject* Function<F, P, N>::defaults[N];
template <w4a4_status (*F)(PyObject* const*), const Param* P, int N>
const char* Function<F, P, N>::title;

using Append = Function<kv_append, kAppend, sizeof(kAppend) / sizeof(Param)>;
using Attention = Function<paged_attention, kAttention, sizeof(kAttention) / sizeof(Param)>;
using Norm = Function<block_norm, kNorm, sizeof(kNorm) / sizeof(Param)>;
using Rope = Function<qk_rope, kRope, sizeof(kRope) / sizeof(Param)>;
using Prompt = Function<prompt_attention, kPrompt, sizeof(kPrompt) / sizeof(Param)>;
using Chunk = Function<chunk_attention, kChunk, sizeof(kChunk) / sizeof(Param)>;

template <class Fn>
PyMethodDef method(const char* name, const char* doc) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(Fn::call)), METH_FASTCALL | METH_KEYWORDS, doc};
}

PyMethodDef methods[] = {
    method<Append>("w4a4_kv_append",
        "w4a4_kv_append(q, k, v, positions, cache, q_out, seqs=None, rope=None, q_gain=None, k_gain=None, eps=1e-06,\n"
        "               interleaved=False, stream=None)\n--\n\n"
        "Keys and values of new tokens into `cache` (a PagedKVCache), q and k normalised (gains given) and rotated\n"
        "(rope given) on the way; the rotated queries go to q_out, which may be q.\n\n"
        "q, q_out [tokens, q_heads, dim], k, v [tokens, kv_heads, dim]: fp16 or bf16, last dimension contiguous\n"
        "(slices of a fused q|k|v output).  positions, seqs: int32 [tokens]; seqs None: token t belongs to sequence\n"
        "t, negative: padding.  rope: fp32 [rows, 2, rot_dim / 2] (w4a4_rope_table).  q_gain, k_gain: [dim]."),
    method<Attention>("w4a4_paged_attention",
        "w4a4_paged_attention(q, cache, lengths, out, lse=None, scale=None, window=0, workspace=None, stream=None)\n"
        "--\n\n"
        "out [seqs, q_heads, dim] = attention of one new token per sequence, q, over the first lengths[b] tokens\n"
        "(int32 [seqs]) that `cache` holds of each, or the last `window` of them.\n\n"
        "scale: of the scores, dim ** -0.5 by default.  lse: fp32 [seqs, q_heads] or None.  workspace: zeroed uint8\n"
        "of w4a4_paged_attention_workspace_bytes, for calls of any shapes that do not overlap; by default the cache\n"
        "object's own."),
    method<Norm>("w4a4_block_norm",
        "w4a4_block_norm(y, r, x, r_out, gate=None, rows_per_gate=0, scale=1.0, post=1, post_gain=None,\n"
        "                post_bias=None, pre=1, pre_gain=None, pre_bias=None, eps=1e-06, stream=None)\n--\n\n"
        "r_out = r + scale * gate * post(y); x = pre(r_out): the norm after a block, its gate and residual scale, the\n"
        "residual addition and the norm before the next block in one pass.\n\n"
        "y, x [rows, width] fp16 or bf16 (x None: not wanted); r, r_out the same type or fp32 (r_out may be r).\n"
        "post, pre: NORM_NONE, NORM_RMS (the default) or NORM_LAYER with gain and bias [width].  gate: [width] or [gates, width],\n"
        "row m under gate row m // rows_per_gate (0: one row for all)."),
    method<Rope>("w4a4_qk_rope",
        "w4a4_qk_rope(q, k, positions, q_out, k_out, rope=None, q_gain=None, k_gain=None, eps=1e-06,\n"
        "             interleaved=False, stream=None)\n--\n\n"
        "q_out, k_out = queries and keys normalised (gains given) and rotated (rope given), without a cache.\n\n"
        "q, q_out [tokens, q_heads, dim], k, k_out [tokens, kv_heads, dim]: fp16 or bf16, last dimension contiguous;\n"
        "q_out may be q, k_out may be k.  positions: int32 [tokens], negative: padding (rows of zeros); None without\n"
        "rope.  rope: fp32 [rows, 2, rot_dim / 2] (w4a4_rope_table).  q_gain, k_gain: [dim]."),
    method<Prompt>("w4a4_prompt_attention",
        "w4a4_prompt_attention(q, k, v, starts, out, lse=None, scale=None, window=0, causal=True, stream=None)\n"
        "--\n\n"
        "out [tokens, q_heads, dim] = attention over prompts packed one behind the other: sequence b is the rows\n"
        "starts[b] .. starts[b + 1] - 1 (int32 [seqs + 1], on the device).  Rows outside all of them stay as they are.\n\n"
        "q [tokens, q_heads, dim], k, v [tokens, kv_heads, dim]: fp16 or bf16, last dimension contiguous (slices of a\n"
        "fused q|k|v output).  causal: a row sees itself and the rows before it, with window > 0 the last `window` of\n"
        "them; else every row of its sequence.  scale: of the scores, dim ** -0.5 by default.  lse: fp32\n"
        "[tokens, q_heads] or None."),
    method<Chunk>("w4a4_chunk_attention",
        "w4a4_chunk_attention(q, cache, starts, lengths, out, lse=None, scale=None, window=0, causal=True,\n"
        "                     workspace=None, stream=None)\n--\n\n"
        "out [tokens, q_heads, dim] = attention of a chunk of new tokens of every sequence over `cache`, which holds them\n"
        "already: rows starts[b] .. starts[b + 1] - 1 (int32 [seqs + 1]) are the last of the lengths[b] tokens\n"
        "(int32 [seqs]) that the cache holds of sequence b.\n\n"
        "causal, window, scale, lse: as for w4a4_prompt_attention.  workspace: as for w4a4_paged_attention, by default\n"
        "the cache object's own."),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    if (!(n_struct = PyUnicode_InternFromString("_struct")) || !(n_device = PyUnicode_InternFromString("device")) ||
        !(n_ws = PyUnicode_InternFromString("_ws")) || !(n_workspace = PyUnicode_InternFromString("workspace")) ||
        !(n_refuse = PyUnicode_InternFromString("_refuse")) || !(n_stream_id = PyUnicode_InternFromString("stream_id")) || !Append::init("w4a4_kv_append") ||
        !Attention::init("w4a4_paged_attention") || !Norm::init("w4a4_block_norm") || !Rope::init("w4a4_qk_rope") ||
        !Prompt::init("w4a4_prompt_attention") || !Chunk::init("w4a4_chunk_attention"))
        return nullptr;
    return PyModule_Create(&module);
}
