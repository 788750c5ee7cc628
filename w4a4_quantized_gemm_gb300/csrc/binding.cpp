// Python entry of the decoder-layer operators (cache append, paged attention, block
// norm): checks the tensors, fills the argument struct of include/w4a4.h and calls the
// C ABI.  A call of one of them takes a dozen tensors, and reading their type, shape,
// strides, device and pointer through Python attributes takes twice as long as the
// launch (5 us beside 2 us on the Grace host), which a decode step's short kernels
// cannot hide; here it is 0.1 us.
//
// Each function takes its arguments by position and returns a w4a4_status as an int
// (W4A4_ERR_INVALID_ARG for a tensor it cannot describe); None stands for NULL.
#include <Python.h>

#include <ATen/core/Tensor.h>
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

const w4a4_kv_cache* cache_of(PyObject* o) {
    return PyBytes_Check(o) && PyBytes_GET_SIZE(o) == sizeof(w4a4_kv_cache)
               ? reinterpret_cast<const w4a4_kv_cache*>(PyBytes_AS_STRING(o))
               : nullptr;
}

// (cache, device, q, k, v, positions, q_out, seqs, rope, q_gain, k_gain, eps, interleaved, stream)
w4a4_status kv_append(PyObject* const* a) {
    const w4a4_kv_cache* c = cache_of(a[0]);
    const int dev = int(PyLong_AsLong(a[1]));
    const at::Tensor* q = tensor(a[2], dev);
    w4a4_kv_append_args x{};
    x.bytes = sizeof(x);
    if (!c || !q || q->dim() != 3 || !type_of(q->scalar_type(), x.dtype)) return W4A4_ERR_INVALID_ARG;
    const ScalarType type = q->scalar_type();
    const int64_t n = q->size(0), heads = q->size(1);
    const void* out = nullptr;
    if (!fits(n) || !fits(heads) ||
        !heads_of(a[2], dev, type, n, heads, c->head_dim, x.q, x.q_token_stride, x.q_head_stride) ||
        !heads_of(a[3], dev, type, n, c->kv_heads, c->head_dim, x.k, x.k_token_stride, x.k_head_stride) ||
        !heads_of(a[4], dev, type, n, c->kv_heads, c->head_dim, x.v, x.v_token_stride, x.v_head_stride) ||
        !vector_of(a[5], dev, ScalarType::Int, n, x.positions) ||
        !heads_of(a[6], dev, type, n, heads, c->head_dim, out, x.out_token_stride, x.out_head_stride) ||
        !vector_of(a[7], dev, ScalarType::Int, n, x.seqs) || !vector_of(a[9], dev, type, c->head_dim, x.q_gain) ||
        !vector_of(a[10], dev, type, c->head_dim, x.k_gain))
        return W4A4_ERR_INVALID_ARG;
    x.q_out = const_cast<void*>(out);
    if (a[8] != Py_None) {
        const at::Tensor* rope = tensor(a[8], dev);
        if (!rope || rope->dim() != 3 || rope->size(1) != 2 || !fits(rope->size(0)) || !fits(2 * rope->size(2)) ||
            !vector_of(a[8], dev, ScalarType::Float, rope->numel(), x.rope))
            return W4A4_ERR_INVALID_ARG;
        x.rope_rows = int32_t(rope->size(0)), x.rot_dim = int32_t(2 * rope->size(2));
        if (!x.rope) return W4A4_ERR_INVALID_ARG;  // an empty table
    }
    x.tokens = int32_t(n), x.q_heads = int32_t(heads);
    x.eps = float(PyFloat_AsDouble(a[11]));
    x.interleaved = PyObject_IsTrue(a[12]);
    cudaStream_t stream;
    if (!stream_of(a[13], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    return w4a4_kv_append(c, &x, stream);
}

// (cache, device, q, lengths, out, lse, scale, window, workspace, stream)
w4a4_status paged_attention(PyObject* const* a) {
    const w4a4_kv_cache* c = cache_of(a[0]);
    const int dev = int(PyLong_AsLong(a[1]));
    const at::Tensor *q = tensor(a[2], dev), *ws = tensor(a[8], dev);
    w4a4_paged_attention_args x{};
    x.bytes = sizeof(x);
    if (!c || !q || !ws || q->dim() != 3 || !type_of(q->scalar_type(), x.dtype) || !ws->is_contiguous())
        return W4A4_ERR_INVALID_ARG;
    const ScalarType type = q->scalar_type();
    const int64_t n = c->seqs, heads = q->size(1);
    const void* out = nullptr;
    if (!fits(heads) || !heads_of(a[2], dev, type, n, heads, c->head_dim, x.q, x.q_token_stride, x.q_head_stride) ||
        !vector_of(a[3], dev, ScalarType::Int, n, x.lengths) ||
        !heads_of(a[4], dev, type, n, heads, c->head_dim, out, x.out_token_stride, x.out_head_stride) ||
        !vector_of(a[5], dev, ScalarType::Float, n * heads, x.lse))
        return W4A4_ERR_INVALID_ARG;
    x.out = const_cast<void*>(out);
    x.workspace = ws->data_ptr(), x.workspace_bytes = uint64_t(ws->nbytes());
    x.scale = float(PyFloat_AsDouble(a[6]));
    const int64_t window = PyLong_AsLongLong(a[7]);
    x.window = int32_t(window < INT32_MAX ? window : INT32_MAX);
    x.q_heads = int32_t(heads);
    cudaStream_t stream;
    if (window < 0 || !stream_of(a[9], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    return w4a4_paged_attention(c, &x, stream);
}

// (y, r, x, r_out, gate, rows_per_gate, scale, post, post_gain, post_bias, pre, pre_gain, pre_bias, eps, stream)
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
    x.post = int32_t(PyLong_AsLong(a[7])), x.pre = int32_t(PyLong_AsLong(a[10]));
    cudaStream_t stream;
    if (!stream_of(a[14], dev, stream) || PyErr_Occurred()) return W4A4_ERR_INVALID_ARG;
    return w4a4_block_norm(&x, stream);
}

template <w4a4_status (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    w4a4_status st = W4A4_ERR_INVALID_ARG;
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        st = F(args);
    } catch (const std::exception&) {  // torch refuses what it is asked about the tensor
    }
    PyErr_Clear();  // an argument that is no number
    return PyLong_FromLong(st);
}

template <w4a4_status (*F)(PyObject* const*), int N>
constexpr PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<kv_append, 14>("kv_append"), method<paged_attention, 10>("paged_attention"),
                         method<block_norm, 15>("block_norm"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
