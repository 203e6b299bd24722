// The serving calls' argument marshalling (awq_gemm_fused, awq_kv_write,
// awq_kv_read, awq_kv_attention) as a CPython extension over torch tensors.
//
// A decode step makes such a call every 5 to 10 us. Checking eight tensors
// attribute by attribute in Python and passing twenty numbers through ctypes
// took 4.9 us of an 8.4 us call (the launch itself is 3.5); here it takes a
// few hundred nanoseconds. Every function checks its tensors and calls the
// library's entry point, whose address the caller passes; it returns the
// status, or None where a tensor is not what the call takes, and the Python
// wrapper then says which and why. No GPU work of its own.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <optional>

#include "../../include/awq.h"

namespace {

using at::Tensor;

// the tensor behind a Python object, or nullptr
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const Tensor& t, at::ScalarType type, int64_t device) {
    return t.scalar_type() == type && t.is_cuda() && t.get_device() == device;
}
bool dense(const Tensor& t, at::ScalarType type, int64_t device) { return on(t, type, device) && t.is_contiguous(); }

int64_t integer(PyObject* o, bool& ok) {
    const int64_t v = PyLong_Check(o) ? PyLong_AsLongLong(o) : (ok = false, 0);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        ok = false;
    }
    return v;
}
void* address(PyObject* o, bool& ok) { return reinterpret_cast<void*>(static_cast<uintptr_t>(integer(o, ok))); }

// fp16 [M, N] with contiguous rows: its address and row stride; None is no tensor
bool rows(PyObject* o, int64_t M, int64_t N, int64_t device, const void*& p, int64_t& stride) {
    p = nullptr;
    stride = 0;
    if (o == Py_None) return true;
    const Tensor* t = tensor(o);
    if (t == nullptr || !on(*t, at::kHalf, device) || t->dim() != 2 || t->size(0) != M || t->size(1) != N ||
        (N > 1 && t->stride(1) != 1))
        return false;
    p = t->data_ptr();
    stride = M > 1 ? t->stride(0) : N;
    return true;
}
bool workspace_of(PyObject* o, int64_t device, void*& p, size_t& bytes) {
    p = nullptr;
    bytes = 0;
    if (o == Py_None) return true;
    const Tensor* t = tensor(o);
    if (t == nullptr || !dense(*t, at::kByte, device)) return false;
    p = t->data_ptr();
    bytes = static_cast<size_t>(t->numel());
    return true;
}
// fp16 [T, heads, D] with contiguous channels; heads < 0 takes any
struct Tokens {
    void* p = nullptr;
    int64_t n = 0, heads = 0, token = 0, head = 0;
};
bool tokens(PyObject* o, int64_t heads, int64_t dim, int64_t device, Tokens& r) {
    const Tensor* t = tensor(o);
    if (t == nullptr || !on(*t, at::kHalf, device) || t->dim() != 3 || t->size(2) != dim || t->stride(2) != 1 ||
        (heads >= 0 && t->size(1) != heads))
        return false;
    r.p = t->data_ptr();
    r.n = t->size(0);
    r.heads = t->size(1);
    r.token = r.n > 1 ? t->stride(0) : 0;
    r.head = r.heads > 1 ? t->stride(1) : 0;
    return true;
}

// The status of an entry point's call, as a Python integer. The interpreter is
// other threads' meanwhile (a launch waits when its queue is full); the
// arguments' tensors are the caller's, who waits for this.
template <class F, class... A>
PyObject* status_of(F entry, A... args) {
    awq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = entry(args...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// gemm_fused(entry, stream, device, x, qweight, scales, zeros, group, bias, act, mul, residual, path, out, workspace)
PyObject* gemm_fused(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 15) Py_RETURN_NONE;
    bool ok = true;
    auto entry = reinterpret_cast<decltype(&awq_gemm_fused)>(address(a[0], ok));
    void* stream = address(a[1], ok);
    const int64_t dev = integer(a[2], ok), group = integer(a[7], ok), act = integer(a[9], ok), path = integer(a[12], ok);
    const Tensor *x = tensor(a[3]), *q = tensor(a[4]), *s = tensor(a[5]), *z = tensor(a[6]), *y = tensor(a[13]);
    if (!ok || !x || !q || !s || !z || !y || group < 1 || group > 1 << 20 || path < 0 || path > 255) Py_RETURN_NONE;
    if (!dense(*x, at::kHalf, dev) || !dense(*q, at::kInt, dev) || !dense(*s, at::kHalf, dev) ||
        !dense(*z, at::kHalf, dev) || !dense(*y, at::kHalf, dev) || x->dim() != 2 || q->dim() != 2 || s->dim() != 2 ||
        z->dim() != 2 || y->dim() != 2)
        Py_RETURN_NONE;
    const int64_t M = x->size(0), K = x->size(1), N = q->size(0), words = q->size(1);
    const int bits = words * 8 == K ? 4 : 8;
    if (words * 32 != K * bits || s->size(0) != N || s->size(1) != K / group || z->size(0) != N ||
        z->size(1) != K / group || y->size(0) != M || y->size(1) != N)
        Py_RETURN_NONE;
    const void* bias = nullptr;
    if (a[8] != Py_None) {
        const Tensor* b = tensor(a[8]);
        if (b == nullptr || !dense(*b, at::kHalf, dev) || b->dim() != 1 || b->size(0) != N) Py_RETURN_NONE;
        bias = b->data_ptr();
    }
    const void *mul, *res;
    int64_t ms, rs;
    void* ws;
    size_t bytes;
    if (!rows(a[10], M, N, dev, mul, ms) || !rows(a[11], M, N, dev, res, rs) || !workspace_of(a[14], dev, ws, bytes))
        Py_RETURN_NONE;
    return status_of(entry, x->data_ptr(), static_cast<const uint32_t*>(q->data_ptr()), s->data_ptr(), z->data_ptr(), M,
                     N, K, static_cast<int>(group), bits, bias, static_cast<int>(act), mul, ms, res, rs, y->data_ptr(),
                     static_cast<int>(path), ws, bytes, stream);
}

// kv_write(entry, stream, device, cache, seqs, heads, dim, k, v)
PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 9) Py_RETURN_NONE;
    bool ok = true;
    auto entry = reinterpret_cast<decltype(&awq_kv_write)>(address(a[0], ok));
    void* stream = address(a[1], ok);
    const int64_t dev = integer(a[2], ok);
    auto* cache = static_cast<const awq_kv_cache*>(address(a[3], ok));
    auto* seqs = static_cast<const awq_kv_seqs*>(address(a[4], ok));
    const int64_t heads = integer(a[5], ok), dim = integer(a[6], ok);
    Tokens k, v;
    if (!ok || !tokens(a[7], heads, dim, dev, k) || !tokens(a[8], heads, dim, dev, v) || k.n != v.n) Py_RETURN_NONE;
    return status_of(entry, cache, seqs, k.p, k.token, k.head, v.p, v.token, v.head, k.n, stream);
}

// kv_read(entry, stream, device, cache, seqs, heads, dim, k, v): k or v may be None, not both
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 9) Py_RETURN_NONE;
    bool ok = true;
    auto entry = reinterpret_cast<decltype(&awq_kv_read)>(address(a[0], ok));
    void* stream = address(a[1], ok);
    const int64_t dev = integer(a[2], ok);
    auto* cache = static_cast<const awq_kv_cache*>(address(a[3], ok));
    auto* seqs = static_cast<const awq_kv_seqs*>(address(a[4], ok));
    const int64_t heads = integer(a[5], ok), dim = integer(a[6], ok);
    Tokens t[2];
    for (int i = 0; i < 2; ++i)
        if (a[7 + i] != Py_None &&
            (!tokens(a[7 + i], heads, dim, dev, t[i]) || !tensor(a[7 + i])->is_contiguous()))
            Py_RETURN_NONE;
    if (!ok || (a[7] == Py_None && a[8] == Py_None) || (a[7] != Py_None && a[8] != Py_None && t[0].n != t[1].n))
        Py_RETURN_NONE;
    return status_of(entry, cache, seqs, t[0].p, t[1].p, a[7] != Py_None ? t[0].n : t[1].n, stream);
}

// kv_attention(entry, stream, device, cache, seqs, dim, q, scale, causal, window, out, lse, workspace)
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 13) Py_RETURN_NONE;
    bool ok = true;
    auto entry = reinterpret_cast<decltype(&awq_kv_attention)>(address(a[0], ok));
    void* stream = address(a[1], ok);
    const int64_t dev = integer(a[2], ok);
    auto* cache = static_cast<const awq_kv_cache*>(address(a[3], ok));
    auto* seqs = static_cast<const awq_kv_seqs*>(address(a[4], ok));
    const int64_t dim = integer(a[5], ok), window = integer(a[9], ok);
    if (!PyFloat_Check(a[7]) || !PyBool_Check(a[8])) ok = false;
    Tokens q, o;
    if (!ok || !tokens(a[6], -1, dim, dev, q) || !tokens(a[10], q.heads, dim, dev, o) || o.n != q.n) Py_RETURN_NONE;
    float* lse = nullptr;
    if (a[11] != Py_None) {
        const Tensor* t = tensor(a[11]);
        if (t == nullptr || !dense(*t, at::kFloat, dev) || t->dim() != 2 || t->size(0) != q.n || t->size(1) != q.heads)
            Py_RETURN_NONE;
        lse = static_cast<float*>(t->data_ptr());
    }
    void* ws;
    size_t bytes;
    if (q.heads > INT32_MAX || !workspace_of(a[12], dev, ws, bytes)) Py_RETURN_NONE;
    return status_of(entry, cache, seqs, q.p, q.token, q.head, q.n, static_cast<int>(q.heads),
                     static_cast<float>(PyFloat_AS_DOUBLE(a[7])), static_cast<int>(a[8] == Py_True), window, o.p, o.token,
                     o.head, lse, ws, bytes, stream);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (...) {     // a tensor without storage, and the like: the wrapper says what is wrong
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}
#define AWQ_CALL(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {AWQ_CALL(gemm_fused), AWQ_CALL(kv_write), AWQ_CALL(kv_read), AWQ_CALL(kv_attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
