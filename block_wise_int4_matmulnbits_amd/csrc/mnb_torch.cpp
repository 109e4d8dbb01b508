// Argument marshalling of the cache, attention and adapter calls for the Python
// binding: checks of torch tensors, their addresses into the C ABI's structures,
// and a workspace of torch's allocator.  These calls are made once for each
// layer and token, where the same steps in Python take longer than the kernels
// (one token's attention: 14.8 us a call in Python).
//
// The library's entry points are given as addresses (bind), so that this module
// links with torch alone.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "mnb.h"

namespace {

using Shape = std::initializer_list<int64_t>;

decltype(&append_kv_int8) g_append;
decltype(&attention_int8) g_attention;
decltype(&mnb_attention_workspace) g_attention_workspace;
decltype(&matmul_lora) g_lora;
decltype(&mnb_lora_workspace) g_lora_workspace;

// A wrong argument: type is TypeError or ValueError.
struct Wrong {
    PyObject* type;
    std::string text;
};

std::string list_of(at::IntArrayRef v)
{
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

const at::Tensor& tensor(const char* name, PyObject* o)
{
    if (!THPVariable_Check(o)) throw Wrong{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

void place(const char* name, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, int64_t index)
{
    if (t.scalar_type() != dtype)
        throw Wrong{PyExc_TypeError, std::string(name) + " must be " + c10::toString(dtype) + ", got " +
                                         c10::toString(t.scalar_type())};
    if (t.sizes() != shape)
        throw Wrong{PyExc_ValueError, std::string(name) + " must be " + list_of(shape) + ", got " + list_of(t.sizes())};
    if (!t.is_cuda() || t.get_device() != index)
        throw Wrong{PyExc_ValueError, std::string(name) + " must be on the GPU of the first argument, got " +
                                          t.device().str()};
}

// A contiguous tensor of this shape and type on GPU `index`.
void* dense(const char* name, PyObject* o, Shape shape, at::ScalarType dtype, int64_t index)
{
    const at::Tensor& t = tensor(name, o);
    place(name, t, at::IntArrayRef(shape.begin(), shape.size()), dtype, index);
    if (!t.is_contiguous()) throw Wrong{PyExc_ValueError, std::string(name) + " must be contiguous"};
    return t.data_ptr();
}

// The same, but for its first dimension: *stride gets the elements from one row to the next.
void* strided(const char* name, const at::Tensor& t, Shape shape, at::ScalarType dtype, int64_t index, int64_t* stride)
{
    place(name, t, at::IntArrayRef(shape.begin(), shape.size()), dtype, index);
    int64_t width = 1;
    for (int64_t d = t.dim() - 1; d > 0; --d) {
        if (t.size(d) != 1 && t.stride(d) != width)
            throw Wrong{PyExc_ValueError, std::string(name) + " must be contiguous but for its first dimension"};
        width *= t.size(d);
    }
    *stride = t.size(0) > 1 ? t.stride(0) : width;
    return t.data_ptr();
}

int code_of(const at::Tensor& t)
{
    if (t.scalar_type() == at::kHalf) return MNB_F16;
    if (t.scalar_type() == at::kBFloat16) return MNB_BF16;
    throw Wrong{PyExc_TypeError, std::string("expected float16 or bfloat16, got ") + c10::toString(t.scalar_type())};
}

void dims(const char* name, const at::Tensor& t, int64_t dim)
{
    if (t.dim() != dim) throw Wrong{PyExc_ValueError, std::string(name) + " must be " + std::to_string(dim) + "-D"};
}

int64_t integer(PyObject* o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

void* address(PyObject* o)
{
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw python_error();
    return p;
}

// starts, lengths, page_table, k_pages, v_pages, k_scales, v_scales
struct Cache {
    mnb_kv_cache cache;
    mnb_kv_batch batch;

    Cache(PyObject* const* a, int64_t tokens, int64_t index)
    {
        const at::Tensor &lengths = tensor("lengths", a[1]), &table = tensor("page_table", a[2]), &k = tensor("k_pages", a[3]);
        dims("lengths", lengths, 1);
        dims("page_table", table, 2);
        dims("k_pages", k, 4);
        const int64_t S = lengths.size(0), W = table.size(1), N = k.size(0), H = k.size(1), P = k.size(2), D = k.size(3);
        cache = mnb_kv_cache{N, P, H, D,
                             static_cast<int8_t*>(dense("k_pages", a[3], {N, H, P, D}, at::kChar, index)),
                             static_cast<int8_t*>(dense("v_pages", a[4], {N, H, D, P}, at::kChar, index)),
                             static_cast<float*>(dense("k_scales", a[5], {N, H}, at::kFloat, index)),
                             static_cast<float*>(dense("v_scales", a[6], {N, H}, at::kFloat, index))};
        batch = mnb_kv_batch{S, tokens, W,
                             static_cast<int32_t*>(dense("starts", a[0], {S + 1}, at::kInt, index)),
                             static_cast<int32_t*>(dense("lengths", a[1], {S}, at::kInt, index)),
                             static_cast<int32_t*>(dense("page_table", a[2], {S, W}, at::kInt, index))};
    }
};

// The caller's workspace, or one of torch's allocator on its current stream.
struct Workspace {
    at::Tensor held;
    void* p = nullptr;
    size_t bytes = 0;

    Workspace(PyObject* o, size_t need, const at::Tensor& like, int64_t index)
    {
        if (o != Py_None) {
            held = tensor("workspace", o);
            if (!held.is_cuda() || held.get_device() != index || !held.is_contiguous())
                throw Wrong{PyExc_ValueError, "workspace must be a contiguous tensor on the GPU of the first argument"};
            bytes = (size_t)held.numel() * held.element_size();
        } else if (need) {
            held = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
            bytes = need;
        }
        if (bytes) p = held.data_ptr();
    }
};

// Runs call() and gives its status; errors in Python's manner.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F call)
{
    HANDLE_TH_ERRORS
    try {
        if (got != want) throw Wrong{PyExc_TypeError, "wrong number of arguments"};
        return PyLong_FromLong(call());
    } catch (const Wrong& w) {
        PyErr_SetString(w.type, w.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// k, v, cos, sin, the cache's seven, q, q_out, interleaved, stream
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 15, [&] {
        const at::Tensor& k = tensor("k", a[0]);
        dims("k", k, 3);
        const int64_t index = k.get_device(), T = k.size(0);
        const int code = code_of(k);
        const at::ScalarType dtype = k.scalar_type();
        Cache c(a + 4, T, index);
        const int64_t H = c.cache.kv_heads, D = c.cache.head_dim;
        int64_t ks, vs, qs = 0, os = 0, heads = 0, rows = 0, rot = 0;
        void *kp = strided("k", k, {T, H, D}, dtype, index, &ks), *qp = nullptr, *op = nullptr;
        void* vp = strided("v", tensor("v", a[1]), {T, H, D}, dtype, index, &vs);
        if ((a[11] == Py_None) != (a[12] == Py_None)) throw Wrong{PyExc_ValueError, "q and q_out go together"};
        if (a[11] != Py_None) {
            const at::Tensor& q = tensor("q", a[11]);
            dims("q", q, 3);
            heads = q.size(1);
            qp = strided("q", q, {T, heads, D}, dtype, index, &qs);
            op = strided("q_out", tensor("q_out", a[12]), {T, heads, D}, dtype, index, &os);
        }
        const float *cp = nullptr, *sp = nullptr;
        if ((a[2] == Py_None) != (a[3] == Py_None)) throw Wrong{PyExc_ValueError, "cos and sin go together"};
        if (a[2] != Py_None) {
            const at::Tensor& cos = tensor("cos", a[2]);
            dims("cos", cos, 2);
            rows = cos.size(0);
            rot = 2 * cos.size(1);
            cp = static_cast<float*>(dense("cos", a[2], {rows, rot / 2}, at::kFloat, index));
            sp = static_cast<float*>(dense("sin", a[3], {rows, rot / 2}, at::kFloat, index));
        }
        const int near = PyObject_IsTrue(a[13]);
        if (near < 0) throw python_error();
        return g_append(&c.cache, &c.batch, code, kp, ks, vp, vs, qp, qs, op, os, heads, cp, sp, rot, rows,
                        near, address(a[14]));
    });
}

// q, the cache's seven, out, scale (or None), max_tokens (or None), workspace (or None), stream
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 13, [&] {
        const at::Tensor& q = tensor("q", a[0]);
        dims("q", q, 3);
        const int64_t index = q.get_device(), T = q.size(0), heads = q.size(1), D = q.size(2);
        const int code = code_of(q);
        Cache c(a + 1, T, index);
        if (D != c.cache.head_dim)
            throw Wrong{PyExc_ValueError, "q must be [tokens, query heads, " + std::to_string(c.cache.head_dim) + "]"};
        int64_t qs, os;
        void* qp = strided("q", q, {T, heads, D}, q.scalar_type(), index, &qs);
        void* op = strided("out", tensor("out", a[8]), {T, heads, D}, q.scalar_type(), index, &os);
        double scale = 1.0 / std::sqrt((double)D);
        if (a[9] != Py_None) {
            scale = PyFloat_AsDouble(a[9]);
            if (scale == -1.0 && PyErr_Occurred()) throw python_error();
        }
        const int64_t most = a[10] == Py_None ? 0 : integer(a[10]);
        const size_t need = g_attention_workspace(T, c.batch.sequences, heads, c.cache.kv_heads, D);
        Workspace ws(a[11], need, q, index);
        return g_attention(&c.cache, &c.batch, code, qp, qs, heads, (float)scale, op, os, most, ws.p, ws.bytes,
                           address(a[12]));
    });
}

// x, ids, A, B, base (or None), out, scaling (or None), workspace (or None), stream
PyObject* py_lora(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        const at::Tensor &x = tensor("x", a[0]), &A = tensor("A", a[2]), &B = tensor("B", a[3]), &out = tensor("out", a[5]);
        dims("x", x, 2);
        dims("A", A, 3);
        dims("B", B, 3);
        dims("out", out, 2);
        const int64_t index = x.get_device(), m = x.size(0), K = x.size(1), E = A.size(0), R = A.size(1), N = B.size(1);
        const int code = code_of(x), out_code = code_of(out);
        int64_t xs, os, bs = 0;
        void* xp = strided("x", x, {m, K}, x.scalar_type(), index, &xs);
        void* op = strided("out", out, {m, N}, out.scalar_type(), index, &os);
        const int32_t* ids = static_cast<int32_t*>(dense("ids", a[1], {m}, at::kInt, index));
        void* Ap = dense("A", a[2], {E, R, K}, x.scalar_type(), index);
        void* Bp = dense("B", a[3], {E, N, R}, x.scalar_type(), index);
        const float* sp = a[6] == Py_None ? nullptr : static_cast<float*>(dense("scaling", a[6], {E}, at::kFloat, index));
        void* bp = a[4] == Py_None ? nullptr
                                   : strided("base", tensor("base", a[4]), {m, N}, out.scalar_type(), index, &bs);
        Workspace ws(a[7], g_lora_workspace(m, K, N, R, E), x, index);
        return g_lora(xp, code, xs, m, K, N, R, E, ids, Ap, Bp, sp, bp, bs, op, os, out_code, ws.p, ws.bytes, address(a[8]));
    });
}

// Addresses of the library's entry points, in the order above.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 5, [&] {
        g_append = reinterpret_cast<decltype(g_append)>(address(a[0]));
        g_attention = reinterpret_cast<decltype(g_attention)>(address(a[1]));
        g_attention_workspace = reinterpret_cast<decltype(g_attention_workspace)>(address(a[2]));
        g_lora = reinterpret_cast<decltype(g_lora)>(address(a[3]));
        g_lora_workspace = reinterpret_cast<decltype(g_lora_workspace)>(address(a[4]));
        return 0;
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {{"append_kv_int8", FAST(py_append)}, {"attention_int8", FAST(py_attention)},
                           {"matmul_lora", FAST(py_lora)}, {"bind", FAST(py_bind)}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "mnb_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mnb_torch() { return PyModule_Create(&g_module); }
