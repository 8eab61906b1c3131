// fastcall.cpp -- the Python binding's short cut for the calls of a decode step.
//
// A decode step makes several calls per layer, each of a few microseconds on the device, and the
// checks and conversions of ~10 tensors take the interpreter 15 to 25 us.  These functions make the
// same checks on the tensors in C++ (about 1 us), allocate the outputs that were not given, and
// call libbsp.  They take the plain case only: where a check fails, an argument is of another kind, a
// stream is given or libbsp refuses the call, they return None without having launched anything,
// and the binding's Python code runs the call and says what is wrong.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "bsp.h"

namespace {

// A call's arguments: unpacks tensors, and remembers whether all of them passed.
struct Args {
    PyObject* const* a;
    c10::DeviceIndex device;
    bool ok = true;

    explicit Args(PyObject* const* args) : a(args), device(c10::cuda::current_device()) {}

    const at::Tensor* tensor(int i, at::ScalarType type, bool contiguous = true)
    {
        if (!ok) return nullptr;
        if (!THPVariable_CheckExact(a[i])) return fail();
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda() || t.scalar_type() != type || t.device().index() != device ||
            t.layout() != at::kStrided || (contiguous && !t.is_contiguous()))
            return fail();
        return &t;
    }
    const at::Tensor* at_least(int i, at::ScalarType type, int64_t n)
    {
        const at::Tensor* t = tensor(i, type);
        return t && t->numel() < n ? fail() : t;
    }
    // nullptr with ok still true: None was given
    const at::Tensor* maybe(int i, at::ScalarType type, int64_t n)
    {
        return a[i] == Py_None ? nullptr : at_least(i, type, n);
    }
    const at::Tensor* fail()
    {
        ok = false;
        return nullptr;
    }
    // a truth value; where asking for it raises, the error is dropped: the Python code meets it again
    bool truth(int i)
    {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) {
            PyErr_Clear();
            ok = false;
        }
        return v > 0;
    }
    bool require(bool b)
    {
        ok = ok && b;
        return ok;
    }
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const
    {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
    }
};

void* data(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

bsp_stream_t current_stream(c10::DeviceIndex d)
{
    return reinterpret_cast<bsp_stream_t>(c10::cuda::getCurrentCUDAStream(d).stream());
}

// C++ exceptions (an allocation that fails) end here: the Python code meets them again.
template <typename F>
PyObject* guarded(F f)
{
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// (x, w_codes, w_sf, w_scale, bias, out, workspace) -> out
PyObject* gemv(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != 7) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a(args);
        const at::Tensor* x = a.tensor(0, at::kBFloat16);
        const at::Tensor* w = a.tensor(1, at::kByte);
        if (!a.require(x && w && x->dim() == 2 && w->dim() == 2)) Py_RETURN_NONE;
        const int64_t M = x->size(0), K = x->size(1), N = w->size(0);
        if (!a.require(w->size(1) == K / 2 && K % 64 == 0)) Py_RETURN_NONE;
        const at::Tensor* sf = a.at_least(2, at::kByte, nvfp4_sf_bytes(N, K, BSP_SF_MMA));
        const at::Tensor* g = a.at_least(3, at::kFloat, 1);
        const at::Tensor* bias = a.maybe(4, at::kBFloat16, N);
        const at::Tensor* out = a.maybe(5, at::kBFloat16, M * N);
        const int64_t need = nvfp4_gemv_workspace_bytes(M, N, K);
        const at::Tensor* ws = a.maybe(6, at::kByte, need);
        if (!a.require(need >= 0)) Py_RETURN_NONE;
        at::Tensor made, room;
        if (!out) out = &(made = a.make({M, N}, at::kBFloat16));
        if (!ws) ws = &(room = a.make({need}, at::kByte));
        if (nvfp4_gemv(data(x), w->data_ptr<uint8_t>(), sf->data_ptr<uint8_t>(),
                       g->data_ptr<float>(), data(bias), data(out), M, N, K, data(ws),
                       ws->numel(), current_stream(a.device)) != BSP_OK)
            Py_RETURN_NONE;
        return THPVariable_Wrap(*out);
    });
}

struct Cache {
    const at::Tensor *k, *v, *ks, *vs, *table, *cu, *len;
    int64_t pages, Hkv, page, D, B, max_pages;
};

// arguments i .. i + 6: k_cache, v_cache, k_scale, v_scale, block_table, cu_new, kv_len
bool unpack_cache(Args& a, int i, Cache& c)
{
    c.k = a.tensor(i, at::kByte);
    c.v = a.tensor(i + 1, at::kByte);
    c.table = a.tensor(i + 4, at::kInt);
    if (!a.require(c.k && c.v && c.table && c.k->dim() == 4 && c.k->sizes() == c.v->sizes() &&
                   c.table->dim() == 2))
        return false;
    c.pages = c.k->size(0);
    c.Hkv = c.k->size(1);
    c.page = c.k->size(2);
    c.D = c.k->size(3);
    c.B = c.table->size(0);
    c.max_pages = c.table->size(1);
    c.ks = a.at_least(i + 2, at::kByte, c.pages * c.Hkv * (c.page / 16));
    c.vs = a.at_least(i + 3, at::kByte, c.pages * c.Hkv * (c.page / 16));
    c.cu = a.at_least(i + 5, at::kInt, c.B + 1);
    c.len = a.at_least(i + 6, at::kInt, c.B);
    return a.ok;
}

// bf16 [T, heads, D] with the heads of a token side by side; T < 0 takes any
const at::Tensor* unpack_heads(Args& a, int i, int64_t T, int64_t D, int64_t& stride)
{
    const at::Tensor* t = a.tensor(i, at::kBFloat16, false);
    if (!t) return nullptr;
    if (t->dim() != 3 || (T >= 0 && t->size(0) != T) || t->size(2) != D ||
        (t->stride(2) != 1 && D > 1) || (t->stride(1) != D && t->size(1) > 1))
        return a.fail();
    stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * D;
    return t;
}

// (k, v, <cache>, q, q_out, inv_freq, interleaved, rope_scale) -> q_out, or True without q
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != 14) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a(args);
        Cache c;
        if (!unpack_cache(a, 2, c)) Py_RETURN_NONE;
        int64_t ks = 0, vs = 0, qs = 0;
        const at::Tensor* k = unpack_heads(a, 0, -1, c.D, ks);
        if (!k) Py_RETURN_NONE;
        const int64_t T = k->size(0);
        const at::Tensor* v = unpack_heads(a, 1, T, c.D, vs);
        if (!a.require(v && k->size(1) == c.Hkv && v->size(1) == c.Hkv)) Py_RETURN_NONE;
        const at::Tensor* q = args[9] == Py_None ? nullptr : unpack_heads(a, 9, T, c.D, qs);
        const int64_t Hq = q ? q->size(1) : 0;
        const at::Tensor* out = q ? a.maybe(10, at::kBFloat16, T * Hq * c.D) : nullptr;
        const at::Tensor* f = a.maybe(11, at::kFloat, 0);
        const int inter = a.truth(12);
        const double rope = PyFloat_Check(args[13]) ? PyFloat_AS_DOUBLE(args[13]) : NAN;
        if (!a.require(PyFloat_Check(args[13]))) Py_RETURN_NONE;
        at::Tensor made;
        if (q && !out) out = &(made = a.make({T, Hq, c.D}, at::kBFloat16));
        if (fp8kv_append(data(q), qs, data(k), ks, data(v), vs, f ? f->data_ptr<float>() : nullptr,
                         f ? 2 * f->numel() : 0, inter, static_cast<float>(rope), data(out),
                         c.k->data_ptr<uint8_t>(), c.v->data_ptr<uint8_t>(),
                         c.ks->data_ptr<uint8_t>(), c.vs->data_ptr<uint8_t>(), c.pages, c.page,
                         c.table->data_ptr<int32_t>(), c.max_pages, c.cu->data_ptr<int32_t>(),
                         c.len->data_ptr<int32_t>(), c.B, T, Hq, c.Hkv, c.D,
                         current_stream(a.device)) != BSP_OK)
            Py_RETURN_NONE;
        if (!q) Py_RETURN_TRUE;
        return THPVariable_Wrap(*out);
    });
}

// (q, <cache>, sm_scale or None, window, out, lse, return_lse, workspace) -> out or (out, lse)
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != 14) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a(args);
        Cache c;
        if (!unpack_cache(a, 1, c)) Py_RETURN_NONE;
        int64_t qs = 0;
        const at::Tensor* q = unpack_heads(a, 0, -1, c.D, qs);
        if (!q) Py_RETURN_NONE;
        const int64_t T = q->size(0), Hq = q->size(1);
        if (!a.require((args[8] == Py_None || PyFloat_Check(args[8])) && PyLong_Check(args[9])))
            Py_RETURN_NONE;
        const double sm = args[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.D))
                                             : PyFloat_AS_DOUBLE(args[8]);
        const int64_t window = PyLong_AsLongLong(args[9]);
        if (window == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        const at::Tensor* out = a.maybe(10, at::kBFloat16, T * Hq * c.D);
        const at::Tensor* lse = a.maybe(11, at::kFloat, T * Hq);
        const bool want = a.truth(12);
        const int64_t need = fp8kv_attention_workspace_bytes(T, Hq, c.Hkv, c.D);
        const at::Tensor* ws = a.maybe(13, at::kByte, need);
        if (!a.require(need >= 0)) Py_RETURN_NONE;
        at::Tensor made, made_lse, room;
        if (!out) out = &(made = a.make({T, Hq, c.D}, at::kBFloat16));
        if (want && !lse) lse = &(made_lse = a.make({T, Hq}, at::kFloat));
        if (!ws) ws = &(room = a.make({need}, at::kByte));
        if (fp8kv_attention(data(q), qs, c.k->data_ptr<uint8_t>(), c.v->data_ptr<uint8_t>(),
                            c.ks->data_ptr<uint8_t>(), c.vs->data_ptr<uint8_t>(), c.pages, c.page,
                            c.table->data_ptr<int32_t>(), c.max_pages, c.cu->data_ptr<int32_t>(),
                            c.len->data_ptr<int32_t>(), c.B, T, Hq, c.Hkv, c.D,
                            static_cast<float>(sm), window, data(out),
                            lse ? lse->data_ptr<float>() : nullptr, data(ws), ws->numel(),
                            current_stream(a.device)) != BSP_OK)
            Py_RETURN_NONE;
        PyObject* first = THPVariable_Wrap(*out);
        if (!want || !first) return first;
        PyObject* second = THPVariable_Wrap(*lse);
        PyObject* both = second ? PyTuple_Pack(2, first, second) : nullptr;
        Py_DECREF(first);
        Py_XDECREF(second);
        return both;
    });
}

PyMethodDef kMethods[] = {
    {"gemv", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(gemv)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL,
     nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attention)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&kModule); }
