// paged_calls.cpp -- the Python side's checks and argument structs of the two paged
// calls that run once or more a layer, as an extension module.  Written in Python
// they took 3.5 to 6 us a call, more than the kernels of a small step; here 0.3.
//
// append(args, dev, workspace, k, v, k_cache, v_cache, slots, positions, q, q_out,
//        sections, stream) and
// attend(args, dev, tokens, workspace, q, k_cache, v_cache, out, score_cap, slopes,
//        lse, stream): args is the address of a struct that holds what stays from
// call to call; it is copied, so threads may share it.  Both return the library's
// status, or raise ValueError for tensors that do not fit.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <exception>
#include <string>

#include "sarathi.h"

namespace {

using Append = int32_t (*)(const sarathi_append_args*, void*);
using Attend = int32_t (*)(const sarathi_paged_args*, void*);
Append lib_append = nullptr;
Attend lib_attend = nullptr;

// A ValueError that unwinds to the entry points.
struct Refused : std::exception {};
template <typename... A>
[[noreturn]] void refuse(const char* format, A... a) {
    PyErr_Format(PyExc_ValueError, format, a...);
    throw Refused();
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse("%s: a tensor is needed", name);
    return THPVariable_Unpack(o);
}
int64_t number(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
void* address(PyObject* o) { return reinterpret_cast<void*>(static_cast<uintptr_t>(number(o))); }

// Every tensor of a call: its type and its device (-1: the CPU, refused at the end).
struct Like {
    at::ScalarType dtype;
    int64_t dev;
};
void like(const char* name, const at::Tensor& t, const Like& l) {
    if (t.scalar_type() != l.dtype || t.get_device() != l.dev)
        refuse("%s: %s on device %lld, not %s on the device of the others (%lld)", name, toString(t.scalar_type()),
               (long long)t.get_device(), toString(l.dtype), (long long)l.dev);
}
Like element_type(const at::Tensor& t, int64_t dev, int32_t* code) {
    const at::ScalarType s = t.scalar_type();
    if (s != at::kBFloat16 && s != at::kHalf) refuse("element type %s: bfloat16 and float16 are built", toString(s));
    *code = s == at::kHalf ? SARATHI_FP16 : SARATHI_BF16;
    return Like{s, dev};
}
// [tokens][heads][d] whose tokens may be strided; the number of tokens.
int64_t token_rows(const char* name, const at::Tensor& t, const Like& l, int64_t heads, int64_t d, int64_t* stride) {
    if (t.dim() != 3 || t.size(1) != heads || t.size(2) != d)
        refuse("%s: the shape is not [tokens][%lld][%lld]", name, (long long)heads, (long long)d);
    like(name, t, l);
    const int64_t n = t.size(0);
    if (n && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)))
        refuse("%s: the heads of a token must be contiguous", name);
    *stride = n > 1 ? t.stride(0) : heads * d;
    return n;
}
int32_t page_pools(const at::Tensor& k, const at::Tensor& v, const Like& l, const sarathi_shape& sh) {
    if (k.dim() != 4 || k.size(1) != sh.num_heads_kv || k.size(2) != sh.page_size || k.size(3) != sh.head_dim)
        refuse("k_cache: the shape is not [num_pages][%d][%d][%d]", sh.num_heads_kv, sh.page_size, sh.head_dim);
    if (v.sizes() != k.sizes()) refuse("v_cache: the shape is not k_cache's");
    like("k_cache", k, l);
    like("v_cache", v, l);
    if (!k.is_contiguous() || !v.is_contiguous()) refuse("k_cache and v_cache must be contiguous");
    if (k.size(0) > INT32_MAX) refuse("k_cache: more than 2^31 - 1 pages");
    return (int32_t)k.size(0);
}
void* flat(const char* name, const at::Tensor& t, const Like& l, int64_t count) {
    like(name, t, l);
    if (t.numel() != count || !t.is_contiguous())
        refuse("%s: a contiguous tensor of %lld elements is needed", name, (long long)count);
    return t.data_ptr();
}
void on_gpu(int64_t dev) {
    if (dev < 0) refuse("tensors must be on a CUDA device");
}
void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse("%zd arguments, not %zd", n, want);
}

// Runs an entry point's body; nothing but a Python error leaves it.
template <typename Body>
PyObject* guarded(Body body) {
    try {
        return PyLong_FromLong(body());
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 13);
        sarathi_append_args x = *static_cast<const sarathi_append_args*>(address(a[0]));
        const int64_t dev = number(a[1]);
        const at::Tensor &ws = tensor("workspace", a[2]), &k = tensor("k", a[3]), &v = tensor("v", a[4]);
        const at::Tensor &kc = tensor("k_cache", a[5]), &vc = tensor("v_cache", a[6]);
        const at::Tensor &slots = tensor("slots", a[7]), &positions = tensor("positions", a[8]);
        const int64_t d = x.shape.head_dim;
        if (ws.nbytes() < 256 || ws.get_device() != dev || !ws.is_contiguous())
            refuse("workspace: contiguous, at least 256 bytes on the device of the others");
        const Like l = element_type(k, dev, &x.dtype), whole{at::kInt, dev};
        const int64_t T = token_rows("k", k, l, x.shape.num_heads_kv, d, &x.k_stride);
        if (token_rows("v", v, l, x.shape.num_heads_kv, d, &x.v_stride) != T)
            refuse("k and v hold different numbers of tokens");
        if (T > INT32_MAX) refuse("more than 2^31 - 1 tokens");
        if ((a[9] == Py_None) != (a[10] == Py_None)) refuse("q and q_out come together");
        if (a[9] != Py_None) {
            const at::Tensor &q = tensor("q", a[9]), &out = tensor("q_out", a[10]);
            if (token_rows("q", q, l, x.shape.num_heads_q, d, &x.q_stride) != T ||
                token_rows("q_out", out, l, x.shape.num_heads_q, d, &x.q_out_stride) != T)
                refuse("q, q_out and k hold different numbers of tokens");
            x.q = q.data_ptr();
            x.q_out = out.data_ptr();
        }
        x.num_pages = page_pools(kc, vc, l, x.shape);
        x.n_axes = 1;
        x.sections[0] = (int32_t)(d / 2);
        if (a[11] != Py_None) {
            const Py_ssize_t axes = PySequence_Size(a[11]);
            if (axes < 0) throw Refused();
            if (axes < 1 || axes > SARATHI_MAX_AXES) refuse("1 to %d sections", SARATHI_MAX_AXES);
            x.n_axes = (int32_t)axes;
            for (Py_ssize_t i = 0; i < axes; ++i) {
                PyObject* item = PySequence_GetItem(a[11], i);
                if (!item) throw Refused();
                const long long s = PyLong_AsLongLong(item);
                Py_DECREF(item);
                if (s == -1 && PyErr_Occurred()) throw Refused();
                if (s < 0 || s > d / 2) refuse("a section of %lld pairs, of %lld", s, (long long)(d / 2));
                x.sections[i] = (int32_t)s;
            }
        }
        x.slots = static_cast<const int32_t*>(flat("slots", slots, whole, T));
        x.positions = static_cast<const int32_t*>(flat("positions", positions, whole, T * x.n_axes));
        if (x.n_axes > 1 && (positions.dim() != 2 || positions.size(0) != x.n_axes))
            refuse("positions: the shape is not [axes][tokens]");
        on_gpu(dev);
        x.tokens = (int32_t)T;
        x.k = k.data_ptr();
        x.v = v.data_ptr();
        x.k_cache = kc.data_ptr();
        x.v_cache = vc.data_ptr();
        x.workspace = ws.data_ptr();
        void* stream = address(a[12]);
        int32_t st;
        Py_BEGIN_ALLOW_THREADS st = lib_append(&x, stream);
        Py_END_ALLOW_THREADS return st;
    });
}

PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 12);
        sarathi_paged_args x = *static_cast<const sarathi_paged_args*>(address(a[0]));
        const int64_t dev = number(a[1]), tokens = number(a[2]);
        const at::Tensor &ws = tensor("workspace", a[3]), &q = tensor("q", a[4]);
        const at::Tensor &kc = tensor("k_cache", a[5]), &vc = tensor("v_cache", a[6]), &out = tensor("out", a[7]);
        const int64_t heads = x.shape.num_heads_q, d = x.shape.head_dim;
        if (ws.get_device() != dev || !ws.is_contiguous())
            refuse("workspace: contiguous, on the device of the others");
        const Like l = element_type(q, dev, &x.dtype), single{at::kFloat, dev};
        int64_t stride;
        if (token_rows("q", q, l, heads, d, &x.q_stride) < tokens)
            refuse("q holds fewer tokens than the plan (%lld)", (long long)tokens);
        if (token_rows("out", out, l, heads, d, &stride) < tokens || stride != heads * d)
            refuse("out: contiguous, at least %lld tokens", (long long)tokens);
        x.num_pages = page_pools(kc, vc, l, x.shape);
        const double cap = PyFloat_AsDouble(a[8]);
        if (cap == -1.0 && PyErr_Occurred()) throw Refused();
        x.score_cap = (float)cap;
        if (cap != 0.0 && x.score_cap == 0.f) refuse("score_cap: too small a number, 0 is no cap");
        if (a[9] != Py_None) x.slopes = static_cast<const float*>(flat("slopes", tensor("slopes", a[9]), single, heads));
        if (a[10] != Py_None) {
            const at::Tensor& lse = tensor("lse", a[10]);
            if (lse.dim() != 2 || lse.size(1) != heads || lse.size(0) < tokens)
                refuse("lse: the shape is not [at least %lld][%lld]", (long long)tokens, (long long)heads);
            x.lse = static_cast<float*>(flat("lse", lse, single, lse.numel()));
        }
        on_gpu(dev);
        x.q = q.data_ptr();
        x.k_cache = kc.data_ptr();
        x.v_cache = vc.data_ptr();
        x.out = out.data_ptr();
        x.workspace = ws.data_ptr();
        x.workspace_bytes = (int64_t)ws.nbytes();
        void* stream = address(a[11]);
        int32_t st;
        Py_BEGIN_ALLOW_THREADS st = lib_attend(&x, stream);
        Py_END_ALLOW_THREADS return st;
    });
}

// bind(torch_version, append, attend): the running torch's version and the library's
// functions.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        count(n, 3);
        const char* version = PyUnicode_AsUTF8(a[0]);
        if (!version) throw Refused();
        if (std::string(version).rfind(TORCH_VERSION, 0) != 0) {
            PyErr_Format(PyExc_RuntimeError, "built for torch " TORCH_VERSION ", not %s: build again", version);
            throw Refused();
        }
        lib_append = reinterpret_cast<Append>(address(a[1]));
        lib_attend = reinterpret_cast<Attend>(address(a[2]));
        return 0;
    });
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_calls() { return PyModule_Create(&module); }
