// host_calls.cpp -- the INT8 path's and the router's marshalling as a CPython module.
//
// Many of these calls take 2 to 4 us on the GPU; the same marshalling in Python (one look at
// each tensor, the outputs, ctypes) takes 7 us of host time.  Each function takes the
// tensors of the Python call of the same name, checks them (dtype, shape, contiguous, on the
// current CUDA device), allocates the outputs and calls the C ABI of include/nvfp4.h on the
// current stream.  It returns the result, the entry point's status as an int when that is
// not NVFP4_OK, or None for anything but the plain case; the caller then takes the Python
// path, which says what is wrong or does what is unusual.
//
// The module does not link the kernels' library: bind() receives the entry points'
// addresses from the process that loaded it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cxxabi.h>

#include <initializer_list>

#include "../../include/nvfp4.h"

namespace {

decltype(&gemm_int8_w8a8) g_gemm = nullptr;
decltype(&gemm_int8_w8a8_grouped) g_grouped = nullptr;
decltype(&int8_quantize_bf16) g_quantize = nullptr;
decltype(&int8_quantize_bf16_routed) g_routed = nullptr;
decltype(&nvfp4_moe_topk) g_topk = nullptr;

const at::Tensor* tensor(PyObject* o) {
    return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool is(const at::Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape, int dev) {
    return t && t->defined() && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type &&
           t->layout() == at::kStrided && t->sizes() == c10::IntArrayRef(shape) && t->is_contiguous();
}

at::Tensor empty(std::initializer_list<int64_t> shape, at::ScalarType type, int dev) {
    return at::detail::empty_cuda(c10::IntArrayRef(shape), type, c10::Device(c10::kCUDA, dev), std::nullopt);
}

bool fits(int64_t v) { return v >= 0 && v <= INT32_MAX; }

// a Python int that fits a C int
bool integer(PyObject* o, int& v) {
    if (!PyLong_CheckExact(o)) return false;
    int overflow = 0;
    const long l = PyLong_AsLongAndOverflow(o, &overflow);
    if (overflow || l < INT32_MIN || l > INT32_MAX) return false;
    v = (int)l;
    return true;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* pa = THPVariable_Wrap(a);
    PyObject* pb = pa ? THPVariable_Wrap(b) : nullptr;
    PyObject* t = pb ? PyTuple_New(2) : nullptr;
    if (!t) {
        Py_XDECREF(pa);
        Py_XDECREF(pb);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, pa);
    PyTuple_SET_ITEM(t, 1, pb);
    return t;
}

// The current device's index and stream, if every call is bound and `t` lives there.
bool here(const at::Tensor* t, bool bound, int& dev, void*& stream) {
    if (!bound || !t || !t->defined() || !t->is_cuda()) return false;
    dev = c10::cuda::current_device();
    if (t->get_device() != dev) return false;
    stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    return true;
}

// `body` returns a new reference, nullptr with a Python error set, or Py_None (borrowed)
// for the caller's own path.  No C++ exception leaves the module.  (What may pass is the
// unwinding by which Python ends a daemon thread that asks for the lock while the interpreter
// is being finalised: to stop it would abort the process.)
template <typename F>
PyObject* guarded(F&& body) {
    try {
        PyObject* r = body();
        if (r == Py_None) Py_INCREF(r);
        return r;
    } catch (abi::__forced_unwind&) {
        throw;
    } catch (...) {  // for example no memory: the Python path meets it again and raises it
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// Runs an entry point without the interpreter's lock (a launch can wait for a full queue).
// The lock is not taken back in a destructor, which the unwinding above may not leave.
template <typename F>
nvfp4_status unlocked(F&& call) {
    PyThreadState* const state = PyEval_SaveThread();
    nvfp4_status s;
    try {
        s = call();
    } catch (...) {
        PyEval_RestoreThread(state);
        throw;
    }
    PyEval_RestoreThread(state);
    return s;
}

PyObject* status(nvfp4_status st) { return PyLong_FromLong((long)st); }

// (A, sA, W, sW)
PyObject* py_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 4) return Py_None;
        const at::Tensor *A = tensor(a[0]), *sA = tensor(a[1]), *W = tensor(a[2]), *sW = tensor(a[3]);
        int dev;
        void* st;
        if (!here(A, g_gemm, dev, st) || A->dim() != 2 || !W || W->dim() != 2) return Py_None;
        const int64_t M = A->size(0), K = A->size(1), N = W->size(0);
        if (!fits(M) || !fits(N) || !fits(K) || !is(A, at::kChar, {M, K}, dev) ||
            !is(sA, at::kFloat, {M}, dev) || !is(W, at::kChar, {N, K}, dev) || !is(sW, at::kFloat, {N}, dev))
            return Py_None;
        at::Tensor y = empty({M, N}, at::kBFloat16, dev);
        const auto *pa = static_cast<const int8_t*>(A->data_ptr()), *pw = static_cast<const int8_t*>(W->data_ptr());
        const auto *psa = static_cast<const float*>(sA->data_ptr()), *psw = static_cast<const float*>(sW->data_ptr());
        void* py = y.data_ptr();
        const nvfp4_status s =
            unlocked([&] { return g_gemm(pa, psa, pw, psw, py, (int)M, (int)N, (int)K, st); });
        return s == NVFP4_OK ? THPVariable_Wrap(y) : status(s);
    });
}

// (A, sA, W, sW, offsets)
PyObject* py_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) return Py_None;
        const at::Tensor *A = tensor(a[0]), *sA = tensor(a[1]), *W = tensor(a[2]), *sW = tensor(a[3]),
                         *off = tensor(a[4]);
        int dev;
        void* st;
        if (!here(A, g_grouped, dev, st) || A->dim() != 2 || !W || W->dim() != 3) return Py_None;
        const int64_t M = A->size(0), K = A->size(1), E = W->size(0), N = W->size(1);
        if (!fits(M) || !fits(N) || !fits(K) || !fits(E) || !is(A, at::kChar, {M, K}, dev) ||
            !is(sA, at::kFloat, {M}, dev) || !is(W, at::kChar, {E, N, K}, dev) ||
            !is(sW, at::kFloat, {E, N}, dev) || !is(off, at::kInt, {E + 1}, dev))
            return Py_None;
        at::Tensor y = empty({M, N}, at::kBFloat16, dev);
        const auto *pa = static_cast<const int8_t*>(A->data_ptr()), *pw = static_cast<const int8_t*>(W->data_ptr());
        const auto *psa = static_cast<const float*>(sA->data_ptr()), *psw = static_cast<const float*>(sW->data_ptr());
        const auto* po = static_cast<const int32_t*>(off->data_ptr());
        void* py = y.data_ptr();
        const nvfp4_status s = unlocked([&] {
            return g_grouped(pa, psa, pw, psw, po, (int)E, (int)M, py, (int)N, (int)K, st);
        });
        return s == NVFP4_OK ? THPVariable_Wrap(y) : status(s);
    });
}

// (x) or (x, dest, k)
PyObject* py_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 1 && n != 3) return Py_None;
        const bool routed = n == 3;
        const at::Tensor *x = tensor(a[0]), *dest = routed ? tensor(a[1]) : nullptr;
        int k = 1, dev;
        void* st;
        if (routed && (!integer(a[2], k) || k < 1)) return Py_None;
        if (!here(x, g_quantize && g_routed, dev, st) || x->dim() != 2) return Py_None;
        const int64_t rows = x->size(0), K = x->size(1);
        if (!fits(rows) || !fits(K) || !fits(rows * k) || !is(x, at::kBFloat16, {rows, K}, dev) ||
            (routed && !is(dest, at::kInt, {rows * k}, dev)))
            return Py_None;
        at::Tensor codes = empty({rows * k, K}, at::kChar, dev);
        at::Tensor scales = empty({rows * k}, at::kFloat, dev);
        int8_t* c = static_cast<int8_t*>(codes.data_ptr());
        float* s = static_cast<float*>(scales.data_ptr());
        const void* px = x->data_ptr();
        const int32_t* pd = routed ? static_cast<const int32_t*>(dest->data_ptr()) : nullptr;
        const nvfp4_status r = unlocked([&] {
            return routed ? g_routed(px, (int)rows, (int)K, pd, k, c, s, st)
                          : g_quantize(px, (int)rows, (int)K, c, s, st);
        });
        return r == NVFP4_OK ? pair(codes, scales) : status(r);
    });
}

// (logits, k, score, bias or None, groups, top_groups, group_top, renormalize, scale)
PyObject* py_topk(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 9) return Py_None;
        const at::Tensor *x = tensor(a[0]), *bias = a[3] == Py_None ? nullptr : tensor(a[3]);
        int k, score, groups, top_groups, group_top, dev;
        void* st;
        if (!integer(a[1], k) || !integer(a[2], score) || !integer(a[4], groups) ||
            !integer(a[5], top_groups) || !integer(a[6], group_top) || !PyBool_Check(a[7]) ||
            !PyFloat_CheckExact(a[8]) || k < 1 || score < 0)
            return Py_None;
        if (!here(x, g_topk, dev, st) || x->dim() != 2) return Py_None;
        const int64_t T = x->size(0), E = x->size(1);
        if (k > E) return Py_None;  // refused there, without outputs of that size
        const bool bf16 = x->scalar_type() == at::kBFloat16;
        if (!fits(T) || !fits(E) || !is(x, bf16 ? at::kBFloat16 : at::kFloat, {T, E}, dev) ||
            (a[3] != Py_None && !is(bias, at::kFloat, {E}, dev)))
            return Py_None;
        at::Tensor ids = empty({T, k}, at::kInt, dev), w = empty({T, k}, at::kFloat, dev);
        const void* px = x->data_ptr();
        const float* pb = bias ? static_cast<const float*>(bias->data_ptr()) : nullptr;
        int32_t* pi = static_cast<int32_t*>(ids.data_ptr());
        float* pw = static_cast<float*>(w.data_ptr());
        const int renorm = a[7] == Py_True;
        const float scale = (float)PyFloat_AS_DOUBLE(a[8]);
        const nvfp4_status r = unlocked([&] {
            return g_topk(px, bf16, (int)T, (int)E, k, score, pb, groups, top_groups, group_top, renorm,
                          scale, pi, pw, st);
        });
        return r == NVFP4_OK ? pair(ids, w) : status(r);
    });
}

// The addresses of gemm_int8_w8a8, gemm_int8_w8a8_grouped, int8_quantize_bf16,
// int8_quantize_bf16_routed and nvfp4_moe_topk in the loaded library.
PyObject* py_bind(PyObject*, PyObject* args) {
    unsigned long long p[5];
    if (!PyArg_ParseTuple(args, "KKKKK", &p[0], &p[1], &p[2], &p[3], &p[4])) return nullptr;
    g_gemm = reinterpret_cast<decltype(g_gemm)>(p[0]);
    g_grouped = reinterpret_cast<decltype(g_grouped)>(p[1]);
    g_quantize = reinterpret_cast<decltype(g_quantize)>(p[2]);
    g_routed = reinterpret_cast<decltype(g_routed)>(p[3]);
    g_topk = reinterpret_cast<decltype(g_topk)>(p[4]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)); }

PyMethodDef methods[] = {
    {"bind", py_bind, METH_VARARGS, nullptr},
    {"gemm", fast<py_gemm>(), METH_FASTCALL, nullptr},
    {"grouped", fast<py_grouped>(), METH_FASTCALL, nullptr},
    {"quantize", fast<py_quantize>(), METH_FASTCALL, nullptr},
    {"topk", fast<py_topk>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_calls", nullptr, -1, methods, nullptr, nullptr, nullptr,
                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host_calls() { return PyModule_Create(&module); }
