// binding.cpp -- the calls of adapters and token log probabilities on torch tensors as
// they mostly come: contiguous, of the types the library takes, on the current device.
// Each function checks that, allocates the results and calls the library's C ABI; for
// anything else it returns None and the Python wrapper, which converts or refuses,
// takes over.  A status other than 0 is returned as an int.  Small calls are bound by
// the host: through ctypes and torch.empty a decode step's 10 us of kernels took 20 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sherry.h"

namespace {

// Reads positional arguments; `ok` turns false at the first that is not ordinary.
struct Args {
    PyObject* const* v;
    bool ok = true;
    c10::DeviceIndex dev;

    explicit Args(PyObject* const* args) : v(args), dev(c10::cuda::device_count() > 0 ? c10::cuda::current_device() : -1) {}

    // a tensor of this type on the current device, or with `optional` None (then undefined)
    at::Tensor tensor(int i, at::ScalarType type, int64_t dim, bool optional = false) {
        if (optional && v[i] == Py_None) return {};
        if (!THPVariable_Check(v[i])) return ok = false, at::Tensor();
        const at::Tensor& t = THPVariable_Unpack(v[i]);
        if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != dim) ok = false;
        return t;
    }
    at::Tensor dense(int i, at::ScalarType type, int64_t dim, bool optional = false) {
        at::Tensor t = tensor(i, type, dim, optional);
        if (ok && t.defined() && !t.is_contiguous()) ok = false;
        return t;
    }
    int64_t integer(int i) {
        if (!PyLong_Check(v[i])) return ok = false, 0;
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return x;
    }
    // the type of a tensor argument, fp32 or bf16
    at::ScalarType type(int i) {
        if (!THPVariable_Check(v[i])) return ok = false, at::kFloat;
        const at::ScalarType t = THPVariable_Unpack(v[i]).scalar_type();
        if (t != at::kFloat && t != at::kBFloat16) ok = false;
        return t;
    }
    at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
        return at::Tensor(at::detail::empty_cuda(size, type, c10::Device(c10::DeviceType::CUDA, dev), std::nullopt));
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T* as(const at::Tensor& t) {
    return static_cast<T*>(ptr(t));
}
bool is(const at::Tensor& t, at::IntArrayRef shape) { return !t.defined() || t.sizes() == shape; }

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

// No C++ exception leaves a call: an allocation that fails raises torch's error
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

// logits [M][V] with rows of unit stride
bool logits_of(Args& a, int i, at::Tensor& z, at::ScalarType& type) {
    type = a.type(i);
    if (a.ok) z = a.tensor(i, type, 2);
    if (!a.ok) return false;
    const int64_t M = z.size(0), V = z.size(1);
    return V >= 1 && V <= SHERRY_MAX_VOCAB && z.stride(1) == 1 && (M <= 1 || z.stride(0) >= V);
}
int64_t row_stride(const at::Tensor& z) { return z.size(0) > 1 ? z.stride(0) : z.size(1); }
int dtype_of(at::ScalarType t) { return t == at::kBFloat16 ? SHERRY_BF16 : SHERRY_F32; }

// (logits, targets or None, top) -> (logp, entropy, stats, top_logp, top_ids)
PyObject* token_logprobs(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) Py_RETURN_NONE;
        Args a(args);
        at::Tensor z;
        at::ScalarType type;
        if (!logits_of(a, 0, z, type)) Py_RETURN_NONE;
        const int64_t M = z.size(0), V = z.size(1);
        const at::Tensor targets = a.dense(1, at::kInt, 1, true);
        const int64_t top = a.integer(2);
        if (!a.ok || !is(targets, {M}) || top < 0 || top > V || top > SHERRY_MAX_TOP) Py_RETURN_NONE;
        at::Tensor logp, best, ids;
        if (targets.defined()) logp = a.empty({M}, at::kFloat);
        const at::Tensor entropy = a.empty({M}, at::kFloat), stats = a.empty({M, 2}, at::kFloat);
        if (top > 0) {
            best = a.empty({M, top}, at::kFloat);
            ids = a.empty({M, top}, at::kInt);
        }
        const int st = sherry_token_logprobs(ptr(z), dtype_of(type), M, V, row_stride(z), as<int32_t>(targets), (int)top,
                                             as<float>(logp), as<float>(entropy), as<float>(stats), as<float>(best),
                                             as<int32_t>(ids), a.stream());
        if (st) return PyLong_FromLong(st);
        return tuple({logp, entropy, stats, best, ids});
    });
}

// (logits, targets, stats, entropy, dlogp, dentropy) -> dlogits
PyObject* token_logprobs_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 6) Py_RETURN_NONE;
        Args a(args);
        at::Tensor z;
        at::ScalarType type;
        if (!logits_of(a, 0, z, type)) Py_RETURN_NONE;
        const int64_t M = z.size(0), V = z.size(1);
        const at::Tensor targets = a.dense(1, at::kInt, 1, true), stats = a.dense(2, at::kFloat, 2),
                         entropy = a.dense(3, at::kFloat, 1, true), g = a.dense(4, at::kFloat, 1, true),
                         h = a.dense(5, at::kFloat, 1, true);
        if (!a.ok || !is(targets, {M}) || !is(stats, {M, 2}) || !is(entropy, {M}) || !is(g, {M}) || !is(h, {M}) ||
            (g.defined() && !targets.defined()) || (h.defined() && !entropy.defined()))
            Py_RETURN_NONE;
        const at::Tensor out = a.empty({M, V}, type);
        const int st = sherry_token_logprobs_backward(ptr(z), dtype_of(type), M, V, row_stride(z), as<int32_t>(targets),
                                                      as<float>(stats), as<float>(entropy), as<float>(g), as<float>(h),
                                                      ptr(out), V, a.stream());
        if (st) return PyLong_FromLong(st);
        return wrap(out);
    });
}

// what the adapters' calls share: X [M][K], the packed planes at i.., A, B, ids, scaling at j..
struct Lora {
    at::Tensor X, idx, sgn, scales, A, B, ids, scaling;
    int64_t M, N, K, n, R;
    int gran, group;

    // a plane of any shape; its elements are counted in read
    static at::Tensor plane(Args& a, int i, at::ScalarType type) {
        if (!THPVariable_Check(a.v[i])) return a.ok = false, at::Tensor();
        return a.dense(i, type, THPVariable_Unpack(a.v[i]).dim());
    }

    bool read(Args& a, int x, int i, int j) {
        X = a.dense(x, at::kBFloat16, 2);
        if (!a.ok) return false;
        idx = plane(a, i, at::kInt);
        sgn = plane(a, i + 1, at::kByte);
        scales = plane(a, i + 2, at::kFloat);
        N = a.integer(i + 3);
        K = a.integer(i + 4);
        gran = (int)a.integer(i + 5);
        group = (int)a.integer(i + 6);
        A = a.dense(j, at::kBFloat16, 3);
        B = a.dense(j + 1, at::kBFloat16, 3);
        ids = a.dense(j + 2, at::kInt, 1);
        scaling = a.dense(j + 3, at::kFloat, 1, true);
        if (!a.ok) return false;
        M = X.size(0);
        n = A.size(0);
        R = A.size(1);
        // the kernels index the planes by the shape and the granularity
        const int64_t count = sherry_num_scales(N, K, gran, group);
        if (count < 0 || idx.numel() != N * (K / 32) || sgn.numel() != idx.numel() || scales.numel() < count) return false;
        return N > 0 && M > 0 && X.size(1) == K && A.size(2) == K && is(B, {n, N, R}) && is(ids, {M}) &&
               is(scaling, {n}) && n >= 1 && n <= SHERRY_MAX_ADAPTERS && R >= 8 && R <= SHERRY_MAX_RANK && R % 8 == 0;
    }
};

// (X, idx, sgn, scales, N, K, granularity, group, A, B, ids, scaling, y dtype, whether U is wanted) -> (Y, U)
PyObject* linear_lora(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject* {
        if (nargs != 14) Py_RETURN_NONE;
        Args a(args);
        Lora l;
        if (!l.read(a, 0, 1, 8)) Py_RETURN_NONE;
        const int yd = (int)a.integer(12), want = PyObject_IsTrue(args[13]);
        // a call that needs a workspace of zeroed tickets has the wrapper's
        if (!a.ok || want < 0 || sherry_linear_lora_needs_tickets(l.M, l.N, l.K, l.gran, l.group)) Py_RETURN_NONE;
        const at::Tensor Y = a.empty({l.M, l.N}, yd == SHERRY_BF16 ? at::kBFloat16 : at::kFloat);
        at::Tensor U, ws;
        if (want) U = a.empty({l.M, l.R}, at::kFloat);
        const size_t wsb = sherry_linear_lora_workspace_bytes(l.M, l.N, l.K, l.gran, l.group, (int)l.n, (int)l.R, yd);
        if (wsb > 0) ws = a.empty({(int64_t)wsb}, at::kByte);
        const int st = sherry_linear_lora(as<uint16_t>(l.X), l.M, l.N, l.K, as<uint32_t>(l.idx), as<uint8_t>(l.sgn),
                                          as<float>(l.scales), l.gran, l.group, as<uint16_t>(l.A), as<uint16_t>(l.B),
                                          as<int32_t>(l.ids), as<float>(l.scaling), (int)l.n, (int)l.R, as<float>(U),
                                          ptr(Y), yd, ptr(ws), wsb, a.stream());
        if (st) return PyLong_FromLong(st);
        return tuple({Y, U});
    });
}

// (dY, X, idx, sgn, scales, N, K, granularity, group, A, B, ids, scaling, U, gradient dtype, need) -> (dX, dA, dB);
// need: 1 for dX, 2 for dA, 4 for dB
PyObject* linear_lora_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return guarded([&]() -> PyObject* {
        if (nargs != 16) Py_RETURN_NONE;
        Args a(args);
        Lora l;
        if (!l.read(a, 1, 2, 9)) Py_RETURN_NONE;
        const at::Tensor dY = a.dense(0, at::kBFloat16, 2), U = a.dense(13, at::kFloat, 2, true);
        const int gd = (int)a.integer(14), need = (int)a.integer(15);
        if (!a.ok || !is(dY, {l.M, l.N}) || reinterpret_cast<uintptr_t>(ptr(dY)) % 16 != 0 || !is(U, {l.M, l.R}) || ((need & 4) && !U.defined())) Py_RETURN_NONE;
        const at::ScalarType type = gd == SHERRY_BF16 ? at::kBFloat16 : at::kFloat;
        at::Tensor dX, dA, dB, ws;
        if (need & 1) dX = a.empty({l.M, l.K}, at::kBFloat16);
        if (need & 2) dA = a.empty({l.n, l.R, l.K}, type);
        if (need & 4) dB = a.empty({l.n, l.N, l.R}, type);
        const size_t wsb = sherry_linear_lora_backward_workspace_bytes(l.M, l.N, l.K, (int)l.n, (int)l.R);
        if (wsb > 0) ws = a.empty({(int64_t)wsb}, at::kByte);
        const int st = sherry_linear_lora_backward(
            as<uint16_t>(dY), as<uint16_t>(l.X), l.M, l.N, l.K, as<uint32_t>(l.idx), as<uint8_t>(l.sgn),
            as<float>(l.scales), l.gran, l.group, as<uint16_t>(l.A), as<uint16_t>(l.B), as<int32_t>(l.ids),
            as<float>(l.scaling), (int)l.n, (int)l.R, as<float>(U), as<uint16_t>(dX), ptr(dA), ptr(dB), gd, ptr(ws), wsb,
            a.stream());
        if (st) return PyLong_FromLong(st);
        return tuple({dX, dA, dB});
    });
}

#define SHERRY_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SHERRY_METHOD(token_logprobs), SHERRY_METHOD(token_logprobs_backward), SHERRY_METHOD(linear_lora),
                         SHERRY_METHOD(linear_lora_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
