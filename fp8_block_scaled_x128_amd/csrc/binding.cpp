// binding.cpp -- Python module `_native`: the short path from torch tensors to the C ABI for the
// operators whose kernels take a few microseconds (routing, token permutation, 4-bit products, the gated
// block, low-rank adapters).
// Each function reads its tensors' types, shapes and addresses directly, launches on the current
// stream of their device (or the given one) and returns the C call's status, or -1 where an
// argument is not what the call takes; the Python layer then finds out which one and raises.
// No output is allocated here.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "fp8gemm.h"

namespace {

constexpr int kRefused = -1;

// Arguments of one call: every tensor on the device of the first, contiguous, of a given type and shape.
struct Call {
    PyObject* const* args;
    Py_ssize_t n;
    int device = -1;
    bool ok = true;

    Call(PyObject* const* a, Py_ssize_t count, Py_ssize_t expected) : args(a), n(count), ok(count == expected) {}

    // Argument i as a tensor, or null: the call is refused (now or before), or it is `optional` and None.
    const at::Tensor* tensor(int i, bool optional = false, bool strided = false) {
        if (!ok) return nullptr;
        if (optional && args[i] == Py_None) return nullptr;
        if (!THPVariable_Check(args[i])) return refuse();
        const at::Tensor& t = THPVariable_Unpack(args[i]);
        if (!t.is_cuda() || (!strided && !t.is_contiguous())) return refuse();
        if (device < 0) device = t.get_device();
        if (t.get_device() != device) return refuse();
        return &t;
    }
    // Address of argument i, a tensor of this type and shape (null if None and optional).
    void* data(int i, at::ScalarType type, std::initializer_list<int64_t> shape, bool optional = false) {
        const at::Tensor* t = tensor(i, optional);
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape)) return refuse();
        return t->data_ptr();
    }
    // Argument i, a bf16 matrix [rows][cols] whose rows are contiguous, `stride` values apart.
    void* matrix(int i, int64_t rows, int64_t cols, int64_t* stride) {
        const at::Tensor* t = tensor(i, false, true);
        if (!t) return nullptr;
        if (t->scalar_type() != at::kBFloat16 || t->dim() != 2 || t->size(0) != rows || t->size(1) != cols ||
            (cols > 1 && t->stride(1) != 1))
            return refuse();
        *stride = rows > 1 && cols > 0 ? t->stride(0) : cols;
        return t->data_ptr();
    }
    int64_t integer(int i) {
        if (!ok) return 0;
        const long long v = PyLong_AsLongLong(args[i]);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return v;
    }
    // A size that the C call takes in 32 bits.
    int32_t small(int i) {
        const int64_t v = integer(i);
        if (v != (int32_t)v) ok = false;
        return (int32_t)v;
    }
    float real(int i) {
        if (!ok) return 0.0f;
        const double v = PyFloat_AsDouble(args[i]);
        if (v == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return (float)v;
    }
    std::nullptr_t refuse() {
        ok = false;
        return nullptr;
    }

    // The C call with the stream: argument i, or the device's current stream if that is None.
    template <typename F>
    PyObject* run(int i, F call) {
        void* stream = nullptr;
        if (ok) {
            if (args[i] == Py_None) stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
            else stream = reinterpret_cast<void*>((intptr_t)integer(i));
        }
        if (!ok) return PyLong_FromLong(kRefused);
        const c10::DeviceIndex current = c10::hip::current_device();
        if (current != device) c10::hip::set_device((c10::DeviceIndex)device);
        int status;
        Py_BEGIN_ALLOW_THREADS;
        status = call(stream);
        Py_END_ALLOW_THREADS;
        if (current != device) c10::hip::set_device(current);
        return PyLong_FromLong(status);
    }
};

// A C++ exception of the tensor library becomes a Python one.
template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

using at::kBFloat16;
using at::kByte;
using at::kFloat;
using at::kInt;

// Type of the router's logits [T][E] (FP8GEMM_F32 or FP8GEMM_BF16), or -1.
int logits_type(const at::Tensor& t) {
    return t.scalar_type() == kFloat ? FP8GEMM_F32 : t.scalar_type() == kBFloat16 ? FP8GEMM_BF16 : -1;
}

// E4M3 codes as float8_e4m3fn or uint8.
void* codes(Call& c, int i, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = c.tensor(i);
    if (!t) return nullptr;
    return c.data(i, t->scalar_type() == kByte ? kByte : at::kFloat8_e4m3fn, shape);
}

// (logits, bias, ids, weights, k, score, n_group, topk_group, group_top, renorm, scale, stream)
PyObject* route_topk(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 12);
        const at::Tensor* x = c.tensor(0);
        if (!x || x->dim() != 2 || logits_type(*x) < 0) return PyLong_FromLong(kRefused);
        const int64_t T = x->size(0), E = x->size(1);
        const int32_t k = c.small(4), score = c.small(5), ng = c.small(6), tg = c.small(7), gt = c.small(8), renorm = c.small(9);
        const float scale = c.real(10);
        void* bias = c.data(1, kFloat, {E}, true);
        void* ids = c.data(2, kInt, {T, k});
        void* w = c.data(3, kFloat, {T, k});
        if (E != (int32_t)E) c.refuse();
        return c.run(11, [&](void* s) {
            return fp8gemm_route_topk(x->data_ptr(), (const float*)bias, (int32_t*)ids, (float*)w, T, (int32_t)E, k,
                                      logits_type(*x), score, ng, tg, gt, renorm, scale, s);
        });
    });
}

// (logits, ids, dweights, dlogits, score, renorm, scale, stream)
PyObject* route_topk_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 8);
        const at::Tensor *x = c.tensor(0), *i = c.tensor(1);
        if (!x || !i || x->dim() != 2 || i->dim() != 2 || logits_type(*x) < 0) return PyLong_FromLong(kRefused);
        const int64_t T = x->size(0), E = x->size(1), k = i->size(1);
        void* ids = c.data(1, kInt, {T, k});
        void* dw = c.data(2, kFloat, {T, k});
        void* dx = c.data(3, x->scalar_type(), {T, E});
        const int32_t score = c.small(4), renorm = c.small(5);
        const float scale = c.real(6);
        if (E != (int32_t)E || k != (int32_t)k) c.refuse();
        return c.run(7, [&](void* s) {
            return fp8gemm_route_topk_backward(x->data_ptr(), (const int32_t*)ids, (const float*)dw, dx, T, (int32_t)E, (int32_t)k,
                                               logits_type(*x), score, renorm, scale, s);
        });
    });
}

// (X, ids, codes, scales, masked_m or m_indices, row_map, G, M_max or M_total, first_expert, masked, stream)
PyObject* moe_dispatch(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 11);
        const at::Tensor *x = c.tensor(0), *i = c.tensor(1);
        if (!x || !i || x->dim() != 2 || i->dim() != 2) return PyLong_FromLong(kRefused);
        const int64_t T = x->size(0), H = x->size(1), k = i->size(1), cap = c.integer(7);
        const int32_t G = c.small(6), first = c.small(8);
        const bool masked = c.small(9) != 0;
        void* X = c.data(0, kBFloat16, {T, H});
        void* ids = c.data(1, kInt, {T, k});
        void* A = masked ? codes(c, 2, {G, cap, H}) : codes(c, 2, {cap, H});
        void* sa = masked ? c.data(3, kFloat, {G, H / 128, cap}) : c.data(3, kFloat, {H / 128, cap});
        void* where = masked ? c.data(4, kInt, {G}) : c.data(4, kInt, {cap});
        void* rows = c.data(5, kInt, {T, k});
        if (k != (int32_t)k) c.refuse();
        return c.run(10, [&](void* s) {
            auto f = masked ? fp8gemm_moe_dispatch_masked : fp8gemm_moe_dispatch_contiguous;
            return f(X, (const int32_t*)ids, A, (float*)sa, (int32_t*)where, (int32_t*)rows, T, H, (int32_t)k, G, cap, first, s);
        });
    });
}

// Pairs [T][k] of a combine from its weights or row map, and the rows of Y ([R][H] or [G][M_max][H]).
bool combine_sizes(Call& c, int iy, int iw, int ir, int64_t* T, int64_t* k, int64_t* R, int64_t* H) {
    const at::Tensor *y = c.tensor(iy), *w = c.tensor(iw, true), *r = c.tensor(ir, true);
    const at::Tensor* pairs = w ? w : r;
    if (!c.ok || !y || !pairs || pairs->dim() != 2 || (y->dim() != 2 && y->dim() != 3) || y->scalar_type() != kBFloat16) return false;
    *T = pairs->size(0);
    *k = pairs->size(1);
    *H = y->size(-1);
    *R = y->dim() == 2 ? y->size(0) : y->size(0) * y->size(1);
    return *k == (int32_t)*k;
}

// (Y, weights, row_map, out, stream)
PyObject* moe_combine(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 5);
        int64_t T, k, R, H;
        if (!combine_sizes(c, 0, 1, 2, &T, &k, &R, &H)) return PyLong_FromLong(kRefused);
        void* Y = c.tensor(0)->data_ptr();               // (a tensor: its sizes were read)
        void* w = c.data(1, kFloat, {T, k}, true);
        void* rows = c.data(2, kInt, {T, k}, true);
        void* out = c.data(3, kBFloat16, {T, H});
        return c.run(4, [&](void* s) {
            return fp8gemm_moe_combine(Y, (const float*)w, (const int32_t*)rows, out, T, H, (int32_t)k, R, s);
        });
    });
}

// (dout, Y, weights, row_map, dY, dweights, stream)
PyObject* moe_combine_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 7);
        int64_t T, k, R, H;
        if (!combine_sizes(c, 1, 2, 3, &T, &k, &R, &H)) return PyLong_FromLong(kRefused);
        const at::Tensor *y = c.tensor(1), *dy = c.tensor(4);
        if (!dy || dy->scalar_type() != kBFloat16 || dy->sizes() != y->sizes()) return PyLong_FromLong(kRefused);
        void* dout = c.data(0, kBFloat16, {T, H});
        void* w = c.data(2, kFloat, {T, k}, true);
        void* rows = c.data(3, kInt, {T, k}, true);
        void* dw = c.data(5, kFloat, {T, k});
        return c.run(6, [&](void* s) {
            return fp8gemm_moe_combine_backward(dout, y->data_ptr(), (const float*)w, (const int32_t*)rows, dy->data_ptr(),
                                                (float*)dw, T, H, (int32_t)k, R, s);
        });
    });
}

// Format and group of 4-bit weights from their scales ([(E)][N][groups]): uint8 is MXFP4 (which has no
// zero points), bf16 INT4.
bool w4_format(const at::Tensor& scales, PyObject* zeros, int64_t K, int32_t* format, int32_t* group) {
    const int64_t groups = scales.size(-1);
    if (groups <= 0 || K % groups != 0) return false;
    *group = (int32_t)(K / groups);
    *format = scales.scalar_type() == kByte ? FP8GEMM_W4_MXFP4 : FP8GEMM_W4_INT4;
    return scales.scalar_type() == kByte ? zeros == Py_None : scales.scalar_type() == kBFloat16;
}

// (X, W, scales, zeros, out, stream)
PyObject* w4_gemv(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 6);
        const at::Tensor *x = c.tensor(0), *w = c.tensor(1), *sc = c.tensor(2);
        if (!x || !w || !sc || x->dim() != 2 || w->dim() != 2 || sc->dim() != 2) return PyLong_FromLong(kRefused);
        const int64_t M = x->size(0), K = x->size(1), N = w->size(0), groups = sc->size(1);
        int32_t format, group;
        if (K % 2 || !w4_format(*sc, args[3], K, &format, &group)) return PyLong_FromLong(kRefused);
        void* X = c.data(0, kBFloat16, {M, K});
        void* W = c.data(1, kByte, {N, K / 2});
        void* S = c.data(2, sc->scalar_type(), {N, groups});
        void* Z = c.data(3, kByte, {N, groups}, true);
        void* Y = c.data(4, kBFloat16, {M, N});
        return c.run(5, [&](void* s) { return fp8gemm_w4_gemv(X, W, S, (const uint8_t*)Z, Y, M, N, K, format, group, s); });
    });
}

// (X, W, scales, zeros, ids, out, first_expert, swiglu, stream)
PyObject* w4_gemv_experts(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 9);
        const at::Tensor *x = c.tensor(0), *w = c.tensor(1), *sc = c.tensor(2), *id = c.tensor(4);
        if (!x || !w || !sc || !id || x->dim() != 2 || w->dim() != 3 || sc->dim() != 3 || id->dim() != 2)
            return PyLong_FromLong(kRefused);
        const int64_t rows = x->size(0), K = x->size(1), E = w->size(0), N = w->size(1), groups = sc->size(2);
        const int64_t T = id->size(0), k = id->size(1);
        const int32_t first = c.small(6), swiglu = c.small(7);
        int32_t format, group;
        if (K % 2 || !w4_format(*sc, args[3], K, &format, &group) || (rows != T && rows != T * k) || (swiglu && N % 2))
            return PyLong_FromLong(kRefused);
        void* X = c.data(0, kBFloat16, {rows, K});
        void* W = c.data(1, kByte, {E, N, K / 2});
        void* S = c.data(2, sc->scalar_type(), {E, N, groups});
        void* Z = c.data(3, kByte, {E, N, groups}, true);
        void* ids = c.data(4, kInt, {T, k});
        void* Y = c.data(5, kBFloat16, {T * k, swiglu ? N / 2 : N});
        if (E != (int32_t)E || k != (int32_t)k) c.refuse();
        return c.run(8, [&](void* s) {
            return fp8gemm_w4_gemv_experts(X, W, S, (const uint8_t*)Z, (const int32_t*)ids, Y, T, (int32_t)k, (int32_t)E, N, K, format,
                                           group, first, rows != T, swiglu, s);
        });
    });
}

// (X, W, out, pre, act, stream)
PyObject* gated_ffn(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 6);
        const at::Tensor *x = c.tensor(0), *w = c.tensor(1);
        if (!x || !w || x->dim() != 2 || w->dim() != 2 || w->size(0) % 2) return PyLong_FromLong(kRefused);
        const int64_t M = x->size(0), K = x->size(1), I = w->size(0) / 2;
        void* X = c.data(0, kBFloat16, {M, K});
        void* W = c.data(1, kBFloat16, {2 * I, K});
        void* H = c.data(2, kBFloat16, {M, I});
        void* pre = c.data(3, kBFloat16, {M, 2 * I}, true);
        const int32_t act = c.small(4);
        return c.run(5, [&](void* s) { return fp8gemm_gated_ffn(X, W, H, pre, M, I, K, act, s); });
    });
}

// (dH, X, W, pre, dpre, dX, dW, act, stream)
PyObject* gated_ffn_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 9);
        const at::Tensor *x = c.tensor(1), *w = c.tensor(2);
        if (!x || !w || x->dim() != 2 || w->dim() != 2 || w->size(0) % 2) return PyLong_FromLong(kRefused);
        const int64_t M = x->size(0), K = x->size(1), I = w->size(0) / 2;
        void* dH = c.data(0, kBFloat16, {M, I});
        void* X = c.data(1, kBFloat16, {M, K});
        void* W = c.data(2, kBFloat16, {2 * I, K});
        void* pre = c.data(3, kBFloat16, {M, 2 * I}, true);
        void* dpre = c.data(4, kBFloat16, {M, 2 * I});
        void* dX = c.data(5, kBFloat16, {M, K}, true);
        void* dW = c.data(6, kBFloat16, {2 * I, K}, true);
        const int32_t act = c.small(7);
        return c.run(8, [&](void* s) { return fp8gemm_gated_ffn_backward(dH, X, W, pre, dpre, dX, dW, M, I, K, act, s); });
    });
}

// (Y, X, A, B, ids, order, scales, out, stream)
PyObject* lora_add(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 9);
        const at::Tensor *x = c.tensor(1, false, true), *ta = c.tensor(2), *tb = c.tensor(3);
        if (!x || !ta || !tb || x->dim() != 2 || ta->dim() != 3 || tb->dim() != 3) return PyLong_FromLong(kRefused);
        const int64_t T = x->size(0), K = x->size(1), L = ta->size(0), R = ta->size(1), N = tb->size(1);
        int64_t ldx = 0, ldy = 0, ldo = 0;
        void* Y = c.matrix(0, T, N, &ldy);
        void* X = c.matrix(1, T, K, &ldx);
        void* A = c.data(2, kBFloat16, {L, R, K});
        void* B = c.data(3, kBFloat16, {L, N, R});
        void* ids = c.data(4, kInt, {T});
        void* order = c.data(5, kInt, {T}, true);
        void* scales = c.data(6, kFloat, {L}, true);
        void* out = c.matrix(7, T, N, &ldo);
        if (L != (int32_t)L || R != (int32_t)R) c.refuse();
        return c.run(8, [&](void* s) {
            return fp8gemm_lora_add(Y, X, A, B, (const int32_t*)ids, (const int32_t*)order, (const float*)scales, out, T, (int32_t)L,
                                    (int32_t)R, K, N, ldx, ldy, ldo, s);
        });
    });
}

#define FP8GEMM_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FP8GEMM_METHOD(route_topk), FP8GEMM_METHOD(route_topk_backward), FP8GEMM_METHOD(moe_dispatch),
                         FP8GEMM_METHOD(moe_combine), FP8GEMM_METHOD(moe_combine_backward), FP8GEMM_METHOD(w4_gemv),
                         FP8GEMM_METHOD(w4_gemv_experts), FP8GEMM_METHOD(gated_ffn), FP8GEMM_METHOD(gated_ffn_backward),
                         FP8GEMM_METHOD(lora_add),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
