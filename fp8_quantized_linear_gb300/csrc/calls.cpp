// The linear layers' calls from Python: the checks of the tensors, the outputs'
// allocation and the C entry points, in one C function per call.
//
// These calls stand in front of kernels of two to fifteen microseconds, and the
// same checks written in Python took longer than that (13 to 20 us a call on
// the GB300's host cores; 4 to 8 us here).  Every error is a Python exception:
// a C++ one does not leave the extension.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <mutex>

#include "fp8linear.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *g_status_error = nullptr;  // called with (status, entry point): the exception

struct Refusal {
    PyObject *type;
    const char *text;
};

[[noreturn]] void value_error(const char *text) { throw Refusal{PyExc_ValueError, text}; }

// The tensor behind an argument (null for None): on device `index` (the first
// one sets it) and contiguous.
const Tensor *tensor(PyObject *o, int &index) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, "expected CUDA tensors"};
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw Refusal{PyExc_TypeError, "expected CUDA tensors"};
    if (index < 0) index = t.get_device();
    if (t.get_device() != index) value_error("tensors are on different devices");
    if (!t.is_contiguous()) value_error("expected contiguous tensors");
    return &t;
}

const Tensor &needed(PyObject *o, int &index) {
    const Tensor *t = tensor(o, index);
    if (t == nullptr) throw Refusal{PyExc_TypeError, "expected CUDA tensors"};
    return *t;
}

void *address(const Tensor *t) { return t == nullptr ? nullptr : t->data_ptr(); }

bool is_codes(const Tensor &t) {
    return t.scalar_type() == ScalarType::Byte || t.scalar_type() == ScalarType::Float8_e4m3fn;
}

bool is_16(ScalarType s) { return s == ScalarType::Half || s == ScalarType::BFloat16; }

int code16(ScalarType s) { return s == ScalarType::Half ? FP8L_F16 : FP8L_BF16; }

bool shaped(const Tensor &t, int64_t rows, int64_t cols) {
    return t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
}

// Other Python threads run while this one allocates and launches: a launch
// waits where the queue of the GPU is full, and what it waits for may need the
// interpreter.  (Nothing below an instance touches a Python object's count.)
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
    Unlocked() = default;
    Unlocked(const Unlocked &) = delete;
    Unlocked &operator=(const Unlocked &) = delete;
};

// The two kernels of a dynamic norm stand behind each other on their stream,
// also where two threads share it (and with it the workspace).
std::mutex g_norm_order;

Tensor empty(at::IntArrayRef size, ScalarType s, int index) {
    return at::detail::empty_cuda(size, s, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(index)),
                                  std::nullopt);
}

// A tensor that this call makes, or the one given.
struct Output {
    Tensor made;
    PyObject *given;
    explicit Output(PyObject *o) : given(o) {}
    void make(bool want, int64_t rows, int64_t cols, ScalarType s, int index) {
        if (given == Py_None && want) made = empty({rows, cols}, s, index);
    }
    void *ptr() const {
        if (made.defined()) return made.data_ptr();
        return given == Py_None ? nullptr : THPVariable_Unpack(given).data_ptr();
    }
    PyObject *result() const {  // a new reference
        if (made.defined()) return THPVariable_Wrap(made);
        Py_INCREF(given);
        return given;
    }
};

// Null, with the exception set, unless status is FP8L_OK.
bool failed(int status, const char *where) {
    if (status == FP8L_OK) return false;
    PyObject *e = PyObject_CallFunction(g_status_error, "is", status, where);
    if (e != nullptr) {
        PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
        Py_DECREF(e);
    }
    return true;
}

struct Epilogue {
    void *bias, *residual;
    int bias_code;
    int64_t width;
};

Epilogue epilogue(const Tensor *bias, const Tensor *residual, bool gated, int64_t M, int64_t N,
                  ScalarType out) {
    Epilogue e{address(bias), address(residual), FP8L_F32, gated ? N / 2 : N};
    if (bias != nullptr) {
        const ScalarType s = bias->scalar_type();
        if (bias->dim() != 1 || bias->size(0) != N || !(is_16(s) || s == ScalarType::Float))
            value_error("bias is [N] of float16, bfloat16 or float32");
        if (is_16(s)) e.bias_code = code16(s);
    }
    if (residual != nullptr && (!shaped(*residual, M, e.width) || residual->scalar_type() != out))
        value_error("residual is [M, N] ([M, N / 2] when gated) of the output's 16-bit type");
    return e;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

unsigned number(PyObject *o) {
    const unsigned long v = PyLong_AsUnsignedLong(o);
    if (v == static_cast<unsigned long>(-1) && PyErr_Occurred()) throw python_error();
    return static_cast<unsigned>(v);
}

#define CALL_BEGIN \
    HANDLE_TH_ERRORS try {
#define CALL_END                          \
    }                                     \
    catch (const Refusal &r) {            \
        PyErr_SetString(r.type, r.text);  \
        return nullptr;                   \
    }                                     \
    END_HANDLE_TH_ERRORS

// linear(a, w, a_scale, w_scale, bias, activation, gated, residual, out_dtype,
//        out_scale, y, ws, flags, per_token)
PyObject *linear(PyObject *, PyObject *const *args, Py_ssize_t count) {
    CALL_BEGIN
    if (count != 14) value_error("14 arguments");
    int index = -1;
    const Tensor &a = needed(args[0], index), &w = needed(args[1], index);
    const Tensor &a_scale = needed(args[2], index), &w_scale = needed(args[3], index);
    const Tensor *bias = tensor(args[4], index), *residual = tensor(args[7], index);
    const Tensor *out_scale = tensor(args[9], index), *y = tensor(args[10], index);
    const Tensor *ws = tensor(args[11], index);
    const bool gated = truth(args[6]);
    unsigned flags = number(args[12]);
    if (a.dim() != 2 || !is_codes(a)) value_error("a is [M, K] E4M3 codes (uint8 or float8_e4m3fn)");
    const int64_t M = a.size(0), K = a.size(1);
    if (w.dim() != 2 || !is_codes(w) || w.size(1) != K)
        value_error("w is [N, K] E4M3 codes (uint8 or float8_e4m3fn) of a's K");
    const int64_t N = w.size(0), scales = w_scale.numel(), tokens = a_scale.numel();
    if (w_scale.scalar_type() != ScalarType::Float || (scales != N && scales != 1))
        value_error("w_scale is float32 with 1 or N entries");
    const bool per_token = args[13] == Py_None ? tokens == M && M != 1 : truth(args[13]);
    if (a_scale.scalar_type() != ScalarType::Float || tokens != (per_token ? M : 1))
        value_error("a_scale is float32 with 1 entry, or M with per_token");
    if (per_token) flags |= FP8L_A_PER_TOKEN;
    ScalarType out = y != nullptr          ? y->scalar_type()
                     : residual != nullptr ? residual->scalar_type()
                                           : ScalarType::BFloat16;
    if (args[8] != Py_None) {
        if (!THPDtype_Check(args[8])) throw Refusal{PyExc_TypeError, "out_dtype is a torch.dtype"};
        out = reinterpret_cast<THPDtype *>(args[8])->scalar_type;
    }
    if (out == ScalarType::Float8_e4m3fn) out = ScalarType::Byte;
    const bool codes = out == ScalarType::Byte;
    if (!codes && !is_16(out)) value_error("out_dtype is float16, bfloat16 or uint8 (E4M3 codes)");
    if (codes) {
        if (out_scale == nullptr || out_scale->scalar_type() != ScalarType::Float || out_scale->numel() != 1)
            value_error("an E4M3 output needs out_scale, one float32");
        if (residual != nullptr) value_error("an E4M3 output takes no residual");
    }
    const Epilogue e = epilogue(bias, residual, gated, M, N, out);
    if (y != nullptr && (!shaped(*y, M, e.width) || !(codes ? is_codes(*y) : y->scalar_type() == out)))
        value_error("y is [M, N] ([M, N / 2] when gated) of out_dtype");
    if (ws != nullptr && (ws->scalar_type() != ScalarType::Byte ||
                          static_cast<size_t>(ws->numel()) < fp8l_workspace_bytes()))
        value_error("ws is a uint8 tensor of fp8l_workspace_bytes() elements");
    const int act = static_cast<int>(number(args[5])) | (gated ? FP8L_ACT_GATED : 0);
    Output result(args[10]);
    int status;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
        result.make(true, M, e.width, out, index);
        status = fp8_linear(
            static_cast<const uint8_t *>(a.data_ptr()), static_cast<const uint8_t *>(w.data_ptr()), M, N, K,
            static_cast<const float *>(a_scale.data_ptr()), static_cast<const float *>(w_scale.data_ptr()),
            scales != 1 ? 1 : 0, e.bias, e.bias_code, act, e.residual,
            codes ? static_cast<const float *>(out_scale->data_ptr()) : nullptr, result.ptr(),
            codes ? FP8L_E4M3 : code16(out), address(ws), flags,
            c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
    }
    if (failed(status, "fp8_linear")) return nullptr;
    return result.result();
    CALL_END
}

// w8a16_linear(x, w, w_scale, bias, activation, gated, residual, y, flags)
PyObject *w8a16_linear(PyObject *, PyObject *const *args, Py_ssize_t count) {
    CALL_BEGIN
    if (count != 9) value_error("9 arguments");
    int index = -1;
    const Tensor &x = needed(args[0], index), &w = needed(args[1], index);
    const Tensor &w_scale = needed(args[2], index);
    const Tensor *bias = tensor(args[3], index), *residual = tensor(args[6], index);
    const Tensor *y = tensor(args[7], index);
    const bool gated = truth(args[5]);
    const unsigned flags = number(args[8]);
    const ScalarType out = x.scalar_type();
    if (x.dim() != 2 || !is_16(out)) value_error("x is [M, K], float16 or bfloat16");
    const int64_t M = x.size(0), K = x.size(1), N = w_scale.numel();
    if (w_scale.scalar_type() != ScalarType::Float) value_error("w_scale is [N] float32");
    if ((flags & FP8L_WEIGHTS_PACKED) != 0u) {
        if (w.scalar_type() != ScalarType::Byte || w.numel() != N * ((K + 63) / 64 * 64))
            value_error("packed weights must be fp8_pack_w8a16_weights output for [N, K]");
    } else if (!is_codes(w) || !shaped(w, N, K)) {
        value_error("w is [N, K] E4M3 codes (uint8 or float8_e4m3fn) of x's K and w_scale's N");
    }
    const Epilogue e = epilogue(bias, residual, gated, M, N, out);
    if (y != nullptr && (!shaped(*y, M, e.width) || y->scalar_type() != out))
        value_error("y is [M, N] ([M, N / 2] when gated) of x's dtype");
    const int code = code16(out), act = static_cast<int>(number(args[4])) | (gated ? FP8L_ACT_GATED : 0);
    Output result(args[7]);
    int status;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
        result.make(true, M, e.width, out, index);
        // scratch of this call, from the stream's memory
        const size_t bytes = fp8_w8a16_linear_workspace_bytes(code, M, N, K, flags);
        Tensor scratch;
        if (bytes > 0) scratch = empty({static_cast<int64_t>(bytes)}, ScalarType::Byte, index);
        status = fp8_w8a16_linear(
            x.data_ptr(), code, static_cast<const uint8_t *>(w.data_ptr()),
            static_cast<const float *>(w_scale.data_ptr()), M, N, K, e.bias, e.bias_code, act, e.residual,
            result.ptr(), bytes > 0 ? scratch.data_ptr() : nullptr, flags,
            c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
    }
    if (failed(status, "fp8_w8a16_linear")) return nullptr;
    return result.result();
    CALL_END
}

// add_rmsnorm_quant(x, residual, gamma, eps, mode, total, q, scale, h, want_h, ws)
//   -> (q, scale, total, h)
PyObject *add_rmsnorm_quant(PyObject *, PyObject *const *args, Py_ssize_t count) {
    CALL_BEGIN
    if (count != 11) value_error("11 arguments");
    int index = -1;
    const Tensor &x = needed(args[0], index), &residual = needed(args[1], index);
    const Tensor &gamma = needed(args[2], index);
    const Tensor *total = tensor(args[5], index), *q = tensor(args[6], index);
    const Tensor *scale = tensor(args[7], index), *h = tensor(args[8], index);
    const Tensor *ws = tensor(args[10], index);
    const double eps = PyFloat_AsDouble(args[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    const int mode = static_cast<int>(number(args[4]));
    const bool codes = mode != FP8L_NQ_NORM_ONLY;
    const ScalarType s = x.scalar_type();
    if (x.dim() != 2 || !is_16(s)) value_error("x is [M, K], float16 or bfloat16");
    const int64_t M = x.size(0), K = x.size(1);
    if (!shaped(residual, M, K) || residual.scalar_type() != s || gamma.dim() != 1 ||
        gamma.size(0) != K || gamma.scalar_type() != s)
        value_error("residual is [M, K] and gamma [K], of x's dtype");
    if (total != nullptr && (!shaped(*total, M, K) || total->scalar_type() != s))
        value_error("total is [M, K] of x's dtype");
    if (h != nullptr && (!shaped(*h, M, K) || h->scalar_type() != s))
        value_error("h is [M, K] of x's dtype");
    const int64_t entries = mode == FP8L_NQ_PER_TOKEN ? M : 1;
    if (codes) {
        if (q != nullptr && (!shaped(*q, M, K) || !is_codes(*q)))
            value_error("q is [M, K] E4M3 codes (uint8 or float8_e4m3fn)");
        if (scale == nullptr && mode == FP8L_NQ_STATIC) value_error("static mode needs a scale tensor");
        if (scale != nullptr && (scale->numel() != entries || scale->scalar_type() != ScalarType::Float))
            value_error("scale is float32 with 1 entry, or M per token");
    }
    if (ws != nullptr && (ws->scalar_type() != ScalarType::Byte ||
                          static_cast<size_t>(ws->numel()) < fp8l_workspace_bytes()))
        value_error("ws is a uint8 tensor of fp8l_workspace_bytes() elements");
    const bool want_h = !codes || truth(args[9]);
    Output total_out(args[5]), q_out(args[6]), h_out(args[8]);
    Tensor made_scale;
    int status;
    {
        const Unlocked unlocked;
        const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
        total_out.make(true, M, K, s, index);
        q_out.make(codes, M, K, ScalarType::Byte, index);
        if (codes && scale == nullptr) made_scale = empty({entries}, ScalarType::Float, index);
        h_out.make(want_h, M, K, s, index);
        void *scale_ptr = scale != nullptr ? scale->data_ptr()
                                           : (made_scale.defined() ? made_scale.data_ptr() : nullptr);
        std::unique_lock<std::mutex> order(g_norm_order, std::defer_lock);
        if (mode == FP8L_NQ_DYNAMIC) order.lock();
        status = fp8_add_rmsnorm_quant(
            x.data_ptr(), residual.data_ptr(), code16(s), gamma.data_ptr(), static_cast<float>(eps), M, K,
            total_out.ptr(), codes ? static_cast<uint8_t *>(q_out.ptr()) : nullptr,
            codes ? static_cast<float *>(scale_ptr) : nullptr, mode, h_out.ptr(), address(ws),
            c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream());
    }
    if (failed(status, "fp8_add_rmsnorm_quant")) return nullptr;
    PyObject *scale_result = args[7];
    if (made_scale.defined())
        scale_result = THPVariable_Wrap(made_scale);
    else
        Py_INCREF(scale_result);
    PyObject *all[4] = {q_out.result(), scale_result, total_out.result(), h_out.result()};
    PyObject *tuple = PyTuple_New(4);
    for (int i = 0; i < 4; ++i) {
        if (tuple != nullptr && all[i] != nullptr)
            PyTuple_SET_ITEM(tuple, i, all[i]);
        else
            Py_XDECREF(all[i]);
    }
    if (PyErr_Occurred()) {
        Py_XDECREF(tuple);
        return nullptr;
    }
    return tuple;
    CALL_END
}

// setup(status_error)
PyObject *setup(PyObject *, PyObject *error) {
    Py_INCREF(error);
    Py_XDECREF(g_status_error);
    g_status_error = error;
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear)), METH_FASTCALL, nullptr},
    {"w8a16_linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(w8a16_linear)),
     METH_FASTCALL, nullptr},
    {"add_rmsnorm_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(add_rmsnorm_quant)),
     METH_FASTCALL, nullptr},
    {"setup", setup, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&kModule); }
