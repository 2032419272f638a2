// torch_calls.cpp -- how Python reaches the operators around the attention: the
// module `_calls`. Each function checks its tensors, allocates the outputs that
// were not given on the current stream, and calls the C entry on that stream. The
// kernels of a decoding step take 2 to 5 us; the same in Python and ctypes took 9
// to 15 us a call, this takes 3 to 6.
#include <Python.h>

#include <algorithm>
#include <cstdint>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gai4.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* error_class;   // Gai4Error(name, status)

#define GAI4_CHECK(condition, ...) TORCH_CHECK_VALUE(condition, "gai4: ", __VA_ARGS__)
constexpr const char* kOffDevice =
    "tensors must live on one CUDA device, and be contiguous where they have no stride argument";

const Tensor& tensor(PyObject* o) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), "gai4: expected a tensor, got ", Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}
bool given(PyObject* o) { return o != Py_None; }

int device_of(const Tensor& t) { return t.is_cuda() ? (int)t.get_device() : -1; }
void on_device(const Tensor& t, int device) { GAI4_CHECK(device >= 0 && device_of(t) == device, kOffDevice); }

gai4_dtype dtype_of(ScalarType t) {
    GAI4_CHECK(t == at::kFloat || t == at::kHalf || t == at::kBFloat16, "unsupported dtype ", t);
    return t == at::kFloat ? GAI4_F32 : t == at::kHalf ? GAI4_F16 : GAI4_BF16;
}
bool is_codes(const Tensor& t) { return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte; }

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

Tensor fresh(at::IntArrayRef shape, ScalarType type, const Tensor& like) {
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// without the interpreter's lock: a full launch queue blocks a call
struct Unlocked {
    PyThreadState* thread = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(thread); }
};
template <typename F>
void call(const char* name, F entry) {
    const gai4_status status = [&] {
        const Unlocked unlocked;
        return entry();
    }();
    if (status == GAI4_OK) return;
    PyObject* e = PyObject_CallFunction(error_class, "si", name, (int)status);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    throw python_error();
}

PyObject* wrapped(const Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
template <typename... Ts>
PyObject* tuple(const Ts&... ts) {
    PyObject* all[] = {wrapped(ts)...};
    PyObject* r = PyTuple_New(sizeof...(Ts));
    if (!r) throw python_error();
    for (size_t i = 0; i < sizeof...(Ts); ++i) PyTuple_SET_ITEM(r, (Py_ssize_t)i, all[i]);
    return r;
}

// [n, heads, d] rows with contiguous heads
struct HeadRows {
    int64_t heads = 0, stride = 0;
    void* data = nullptr;
};
HeadRows head_rows(const Tensor& t, int64_t n, int64_t d, ScalarType type, int device, const char* what) {
    GAI4_CHECK(t.dim() == 3 && t.size(0) == n && t.size(2) == d && t.scalar_type() == type &&
                   (t.stride(2) == 1 || d == 1) && (t.stride(1) == d || t.size(1) <= 1),
               what, " must be [tokens, heads, head_dim] of q's type, heads contiguous within a token");
    on_device(t, device);
    const int64_t heads = t.size(1);
    return {heads, n > 1 ? t.stride(0) : heads * d, t.data_ptr()};
}

// [rows, cols] with contiguous columns
int64_t row_stride(const Tensor& t, int device, const char* what) {
    GAI4_CHECK(t.dim() == 2 && (t.stride(1) == 1 || t.size(1) <= 1), what, " must be [rows, columns], columns contiguous");
    on_device(t, device);
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

// a contiguous operand or output
void* whole(const Tensor& t, at::IntArrayRef shape, ScalarType type, int device, const char* what) {
    GAI4_CHECK(t.sizes() == shape && t.scalar_type() == type, what, " must be ", type, " of shape ", shape);
    on_device(t, device);
    GAI4_CHECK(t.is_contiguous(), kOffDevice);
    return t.data_ptr();
}

// codes [rows, cols] and scales [scale_rows, ceil(cols / 128)], made where they are not given
void fp8_outputs(PyObject* codes_arg, PyObject* scales_arg, const Tensor& x, int64_t scale_rows, int device, Tensor& codes,
                 Tensor& scales) {
    const int64_t rows = x.size(0), cols = x.size(1), blocks = (cols + 127) / 128;
    if (given(codes_arg)) {
        codes = tensor(codes_arg);
        GAI4_CHECK(is_codes(codes) && codes.sizes() == x.sizes() && codes.is_contiguous() && device_of(codes) == device,
                   "codes must be float8_e4m3fn (or uint8) [rows, cols], contiguous, on x's device");
    } else {
        codes = fresh({rows, cols}, at::kFloat8_e4m3fn, x);
    }
    if (given(scales_arg)) {
        scales = tensor(scales_arg);
        whole(scales, {scale_rows, blocks}, at::kFloat, device, "scales");
    } else {
        scales = fresh({scale_rows, blocks}, at::kFloat, x);
    }
}

#define GAI4_ARGUMENTS(n)                                                     \
    HANDLE_TH_ERRORS                                                          \
    if (count != n) {                                                         \
        PyErr_SetString(PyExc_TypeError, "gai4: wrong number of arguments"); \
        return nullptr;                                                       \
    }

// q, k, positions, inv_freq, interleaved, mscale, q_out, k_out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t count) {
    GAI4_ARGUMENTS(8)
    const Tensor &q = tensor(a[0]), &positions = tensor(a[2]), &inv_freq = tensor(a[3]);
    GAI4_CHECK(q.dim() == 3, "q must be [tokens, heads, head_dim]");
    const int64_t n = q.size(0), d = q.size(2);
    const ScalarType type = q.scalar_type();
    const int device = device_of(q);
    GAI4_CHECK(positions.dim() == 1 && positions.size(0) == n && positions.scalar_type() == at::kInt &&
                   inv_freq.dim() == 1 && inv_freq.scalar_type() == at::kDouble,
               "positions must be int32 [tokens], inv_freq float64 [rot_dim / 2]");
    on_device(positions, device);
    on_device(inv_freq, device);
    GAI4_CHECK(positions.is_contiguous() && inv_freq.is_contiguous(), kOffDevice);
    const HeadRows from = head_rows(q, n, d, type, device, "q");
    Tensor q_out = given(a[6]) ? tensor(a[6]) : fresh(q.sizes(), type, q), k_out;
    const HeadRows to = head_rows(q_out, n, d, type, device, "q_out");
    GAI4_CHECK(to.heads == from.heads, "q_out must have q's shape");
    HeadRows k_from, k_to;
    if (given(a[1])) {
        const Tensor& k = tensor(a[1]);
        k_from = head_rows(k, n, d, type, device, "k");
        k_out = given(a[7]) ? tensor(a[7]) : fresh(k.sizes(), type, k);
        k_to = head_rows(k_out, n, d, type, device, "k_out");
        GAI4_CHECK(k_to.heads == k_from.heads, "k_out must have k's shape");
    }
    const float mscale = (float)number(a[5]);
    const bool interleaved = truth(a[4]);
    const gai4_dtype dtype = dtype_of(type);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    call("gai4_rope", [&] {
        return gai4_rope(from.data, from.stride, to.data, to.stride, k_from.data, k_from.stride, k_to.data, k_to.stride,
                         static_cast<const int32_t*>(positions.data_ptr()),
                         static_cast<const double*>(inv_freq.data_ptr()), mscale, dtype, n, from.heads, k_from.heads,
                         (int)std::min<int64_t>(d, INT32_MAX), (int)std::min<int64_t>(2 * inv_freq.size(0), INT32_MAX),
                         interleaved, stream_of(device));
    });
    return tuple(q_out, k_out);
    END_HANDLE_TH_ERRORS
}

// x, gain, eps, residual, fp8, out, residual_out, codes, scales
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t count) {
    GAI4_ARGUMENTS(9)
    const Tensor& x = tensor(a[0]);
    const int device = device_of(x);
    const ScalarType type = x.scalar_type();
    const int64_t x_stride = row_stride(x, device, "x"), rows = x.size(0), cols = x.size(1);
    const bool fp8 = truth(a[4]);
    Tensor out, residual_out, codes, scales;
    const void *residual = nullptr, *gain = nullptr;
    int64_t r_stride = 0;
    if (given(a[3])) {
        const Tensor& r = tensor(a[3]);
        GAI4_CHECK(r.sizes() == x.sizes() && r.scalar_type() == type, "residual must have x's shape and type");
        r_stride = row_stride(r, device, "residual");
        residual = r.data_ptr();
    }
    if (given(a[1])) gain = whole(tensor(a[1]), {cols}, type, device, "gain");
    if (given(a[6])) {
        residual_out = tensor(a[6]);
        whole(residual_out, x.sizes(), type, device, "residual_out");
    } else if (given(a[3])) {
        residual_out = fresh(x.sizes(), type, x);
    }
    if (given(a[5])) {
        out = tensor(a[5]);
        whole(out, x.sizes(), type, device, "out");
    } else if (!fp8) {
        out = fresh(x.sizes(), type, x);
    }
    if (fp8)
        fp8_outputs(a[7], a[8], x, rows, device, codes, scales);
    else
        GAI4_CHECK(!given(a[7]) && !given(a[8]), "codes and scales are outputs of fp8=True");
    const float eps = (float)number(a[2]);
    const gai4_dtype dtype = dtype_of(type);
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    const auto data = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    call("gai4_rms_norm", [&] {
        return gai4_rms_norm(x.data_ptr(), x_stride, residual, r_stride, gain, data(out), data(residual_out),
                             static_cast<uint8_t*>(data(codes)), static_cast<float*>(data(scales)), dtype, rows, cols, eps,
                             stream_of(device));
    });
    return tuple(out, residual_out, codes, scales);
    END_HANDLE_TH_ERRORS
}

// x, codes, scales
PyObject* quantize_x_fp8(PyObject*, PyObject* const* a, Py_ssize_t count) {
    GAI4_ARGUMENTS(3)
    const Tensor& x = tensor(a[0]);
    const int device = device_of(x);
    const int64_t stride = row_stride(x, device, "x");
    Tensor codes, scales;
    fp8_outputs(a[1], a[2], x, x.size(0), device, codes, scales);
    const gai4_dtype dtype = dtype_of(x.scalar_type());
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    call("gai4_quantize_x_fp8", [&] {
        return gai4_quantize_x_fp8(x.data_ptr(), stride, static_cast<uint8_t*>(codes.data_ptr()),
                                   static_cast<float*>(scales.data_ptr()), dtype, x.size(0), x.size(1),
                                   stream_of(device));
    });
    return tuple(codes, scales);
    END_HANDLE_TH_ERRORS
}

// w, codes, scales
PyObject* quantize_fp8(PyObject*, PyObject* const* a, Py_ssize_t count) {
    GAI4_ARGUMENTS(3)
    const Tensor& w = tensor(a[0]);
    const int device = device_of(w);
    GAI4_CHECK(w.dim() == 2, "w must be [N, K]");
    on_device(w, device);
    GAI4_CHECK(w.is_contiguous(), kOffDevice);
    Tensor codes, scales;
    fp8_outputs(a[1], a[2], w, (w.size(0) + 127) / 128, device, codes, scales);
    const gai4_dtype dtype = dtype_of(w.scalar_type());
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    call("gai4_quantize_fp8", [&] {
        return gai4_quantize_fp8(w.data_ptr(), static_cast<uint8_t*>(codes.data_ptr()),
                                 static_cast<float*>(scales.data_ptr()), dtype, w.size(0), w.size(1), stream_of(device));
    });
    return tuple(codes, scales);
    END_HANDLE_TH_ERRORS
}

// w_codes, w_scales, x_codes, x_scales, out, dtype
PyObject* fp8_mm_t(PyObject*, PyObject* const* a, Py_ssize_t count) {
    GAI4_ARGUMENTS(6)
    const Tensor &w = tensor(a[0]), &ws = tensor(a[1]), &x = tensor(a[2]), &xs = tensor(a[3]);
    GAI4_CHECK(w.dim() == 2 && x.dim() == 2 && ws.dim() == 2 && xs.dim() == 2 && x.size(1) == w.size(1) &&
                   xs.size(0) == x.size(0) && ws.size(0) == (w.size(0) + 127) / 128 &&
                   xs.size(1) == (w.size(1) + 127) / 128 && ws.size(1) == xs.size(1) &&
                   xs.scalar_type() == at::kFloat && ws.scalar_type() == at::kFloat && is_codes(w) && is_codes(x),
               "codes e4m3 [N, K] and [M, K], scales float32 [ceil(N / 128), ceil(K / 128)] and [M, ceil(K / 128)]");
    const int64_t M = x.size(0), N = w.size(0);
    const int device = device_of(x);
    for (const Tensor* t : {&w, &ws, &x, &xs}) {
        on_device(*t, device);
        GAI4_CHECK(t->is_contiguous(), kOffDevice);
    }
    Tensor out;
    if (given(a[4])) {
        out = tensor(a[4]);
        whole(out, {M, N}, out.scalar_type(), device, "out");
    } else {
        TORCH_CHECK_TYPE(THPDtype_Check(a[5]), "gai4: dtype must be a torch.dtype");
        const ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
        dtype_of(type);
        out = fresh({M, N}, type, x);
    }
    const gai4_dtype dtype = dtype_of(out.scalar_type());
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    call("gai4_fp8_mm_t", [&] {
        return gai4_fp8_mm_t(static_cast<const uint8_t*>(w.data_ptr()), static_cast<const float*>(ws.data_ptr()),
                             static_cast<const uint8_t*>(x.data_ptr()), static_cast<const float*>(xs.data_ptr()),
                             out.data_ptr(), dtype, M, N, w.size(1), stream_of(device));
    });
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(error_class, cls);
    Py_RETURN_NONE;
}

template <PyObject* (*fn)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn));
}

PyMethodDef methods[] = {
    {"rope", fast<rope>(), METH_FASTCALL, nullptr},
    {"rms_norm", fast<rms_norm>(), METH_FASTCALL, nullptr},
    {"quantize_x_fp8", fast<quantize_x_fp8>(), METH_FASTCALL, nullptr},
    {"quantize_fp8", fast<quantize_fp8>(), METH_FASTCALL, nullptr},
    {"fp8_mm_t", fast<fp8_mm_t>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
