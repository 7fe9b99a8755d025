// torch_binding.cpp -- the Python calls of the 8-bit operators, of routing from
// logits, the product with an epilogue and the sum of experts' rows: argument checks,
// the outputs' allocation and the C ABI call (include/moe.h), in C++.
//
// These operators take a few microseconds on the GPU at decode sizes, less than
// the same steps cost as Python statements (measured on the GB300 host, a norm
// of one token: four torch.empty 6.3 us, checks and arguments 3.5 us, a ctypes
// call 1.3 us beside the launch's 2). A CPython module over PyTorch's tensors:
// lib.py has the signatures and the documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/moe.h"

namespace {

using at::Tensor;

constexpr int64_t kBlock = 128;   // values that share one scale

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// What is wrong with an argument; raised as ValueError.
struct BadArgument : std::runtime_error {
    using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const char* name, const Tensor& t, const std::string& want)
{
    std::ostringstream s;
    s << name << ": expected " << want << ", got " << t.scalar_type() << " " << t.sizes() << " with strides "
      << t.strides() << " on " << t.device();
    throw BadArgument(s.str());
}

bool is_size(const Tensor& t, std::initializer_list<int64_t> size)
{
    return t.sizes() == at::IntArrayRef(size);
}

std::string described(const char* what, at::ScalarType type, std::initializer_list<int64_t> size, at::Device dev)
{
    std::ostringstream s;
    s << what << " " << type << " tensor of shape " << at::IntArrayRef(size) << " on " << dev;
    return s.str();
}

void expect(const char* name, const Tensor& t, at::ScalarType type, std::initializer_list<int64_t> size, at::Device dev)
{
    if (t.scalar_type() != type || !is_size(t, size) || t.device() != dev || !t.is_contiguous())
        refuse(name, t, described("a contiguous", type, size, dev));
}

// Rows of contiguous elements, any row stride.
void expect_rows(const char* name, const Tensor& t, at::ScalarType type, int64_t rows, int64_t cols, at::Device dev)
{
    if (t.scalar_type() != type || !is_size(t, {rows, cols}) || t.device() != dev || (cols > 1 && t.stride(1) != 1))
        refuse(name, t, described("rows of contiguous elements in a", type, {rows, cols}, dev));
}

const Tensor& tensor_of(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) throw BadArgument(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

std::optional<Tensor> optional_of(PyObject* o, const char* name)
{
    if (o == Py_None) return std::nullopt;
    return tensor_of(o, name);
}

int64_t dim(const Tensor& t, const char* name, int64_t d, int64_t of)
{
    if (t.dim() != of) throw BadArgument(std::string(name) + ": expected " + std::to_string(of) + " dimensions, got " +
                                         std::to_string(t.dim()));
    return t.size(d);
}

void* ptr(const std::optional<Tensor>& t) { return t ? t->data_ptr() : nullptr; }

// The device and stream of a call: the tensors' device, and the stream given (a
// handle, as an int) or the current one. Outputs are allocated on that stream.
struct Launch {
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard on;
    moe_stream_t stream = nullptr;

    Launch(at::Device dev, PyObject* handle)
    {
        if (!dev.is_cuda()) throw BadArgument("expected CUDA tensors");
        device.set_device(dev);
        if (handle != Py_None) {
            const auto raw = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(handle));
            if (PyErr_Occurred()) throw BadArgument("stream: expected a stream's handle");
            on.reset_stream(c10::cuda::getStreamFromExternal(raw, dev.index()).unwrap());
            stream = reinterpret_cast<moe_stream_t>(raw);
        } else {
            stream = reinterpret_cast<moe_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
        }
    }
};

Tensor empty(std::initializer_list<int64_t> size, at::ScalarType type, at::Device dev)
{
    return Tensor(at::detail::empty_cuda(at::IntArrayRef(size), type, dev, std::nullopt));
}

// A status as the Python int that lib.py turns into MoeError.
PyObject* failed(moe_status s) { return PyLong_FromLong(s); }

PyObject* wrap(const std::optional<Tensor>& t)
{
    if (!t) Py_RETURN_NONE;
    return THPVariable_Wrap(*t);
}

PyObject* tuple_of(std::initializer_list<std::optional<Tensor>> ts)
{
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const auto& t : ts) {
        PyObject* o = r ? wrap(t) : nullptr;
        if (!o) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// add_rmsnorm_fp8(x, weight, residual, eps, want_y, sum_out, stream)
PyObject* add_rmsnorm_fp8(PyObject* const* a)
{
    const Tensor& x = tensor_of(a[0], "x");
    const std::optional<Tensor> weight = optional_of(a[1], "weight"), residual = optional_of(a[2], "residual");
    std::optional<Tensor> sum = optional_of(a[5], "sum_out");
    const double eps = PyFloat_AsDouble(a[3]);
    const int want_y = PyObject_IsTrue(a[4]);
    if (PyErr_Occurred()) return nullptr;
    const int64_t T = dim(x, "x", 0, 2), H = x.size(1);
    const at::ScalarType type = x.scalar_type();
    moe_dtype code;
    if (type == at::kBFloat16) code = MOE_BF16;
    else if (type == at::kHalf) code = MOE_FP16;
    else if (type == at::kFloat) code = MOE_FP32;
    else refuse("x", x, "a bf16, fp16 or fp32 tensor");
    const at::Device dev = x.device();
    expect_rows("x", x, type, T, H, dev);
    if (weight) expect("weight", *weight, type, {H}, dev);
    if (residual) expect_rows("residual", *residual, type, T, H, dev);
    if (sum) expect_rows("sum_out", *sum, type, T, H, dev);
    const Launch launch(dev, a[6]);
    if (residual && !sum) sum = empty({T, H}, type, dev);
    std::optional<Tensor> y;
    if (want_y) y = empty({T, H}, type, dev);
    const Tensor q = empty({T, H}, at::kFloat8_e4m3fn, dev);
    const Tensor scale = empty({T, blocks_of(H)}, at::kFloat, dev);
    if (H > INT32_MAX) return failed(MOE_ERR_UNSUPPORTED);
    const moe_status s = moe_add_rmsnorm_fp8(T, (int32_t)H, code, x.data_ptr(), x.stride(0), ptr(residual),
                                             residual ? residual->stride(0) : 0, ptr(weight), (float)eps, ptr(sum),
                                             sum ? sum->stride(0) : 0, ptr(y), static_cast<moe_e4m3*>(q.data_ptr()),
                                             static_cast<float*>(scale.data_ptr()), launch.stream);
    if (s != MOE_OK) return failed(s);
    return tuple_of({sum, y, q, scale});
}

// The sizes and the shared checks of the two products.
struct Product {
    int64_t R, K, N, G;

    Product(const Tensor& a, const Tensor& a_scale, const Tensor& w, const std::optional<Tensor>& offsets,
            const Tensor& ws)
        : R(dim(a, "a", 0, 2)), K(a.size(1)), N(dim(w, "w", 1, 3)), G(w.size(0))
    {
        const at::Device dev = a.device();
        expect("a", a, at::kFloat8_e4m3fn, {R, K}, dev);
        expect("a_scale", a_scale, at::kFloat, {R, blocks_of(K)}, dev);
        if (offsets) expect("offsets", *offsets, at::kInt, {G + 1}, dev);
        if (ws.scalar_type() != at::kByte || ws.device() != dev || !ws.is_contiguous())
            refuse("ws", ws, "a contiguous uint8 tensor on the same device");
    }

    void weight(const char* name, const Tensor& w, const char* scale_name, const Tensor& scale, at::Device dev) const
    {
        expect(name, w, at::kFloat8_e4m3fn, {G, N, K}, dev);
        expect(scale_name, scale, at::kFloat, {G, blocks_of(N), blocks_of(K)}, dev);
    }

    bool fits() const { return K <= INT32_MAX && N <= INT32_MAX && G <= INT32_MAX; }
};

const moe_e4m3* e4m3(const Tensor& t) { return static_cast<const moe_e4m3*>(t.data_ptr()); }
const float* f32(const Tensor& t) { return static_cast<const float*>(t.data_ptr()); }

// fp8_matmul(a, a_scale, w, w_scale, ws, offsets, bf16, out, stream)
PyObject* fp8_matmul(PyObject* const* a)
{
    const Tensor &A = tensor_of(a[0], "a"), &a_scale = tensor_of(a[1], "a_scale"), &w = tensor_of(a[2], "w"),
                 &w_scale = tensor_of(a[3], "w_scale"), &ws = tensor_of(a[4], "ws");
    const std::optional<Tensor> offsets = optional_of(a[5], "offsets");
    const int bf16 = PyObject_IsTrue(a[6]);
    if (bf16 < 0) return nullptr;
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
    const at::Device dev = A.device();
    const Product p(A, a_scale, w, offsets, ws);
    p.weight("w", w, "w_scale", w_scale, dev);
    std::optional<Tensor> out = optional_of(a[7], "out");
    if (out) expect("out", *out, type, {p.R, p.N}, dev);
    const Launch launch(dev, a[8]);
    if (!out) out = empty({p.R, p.N}, type, dev);
    if (!p.fits()) return failed(MOE_ERR_UNSUPPORTED);
    const moe_status s = moe_fp8_matmul(p.R, (int32_t)p.K, (int32_t)p.N, (int32_t)p.G, e4m3(A), f32(a_scale),
                                        static_cast<const int32_t*>(ptr(offsets)), e4m3(w), f32(w_scale),
                                        bf16 ? MOE_BF16 : MOE_FP32, out->data_ptr(), ws.data_ptr(),
                                        (size_t)ws.numel(), launch.stream);
    if (s != MOE_OK) return failed(s);
    return wrap(out);
}

// fp8_gated(a, a_scale, w1, w1_scale, w3, w3_scale, ws, offsets, stream)
PyObject* fp8_gated(PyObject* const* a)
{
    const Tensor &A = tensor_of(a[0], "a"), &a_scale = tensor_of(a[1], "a_scale"), &w1 = tensor_of(a[2], "w1"),
                 &w1_scale = tensor_of(a[3], "w1_scale"), &w3 = tensor_of(a[4], "w3"),
                 &w3_scale = tensor_of(a[5], "w3_scale"), &ws = tensor_of(a[6], "ws");
    const std::optional<Tensor> offsets = optional_of(a[7], "offsets");
    const at::Device dev = A.device();
    const Product p(A, a_scale, w1, offsets, ws);
    p.weight("w1", w1, "w1_scale", w1_scale, dev);
    p.weight("w3", w3, "w3_scale", w3_scale, dev);
    const Launch launch(dev, a[8]);
    const Tensor h = empty({p.R, p.N}, at::kFloat8_e4m3fn, dev);
    const Tensor scale = empty({p.R, blocks_of(p.N)}, at::kFloat, dev);
    if (!p.fits()) return failed(MOE_ERR_UNSUPPORTED);
    const moe_status s = moe_fp8_gated(p.R, (int32_t)p.K, (int32_t)p.N, (int32_t)p.G, e4m3(A), f32(a_scale),
                                       static_cast<const int32_t*>(ptr(offsets)), e4m3(w1), f32(w1_scale), e4m3(w3),
                                       f32(w3_scale), static_cast<moe_e4m3*>(h.data_ptr()),
                                       static_cast<float*>(scale.data_ptr()), ws.data_ptr(), (size_t)ws.numel(),
                                       launch.stream);
    if (s != MOE_OK) return failed(s);
    return tuple_of({h, scale});
}

// The moe_dtype of a tensor's type.
moe_dtype code_of(const char* name, const Tensor& t, bool with_f32 = true)
{
    switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_BF16;
    case at::kHalf: return MOE_FP16;
    case at::kFloat:
        if (with_f32) return MOE_FP32;
        [[fallthrough]];
    default: refuse(name, t, with_f32 ? "a bf16, fp16 or fp32 tensor" : "a bf16 or fp16 tensor");
    }
}

int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw BadArgument("expected whole numbers");
    return v;
}

int32_t small_integer(PyObject* o, const char* name)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) throw BadArgument(std::string(name) + ": out of range");
    return (int32_t)v;
}

// route_logits(logits, k, sigmoid, bias, groups, top_groups, group_top, renormalize, scale, topk_idx, topk_w, stream)
PyObject* route_logits(PyObject* const* a)
{
    const Tensor& logits = tensor_of(a[0], "logits");
    const std::optional<Tensor> bias = optional_of(a[3], "bias");
    std::optional<Tensor> idx = optional_of(a[9], "topk_idx"), w = optional_of(a[10], "topk_w");
    const int32_t k = small_integer(a[1], "k");
    const int sigmoid = PyObject_IsTrue(a[2]), renorm = PyObject_IsTrue(a[7]);
    const double scale = PyFloat_AsDouble(a[8]);
    moe_scoring c{};
    c.groups = small_integer(a[4], "groups");
    c.top_groups = small_integer(a[5], "top_groups");
    c.group_top = small_integer(a[6], "group_top");
    if (PyErr_Occurred()) return nullptr;
    c.scores = sigmoid ? MOE_SCORES_SIGMOID : MOE_SCORES_SOFTMAX;
    c.renormalize = renorm;
    c.scale = (float)scale;
    const int64_t T = dim(logits, "logits", 0, 2), E = logits.size(1);
    const moe_dtype code = code_of("logits", logits);
    const at::Device dev = logits.device();
    expect_rows("logits", logits, logits.scalar_type(), T, E, dev);
    if (bias) expect("bias", *bias, at::kFloat, {E}, dev);
    if (idx) expect("topk_idx", *idx, at::kInt, {T, k}, dev);
    if (w) expect("topk_w", *w, at::kFloat, {T, k}, dev);
    if (k <= 0) return failed(MOE_ERR_INVALID_ARG);
    if (E > INT32_MAX || k > E) return failed(E > INT32_MAX ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG);
    const Launch launch(dev, a[11]);
    // (a block of memory each, 0.5 us more than one for both: they are stored and kept apart)
    if (!idx) idx = empty({T, k}, at::kInt, dev);
    if (!w) w = empty({T, k}, at::kFloat, dev);
    c.bias = static_cast<const float*>(ptr(bias));
    const moe_status s = moe_route_logits(T, (int32_t)E, k, code, logits.data_ptr(), logits.stride(0), &c,
                                          static_cast<int32_t*>(idx->data_ptr()), static_cast<float*>(w->data_ptr()),
                                          launch.stream);
    if (s != MOE_OK) return failed(s);
    return tuple_of({idx, w});
}

// linear(a, w, ws, bias, activation, residual, offsets, f32, out, stream)
PyObject* linear(PyObject* const* a)
{
    const Tensor &A = tensor_of(a[0], "a"), &w = tensor_of(a[1], "w"), &ws = tensor_of(a[2], "ws");
    const std::optional<Tensor> bias = optional_of(a[3], "bias"), residual = optional_of(a[5], "residual"),
                                offsets = optional_of(a[6], "offsets");
    std::optional<Tensor> out = optional_of(a[8], "out");
    moe_epilogue e{};
    e.activation = (moe_activation)small_integer(a[4], "activation");
    const int f32 = PyObject_IsTrue(a[7]);
    if (f32 < 0) return nullptr;
    const int64_t R = dim(A, "a", 0, 2), K = A.size(1), N = dim(w, "w", 2, 3), G = w.size(0);
    const moe_dtype code = code_of("a", A, false);
    const at::ScalarType type = A.scalar_type(), out_type = f32 ? at::kFloat : type;
    const at::Device dev = A.device();
    expect_rows("a", A, type, R, K, dev);
    // [G, K, N] with contiguous n, or the view of [G, N, K] with contiguous k (one column may be either)
    const bool kn = w.is_contiguous(), nk = (!kn || N % 8) && w.transpose(1, 2).is_contiguous();
    if (w.scalar_type() != type || !is_size(w, {G, K, N}) || w.device() != dev || !(kn || nk))
        refuse("w", w, described("(contiguous, or the transpose of a contiguous) a", type, {G, K, N}, dev));
    if (bias) expect("bias", *bias, bias->scalar_type() == at::kFloat ? at::kFloat : type, {G, N}, dev);
    if (residual) expect_rows("residual", *residual, out_type, R, N, dev);
    if (offsets) expect("offsets", *offsets, at::kInt, {G + 1}, dev);
    if (out) expect_rows("out", *out, out_type, R, N, dev);
    if (ws.scalar_type() != at::kByte || ws.device() != dev || !ws.is_contiguous())
        refuse("ws", ws, "a contiguous uint8 tensor on the same device");
    if (K > INT32_MAX || N > INT32_MAX || G > INT32_MAX) return failed(MOE_ERR_UNSUPPORTED);
    const Launch launch(dev, a[9]);
    if (!out) out = empty({R, N}, out_type, dev);
    e.bias = ptr(bias);
    e.bias_dtype = bias && bias->scalar_type() != at::kFloat ? code : MOE_FP32;
    e.residual = ptr(residual);
    e.residual_stride = residual ? residual->stride(0) : 0;
    const moe_status s = moe_linear(R, (int32_t)K, (int32_t)N, (int32_t)G, code, A.data_ptr(), A.stride(0),
                                    static_cast<const int32_t*>(ptr(offsets)), w.data_ptr(),
                                    nk ? MOE_WEIGHT_NK : MOE_WEIGHT_KN, &e, f32 ? MOE_FP32 : code, out->data_ptr(),
                                    out->stride(0), ws.data_ptr(), (size_t)ws.numel(), launch.stream);
    if (s != MOE_OK) return failed(s);
    return wrap(out);
}

// combine_rows(y, inv_pos, topk_w, residual, out_dtype's code, out, stream)
PyObject* combine_rows(PyObject* const* a)
{
    const Tensor &y = tensor_of(a[0], "y"), &inv = tensor_of(a[1], "inv_pos"), &w = tensor_of(a[2], "topk_w");
    const std::optional<Tensor> residual = optional_of(a[3], "residual");
    std::optional<Tensor> out = optional_of(a[5], "out");
    const int32_t out_code = small_integer(a[4], "out_dtype");
    const int64_t R = dim(y, "y", 0, 2), H = y.size(1), T = dim(w, "topk_w", 0, 2), k = w.size(1);
    const moe_dtype code = code_of("y", y), oc = out_code < 0 ? code : (moe_dtype)out_code;
    const at::ScalarType type = y.scalar_type();
    const at::ScalarType out_type = oc == MOE_BF16 ? at::kBFloat16 : oc == MOE_FP16 ? at::kHalf : at::kFloat;
    const at::Device dev = y.device();
    expect_rows("y", y, type, R, H, dev);
    expect("topk_w", w, at::kFloat, {T, k}, dev);
    if (inv.scalar_type() != at::kInt || inv.numel() != T * k || inv.device() != dev || !inv.is_contiguous())
        refuse("inv_pos", inv, described("T * k values in a contiguous", at::kInt, {T, k}, dev));
    if (residual) expect_rows("residual", *residual, out_type, T, H, dev);
    if (out) expect_rows("out", *out, out_type, T, H, dev);
    if (H > INT32_MAX || k > INT32_MAX) return failed(MOE_ERR_UNSUPPORTED);
    const Launch launch(dev, a[6]);
    if (!out) out = empty({T, H}, out_type, dev);
    const moe_status s = moe_combine_rows(T, (int32_t)H, (int32_t)k, R, code, y.data_ptr(), y.stride(0),
                                          static_cast<const int32_t*>(inv.data_ptr()), f32(w), oc, ptr(residual),
                                          residual ? residual->stride(0) : 0, out->data_ptr(), out->stride(0),
                                          launch.stream);
    if (s != MOE_OK) return failed(s);
    return wrap(out);
}

// A method of N positional arguments: C++ exceptions become Python's.
template <int N, PyObject* (*F)(PyObject* const*)>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        return F(args);
    } catch (const BadArgument& e) {
        PyErr_Clear();
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS   // PyTorch's own (out of memory among them) and the standard ones
}

#define FAST(n, f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<n, f>)), METH_FASTCALL, nullptr

PyMethodDef methods[] = {{"add_rmsnorm_fp8", FAST(7, add_rmsnorm_fp8)},
                         {"fp8_matmul", FAST(9, fp8_matmul)},
                         {"fp8_gated", FAST(9, fp8_gated)},
                         {"route_logits", FAST(12, route_logits)},
                         {"linear", FAST(10, linear)},
                         {"combine_rows", FAST(7, combine_rows)},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
