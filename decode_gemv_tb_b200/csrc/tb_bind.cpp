// tb_bind.cpp -- Python calls of the 4-bit and expert-layer entry points.
//
// The smallest of these calls run four or five microseconds on the GPU.
// Checked in Python and passed through ctypes they cost 8 to 11 of host time
// each, so eager decoding waited for the host; read here, a call takes 2.9 to
// 3.8 (tb_moe, two launches: 5.2), nearly all of it the launch.  The checks are
// those of the other bindings: shapes, strides and types that a raw pointer
// cannot show, and one device, the current one.  Everything else is left to
// the library's own checks, whose status becomes the same exception.
//
// Functions take their arguments by position, tensors where the C interface
// takes pointers, None for an absent optional tensor or for the current
// stream, and return None.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <stdexcept>
#include <string>

#include "tb.h"

namespace {

// the library's entry points (the caller has loaded it) and the exception to raise
decltype(&tb_mx4_quantize) f_quantize;
decltype(&tb_mx4_dequantize) f_dequantize;
decltype(&tb_mx4_gemm) f_gemm;
decltype(&tb_moe_route) f_route;
decltype(&tb_moe) f_moe;
decltype(&tb_status_string) f_status_string;
PyObject* g_error = nullptr;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

using Args = PyObject* const*;

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused("sizes and flags must be integers of 64 bits");
    }
    return v;
}
bool truth(PyObject* o, const char* name) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        throw Refused(std::string(name) + " must be true or false");
    }
    return v != 0;
}
unsigned flag_bits(PyObject* o) {
    const int64_t v = integer(o);
    if (v < 0 || v > 0xFFFFFFFFll) throw Refused("flags must fit in 32 bits");
    return (unsigned)v;
}
std::string shape(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}
// row stride of a [rows][cols] tensor whose rows are contiguous (a single row's stride reaches nothing)
int64_t rows(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        throw Refused(std::string(name) + " must be [" + std::to_string(rows) + "][" + std::to_string(cols) + "], got " +
                      shape(t));
    if (t.stride(1) != 1 && cols > 1) throw Refused(std::string(name) + "'s rows must be contiguous");
    return rows > 1 ? t.stride(0) : cols;
}
void matrix(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) throw Refused(std::string(name) + " must have two dimensions, got " + shape(t));
}
int64_t bf16_rows(const at::Tensor& t, const char* name, int64_t r, int64_t c) {
    const auto d = t.scalar_type();
    if (d != at::kBFloat16 && d != at::kShort && d != at::kUInt16)
        throw Refused(std::string(name) + " must hold bf16 bit patterns");
    return rows(t, name, r, c);
}
template <class T>
T* bytes(const at::Tensor& t, const char* name, int64_t need) {
    if (t.scalar_type() != at::kByte || t.numel() < need)
        throw Refused(std::string(name) + " must hold at least " + std::to_string(need) + " bytes as uint8");
    if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
    return static_cast<T*>(t.data_ptr());
}
template <class T>
T* pairs(const at::Tensor& t, const char* name, at::ScalarType d, int64_t T_, int64_t k) {
    if (t.scalar_type() != d || t.dim() != 2 || t.size(0) != T_ || t.size(1) != k || !t.is_contiguous())
        throw Refused(std::string(name) + " must be contiguous [" + std::to_string(T_) + "][" + std::to_string(k) + "] " +
                      c10::toString(d) + ", got " + shape(t) + " " + c10::toString(t.scalar_type()));
    return static_cast<T*>(t.data_ptr());
}
tb_dtype_t dtype(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kFloat) return TB_F32;
    if (t.scalar_type() == at::kBFloat16) return TB_BF16;
    throw Refused(std::string(name) + " must be float32 or bfloat16, got " + c10::toString(t.scalar_type()));
}
void mx4_shape(int64_t N, int64_t K) {
    if (N < 1 || K < 32 || K % 32 != 0 || N > INT_MAX || K > INT_MAX)
        throw Refused("MX4 needs N >= 1 and K a positive multiple of 32, both below 2^31, got " + std::to_string(N) + " x " +
                      std::to_string(K));
}
int64_t code_bytes(int64_t N, int64_t K) { return N * (K / 2); }
int64_t scale_bytes(int64_t N, int64_t K) { return 512 * ((N + 127) / 128) * ((K + 127) / 128); }

// the library launches on the current device: every tensor has to live there
template <class... Ts>
int same_device(const at::Tensor& first, const Ts&... rest) {
    if (!first.is_cuda()) throw Refused("tensors must be CUDA tensors");
    const int dev = first.get_device(), cur = c10::cuda::current_device();
    if (dev != cur)
        throw Refused("tensors on cuda:" + std::to_string(dev) + ", but the current device is cuda:" + std::to_string(cur));
    for (const at::Tensor* t : {&first, &rest...})
        if (!t->is_cuda() || t->get_device() != dev)
            throw Refused("tensors on different devices: cuda:" + std::to_string(dev) + " and " + t->device().str());
    return dev;
}
tb_stream_t stream(PyObject* o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused("stream must be a stream's address or None");
    }
    return p;
}
void check(tb_status_t s, const char* what) {
    if (s == TB_OK) return;
    static const char* const names[] = {"TB_OK",        "TB_ERR_ARG", "TB_ERR_SHAPE", "TB_ERR_ALIGN", "TB_ERR_UNSUPPORTED",
                                        "TB_ERR_CUDA", "TB_ERR_TIMEOUT"};
    throw Refused(std::string(what) + ": " + ((unsigned)s < 7 ? names[s] : "?") + " (" + f_status_string(s) + ")");
}

// (W, codes, scales, bad_count or None, stream)
void quantize(Args a) {
    const at::Tensor &W = tensor(a[0], "W"), &codes = tensor(a[1], "codes"), &scales = tensor(a[2], "scales");
    matrix(W, "W");
    const int64_t N = W.size(0), K = W.size(1), ldw = rows(W, "W", N, K);
    mx4_shape(N, K);
    int dev;
    int32_t* bad = nullptr;
    if (a[3] == Py_None) {
        dev = same_device(W, codes, scales);
    } else {
        const at::Tensor& b = tensor(a[3], "bad_count");
        dev = same_device(W, codes, scales, b);
        if (b.scalar_type() != at::kInt || b.numel() < 1) throw Refused("bad_count must be int32");
        bad = static_cast<int32_t*>(b.data_ptr());
    }
    check(f_quantize(W.data_ptr(), dtype(W, "weights"), ldw, N, K, bytes<void>(codes, "codes", code_bytes(N, K)),
                     bytes<uint8_t>(scales, "scales", scale_bytes(N, K)), bad, stream(a[4], dev)),
          "tb_mx4_quantize");
}

// (codes, scales, N, K, W, stream)
void dequantize(Args a) {
    const at::Tensor &codes = tensor(a[0], "codes"), &scales = tensor(a[1], "scales"), &W = tensor(a[4], "W");
    const int64_t N = integer(a[2]), K = integer(a[3]);
    mx4_shape(N, K);
    const int dev = same_device(codes, scales, W);
    const int64_t ldw = rows(W, "W", N, K);
    check(f_dequantize(bytes<void>(codes, "codes", code_bytes(N, K)), bytes<uint8_t>(scales, "scales", scale_bytes(N, K)),
                       N, K, W.data_ptr(), dtype(W, "W"), ldw, stream(a[5], dev)),
          "tb_mx4_dequantize");
}

// (w_codes, w_scales, x_codes, x_scales, M, N, K, Y, flags, stream)
void gemm(Args a) {
    const at::Tensor &wc = tensor(a[0], "w_codes"), &ws = tensor(a[1], "w_scales"), &xc = tensor(a[2], "x_codes"),
                     &xs = tensor(a[3], "x_scales"), &Y = tensor(a[7], "Y");
    const int64_t M = integer(a[4]), N = integer(a[5]), K = integer(a[6]);
    mx4_shape(N, K);
    mx4_shape(M, K);
    const int dev = same_device(wc, ws, xc, xs, Y);
    const int64_t ldy = rows(Y, "Y", M, N);
    check(f_gemm(bytes<void>(wc, "w_codes", code_bytes(N, K)), bytes<uint8_t>(ws, "w_scales", scale_bytes(N, K)),
                 bytes<void>(xc, "x_codes", code_bytes(M, K)), bytes<uint8_t>(xs, "x_scales", scale_bytes(M, K)),
                 Y.data_ptr(), dtype(Y, "Y"), ldy, M, N, K, flag_bits(a[8]), stream(a[9], dev)),
          "tb_mx4_gemm");
}

// (x, router, k, renormalize, ids, weights, stream)
void route(Args a) {
    const at::Tensor &x = tensor(a[0], "x"), &r = tensor(a[1], "router"), &ids = tensor(a[4], "ids"),
                     &w = tensor(a[5], "weights");
    matrix(x, "x");
    matrix(r, "router");
    const int64_t T = x.size(0), H = x.size(1), E = r.size(0), k = integer(a[2]), ldx = bf16_rows(x, "x", T, H);
    const bool renormalize = truth(a[3], "renormalize");
    if (bf16_rows(r, "router", E, H) != H) throw Refused("router must be contiguous");
    const int dev = same_device(x, r, ids, w);
    if (k < 1 || k > TB_MOE_MAX_TOPK) check(TB_ERR_ARG, "tb_moe_route");
    check(f_route(static_cast<const uint16_t*>(x.data_ptr()), ldx, static_cast<const uint16_t*>(r.data_ptr()), T, E, H,
                  (int)k, renormalize, pairs<int32_t>(ids, "ids", at::kInt, T, k),
                  pairs<float>(w, "weights", at::kFloat, T, k), stream(a[6], dev)),
          "tb_moe_route");
}

// (layer's address, its H, its device, x, ids, weights, y, workspace, flags, stream)
void moe(Args a) {
    const auto* layer = static_cast<const tb_moe_t*>(PyLong_AsVoidPtr(a[0]));
    const int64_t H = integer(a[1]), home = integer(a[2]);
    const at::Tensor &x = tensor(a[3], "x"), &ids = tensor(a[4], "ids"), &w = tensor(a[5], "weights"),
                     &y = tensor(a[6], "y"), &ws = tensor(a[7], "workspace");
    matrix(ids, "ids");
    const int64_t T = ids.size(0), k = ids.size(1), ldx = bf16_rows(x, "x", T, H);
    const int dev = same_device(x, ids, w, y, ws);
    if (dev != home) throw Refused("x on cuda:" + std::to_string(dev) + ", the layer on cuda:" + std::to_string(home));
    const int64_t ldy = rows(y, "y", T, H);
    if (k > TB_MOE_MAX_TOPK) check(TB_ERR_ARG, "tb_moe");
    const size_t size = (size_t)ws.numel() * ws.element_size();
    if (!ws.is_contiguous()) throw Refused("workspace must be contiguous");
    check(f_moe(layer, static_cast<const uint16_t*>(x.data_ptr()), ldx, pairs<int32_t>(ids, "ids", at::kInt, T, k),
                pairs<float>(w, "weights", at::kFloat, T, k), T, (int)k, y.data_ptr(), dtype(y, "y"), ldy,
                flag_bits(a[8]), ws.data_ptr(), size, stream(a[9], dev)),
          "tb_moe");
}

// no C++ exception leaves a call
template <void (*F)(Args), int N>
PyObject* call(PyObject*, Args args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        F(args);
    } catch (const std::exception& e) {
        PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

// (exception class, addresses of tb_mx4_quantize, tb_mx4_dequantize, tb_mx4_gemm, tb_moe_route, tb_moe,
// tb_status_string)
PyObject* init(PyObject*, Args a, Py_ssize_t n) {
    if (n != 7) {
        PyErr_Format(PyExc_TypeError, "7 arguments expected, got %zd", n);
        return nullptr;
    }
    void* p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    f_quantize = reinterpret_cast<decltype(f_quantize)>(p[0]);
    f_dequantize = reinterpret_cast<decltype(f_dequantize)>(p[1]);
    f_gemm = reinterpret_cast<decltype(f_gemm)>(p[2]);
    f_route = reinterpret_cast<decltype(f_route)>(p[3]);
    f_moe = reinterpret_cast<decltype(f_moe)>(p[4]);
    f_status_string = reinterpret_cast<decltype(f_status_string)>(p[5]);
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, Args, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<init>("init"),
                         method<call<quantize, 5>>("mx4_quantize"),
                         method<call<dequantize, 6>>("mx4_dequantize"),
                         method<call<gemm, 10>>("mx4_gemm"),
                         method<call<route, 7>>("moe_route"),
                         method<call<moe, 10>>("moe"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tb_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and Python whose headers this was compiled with (no other may run it)
PyMODINIT_FUNC PyInit__tb_bind(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", TB_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
