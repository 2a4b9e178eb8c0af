// The calls of the linear layers and norms from Python: checks of the tensors,
// new outputs and the C ABI call in one step.  A one-row norm runs in 4 us on the
// device; marshalled in Python it took 15 us of host time, here under 7.
//
// The C ABI's addresses come from the binding (which chooses the library), as do
// the exceptions that a status other than ok and a lack of memory raise.  Wrong types, shapes
// and layouts raise AssertionError, tensors off the current device ValueError.
#include <Python.h>

#include <string>
#include <tuple>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp4attn.h"

namespace {

struct Refused {
    PyObject* type;
    std::string what;
};

struct Library {
    decltype(&fp4attn_quantize_rows) quantize_rows;
    decltype(&fp4attn_dequant_rows) dequant_rows;
    decltype(&fp4attn_gemm) gemm;
    decltype(&fp4attn_linear) linear;
    decltype(&fp4attn_linear_backward) linear_backward;
    decltype(&fp4attn_norm_gate) norm_gate;
    decltype(&fp4attn_norm_gate_backward) norm_gate_backward;
} lib;
PyObject* error_class = nullptr;
PyObject* out_of_memory_class = nullptr;  // torch's, which an output without room raises

void require(bool ok, const std::string& what) {
    if (!ok) throw Refused{PyExc_AssertionError, what};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    require(THPVariable_Check(o), std::string(what) + " is a tensor");
    return THPVariable_Unpack(o);
}
bool absent(PyObject* o) { return o == Py_None; }
struct Failed {};  // a Python exception is set
bool flag(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Failed{};
    return v == 1;
}

// The current device, which every tensor of a call has to be on: the library
// launches there, one elsewhere would be reached by address only.
struct Device {
    int index = c10::cuda::current_device();
    void check(const at::Tensor& t) const {
        if (!t.is_cuda() || t.get_device() != index)
            throw Refused{PyExc_ValueError, "tensor on " + t.device().str() + ": the library runs on the current CUDA device"};
    }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream(); }
};
// Made from the first tensor, so that one on the CPU is refused before CUDA is asked for anything.
Device current_device_of(const at::Tensor& t) {
    if (!t.is_cuda())
        throw Refused{PyExc_ValueError, "tensor on " + t.device().str() + ": the library runs on the current CUDA device"};
    Device d;
    d.check(t);
    return d;
}

struct Rows {
    void* p = nullptr;
    int64_t ld = 0;
};
Rows rows_of(const at::Tensor& t, const Device& d, const char* what, at::ScalarType type, int64_t rows, int64_t cols) {
    if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        throw Refused{PyExc_AssertionError, std::string(what) + " is " + at::toString(type) + " [" + std::to_string(rows) + ", " +
                                                std::to_string(cols) + "]"};
    d.check(t);
    require(cols <= 1 || t.stride(1) == 1, std::string(what) + ": rows must be contiguous");
    return {t.data_ptr(), t.stride(0)};
}
Rows rows_of(PyObject* o, const Device& d, const char* what, at::ScalarType type, int64_t rows, int64_t cols) {
    return absent(o) ? Rows{nullptr, cols} : rows_of(tensor(o, what), d, what, type, rows, cols);
}

struct PackedRows {
    int64_t rows, K;
    uint8_t *codes, *scales;
};
int64_t scale_bytes(int64_t rows, int64_t K) { return (rows + 127) / 128 * ((K + 63) / 64) * 512; }
PackedRows packed_of(const at::Tensor& c, const at::Tensor& s, const Device& d, const char* what) {
    require(c.scalar_type() == at::kByte && c.dim() == 2 && c.is_contiguous(), std::string(what) + ": codes are uint8 [rows, K/2]");
    const int64_t rows = c.size(0), K = 2 * c.size(1);
    require(s.scalar_type() == at::kByte && s.is_contiguous() && s.numel() == scale_bytes(rows, K),
            std::string(what) + ": scale tiles of [" + std::to_string(rows) + ", " + std::to_string(K) + "]");
    d.check(c);
    d.check(s);
    return {rows, K, static_cast<uint8_t*>(c.data_ptr()), static_cast<uint8_t*>(s.data_ptr())};
}
float* gscale_of(PyObject* o, const Device& d) {
    if (absent(o)) return nullptr;
    const at::Tensor& t = tensor(o, "a scale");
    require(t.scalar_type() == at::kFloat && t.numel() == 1, "a scale is one fp32 on the device");
    d.check(t);
    return static_cast<float*>(t.data_ptr());
}
const void* vector_of(PyObject* o, int64_t n, const Device& d, const char* what) {
    if (absent(o)) return nullptr;
    const at::Tensor& t = tensor(o, what);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
        throw Refused{PyExc_AssertionError, std::string(what) + " is bf16 [" + std::to_string(n) + "]"};
    d.check(t);
    return t.data_ptr();
}
struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
};
Workspace workspace_of(PyObject* o, const Device& d) {
    if (absent(o)) return {};
    const at::Tensor& t = tensor(o, "a workspace");
    require(t.scalar_type() == at::kByte && t.is_contiguous(), "a workspace is contiguous uint8");
    d.check(t);
    return {t.data_ptr(), (size_t)t.numel()};
}
int type_of(const at::Tensor& t) {
    const at::ScalarType s = t.scalar_type();
    require(s == at::kBFloat16 || s == at::kFloat, "rows are bf16 or fp32");
    return s == at::kFloat ? FP4ATTN_F32 : FP4ATTN_BF16;
}

// per-sample vectors [groups, C] or [C] of one sample
struct Vectors {
    fp4attn_norm_vectors v{};
    int64_t groups = -1;
    void sample(PyObject* o, int64_t C, const Device& d, const void*& p, int64_t& ld) {
        if (absent(o)) return;
        const at::Tensor& t = tensor(o, "gate, scale and shift");
        const int64_t n = t.dim();
        if (t.scalar_type() != at::kBFloat16 || n < 1 || n > 2 || t.size(n - 1) != C || (C > 1 && t.stride(n - 1) != 1))
            throw Refused{PyExc_AssertionError, "gate, scale and shift are bf16 [groups, " + std::to_string(C) + "]"};
        const int64_t g = n == 2 ? t.size(0) : 1;
        if (groups < 0) groups = g;
        require(groups == g, "gate, scale and shift share the number of samples");
        d.check(t);
        p = t.data_ptr();
        ld = n == 2 ? t.stride(0) : C;
    }
    int64_t count() const { return groups < 0 ? 1 : groups; }
};
Vectors vectors_of(PyObject* post, PyObject* gate, PyObject* pre, PyObject* scale, PyObject* shift, PyObject* groups, int64_t C,
                   const Device& d) {
    Vectors v;
    if (!absent(groups)) {
        v.groups = PyLong_AsLongLong(groups);
        require(!PyErr_Occurred() && v.groups >= 0, "groups is a number of samples");
    }
    v.v.post_weight = vector_of(post, C, d, "post_weight");
    v.v.pre_weight = vector_of(pre, C, d, "pre_weight");
    v.sample(gate, C, d, v.v.gate, v.v.gate_stride);
    v.sample(scale, C, d, v.v.scale, v.v.scale_stride);
    v.sample(shift, C, d, v.v.shift, v.v.shift_stride);
    return v;
}

void check(int status, const char* where) {
    if (status == FP4ATTN_OK) return;
    PyObject* e = PyObject_CallFunction(error_class, "is", status, where);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    throw Failed{};
}

PyObject* none() { Py_RETURN_NONE; }
PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : none(); }
template <typename... T>
PyObject* tuple_of(const T&... t) {
    PyObject* out = PyTuple_New(sizeof...(T));
    if (!out) throw Failed{};
    Py_ssize_t i = 0;
    for (PyObject* o : {wrap(t)...}) PyTuple_SET_ITEM(out, i++, o);
    return out;
}
at::Tensor made(const at::Tensor& like, at::IntArrayRef size, at::ScalarType type) {
    return at::empty(size, like.options().dtype(type));
}
// A caller's output, or a new one.
at::Tensor given_or_made(PyObject* o, const char* what, const at::Tensor& like, at::IntArrayRef size, at::ScalarType type) {
    return absent(o) ? made(like, size, type) : tensor(o, what);
}

PyObject* quantize_rows(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const Device d = current_device_of(x);
    const int type = type_of(x);
    require(x.dim() == 2, "x is [rows, K]");
    const int64_t rows = x.size(0), K = x.size(1);
    const Rows xr = rows_of(x, d, "x", x.scalar_type(), rows, K);
    const bool dynamic = flag(a[2]);
    const at::Tensor codes = given_or_made(a[3], "codes", x, {rows, K / 2}, at::kByte);
    const at::Tensor scales = given_or_made(a[4], "scales", x, {scale_bytes(rows, K)}, at::kByte);
    PackedRows out{rows, K, static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr())};
    if (K % 2 == 0) {  // an odd K is the library's to refuse
        out = packed_of(codes, scales, d, "output");
        require(out.rows == rows && out.K == K, "output: packed rows of x's size");
    }
    at::Tensor g;
    if (!absent(a[1]))
        g = tensor(a[1], "a scale");
    else if (dynamic)
        g = made(x, {1}, at::kFloat);
    float* gp = absent(a[1]) ? (dynamic ? static_cast<float*>(g.data_ptr()) : nullptr) : gscale_of(a[1], d);
    const Workspace ws = workspace_of(a[5], d);
    check(lib.quantize_rows(xr.p, type, xr.ld, rows, K, gp, dynamic ? FP4ATTN_DYNAMIC_GSCALE : 0u, out.codes, out.scales, ws.p,
                            ws.bytes, d.stream()),
          "fp4attn_quantize_rows");
    return tuple_of(codes, scales, g);
}

PyObject* dequant_rows(PyObject* const* a) {
    const at::Tensor& codes = tensor(a[0], "codes");
    const Device d = current_device_of(codes);
    const PackedRows r = packed_of(codes, tensor(a[1], "scales"), d, "rows");
    const at::Tensor out = made(codes, {r.rows, r.K}, flag(a[3]) ? at::kFloat : at::kBFloat16);
    check(lib.dequant_rows(r.codes, r.scales, gscale_of(a[2], d), r.rows, r.K, out.data_ptr(), type_of(out), d.stream()),
          "fp4attn_dequant_rows");
    return wrap(out);
}

PyObject* gemm(PyObject* const* a) {
    const at::Tensor& xc = tensor(a[0], "x");
    const Device d = current_device_of(xc);
    const PackedRows x = packed_of(xc, tensor(a[1], "x"), d, "x"), w = packed_of(tensor(a[2], "w"), tensor(a[3], "w"), d, "w");
    require(x.K == w.K, "x and w share K");
    const at::Tensor y = given_or_made(a[7], "y", xc, {x.rows, w.rows}, at::kBFloat16);
    const Rows yr = rows_of(y, d, "y", at::kBFloat16, x.rows, w.rows);
    const Workspace ws = workspace_of(a[8], d);
    check(lib.gemm(x.codes, x.scales, gscale_of(a[4], d), w.codes, w.scales, gscale_of(a[5], d),
                   vector_of(a[6], w.rows, d, "bias"), x.rows, w.rows, x.K, yr.p, yr.ld, ws.p, ws.bytes, d.stream()),
          "fp4attn_gemm");
    return wrap(y);
}

PyObject* linear(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const Device d = current_device_of(x);
    const PackedRows w = packed_of(tensor(a[1], "w"), tensor(a[2], "w"), d, "w");
    const int64_t M = x.dim() ? x.size(0) : 0;
    const Rows xr = rows_of(x, d, "x", at::kBFloat16, M, w.K);
    const at::Tensor y = given_or_made(a[7], "y", x, {M, w.rows}, at::kBFloat16);
    const Rows yr = rows_of(y, d, "y", at::kBFloat16, M, w.rows);
    const Workspace ws = workspace_of(a[8], d);
    check(lib.linear(xr.p, xr.ld, gscale_of(a[4], d), flag(a[5]) ? FP4ATTN_DYNAMIC_GSCALE : 0u, w.codes, w.scales,
                     gscale_of(a[3], d), vector_of(a[6], w.rows, d, "bias"), M, w.rows, w.K, yr.p, yr.ld, ws.p, ws.bytes,
                     d.stream()),
          "fp4attn_linear");
    return wrap(y);
}

PyObject* linear_backward(PyObject* const* a) {
    const at::Tensor& dy = tensor(a[0], "dy");
    const Device d = current_device_of(dy);
    const PackedRows x = packed_of(tensor(a[1], "x"), tensor(a[2], "x"), d, "x"),
                     w = packed_of(tensor(a[3], "w"), tensor(a[4], "w"), d, "w");
    require(x.K == w.K, "x and w share K");
    const Rows r = rows_of(dy, d, "dy", at::kBFloat16, x.rows, w.rows);
    at::Tensor dx, dw, db;
    if (flag(a[7])) dx = made(dy, {x.rows, x.K}, at::kBFloat16);
    if (flag(a[8])) dw = made(dy, {w.rows, x.K}, at::kBFloat16);
    if (flag(a[9])) db = made(dy, {w.rows}, at::kFloat);
    auto at_or_null = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    const Workspace ws = workspace_of(a[10], d);
    check(lib.linear_backward(r.p, r.ld, x.codes, x.scales, gscale_of(a[5], d), w.codes, w.scales, gscale_of(a[6], d), x.rows,
                              w.rows, x.K, at_or_null(dx), x.K, at_or_null(dw), static_cast<float*>(at_or_null(db)), ws.p,
                              ws.bytes, d.stream()),
          "fp4attn_linear_backward");
    return tuple_of(dx, dw, db);
}

PyObject* norm_gate(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const Device d = current_device_of(x);
    const int type = type_of(x);
    require(x.dim() == 2, "x is [rows, C]");
    const int64_t rows = x.size(0), C = x.size(1);
    const Rows xr = rows_of(x, d, "x", x.scalar_type(), rows, C), hr = rows_of(a[1], d, "h", at::kBFloat16, rows, C);
    const Vectors v = vectors_of(a[2], a[3], a[4], a[5], a[6], a[9], C, d);
    const double eps = PyFloat_AsDouble(a[7]);
    const unsigned long flags = PyLong_AsUnsignedLongMask(a[8]);
    require(!PyErr_Occurred(), "eps is a number, flags a bit mask");
    at::Tensor y, z, codes, scales;
    if (!absent(a[14]))
        y = tensor(a[14], "y");
    else if (flag(a[10]))
        y = made(x, {rows, C}, x.scalar_type());
    Rows yr{nullptr, C};
    if (y.defined()) yr = rows_of(y, d, "y", x.scalar_type(), rows, C);
    const bool quantize = flag(a[12]);
    const float* gz = nullptr;
    if (quantize) {
        codes = made(x, {rows, C / 2}, at::kByte);
        scales = made(x, {scale_bytes(rows, C)}, at::kByte);
        gz = gscale_of(a[13], d);
        require(absent(a[15]), "z is either bf16 rows or NVFP4 rows");
    } else if (!absent(a[15])) {
        z = tensor(a[15], "z");
    } else if (flag(a[11])) {
        z = made(x, {rows, C}, at::kBFloat16);
    }
    Rows zr{nullptr, C};
    if (z.defined()) zr = rows_of(z, d, "z", at::kBFloat16, rows, C);
    const Workspace ws = workspace_of(a[16], d);
    check(lib.norm_gate(xr.p, type, xr.ld, hr.p, hr.ld, &v.v, rows, C, v.count(), (float)eps, (uint32_t)flags, yr.p, yr.ld,
                        zr.p, zr.ld, quantize ? static_cast<uint8_t*>(codes.data_ptr()) : nullptr,
                        quantize ? static_cast<uint8_t*>(scales.data_ptr()) : nullptr, gz, ws.p, ws.bytes, d.stream()),
          "fp4attn_norm_gate");
    return quantize ? tuple_of(y, codes, scales) : tuple_of(y, z);
}

PyObject* norm_gate_backward(PyObject* const* a) {
    const at::Tensor& y = tensor(a[2], "y");
    const Device d = current_device_of(y);
    const int type = type_of(y);
    require(y.dim() == 2, "y is [rows, C]");
    const int64_t rows = y.size(0), C = y.size(1);
    const Rows yr = rows_of(y, d, "y", y.scalar_type(), rows, C),
               dzr = rows_of(tensor(a[0], "dz"), d, "dz", at::kBFloat16, rows, C),
               dyr = rows_of(a[1], d, "dy", y.scalar_type(), rows, C), hr = rows_of(a[3], d, "h", at::kBFloat16, rows, C);
    const Vectors v = vectors_of(a[4], a[5], a[6], a[7], Py_None, a[10], C, d);
    const double eps = PyFloat_AsDouble(a[8]);
    const unsigned long flags = PyLong_AsUnsignedLongMask(a[9]);
    require(!PyErr_Occurred(), "eps is a number, flags a bit mask");
    const int64_t G = v.count();
    const bool branch = hr.p != nullptr || !absent(a[3]);
    const at::Tensor dx = made(y, {rows, C}, y.scalar_type()), dshift = made(y, {G, C}, at::kFloat),
                     dscale = made(y, {G, C}, at::kFloat), dpre = made(y, {C}, at::kFloat);
    at::Tensor dh, dgate, dpost;
    if (branch) {
        dh = made(y, {rows, C}, at::kBFloat16);
        dgate = made(y, {G, C}, at::kFloat);
        dpost = made(y, {C}, at::kFloat);
    }
    auto at_or_null = [](const at::Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; };
    const Workspace ws = workspace_of(a[11], d);
    check(lib.norm_gate_backward(dzr.p, dzr.ld, dyr.p, dyr.ld, yr.p, yr.ld, type, hr.p, hr.ld, &v.v, rows, C, G, (float)eps,
                                 (uint32_t)flags, dx.data_ptr(), C, branch ? dh.data_ptr() : nullptr, C, at_or_null(dshift),
                                 at_or_null(dscale), at_or_null(dgate), at_or_null(dpre), at_or_null(dpost), ws.p, ws.bytes,
                                 d.stream()),
          "fp4attn_norm_gate_backward");
    return tuple_of(dx, dh, dshift, dscale, dgate, dpre, dpost);
}

// No C++ exception leaves for Python as one.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& e) {
        PyErr_Clear();
        PyErr_SetString(e.type, e.what.c_str());
    } catch (const Failed&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(out_of_memory_class, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown exception");
    }
    return nullptr;
}

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "two exception classes and seven addresses expected");
        return nullptr;
    }
    void* p[7];
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(args[2 + i]);
        if (PyErr_Occurred()) return nullptr;
    }
    lib = {reinterpret_cast<decltype(lib.quantize_rows)>(p[0]),   reinterpret_cast<decltype(lib.dequant_rows)>(p[1]),
           reinterpret_cast<decltype(lib.gemm)>(p[2]),            reinterpret_cast<decltype(lib.linear)>(p[3]),
           reinterpret_cast<decltype(lib.linear_backward)>(p[4]), reinterpret_cast<decltype(lib.norm_gate)>(p[5]),
           reinterpret_cast<decltype(lib.norm_gate_backward)>(p[6])};
    Py_INCREF(args[0]);
    Py_INCREF(args[1]);
    Py_XDECREF(error_class);
    Py_XDECREF(out_of_memory_class);
    error_class = args[0];
    out_of_memory_class = args[1];
    Py_RETURN_NONE;
}

#define FP4ATTN_METHOD(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    FP4ATTN_METHOD(quantize_rows, 6),
    FP4ATTN_METHOD(dequant_rows, 4),
    FP4ATTN_METHOD(gemm, 9),
    FP4ATTN_METHOD(linear, 9),
    FP4ATTN_METHOD(linear_backward, 11),
    FP4ATTN_METHOD(norm_gate, 17),
    FP4ATTN_METHOD(norm_gate_backward, 12),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module_def); }
