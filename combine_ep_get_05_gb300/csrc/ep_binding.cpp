// ep_binding.cpp -- Python binding of the norm, the E4M3 sort and the gradients
// (module _ep_binding; combine_ep_get_05_gb300/_lib.py wraps it).
//
// These calls are a few microseconds of GPU work where a batch is small, and checking ten
// tensors from Python took longer than that (norm of one token: 7.2 us of host time a call,
// 3 us of them in the library and its launch). Here the arguments are read from the tensors
// themselves. Every argument is checked as in _lib.py's _check, with the same messages
// (ValueError); a status other than EP_OK is returned to the caller, which raises EpError.
// The library's entry points come in by address (bind), so that it is loaded in one place.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <limits>
#include <string>

#include "ep.h"

namespace {

struct Refused {};  // a Python exception has been set

[[noreturn]] void refuse(const char* format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(PyExc_ValueError, format, args);
    va_end(args);
    throw Refused();
}

std::string dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kByte: return "torch.uint8";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        default: return c10::toString(t);
    }
}

using Shape = std::initializer_list<int64_t>;

std::string shape_name(c10::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

// the tensor behind an argument, or nullptr for None
const at::Tensor* tensor_of(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse("%s must be a torch.Tensor, got %s", name, Py_TYPE(o)->tp_name);
    return &THPVariable_Unpack(o);
}

const at::Tensor& required(PyObject* o, const char* name) {
    const at::Tensor* t = tensor_of(o, name);
    if (t == nullptr) refuse("%s is required", name);
    return *t;
}

// the sizes of a tensor that sets the call's dimensions
int32_t dim(const at::Tensor& t, const char* name, int64_t dims, int64_t i) {
    if (t.dim() != dims)
        refuse("%s must have %d dimensions, got %d", name, static_cast<int>(dims), static_cast<int>(t.dim()));
    const int64_t n = t.size(i);
    if (n > std::numeric_limits<int32_t>::max()) refuse("%s is too large", name);
    return static_cast<int32_t>(n);
}

int32_t integer(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
        refuse("%s is too large", name);
    return static_cast<int32_t>(v);
}

// the device that the call of this thread launches on, asked for once a call
thread_local int t_device = -1;

void check(const at::Tensor& t, const char* name, at::ScalarType dtype, Shape shape) {
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (t_device < 0) t_device = c10::cuda::current_device();
    if (t.get_device() != t_device)
        refuse("%s must be on the current device, cuda:%d, got cuda:%d", name, t_device,
               static_cast<int>(t.get_device()));
    if (t.scalar_type() != dtype)
        refuse("%s must be %s, got %s", name, dtype_name(dtype).c_str(), dtype_name(t.scalar_type()).c_str());
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    const c10::IntArrayRef want(shape.begin(), shape.size());
    if (t.sizes() != want)
        refuse("%s must have shape %s, got %s", name, shape_name(want).c_str(), shape_name(t.sizes()).c_str());
}

// The address of a tensor that the call reads, or writes: asking to write copies the
// memory of a lazily cloned tensor, asking to read does not.
const void* reads(const at::Tensor& t, const char* name, at::ScalarType dtype, Shape shape) {
    check(t, name, dtype, shape);
    return t.const_data_ptr();
}

const void* reads(PyObject* o, const char* name, at::ScalarType dtype, Shape shape) {
    return reads(required(o, name), name, dtype, shape);
}

const void* reads_or_null(PyObject* o, const char* name, at::ScalarType dtype, Shape shape) {
    const at::Tensor* t = tensor_of(o, name);
    return t == nullptr ? nullptr : reads(*t, name, dtype, shape);
}

void* writes(const at::Tensor& t, const char* name, at::ScalarType dtype, Shape shape) {
    check(t, name, dtype, shape);
    return t.mutable_data_ptr();
}

void* writes(PyObject* o, const char* name, at::ScalarType dtype, Shape shape) {
    return writes(required(o, name), name, dtype, shape);
}

void* writes_or_null(PyObject* o, const char* name, at::ScalarType dtype, Shape shape) {
    const at::Tensor* t = tensor_of(o, name);
    return t == nullptr ? nullptr : writes(*t, name, dtype, shape);
}

// the type of E4M3 codes: bytes, or torch's own
at::ScalarType code_type(PyObject* o, const char* name) {
    return required(o, name).scalar_type() == at::kFloat8_e4m3fn ? at::kFloat8_e4m3fn : at::kByte;
}

void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
    if (handle == nullptr) throw Refused();
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (p == nullptr && PyErr_Occurred()) throw Refused();
    return p;
}

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return static_cast<float>(v);
}

template <typename T>
T* as(void* p) {
    return static_cast<T*>(p);
}

template <typename T>
const T* as(const void* p) {
    return static_cast<const T*>(p);
}

// the library's entry points
struct {
    decltype(&ep_rmsnorm) rmsnorm;
    decltype(&ep_rmsnorm_bwd) rmsnorm_bwd;
    decltype(&ep_dispatch_permuted_fp8) dispatch_permuted_fp8;
    decltype(&ep_dispatch_permuted_fp8_ll) dispatch_permuted_fp8_ll;
    decltype(&ep_dispatch_permuted_bwd) dispatch_permuted_bwd;
    decltype(&ep_combine_permuted_bwd) combine_permuted_bwd;
} g_ep;

template <typename F>
void take(F*& to, PyObject* addresses, const char* name) {
    PyObject* v = PyDict_GetItemString(addresses, name);  // borrowed
    if (v == nullptr) refuse("no address for %s", name);
    to = reinterpret_cast<F*>(PyLong_AsVoidPtr(v));
    if (to == nullptr) refuse("no address for %s", name);
}

ep_status_t bind(PyObject* const* a) {
    take(g_ep.rmsnorm, a[0], "ep_rmsnorm");
    take(g_ep.rmsnorm_bwd, a[0], "ep_rmsnorm_bwd");
    take(g_ep.dispatch_permuted_fp8, a[0], "ep_dispatch_permuted_fp8");
    take(g_ep.dispatch_permuted_fp8_ll, a[0], "ep_dispatch_permuted_fp8_ll");
    take(g_ep.dispatch_permuted_bwd, a[0], "ep_dispatch_permuted_bwd");
    take(g_ep.combine_permuted_bwd, a[0], "ep_combine_permuted_bwd");
    return EP_OK;
}

// The library's call itself, with other Python threads let through: a launch waits while the
// stream's queue is full. Its arguments are C values by then; `launch` touches no Python object.
template <typename Launch>
ep_status_t launched(Launch launch) {
    PyThreadState* const state = PyEval_SaveThread();
    const ep_status_t status = launch();
    PyEval_RestoreThread(state);
    return status;
}

// the residual stream's type, that of `t`; bf16 where there is no stream
at::ScalarType stream_type(const at::Tensor* t) {
    const at::ScalarType type = t == nullptr ? at::kBFloat16 : t->scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat)
        refuse("the residual stream must be bfloat16 or float32, got %s", dtype_name(type).c_str());
    return type;
}

ep_dtype_t ep_type(at::ScalarType t) { return t == at::kFloat ? EP_DTYPE_F32 : EP_DTYPE_BF16; }

// x, residual, weight, eps, residual_out, y, y_q, y_scales, stream
ep_status_t rmsnorm(PyObject* const* a) {
    const at::Tensor *x = tensor_of(a[0], "x"), *residual = tensor_of(a[1], "residual");
    if (x == nullptr && residual == nullptr) refuse("x or residual is required");
    const at::Tensor& in = x != nullptr ? *x : *residual;
    const char* const name = x != nullptr ? "x" : "residual";
    const int32_t T = dim(in, name, 2, 0), H = dim(in, name, 2, 1);
    const at::Tensor* out = tensor_of(a[4], "residual_out");
    const at::ScalarType type = stream_type(residual != nullptr ? residual : out);
    if (out != nullptr && out->scalar_type() != type)
        refuse("the residual stream must be of one type, got %s and %s", dtype_name(type).c_str(),
               dtype_name(out->scalar_type()).c_str());
    const void* const px = reads_or_null(a[0], "x", at::kBFloat16, {T, H});
    const void* const pr = reads_or_null(a[1], "residual", type, {T, H});
    const at::Tensor& w = required(a[2], "weight");
    const at::ScalarType wtype = w.scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
    const void* const pw = reads(w, "weight", wtype, {H});
    void* const po = writes_or_null(a[4], "residual_out", type, {T, H});
    void* const py = writes_or_null(a[5], "y", at::kBFloat16, {T, H});
    void *pq = nullptr, *ps = nullptr;
    if (a[6] != Py_None) {
        pq = writes(a[6], "y_q", code_type(a[6], "y_q"), {T, H});
        ps = writes(a[7], "y_scales", at::kFloat, {T, H / 128});
    } else {
        ps = writes_or_null(a[7], "y_scales", at::kFloat, {T, H / 128});
    }
    const float eps = number(a[3]);
    void* const stream = stream_of(a[8]);
    return launched([&] {
        return g_ep.rmsnorm(px, pr, pw, ep_type(type), ep_type(wtype), eps, T, H, po, py, as<uint8_t>(pq),
                            as<float>(ps), stream);
    });
}

// dy, z, weight, dz_in, eps, dz, dx, dweight, workspace, stream
ep_status_t rmsnorm_bwd(PyObject* const* a) {
    const at::Tensor& z = required(a[1], "z");
    const int32_t T = dim(z, "z", 2, 0), H = dim(z, "z", 2, 1);
    const at::ScalarType type = stream_type(&z);
    const void* const pdy = reads(a[0], "dy", at::kBFloat16, {T, H});
    const void* const pz = reads(z, "z", type, {T, H});
    const at::Tensor& w = required(a[2], "weight");
    const at::ScalarType wtype = w.scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
    const void* const pw = reads(w, "weight", wtype, {H});
    const void* const pin = reads_or_null(a[3], "dz_in", type, {T, H});
    void* const pdz = writes(a[5], "dz", type, {T, H});
    void* const pdx = writes_or_null(a[6], "dx", at::kBFloat16, {T, H});
    void* const pdw = writes_or_null(a[7], "dweight", at::kFloat, {H});
    const at::Tensor* ws = pdw != nullptr ? &required(a[8], "workspace") : tensor_of(a[8], "workspace");
    const int64_t bytes = ws == nullptr ? 0 : ws->numel();
    void* const pws = ws == nullptr ? nullptr : writes(*ws, "workspace", at::kByte, {bytes});
    const float eps = number(a[4]);
    void* const stream = stream_of(a[9]);
    return launched([&] {
        return g_ep.rmsnorm_bwd(pdy, pz, pw, pin, ep_type(type), ep_type(wtype), eps, T, H, pdz, pdx, as<float>(pdw),
                                pws, static_cast<size_t>(bytes), stream);
    });
}

// x_q, x_scales, topk_idx, topk_w, expert_offsets, expert_slot, num_experts, num_ranks, max_rows,
// perm_q, perm_scales, perm_src, perm_w, status, stream; the one-launch form writes the layout
ep_status_t sort_fp8(PyObject* const* a, bool one_launch) {
    const at::Tensor& q = required(a[0], "x_q");
    const int32_t T = dim(q, "x_q", 2, 0), H = dim(q, "x_q", 2, 1);
    const int32_t k = dim(required(a[2], "topk_idx"), "topk_idx", 2, 1);
    const int32_t E = integer(a[6], "num_experts"), R = integer(a[7], "num_ranks"), M = integer(a[8], "max_rows");
    auto* const pq = as<uint8_t>(reads(a[0], "x_q", code_type(a[0], "x_q"), {T, H}));
    auto* const ps = as<float>(reads(a[1], "x_scales", at::kFloat, {T, H / 128}));
    auto* const idx = as<int64_t>(reads(a[2], "topk_idx", at::kLong, {T, k}));
    auto* const w = as<float>(reads_or_null(a[3], "topk_w", at::kFloat, {T, k}));
    // the layout: written by the one-launch form, read by the other
    const int32_t *off = nullptr, *slot = nullptr;
    int32_t *off_out = nullptr, *slot_out = nullptr;
    if (one_launch) {
        off_out = as<int32_t>(writes(a[4], "expert_offsets", at::kInt, {static_cast<int64_t>(E) + 1}));
        slot_out = as<int32_t>(writes(a[5], "expert_slot", at::kInt, {T, k}));
    } else {
        off = as<int32_t>(reads(a[4], "expert_offsets", at::kInt, {static_cast<int64_t>(E) + 1}));
        slot = as<int32_t>(reads(a[5], "expert_slot", at::kInt, {T, k}));
    }
    auto* const oq = as<uint8_t>(writes(a[9], "perm_q", code_type(a[9], "perm_q"), {R, M, H}));
    auto* const os = as<float>(writes(a[10], "perm_scales", at::kFloat, {R, M, H / 128}));
    auto* const src = as<int32_t>(writes_or_null(a[11], "perm_src", at::kInt, {R, M}));
    auto* const pw = as<float>(writes_or_null(a[12], "perm_w", at::kFloat, {R, M}));
    auto* const status = as<int32_t>(writes_or_null(a[13], "status", at::kInt, {1}));
    void* const stream = stream_of(a[14]);
    return launched([&] {
        if (one_launch)
            return g_ep.dispatch_permuted_fp8_ll(pq, ps, idx, w, T, H, k, E, R, M, off_out, slot_out, oq, os, src, pw,
                                                 status, stream);
        return g_ep.dispatch_permuted_fp8(pq, ps, idx, w, off, slot, T, H, k, E, R, M, oq, os, src, pw, status,
                                          stream);
    });
}

ep_status_t dispatch_permuted_fp8(PyObject* const* a) { return sort_fp8(a, false); }
ep_status_t dispatch_permuted_fp8_ll(PyObject* const* a) { return sort_fp8(a, true); }

// dperm_x, dperm_w, dx_in, topk_idx, expert_offsets, expert_slot, num_experts, dx, dtopk_w, status, stream
ep_status_t dispatch_permuted_bwd(PyObject* const* a) {
    const at::Tensor &d = required(a[0], "dperm_x"), &ids = required(a[3], "topk_idx");
    const int32_t R = dim(d, "dperm_x", 3, 0), M = dim(d, "dperm_x", 3, 1), H = dim(d, "dperm_x", 3, 2);
    const int32_t T = dim(ids, "topk_idx", 2, 0), k = dim(ids, "topk_idx", 2, 1), E = integer(a[6], "num_experts");
    const void* const pd = reads(d, "dperm_x", at::kBFloat16, {R, M, H});
    auto* const pw = as<float>(a[8] != Py_None ? reads(a[1], "dperm_w", at::kFloat, {R, M})
                                               : reads_or_null(a[1], "dperm_w", at::kFloat, {R, M}));
    const void* const add = reads_or_null(a[2], "dx_in", at::kBFloat16, {T, H});
    auto* const idx = as<int64_t>(reads(ids, "topk_idx", at::kLong, {T, k}));
    auto* const off = as<int32_t>(reads(a[4], "expert_offsets", at::kInt, {static_cast<int64_t>(E) + 1}));
    auto* const slot = as<int32_t>(reads(a[5], "expert_slot", at::kInt, {T, k}));
    void* const dx = writes(a[7], "dx", at::kBFloat16, {T, H});
    auto* const dw = as<float>(writes_or_null(a[8], "dtopk_w", at::kFloat, {T, k}));
    auto* const status = as<int32_t>(writes_or_null(a[9], "status", at::kInt, {1}));
    void* const stream = stream_of(a[10]);
    return launched([&] {
        return g_ep.dispatch_permuted_bwd(pd, pw, add, idx, off, slot, T, H, k, E, R, M, dx, dw, status, stream);
    });
}

// dout, y, topk_idx, topk_w, expert_offsets, expert_slot, num_experts, dy, dtopk_w, status, stream
ep_status_t combine_permuted_bwd(PyObject* const* a) {
    const at::Tensor &d = required(a[7], "dy"), &ids = required(a[2], "topk_idx");
    const int32_t R = dim(d, "dy", 3, 0), M = dim(d, "dy", 3, 1), H = dim(d, "dy", 3, 2);
    const int32_t T = dim(ids, "topk_idx", 2, 0), k = dim(ids, "topk_idx", 2, 1), E = integer(a[6], "num_experts");
    const void* const dout = reads(a[0], "dout", at::kBFloat16, {T, H});
    const void* const y = a[8] != Py_None ? reads(a[1], "y", at::kBFloat16, {R, M, H})
                                          : reads_or_null(a[1], "y", at::kBFloat16, {R, M, H});
    auto* const idx = as<int64_t>(reads(ids, "topk_idx", at::kLong, {T, k}));
    auto* const w = as<float>(reads_or_null(a[3], "topk_w", at::kFloat, {T, k}));
    auto* const off = as<int32_t>(reads(a[4], "expert_offsets", at::kInt, {static_cast<int64_t>(E) + 1}));
    auto* const slot = as<int32_t>(reads(a[5], "expert_slot", at::kInt, {T, k}));
    void* const dy = writes(d, "dy", at::kBFloat16, {R, M, H});
    auto* const dw = as<float>(writes_or_null(a[8], "dtopk_w", at::kFloat, {T, k}));
    auto* const status = as<int32_t>(writes_or_null(a[9], "status", at::kInt, {1}));
    void* const stream = stream_of(a[10]);
    return launched([&] {
        return g_ep.combine_permuted_bwd(dout, y, idx, w, off, slot, T, H, k, E, R, M, dy, dw, status, stream);
    });
}

// A call: the number of arguments, then the function; no C++ exception leaves it.
template <ep_status_t (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", kArgs, n);
        return nullptr;
    }
    t_device = -1;
    try {
        return PyLong_FromLong(kCall(args));
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <ep_status_t (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyMethodDef method(const char* name) {
    auto* const f = reinterpret_cast<void (*)()>(call<kCall, kArgs>);
    return {name, reinterpret_cast<PyCFunction>(f), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<bind, 1>("bind"),
    method<rmsnorm, 9>("rmsnorm"),
    method<rmsnorm_bwd, 10>("rmsnorm_bwd"),
    method<dispatch_permuted_fp8, 15>("dispatch_permuted_fp8"),
    method<dispatch_permuted_fp8_ll, 15>("dispatch_permuted_fp8_ll"),
    method<dispatch_permuted_bwd, 11>("dispatch_permuted_bwd"),
    method<combine_permuted_bwd, 11>("combine_permuted_bwd"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ep_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr,
                        nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ep_binding(void) { return PyModule_Create(&g_module); }
