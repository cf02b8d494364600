// Argument marshalling of the operators whose calls take only microseconds on the GPU: a Python
// module in C++, since reading a tensor's attributes and allocating outputs from Python took longer
// than the kernels (one norm of a row: 18 us of host time from Python).  Nothing is computed here:
// every function checks its tensors, allocates outputs and calls the C ABI through the addresses
// that bind() was given.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <string>

#include "../../include/gbgemm.h"

namespace {

decltype(&gb_gemm_linear_w4) f_linear_w4;
decltype(&gb_gemm_ffn_gated_w4) f_ffn_gated_w4;
decltype(&gb_dropout) f_dropout;
decltype(&gb_add_rms_norm) f_norm;
decltype(&gb_add_rms_norm_q8) f_norm_q8;
decltype(&gb_add_rms_norm_backward) f_norm_bwd;
decltype(&gb_add_rms_norm_backward_workspace_bytes) f_norm_bwd_ws;
decltype(&gb_add_layer_norm) f_layer_norm;
decltype(&gb_add_layer_norm_backward) f_layer_norm_bwd;
decltype(&gb_add_layer_norm_backward_workspace_bytes) f_layer_norm_bwd_ws;
decltype(&gb_moe_ffn_gated) f_moe;
decltype(&gb_moe_ffn_gated_workspace_bytes) f_moe_ws;
decltype(&gb_lora) f_lora;
decltype(&gb_lora_workspace_bytes) f_lora_ws;
decltype(&gb_last_error) f_last_error;
PyObject* g_error;   // the package's GBError
PyObject* g_device;  // gives the current device's number
PyObject* g_stream;  // and of a device's number its current stream's handle: what every call runs on

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kE4m3 = at::kFloat8_e4m3fn;

// A Python error that is set already.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw Raised{};
}

std::string shape_of(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

void check(gb_status_t status) {
    if (status == GB_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(status), f_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + ": expected a tensor, got " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

struct Arg {
    void* p = nullptr;
    int64_t ld = 0;
};

// The device that the call runs on: the current one, asked for once in a call.
thread_local int64_t t_device;

int64_t device() {
    if (t_device < 0) {
        PyObject* o = PyObject_CallNoArgs(g_device);
        if (!o) throw Raised{};
        t_device = PyLong_AsLongLong(o);
        Py_DECREF(o);
        if (t_device < 0) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "no current CUDA device");
            throw Raised{};
        }
    }
    return t_device;
}

void check_device(const at::Tensor& t, const char* name) {
    if (t.get_device() != device())
        raise(PyExc_ValueError, std::string(name) + ": on " + t.device().str() + ", the current device is cuda:" +
                                    std::to_string(device()));
}

void check_type(const at::Tensor& t, const char* name, at::ScalarType type) {
    if (t.scalar_type() == type && t.is_cuda()) return check_device(t, name);
    raise(PyExc_TypeError, std::string(name) + ": expected a CUDA " + c10::toString(type) + " tensor, got " +
                               c10::toString(t.scalar_type()) + " on " + t.device().str());
}

// A [rows, cols] matrix with a contiguous last dimension: its address and leading dimension.
Arg matrix(const at::Tensor& t, const char* name, at::ScalarType type, int64_t rows, int64_t cols) {
    check_type(t, name, type);
    const auto s = t.sizes();
    if (s.size() != 2 || s[0] != rows || s[1] != cols)
        raise(PyExc_ValueError, std::string(name) + ": expected shape (" + std::to_string(rows) + ", " +
                                    std::to_string(cols) + "), got " + shape_of(s));
    const auto st = t.strides();
    if (cols > 1 && st[1] != 1) raise(PyExc_ValueError, std::string(name) + ": expected a contiguous last dimension");
    // (one row's stride is arbitrary: at least its width)
    return {t.data_ptr(), rows > 1 ? st[0] : std::max<int64_t>({st[0], cols, 1})};
}

Arg matrix(PyObject* o, const char* name, at::ScalarType type, int64_t rows, int64_t cols) {
    if (o == Py_None) return {};
    return matrix(tensor(o, name), name, type, rows, cols);
}

// A matrix for each of `count` experts or adapters: [count, rows, cols] with a contiguous last dimension.
struct Stack {
    void* p;
    int64_t ld, apart;
};

Stack stack(PyObject* o, const char* name, int64_t count, int64_t rows, int64_t cols) {
    const at::Tensor& t = tensor(o, name);
    check_type(t, name, kBf16);
    const auto s = t.sizes();
    if (s.size() != 3 || s[0] != count || s[1] != rows || s[2] != cols)
        raise(PyExc_ValueError, std::string(name) + ": expected shape (" + std::to_string(count) + ", " +
                                    std::to_string(rows) + ", " + std::to_string(cols) + "), got " + shape_of(s));
    const auto st = t.strides();
    if (cols > 1 && st[2] != 1) raise(PyExc_ValueError, std::string(name) + ": expected a contiguous last dimension");
    return {t.data_ptr(), rows > 1 ? st[1] : std::max<int64_t>({st[1], cols, 1}), st[0]};
}

void* vector(PyObject* o, const char* name, at::ScalarType type, int64_t n) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    check_type(t, name, type);
    if (t.dim() != 1 || t.size(0) != n)
        raise(PyExc_ValueError, std::string(name) + ": expected shape (" + std::to_string(n) + ",), got " + shape_of(t.sizes()));
    if (n > 1 && t.stride(0) != 1) raise(PyExc_ValueError, std::string(name) + ": expected a contiguous last dimension");
    return t.data_ptr();
}

int64_t number(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
uint64_t word(PyObject* o) {  // modulo 2^64
    const uint64_t v = PyLong_AsUnsignedLongLongMask(o);
    if (v == ~uint64_t(0) && PyErr_Occurred()) throw Raised{};
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

// (rows, columns) of a matrix that gives a call its sizes.
std::pair<int64_t, int64_t> sizes(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) raise(PyExc_ValueError, std::string(name) + ": expected a 2-D tensor, got shape " + shape_of(t.sizes()));
    return {t.size(0), t.size(1)};
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// An output: the caller's tensor, or a new one.
struct Out {
    PyObject* given = nullptr;
    at::Tensor made;
    Arg arg;
    Out(PyObject* o, const char* name, at::ScalarType type, int64_t rows, int64_t cols, const at::Tensor& like) {
        if (o != Py_None) {
            given = o;
            arg = matrix(tensor(o, name), name, type, rows, cols);
        } else {
            made = make({rows, cols}, type, like);
            arg = {made.data_ptr(), std::max<int64_t>(cols, 1)};
        }
    }
    PyObject* object() { return given ? Py_NewRef(given) : THPVariable_Wrap(std::move(made)); }
};

// A call's workspace: the caller's tensor, or a new one.
at::Tensor scratch(PyObject* o, size_t need, const at::Tensor& like) {
    if (o == Py_None) return make({std::max<int64_t>(need, 1)}, at::kByte, like);
    const at::Tensor& t = tensor(o, "workspace");
    if (!t.is_cuda()) raise(PyExc_TypeError, "workspace: expected a CUDA tensor");
    check_device(t, "workspace");
    if (!t.is_contiguous() || t.nbytes() < need)
        raise(PyExc_ValueError, "workspace holds " + std::to_string(t.nbytes()) + " contiguous bytes, " +
                                    std::to_string(need) + " needed");
    return t;
}

// seed and offset as numbers, or a CUDA int64 tensor {seed, offset} in the place of the seed.
struct Seed {
    uint64_t seed = 0, offset = 0;
    void* state = nullptr;
    Seed(PyObject* s, PyObject* o) {
        if (PyLong_Check(s)) {
            seed = word(s);
            offset = word(o);
        } else {
            state = vector(s, "seed", at::kLong, 2);
            if (!state) raise(PyExc_TypeError, "seed: expected a number or a CUDA int64 tensor {seed, offset}");
        }
    }
};

struct Activations {
    Arg x, scale;
    int type = GB_X_BF16;
};

Activations activations(const at::Tensor& X, PyObject* x_scale, int64_t M, int64_t K) {
    Activations a;
    if (X.scalar_type() != kE4m3) {
        if (x_scale != Py_None) raise(PyExc_ValueError, "x_scale: only float8_e4m3fn X has scales");
        a.x = matrix(X, "X", kBf16, M, K);
        return a;
    }
    if (x_scale == Py_None) raise(PyExc_ValueError, "x_scale: float8_e4m3fn X needs its scales");
    a.x = matrix(X, "X", kE4m3, M, K);
    const at::Tensor& s = tensor(x_scale, "x_scale");
    a.type = GB_X_E4M3_ROW_SCALE;
    if (s.dim() == 1) {
        check_type(s, "x_scale", at::kFloat);
        if (s.size(0) != M) raise(PyExc_ValueError, "x_scale: expected shape (" + std::to_string(M) + ",), got " + shape_of(s.sizes()));
        // (an expanded scale has a stride of 0: its storage ends after one element)
        if (M > 1 && s.stride(0) < 1)
            raise(PyExc_ValueError, "x_scale: expected a scale of its own for each row, got stride " + std::to_string(s.stride(0)));
        a.scale = {s.data_ptr(), std::max<int64_t>(s.stride(0), 1)};  // (a row's scale each stride)
        return a;
    }
    const int64_t groups = (K + 127) / 128;
    const bool by_group = groups > 1 && s.dim() == 2 && s.size(1) == groups;
    if (by_group) a.type = GB_X_E4M3_GROUP_SCALE;
    a.scale = matrix(s, "x_scale", at::kFloat, M, by_group ? groups : 1);
    return a;
}

struct Weights {
    Arg q, s, z;
};

Weights weights(PyObject* q, PyObject* s, PyObject* z, const char* const (&names)[3], int64_t N, int64_t K, int64_t groups) {
    return {matrix(tensor(q, names[0]), names[0], at::kByte, N, K / 2),
            matrix(tensor(s, names[1]), names[1], kBf16, N, groups), matrix(z, names[2], at::kByte, N, groups)};
}

int64_t group_of(PyObject* o) {
    const int64_t g = number(o);
    if (g != 32 && g != 64 && g != 128) raise(PyExc_ValueError, "group must be 32, 64 or 128");
    return g;
}

void* address(PyObject* o) { return reinterpret_cast<void*>(static_cast<uintptr_t>(word(o))); }

void* current_stream() {
    PyObject* number = PyLong_FromLongLong(device());
    PyObject* handle = number ? PyObject_CallOneArg(g_stream, number) : nullptr;
    Py_XDECREF(number);
    if (!handle) throw Raised{};
    const uint64_t v = PyLong_AsUnsignedLongLongMask(handle);
    Py_DECREF(handle);
    if (v == ~uint64_t(0) && PyErr_Occurred()) throw Raised{};
    return reinterpret_cast<void*>(static_cast<uintptr_t>(v));
}

template <int N>
void expect(Py_ssize_t n) {
    if (n != N) raise(PyExc_TypeError, "expected " + std::to_string(N) + " arguments, got " + std::to_string(n));
}

// A C function, without Python's lock: a launch waits for room where many are queued, and other threads'
// Python code runs meanwhile.
template <class F, class... A>
gb_status_t unlocked(F f, A... args) {
    PyThreadState* state = PyEval_SaveThread();
    const gb_status_t status = f(args...);
    PyEval_RestoreThread(state);
    return status;
}

using Args = PyObject* const*;

// X, Wq, scales, bias, R, act, zeros, group, x_scale, out
PyObject* linear_w4(Args a, Py_ssize_t n) {
    expect<10>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [M, K] = sizes(X, "X");
    const int64_t N = sizes(tensor(a[1], "Wq"), "Wq").first, group = group_of(a[7]);
    const Activations x = activations(X, a[8], M, K);
    const Weights w = weights(a[1], a[2], a[6], {"Wq", "scales", "zeros"}, N, K, (K + group - 1) / group);
    const void* bias = vector(a[3], "bias", kBf16, N);
    const Arg r = matrix(a[4], "R", kBf16, M, N);
    Out out(a[9], "out", kBf16, M, N, X);
    check(unlocked(f_linear_w4, x.x.p, x.x.ld, x.type, static_cast<float*>(x.scale.p), x.scale.ld, w.q.p, w.q.ld, w.s.p,
                   w.s.ld, w.z.p, w.z.ld, static_cast<int>(group), bias, r.p, r.ld, static_cast<int>(number(a[5])),
                   out.arg.p, out.arg.ld, M, N, K, current_stream()));
    return out.object();
}

// X, W1q, scales1, W3q, scales3, zeros1, zeros3, group, x_scale, out
PyObject* ffn_gated_w4(Args a, Py_ssize_t n) {
    expect<10>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [M, K] = sizes(X, "X");
    const int64_t N = sizes(tensor(a[1], "W1q"), "W1q").first, group = group_of(a[7]), groups = (K + group - 1) / group;
    const Activations x = activations(X, a[8], M, K);
    const Weights u = weights(a[1], a[2], a[5], {"W1q", "scales1", "zeros1"}, N, K, groups);
    const Weights v = weights(a[3], a[4], a[6], {"W3q", "scales3", "zeros3"}, N, K, groups);
    Out out(a[9], "out", kBf16, M, N, X);
    check(unlocked(f_ffn_gated_w4, x.x.p, x.x.ld, x.type, static_cast<float*>(x.scale.p), x.scale.ld, u.q.p, u.q.ld,
                   u.s.p, u.s.ld, u.z.p, u.z.ld, v.q.p, v.q.ld, v.s.p, v.s.ld, v.z.p, v.z.ld, static_cast<int>(group),
                   out.arg.p, out.arg.ld, M, N, K, current_stream()));
    return out.object();
}

// X, p, seed, offset, R, out
PyObject* dropout(Args a, Py_ssize_t n) {
    expect<6>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [M, N] = sizes(X, "X");
    const Arg x = matrix(X, "X", kBf16, M, N), r = matrix(a[4], "R", kBf16, M, N);
    const Seed seed(a[2], a[3]);
    Out out(a[5], "out", kBf16, M, N, X);
    check(unlocked(f_dropout, x.p, x.ld, r.p, r.ld, real(a[1]), seed.seed, seed.offset, seed.state, out.arg.p,
                   out.arg.ld, M, N, current_stream()));
    return out.object();
}

// A tuple of new references (of which one may be null: an error that is set already).
template <class... O>
PyObject* tuple(O... objects) {
    PyObject* all[] = {objects...};
    bool fine = true;
    for (PyObject* o : all) fine &= o != nullptr;
    PyObject* t = fine ? PyTuple_New(sizeof...(objects)) : nullptr;
    if (!t) {
        for (PyObject* o : all) Py_XDECREF(o);
        throw Raised{};
    }
    for (size_t i = 0; i < sizeof...(objects); ++i) PyTuple_SET_ITEM(t, i, all[i]);
    return t;
}

// X, weight, R, eps, p, seed, offset, out, h
PyObject* add_rms_norm(Args a, Py_ssize_t n) {
    expect<9>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [M, D] = sizes(X, "X");
    const Arg x = matrix(X, "X", kBf16, M, D), r = matrix(a[2], "R", kBf16, M, D);
    const void* w = vector(a[1], "weight", kBf16, D);
    const double p = real(a[4]);
    const Seed seed(a[5], a[6]);
    Out out(a[7], "out", kBf16, M, D, X);
    const bool same = a[8] == Py_None && !r.p && a[2] == Py_None && p == 0.0;  // H is X itself
    Out h(same ? a[0] : a[8], "h", kBf16, M, D, X);
    at::Tensor rstd = make({M}, at::kFloat, X);
    check(unlocked(f_norm, x.p, x.ld, r.p, r.ld, w, real(a[3]), p, seed.seed, seed.offset, seed.state,
                   same ? nullptr : h.arg.p, h.arg.ld, out.arg.p, out.arg.ld, static_cast<float*>(rstd.data_ptr()), M, D,
                   current_stream()));
    return tuple(out.object(), h.object(), THPVariable_Wrap(std::move(rstd)));
}

// X, weight, R, eps, scale_group, out, h
PyObject* add_rms_norm_q8(Args a, Py_ssize_t n) {
    expect<7>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [M, D] = sizes(X, "X");
    const Arg x = matrix(X, "X", kBf16, M, D), r = matrix(a[2], "R", kBf16, M, D);
    const void* w = vector(a[1], "weight", kBf16, D);
    // (what is no int is no group either: the C call refuses it)
    const int64_t group = std::clamp<int64_t>(number(a[4]), -1, INT_MAX), scales = group > 0 ? (D + group - 1) / group : 1;
    Out out(a[5], "out", kE4m3, M, D, X);
    const bool same = a[6] == Py_None && a[2] == Py_None;  // H is X itself
    Out h(same ? a[0] : a[6], "h", kBf16, M, D, X);
    at::Tensor scale = make({M, scales}, at::kFloat, X);
    check(unlocked(f_norm_q8, x.p, x.ld, r.p, r.ld, w, real(a[3]), static_cast<int>(group), same ? nullptr : h.arg.p,
                   h.arg.ld, out.arg.p, out.arg.ld, static_cast<float*>(scale.data_ptr()), std::max<int64_t>(scales, 1),
                   M, D, current_stream()));
    return tuple(out.object(), THPVariable_Wrap(std::move(scale)), h.object());
}

// dY, H, weight, rstd, dH, p, seed, offset, workspace
PyObject* add_rms_norm_backward(Args a, Py_ssize_t n) {
    expect<9>(n);
    const at::Tensor& dY = tensor(a[0], "dY");
    const auto [M, D] = sizes(dY, "dY");
    const Arg dy = matrix(dY, "dY", kBf16, M, D), h = matrix(tensor(a[1], "H"), "H", kBf16, M, D);
    const void* w = vector(a[2], "weight", kBf16, D);
    const void* rstd = vector(a[3], "rstd", at::kFloat, M);
    const Arg dh = matrix(a[4], "dH", kBf16, M, D);
    const double p = real(a[5]);
    const Seed seed(a[6], a[7]);
    size_t need = 0;
    check(f_norm_bwd_ws(M, D, &need));
    const at::Tensor workspace = scratch(a[8], need, dY);
    at::Tensor dR = make({M, D}, kBf16, dY), dX = p > 0.0 ? make({M, D}, kBf16, dY) : dR;
    at::Tensor dweight = make({D}, at::kFloat, dY);
    const int64_t ld = std::max<int64_t>(D, 1);
    check(unlocked(f_norm_bwd, dy.p, dy.ld, h.p, h.ld, w, static_cast<const float*>(rstd), dh.p, dh.ld, p, seed.seed,
                   seed.offset, seed.state, dR.data_ptr(), ld, dX.data_ptr(), ld, static_cast<float*>(dweight.data_ptr()),
                   workspace.data_ptr(), workspace.nbytes(), M, D, current_stream()));
    PyObject* x = THPVariable_Wrap(dX);
    return tuple(x, p > 0.0 ? THPVariable_Wrap(dR) : Py_XNewRef(x), THPVariable_Wrap(std::move(dweight)));
}

// X, weight, bias, R, eps, p, seed, offset, out, h
PyObject* add_layer_norm(Args a, Py_ssize_t n) {
    expect<10>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [M, D] = sizes(X, "X");
    const Arg x = matrix(X, "X", kBf16, M, D), r = matrix(a[3], "R", kBf16, M, D);
    const void* w = vector(a[1], "weight", kBf16, D);
    const void* b = vector(a[2], "bias", kBf16, D);
    const double p = real(a[5]);
    const Seed seed(a[6], a[7]);
    Out out(a[8], "out", kBf16, M, D, X);
    const bool same = a[9] == Py_None && a[3] == Py_None && p == 0.0;  // H is X itself
    Out h(same ? a[0] : a[9], "h", kBf16, M, D, X);
    at::Tensor mean = make({M}, at::kFloat, X), rstd = make({M}, at::kFloat, X);
    check(unlocked(f_layer_norm, x.p, x.ld, r.p, r.ld, w, b, real(a[4]), p, seed.seed, seed.offset, seed.state,
                   same ? nullptr : h.arg.p, h.arg.ld, out.arg.p, out.arg.ld, static_cast<float*>(mean.data_ptr()),
                   static_cast<float*>(rstd.data_ptr()), M, D, current_stream()));
    return tuple(out.object(), h.object(), THPVariable_Wrap(std::move(mean)), THPVariable_Wrap(std::move(rstd)));
}

// dY, H, weight, mean, rstd, dH, p, seed, offset, workspace
PyObject* add_layer_norm_backward(Args a, Py_ssize_t n) {
    expect<10>(n);
    const at::Tensor& dY = tensor(a[0], "dY");
    const auto [M, D] = sizes(dY, "dY");
    const Arg dy = matrix(dY, "dY", kBf16, M, D), h = matrix(tensor(a[1], "H"), "H", kBf16, M, D);
    const void* w = vector(a[2], "weight", kBf16, D);
    const void* mean = vector(a[3], "mean", at::kFloat, M);
    const void* rstd = vector(a[4], "rstd", at::kFloat, M);
    const Arg dh = matrix(a[5], "dH", kBf16, M, D);
    const double p = real(a[6]);
    const Seed seed(a[7], a[8]);
    size_t need = 0;
    check(f_layer_norm_bwd_ws(M, D, &need));
    const at::Tensor workspace = scratch(a[9], need, dY);
    at::Tensor dR = make({M, D}, kBf16, dY), dX = p > 0.0 ? make({M, D}, kBf16, dY) : dR;
    at::Tensor dweight = make({D}, at::kFloat, dY), dbias = make({D}, at::kFloat, dY);
    const int64_t ld = std::max<int64_t>(D, 1);
    check(unlocked(f_layer_norm_bwd, dy.p, dy.ld, h.p, h.ld, w, static_cast<const float*>(mean),
                   static_cast<const float*>(rstd), dh.p, dh.ld, p, seed.seed, seed.offset, seed.state, dR.data_ptr(), ld,
                   dX.data_ptr(), ld, static_cast<float*>(dweight.data_ptr()), static_cast<float*>(dbias.data_ptr()),
                   workspace.data_ptr(), workspace.nbytes(), M, D, current_stream()));
    PyObject* x = THPVariable_Wrap(dX);
    return tuple(x, p > 0.0 ? THPVariable_Wrap(dR) : Py_XNewRef(x), THPVariable_Wrap(std::move(dweight)),
                 THPVariable_Wrap(std::move(dbias)));
}

// X, router, W1, W3, W2, top_k, R, renormalize, out, workspace
PyObject* moe_ffn_gated(Args a, Py_ssize_t n) {
    expect<10>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [T, D] = sizes(X, "X");
    const Arg x = matrix(X, "X", kBf16, T, D), r = matrix(a[6], "R", kBf16, T, D);
    const at::Tensor& router = tensor(a[1], "router");
    const int64_t E = sizes(router, "router").first;
    const Arg g = matrix(router, "router", kBf16, E, D);
    const at::Tensor& W1 = tensor(a[2], "W1");
    if (W1.dim() != 3) raise(PyExc_ValueError, "W1: expected a 3-D tensor, got shape " + shape_of(W1.sizes()));
    const int64_t I = W1.size(1);
    const Stack w1 = stack(a[2], "W1", E, I, D), w3 = stack(a[3], "W3", E, I, D), w2 = stack(a[4], "W2", E, D, I);
    const int top = static_cast<int>(std::clamp<int64_t>(number(a[5]), INT_MIN, INT_MAX));
    const int renormalize = PyObject_IsTrue(a[7]);
    if (renormalize < 0) throw Raised{};
    size_t need = 0;
    check(f_moe_ws(T, I, E, top, &need));
    const at::Tensor workspace = scratch(a[9], need, X);
    Out out(a[8], "out", kBf16, T, D, X);
    at::Tensor ids = make({T, top}, at::kInt, X), weights = make({T, top}, at::kFloat, X);
    check(unlocked(f_moe, x.p, x.ld, g.p, g.ld, w1.p, w1.ld, w1.apart, w3.p, w3.ld, w3.apart, w2.p, w2.ld, w2.apart, r.p,
                   r.ld, top, renormalize, out.arg.p, out.arg.ld, static_cast<int32_t*>(ids.data_ptr()),
                   static_cast<float*>(weights.data_ptr()), workspace.data_ptr(), workspace.nbytes(), T, D, I, E,
                   current_stream()));
    return tuple(out.object(), THPVariable_Wrap(std::move(ids)), THPVariable_Wrap(std::move(weights)));
}

// X, A, B, ids, scale, R, act, out, workspace
PyObject* lora(Args a, Py_ssize_t n) {
    expect<9>(n);
    const at::Tensor& X = tensor(a[0], "X");
    const auto [M, K] = sizes(X, "X");
    const at::Tensor &A = tensor(a[1], "A"), &B = tensor(a[2], "B");
    if (A.dim() != 3) raise(PyExc_ValueError, "A: expected a 3-D tensor, got shape " + shape_of(A.sizes()));
    if (B.dim() != 3) raise(PyExc_ValueError, "B: expected a 3-D tensor, got shape " + shape_of(B.sizes()));
    const int64_t adapters = A.size(0), rank = A.size(1), N = B.size(1);
    const Arg x = matrix(X, "X", kBf16, M, K), r = matrix(a[5], "R", kBf16, M, N);
    const Stack down = stack(a[1], "A", adapters, rank, K), up = stack(a[2], "B", adapters, N, rank);
    tensor(a[3], "ids");
    const void* ids = vector(a[3], "ids", at::kInt, M);
    const void* scale = vector(a[4], "scale", at::kFloat, adapters);
    size_t need = 0;
    check(f_lora_ws(M, N, K, rank, &need));
    const at::Tensor workspace = scratch(a[8], need, X);
    Out out(a[7], "out", kBf16, M, N, X);
    check(unlocked(f_lora, x.p, x.ld, down.p, down.ld, down.apart, up.p, up.ld, up.apart, static_cast<const int32_t*>(ids),
                   static_cast<const float*>(scale), r.p, r.ld, static_cast<int>(number(a[6])), out.arg.p, out.arg.ld,
                   workspace.data_ptr(), workspace.nbytes(), M, N, K, rank, adapters, current_stream()));
    return out.object();
}

// GBError, the two functions, then the addresses of the C functions in the order of the declarations above
PyObject* bind(Args a, Py_ssize_t n) {
    constexpr int count = 15;
    expect<count + 3>(n);
    void* at[count];
    for (int i = 0; i < count; ++i) at[i] = address(a[i + 3]);
    f_linear_w4 = reinterpret_cast<decltype(f_linear_w4)>(at[0]);
    f_ffn_gated_w4 = reinterpret_cast<decltype(f_ffn_gated_w4)>(at[1]);
    f_dropout = reinterpret_cast<decltype(f_dropout)>(at[2]);
    f_norm = reinterpret_cast<decltype(f_norm)>(at[3]);
    f_norm_q8 = reinterpret_cast<decltype(f_norm_q8)>(at[4]);
    f_norm_bwd = reinterpret_cast<decltype(f_norm_bwd)>(at[5]);
    f_norm_bwd_ws = reinterpret_cast<decltype(f_norm_bwd_ws)>(at[6]);
    f_layer_norm = reinterpret_cast<decltype(f_layer_norm)>(at[7]);
    f_layer_norm_bwd = reinterpret_cast<decltype(f_layer_norm_bwd)>(at[8]);
    f_layer_norm_bwd_ws = reinterpret_cast<decltype(f_layer_norm_bwd_ws)>(at[9]);
    f_moe = reinterpret_cast<decltype(f_moe)>(at[10]);
    f_moe_ws = reinterpret_cast<decltype(f_moe_ws)>(at[11]);
    f_lora = reinterpret_cast<decltype(f_lora)>(at[12]);
    f_lora_ws = reinterpret_cast<decltype(f_lora_ws)>(at[13]);
    f_last_error = reinterpret_cast<decltype(f_last_error)>(at[14]);
    g_error = Py_NewRef(a[0]);
    g_device = Py_NewRef(a[1]);
    g_stream = Py_NewRef(a[2]);
    return Py_NewRef(Py_None);
}

template <PyObject* (*F)(Args, Py_ssize_t)>
PyObject* entry(PyObject*, Args a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    t_device = -1;
    try {
        return F(a, n);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(Args, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),
                         method<linear_w4>("linear_w4"),
                         method<ffn_gated_w4>("ffn_gated_w4"),
                         method<dropout>("dropout"),
                         method<add_rms_norm>("add_rms_norm"),
                         method<add_rms_norm_q8>("add_rms_norm_q8"),
                         method<add_rms_norm_backward>("add_rms_norm_backward"),
                         method<add_layer_norm>("add_layer_norm"),
                         method<add_layer_norm_backward>("add_layer_norm_backward"),
                         method<moe_ffn_gated>("moe_ffn_gated"),
                         method<lora>("lora"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gbgemm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gbgemm_torch() { return PyModule_Create(&module); }
