// binding.cpp -- argument checks and calls of the norm and *_act entry points for Python.
//
// A call of these on a few rows takes the GPU 3 us, and marshalling its arguments in Python
// and ctypes takes 6; here it takes under one.  Each function checks its tensors (dtype,
// shape, contiguity, overlap, then device), takes the current stream unless it is given one,
// and calls the C ABI through an address that the package hands over at load time; it returns
// the call's status.  TypeError: not a tensor, wrong dtype or device; ValueError: the rest.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <cstdlib>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "nvfp4.h"

namespace {

struct type_error : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct value_error : std::runtime_error {
    using std::runtime_error::runtime_error;
};

// The C ABI entry points, in the order of set_entries.
struct Entries {
    decltype(&int8_rmsnorm_quantize) int8_norm = nullptr;
    decltype(&nvfp4_rmsnorm_quantize) nvfp4_norm = nullptr;
    decltype(&int8_gemm_act) int8_gemm = nullptr;
    decltype(&nvfp4_gemm_act) nvfp4_gemm = nullptr;
    decltype(&int8_linear_act) int8_linear = nullptr;
    decltype(&nvfp4_linear_act) nvfp4_linear = nullptr;
    decltype(&nvfp4_scale_bytes) scale_bytes = nullptr;
    decltype(&nvfp4_prepared_scale_bytes) prepared_bytes = nullptr;
} entries;

const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw type_error(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

std::string shape_text(std::initializer_list<int64_t> shape) {
    std::string s = "[";
    for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
    return s + "]";
}

// The address of a tensor that has to be exactly this (nullptr stays nullptr), on the device
// of `like`.
void* need(const at::Tensor* t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
           const at::Tensor& like) {
    if (!t) return nullptr;
    if (t->scalar_type() != type)
        throw type_error(std::string(name) + " must be a " + c10::toString(type) + " tensor");
    if (!t->sizes().equals(at::IntArrayRef(shape.begin(), shape.size())) || !t->is_contiguous())
        throw value_error(std::string(name) + " must be a contiguous tensor of shape " + shape_text(shape));
    if (t->device() != like.device())
        throw type_error(std::string(name) + " must be on " + like.device().str());
    return t->data_ptr();
}

// The address of a packed uint8 buffer of at least `least` bytes.
void* need_bytes(const at::Tensor* t, const char* name, int64_t least, const at::Tensor& like) {
    if (t->scalar_type() != at::kByte) throw type_error(std::string(name) + " must be a Byte tensor");
    if (t->numel() < least || !t->is_contiguous())
        throw value_error(std::string(name) + " must be contiguous and hold at least " +
                          std::to_string(least) + " bytes");
    if (t->device() != like.device())
        throw type_error(std::string(name) + " must be on " + like.device().str());
    return t->data_ptr();
}

// The address of n row scales; of none there may be one, as int8_quantize_rows returns it.
void* need_scales(const at::Tensor* t, const char* name, int64_t n, const at::Tensor& like) {
    return need(t, name, at::kFloat, {n == 0 && t->dim() == 1 && t->size(0) == 1 ? 1 : n}, like);
}

// The address of a float32 tensor of one element, of whatever shape.
void* need_scalar(const at::Tensor* t, const char* name, const at::Tensor& like) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kFloat)
        throw type_error(std::string(name) + " must be a " + c10::toString(at::kFloat) + " tensor");
    if (t->numel() != 1) throw value_error(std::string(name) + " must be a tensor of one element");
    if (t->device() != like.device())
        throw type_error(std::string(name) + " must be on " + like.device().str());
    return t->data_ptr();
}

// A buffer and its name in a refusal.
struct Named {
    const char* name;
    const void* p;
    int64_t bytes;
};

// Whether two buffers share bytes.
bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

void need_2d(const at::Tensor& t, const char* name, at::ScalarType type) {
    if (t.scalar_type() != type)
        throw type_error(std::string(name) + " must be a " + c10::toString(type) + " tensor");
    if (t.dim() != 2 || !t.is_contiguous())
        throw value_error(std::string(name) + " must be a contiguous 2-D tensor");
}

// The library launches on the current device, so that is where the tensors have to be.
void on_current_device(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) throw type_error(std::string(name) + " must be a CUDA tensor");
    if (t.device().index() != c10::cuda::current_device())
        throw value_error(std::string(name) + " is on " + t.device().str() +
                          ", which is not the current device");
}

void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    void* s = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw type_error("stream must be a stream's handle");
    return s;
}

double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw type_error(std::string(name) + " must be a number");
    return v;
}

int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw type_error(std::string(name) + " must be an integer");
    return v;
}

int int32(PyObject* o, const char* name) {
    const int64_t v = integer(o, name);
    if (v != (int)v) throw value_error(std::string(name) + " is out of range");
    return (int)v;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
    try {
        if (n != want) throw type_error("wrong number of arguments");
        if (!entries.int8_norm) throw std::runtime_error("the CUDA library has not been loaded");
        return PyLong_FromLong(body());
    } catch (const type_error& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const value_error& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// --- norms ------------------------------------------------------------------------------

struct NormArgs {
    const at::Tensor* x;
    void *px, *residual, *weight, *h, *n;
    int64_t R, K;
};

NormArgs norm_args(PyObject* x, PyObject* weight, PyObject* residual, PyObject* h, PyObject* n) {
    NormArgs a;
    a.x = tensor(x, "x");
    need_2d(*a.x, "x", at::kBFloat16);
    a.R = a.x->size(0);
    a.K = a.x->size(1);
    a.px = a.x->data_ptr();
    a.residual = need(tensor(residual, "residual", true), "residual", at::kBFloat16, {a.R, a.K}, *a.x);
    a.weight = need(tensor(weight, "weight", true), "weight", at::kBFloat16, {a.K}, *a.x);
    a.h = need(tensor(h, "residual_out", true), "residual_out", at::kBFloat16, {a.R, a.K}, *a.x);
    a.n = need(tensor(n, "norm_out", true), "norm_out", at::kBFloat16, {a.R, a.K}, *a.x);
    if (a.h && !a.residual && a.R) throw value_error("residual_out needs a residual");
    const int64_t bytes = 2 * a.R * a.K;
    for (void* in : {a.px, a.residual})
        if (in != a.h && overlap(in, bytes, a.h, bytes))
            throw value_error("residual_out must be x or residual itself or not overlap them");
    for (void* other : {a.px, a.residual, a.h})
        if (overlap(other, bytes, a.n, bytes)) throw value_error("norm_out must not overlap the other tensors");
    if (overlap(a.weight, 2 * a.K, a.h, bytes) || overlap(a.weight, 2 * a.K, a.n, bytes))
        throw value_error("weight must not overlap the outputs");
    return a;
}

void codes_apart(const NormArgs& a, const Named& codes, const Named& scales) {
    const int64_t bytes = 2 * a.R * a.K;
    for (const Named* o : {&codes, &scales}) {
        for (const void* t : {a.px, a.residual, a.h, a.n})
            if (overlap(o->p, o->bytes, t, bytes))
                throw value_error(std::string(o->name) + " must not overlap the other tensors");
        if (overlap(o->p, o->bytes, a.weight, 2 * a.K))
            throw value_error(std::string(o->name) + " must not overlap the other tensors");
    }
    if (overlap(codes.p, codes.bytes, scales.p, scales.bytes))
        throw value_error(std::string(scales.name) + " must not overlap the other tensors");
}

// The device scalars: the scales that are read stay out of the outputs' bytes, alpha_out out of
// every other tensor's.
void scalars_apart(const NormArgs& a, const Named& codes, const Named& scales, const void* gsf,
                   const void* gsf_w, const void* alpha) {
    const int64_t bytes = 2 * a.R * a.K;
    const Named outputs[] = {{"residual_out", a.h, bytes}, {"norm_out", a.n, bytes}, codes, scales};
    const Named inputs[] = {{"x", a.px, bytes}, {"residual", a.residual, bytes},
                            {"weight", a.weight, 2 * a.K}, {"gsf", gsf, 4}, {"gsf_w", gsf_w, 4}};
    const auto apart = [](const Named& s, const Named& t) {
        if (overlap(s.p, s.bytes, t.p, t.bytes))
            throw value_error(std::string(s.name) + " must not overlap " + t.name);
    };
    for (const Named& o : outputs) {
        apart({"gsf", gsf, 4}, o);
        apart({"gsf_w", gsf_w, 4}, o);
        apart({"alpha_out", alpha, 4}, o);
    }
    for (const Named& i : inputs) apart({"alpha_out", alpha, 4}, i);
}

// (x, weight, eps, residual, codes, scales, residual_out, norm_out, stream)
PyObject* py_int8_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> int {
        const NormArgs a = norm_args(v[0], v[1], v[3], v[6], v[7]);
        void* q = need(tensor(v[4], "codes"), "codes", at::kChar, {a.R, a.K}, *a.x);
        void* s = need(tensor(v[5], "scales"), "scales", at::kFloat, {a.R}, *a.x);
        codes_apart(a, {"codes", q, a.R * a.K}, {"scales", s, 4 * a.R});
        const double eps = number(v[2], "eps");
        on_current_device(*a.x, "x");
        if (a.R == 0) return NVFP4_OK;           // an empty tensor has no address
        return entries.int8_norm(a.px, a.residual, a.weight, eps, a.R, a.K, static_cast<int8_t*>(q),
                                 static_cast<float*>(s), a.h, a.n, stream_of(v[8]));
    });
}

// (x, weight, eps, residual, gsf, packed, scales, gsf_w, alpha_out, residual_out, norm_out, stream)
PyObject* py_nvfp4_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> int {
        const NormArgs a = norm_args(v[0], v[1], v[3], v[9], v[10]);
        void* gsf = need_scalar(tensor(v[4], "gsf"), "gsf", *a.x);
        void* packed = need(tensor(v[5], "packed"), "packed", at::kByte, {a.R, a.K / 2}, *a.x);
        const int64_t sf_bytes = (int64_t)entries.scale_bytes(a.R, a.K);
        void* sf = need_bytes(tensor(v[6], "scales"), "scales", sf_bytes, *a.x);
        const Named codes{"packed", packed, a.R * (a.K / 2)}, scales{"scales", sf, sf_bytes};
        codes_apart(a, codes, scales);
        void* gsf_w = need_scalar(tensor(v[7], "gsf_w", true), "gsf_w", *a.x);
        void* alpha = need_scalar(tensor(v[8], "alpha_out", true), "alpha_out", *a.x);
        scalars_apart(a, codes, scales, gsf, gsf_w, alpha);
        const double eps = number(v[2], "eps");
        on_current_device(*a.x, "x");
        if (a.R == 0) return NVFP4_OK;
        return entries.nvfp4_norm(a.px, a.residual, a.weight, eps, a.R, a.K, static_cast<float*>(gsf),
                                  static_cast<uint8_t*>(packed), static_cast<uint8_t*>(sf),
                                  static_cast<float*>(gsf_w), static_cast<float*>(alpha), a.h, a.n,
                                  stream_of(v[11]));
    });
}

// --- products -----------------------------------------------------------------------------

struct EpilogueArgs {
    void *bias, *residual, *y;
    int act;
};

EpilogueArgs epilogue_args(PyObject* bias, PyObject* act, PyObject* residual, PyObject* y, int64_t M,
                           int64_t N, const at::Tensor& like) {
    EpilogueArgs e;
    e.act = int32(act, "activation");
    const int64_t cols = (e.act & NVFP4_ACT_GATED) ? N / 2 : N;
    e.bias = need(tensor(bias, "bias", true), "bias", at::kBFloat16, {N}, like);
    e.y = need(tensor(y, "out"), "out", at::kBFloat16, {M, cols}, like);
    e.residual = need(tensor(residual, "residual", true), "residual", at::kBFloat16, {M, cols}, like);
    if (e.residual != e.y && overlap(e.residual, 2 * M * cols, e.y, 2 * M * cols))
        throw value_error("residual must be out itself or not overlap it");
    return e;
}

void not_over(const EpilogueArgs& e, int64_t M, int64_t N, std::initializer_list<Named> operands) {
    const int64_t cols = (e.act & NVFP4_ACT_GATED) ? N / 2 : N;
    for (const Named& o : operands)
        if (overlap(e.y, 2 * M * cols, o.p, o.bytes))
            throw value_error(std::string("out must not overlap ") + o.name);
    if (overlap(e.y, 2 * M * cols, e.bias, 2 * N)) throw value_error("out must not overlap bias");
}

// A linear's workspace receives x's codes before the product reads its operands, and holds
// them while out is written.
void workspace_apart(const EpilogueArgs& e, int64_t M, int64_t N, const at::Tensor& x, const at::Tensor& ws,
                     std::initializer_list<Named> operands) {
    const int64_t cols = (e.act & NVFP4_ACT_GATED) ? N / 2 : N;
    const void* p = ws.data_ptr();
    const auto apart = [&](const Named& o) {
        if (overlap(p, ws.numel(), o.p, o.bytes))
            throw value_error(std::string("workspace must not overlap ") + o.name);
    };
    for (const Named& o : operands) apart(o);
    apart({"x", x.data_ptr(), 2 * x.numel()});
    apart({"bias", e.bias, 2 * N});
    apart({"residual", e.residual, 2 * M * cols});
}

// (a, sa, b, sb, bias, activation, residual, out, stream)
PyObject* py_int8_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> int {
        const at::Tensor &a = *tensor(v[0], "a"), &b = *tensor(v[2], "b");
        need_2d(a, "a", at::kChar);
        const int64_t M = a.size(0), K = a.size(1), N = b.dim() == 2 ? b.size(0) : 0;
        void* pb = need(&b, "b", at::kChar, {N, K}, a);
        void* sa = need_scales(tensor(v[1], "sa"), "sa", M, a);
        void* sb = need_scales(tensor(v[3], "sb"), "sb", N, a);
        const EpilogueArgs e = epilogue_args(v[4], v[5], v[6], v[7], M, N, a);
        not_over(e, M, N, {{"a", a.data_ptr(), M * K}, {"b", pb, N * K}, {"sa", sa, 4 * M}, {"sb", sb, 4 * N}});
        on_current_device(a, "a");
        if (M == 0 || N == 0) return NVFP4_OK;
        return entries.int8_gemm(static_cast<int8_t*>(a.data_ptr()), static_cast<float*>(sa),
                                 static_cast<int8_t*>(pb), static_cast<float*>(sb), e.bias, e.act,
                                 e.residual, e.y, M, N, K, stream_of(v[8]));
    });
}

// (a, sfa, b, sfb, prepared, alpha, bias, activation, residual, out, M, N, K, stream)
PyObject* py_nvfp4_gemm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> int {
        const int64_t M = integer(v[10], "M"), N = integer(v[11], "N"), K = integer(v[12], "K");
        if (M < 0 || N < 0 || K < 0) return NVFP4_ERR_INVALID_ARG;
        const at::Tensor& a = *tensor(v[0], "a");
        const int prepared = int32(v[4], "prepared");
        void* pa = need_bytes(&a, "a", M * (K / 2), a);
        const int64_t sfa_bytes = (int64_t)entries.scale_bytes(M, K);
        void* sfa = need_bytes(tensor(v[1], "sfa"), "sfa", sfa_bytes, a);
        void* b = need_bytes(tensor(v[2], "b"), "b", N * (K / 2), a);
        const int64_t sfb_bytes = (int64_t)(prepared ? entries.prepared_bytes(N, K) : entries.scale_bytes(N, K));
        void* sfb = need_bytes(tensor(v[3], "sfb"), "sfb", sfb_bytes, a);
        void* alpha = need_scalar(tensor(v[5], "alpha"), "alpha", a);
        const EpilogueArgs e = epilogue_args(v[6], v[7], v[8], v[9], M, N, a);
        not_over(e, M, N, {{"a", pa, M * (K / 2)}, {"b", b, N * (K / 2)}, {"sfa", sfa, sfa_bytes},
                           {"sfb", sfb, sfb_bytes}, {"alpha", alpha, 4}});
        on_current_device(a, "a");
        if (M == 0 || N == 0) return NVFP4_OK;
        return entries.nvfp4_gemm(static_cast<uint8_t*>(pa), static_cast<uint8_t*>(sfa),
                                  static_cast<uint8_t*>(b), static_cast<uint8_t*>(sfb), prepared,
                                  static_cast<float*>(alpha), e.bias, e.act, e.residual, e.y, M, N, K,
                                  stream_of(v[13]));
    });
}

// (x, wq, sw, bias, activation, residual, workspace, out, stream)
PyObject* py_int8_linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> int {
        const at::Tensor &x = *tensor(v[0], "x"), &w = *tensor(v[1], "wq");
        need_2d(x, "x", at::kBFloat16);
        const int64_t M = x.size(0), K = x.size(1), N = w.dim() == 2 ? w.size(0) : 0;
        void* wq = need(&w, "wq", at::kChar, {N, K}, x);
        void* sw = need_scales(tensor(v[2], "sw"), "sw", N, x);
        const EpilogueArgs e = epilogue_args(v[3], v[4], v[5], v[7], M, N, x);
        const at::Tensor* ws = tensor(v[6], "workspace");
        void* pws = need_bytes(ws, "workspace", 0, x);
        not_over(e, M, N, {{"wq", wq, N * K}, {"sw", sw, 4 * N}, {"workspace", pws, ws->numel()}});
        workspace_apart(e, M, N, x, *ws, {{"wq", wq, N * K}, {"sw", sw, 4 * N}});
        on_current_device(x, "x");
        if (M == 0 || N == 0) return NVFP4_OK;
        return entries.int8_linear(x.data_ptr(), M, K, static_cast<int8_t*>(wq), static_cast<float*>(sw), N,
                                   e.bias, e.act, e.residual, pws, (size_t)ws->numel(), e.y, stream_of(v[8]));
    });
}

// (x, w_packed, w_sf, prepared, gsf_w, N, bias, gsf_x, rotate_group, activation, residual,
//  workspace, out, stream)
PyObject* py_nvfp4_linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> int {
        const at::Tensor& x = *tensor(v[0], "x");
        need_2d(x, "x", at::kBFloat16);
        const int64_t M = x.size(0), K = x.size(1), N = integer(v[5], "N");
        if (N < 0) return NVFP4_ERR_INVALID_ARG;
        const int prepared = int32(v[3], "prepared");
        void* w = need_bytes(tensor(v[1], "w_packed"), "w_packed", N * (K / 2), x);
        const int64_t sf_bytes = (int64_t)(prepared ? entries.prepared_bytes(N, K) : entries.scale_bytes(N, K));
        void* sf = need_bytes(tensor(v[2], "w_sf"), "w_sf", sf_bytes, x);
        void* gsf_w = need_scalar(tensor(v[4], "gsf_w"), "gsf_w", x);
        void* gsf_x = need_scalar(tensor(v[7], "gsf_x", true), "gsf_x", x);
        const EpilogueArgs e = epilogue_args(v[6], v[9], v[10], v[12], M, N, x);
        const at::Tensor* ws = tensor(v[11], "workspace");
        void* pws = need_bytes(ws, "workspace", 0, x);
        not_over(e, M, N, {{"w_packed", w, N * (K / 2)}, {"w_sf", sf, sf_bytes}, {"gsf_w", gsf_w, 4},
                           {"gsf_x", gsf_x, 4}, {"workspace", pws, ws->numel()}});
        workspace_apart(e, M, N, x, *ws, {{"w_packed", w, N * (K / 2)}, {"w_sf", sf, sf_bytes},
                                          {"gsf_w", gsf_w, 4}, {"gsf_x", gsf_x, 4}});
        const int group = int32(v[8], "rotate_group");
        on_current_device(x, "x");
        if (M == 0 || N == 0) return NVFP4_OK;
        return entries.nvfp4_linear(x.data_ptr(), M, K, static_cast<uint8_t*>(w), static_cast<uint8_t*>(sf),
                                    prepared, static_cast<float*>(gsf_w), N, e.bias,
                                    static_cast<float*>(gsf_x), group, e.act, e.residual, pws,
                                    (size_t)ws->numel(), e.y, stream_of(v[13]));
    });
}

// The addresses of the entry points, in the order of Entries.
PyObject* py_set_entries(PyObject*, PyObject* const* v, Py_ssize_t n) {
    void* p[8];
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "eight addresses are wanted");
        return nullptr;
    }
    for (int i = 0; i < 8; ++i) {
        p[i] = PyLong_AsVoidPtr(v[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    entries.int8_norm = reinterpret_cast<decltype(entries.int8_norm)>(p[0]);
    entries.nvfp4_norm = reinterpret_cast<decltype(entries.nvfp4_norm)>(p[1]);
    entries.int8_gemm = reinterpret_cast<decltype(entries.int8_gemm)>(p[2]);
    entries.nvfp4_gemm = reinterpret_cast<decltype(entries.nvfp4_gemm)>(p[3]);
    entries.int8_linear = reinterpret_cast<decltype(entries.int8_linear)>(p[4]);
    entries.nvfp4_linear = reinterpret_cast<decltype(entries.nvfp4_linear)>(p[5]);
    entries.scale_bytes = reinterpret_cast<decltype(entries.scale_bytes)>(p[6]);
    entries.prepared_bytes = reinterpret_cast<decltype(entries.prepared_bytes)>(p[7]);
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("set_entries", py_set_entries),
                         FAST("int8_rmsnorm_quantize", py_int8_norm),
                         FAST("nvfp4_rmsnorm_quantize", py_nvfp4_norm),
                         FAST("int8_gemm_act", py_int8_gemm),
                         FAST("nvfp4_gemm_act", py_nvfp4_gemm),
                         FAST("int8_linear_act", py_int8_linear),
                         FAST("nvfp4_linear_act", py_nvfp4_linear),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for_torch", BUILT_FOR_TORCH) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
