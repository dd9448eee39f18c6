// lm_binding.cpp - the Python side of the language-model operators (module
// zero_optimizer_step_rs_gb300._lm): checks the tensors, turns them into the C
// entry points' arguments and calls these.  lm.py holds the signatures and the
// documentation.
//
// The small calls of these operators take 2 to 5 microseconds on the GPU, less
// than attribute access and ctypes take in Python for six to nine tensors (4 to 5
// microseconds a call measured on the Arm host of a GB300); here the same checks
// are a few loads each.
//
// The entry points' addresses come from binding.py (bind()), so that there is
// one place that finds and loads the library.  Every function takes its arguments
// by position, None for those left out, and returns the status code; a tensor of
// the wrong type raises TypeError, of the wrong shape, stride or device
// ValueError.  All of a call's tensors lie on one device, which is the current
// one while the entry point runs: a kernel is launched on the current device, and
// every device's default stream has the same null handle.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <vector>

#include "zero_step.h"

namespace {

struct Entries {
    decltype(&zero_embed) embed;
    decltype(&zero_embed_grad) embed_grad;
    decltype(&zero_norm) norm;
    decltype(&zero_norm_replay) norm_replay;
    decltype(&zero_norm_grad) norm_grad;
    decltype(&zero_xent) xent;
    decltype(&zero_xent_grad) xent_grad;
    decltype(&zero_layer_norm) layer_norm;
    decltype(&zero_layer_norm_grad) layer_norm_grad;
    decltype(&zero_preference) preference;
    decltype(&zero_preference_grad) preference_grad;
    decltype(&zero_policy) policy;
    decltype(&zero_policy_grad) policy_grad;
    decltype(&zero_grad_norm) grad_norm;
    decltype(&zero_grad_clip) grad_clip;
} lib = {};

// A Python error that has been set; leaves a function on the way out.
struct Raised {};

[[noreturn]] void raise_set() { throw Raised{}; }

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: expected a tensor", name);
        raise_set();
    }
    return THPVariable_Unpack(o);
}

// The device that a call's tensors lie on: the first one's, which is made the
// current one until the call ends, and which the others are held to.
class Call {
public:
    void on_device(const at::Tensor& t, const char* name)
    {
        if (!t.is_cuda()) {
            PyErr_Format(PyExc_ValueError, "%s: must be a CUDA tensor", name);
            raise_set();
        }
        const c10::DeviceIndex d = t.get_device();
        if (d == device_) return;
        if (device_ >= 0) {
            PyErr_Format(PyExc_ValueError, "%s: tensors on different devices, cuda:%d and cuda:%d",
                         name, (int)device_, (int)d);
            raise_set();
        }
        device_ = d;
    }
    // Once every tensor has been seen.
    void make_current()
    {
        if (device_ != c10::cuda::current_device()) guard_.set_index(device_);
    }
    c10::DeviceIndex device() const { return device_; }

private:
    c10::DeviceIndex device_ = -1;
    c10::cuda::OptionalCUDAGuard guard_;
};

const at::Tensor& typed(Call& c, PyObject* o, at::ScalarType type, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type) {
        PyErr_Format(PyExc_TypeError, "%s: expected torch.%s, got %s", name,
                     type == at::kBFloat16 ? "bfloat16"
                     : type == at::kFloat  ? "float32"
                     : type == at::kChar   ? "int8"
                                           : "int32",
                     c10::toString(t.scalar_type()));
        raise_set();
    }
    c.on_device(t, name);
    return t;
}

[[noreturn]] void wrong_shape(const char* name, long long a, long long b)
{
    if (b < 0) PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld,)", name, a);
    else PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld, %lld)", name, a, b);
    raise_set();
}

// A [T, D] bf16 matrix with contiguous columns.
struct Rows {
    uint16_t* p = nullptr;
    int64_t ld = 0;
};

Rows rows(Call& c, PyObject* o, int64_t T, int64_t D, const char* name)
{
    const at::Tensor& t = typed(c, o, at::kBFloat16, name);
    if (t.dim() != 2 || t.size(0) != T || t.size(1) != D) wrong_shape(name, T, D);
    if (t.stride(1) != 1 && D > 1) {
        PyErr_Format(PyExc_ValueError, "%s: columns must be contiguous", name);
        raise_set();
    }
    return {static_cast<uint16_t*>(t.data_ptr()), T > 1 ? t.stride(0) : D};
}

Rows rows_or_none(Call& c, PyObject* o, int64_t T, int64_t D, const char* name)
{
    return o == Py_None ? Rows{} : rows(c, o, T, D, name);
}

// A contiguous tensor of that shape: a matrix, or a vector (b < 0).
template <typename E>
E* dense(Call& c, PyObject* o, at::ScalarType type, int64_t a, int64_t b, const char* name)
{
    const at::Tensor& t = typed(c, o, type, name);
    const bool fits = b < 0 ? t.dim() == 1 && t.size(0) == a
                            : t.dim() == 2 && t.size(0) == a && t.size(1) == b;
    if (!fits) wrong_shape(name, a, b);
    if (!t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s: tensor must be contiguous", name);
        raise_set();
    }
    return static_cast<E*>(t.data_ptr());
}

// The two sizes of a matrix that others are measured by.
void sizes(PyObject* o, int64_t& a, int64_t& b, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) {
        PyErr_Format(PyExc_ValueError, "%s: expected a matrix, got %lld dimensions", name,
                     (long long)t.dim());
        raise_set();
    }
    a = t.size(0);
    b = t.size(1);
}

struct Ids {
    const void* p;
    int32_t bytes;
    int64_t n;
};

Ids ids(Call& c, PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    const bool wide = t.scalar_type() == at::kLong;
    if (!wide && t.scalar_type() != at::kInt) {
        PyErr_Format(PyExc_TypeError, "%s: expected int32 or int64, got %s", name,
                     c10::toString(t.scalar_type()));
        raise_set();
    }
    c.on_device(t, name);
    if (t.dim() != 1 || !t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s: expected a contiguous vector", name);
        raise_set();
    }
    return {t.data_ptr(), wide ? 8 : 4, t.size(0)};
}

// A vector that may be left out.
template <typename E>
E* dense_or_none(Call& c, PyObject* o, at::ScalarType type, int64_t n, const char* name)
{
    return o == Py_None ? nullptr : dense<E>(c, o, type, n, -1, name);
}

struct Scratch {
    void* p;
    int64_t bytes;
};

Scratch scratch(Call& c, PyObject* o)
{
    const at::Tensor& t = tensor(o, "scratch");
    c.on_device(t, "scratch");
    if (!t.is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "scratch: must be contiguous");
        raise_set();
    }
    return {t.data_ptr(), (int64_t)t.nbytes()};
}

Scratch scratch_or_none(Call& c, PyObject* o)
{
    return o == Py_None ? Scratch{nullptr, 0} : scratch(c, o);
}

int32_t* status(Call& c, PyObject* o)
{
    if (o == Py_None) return nullptr;
    const at::Tensor& t = typed(c, o, at::kInt, "dev_status");
    if (t.numel() < 1) {
        PyErr_SetString(PyExc_ValueError, "dev_status: need 1 element");
        raise_set();
    }
    return static_cast<int32_t*>(t.data_ptr());
}

// The last of a call's arguments.  None: the current stream of the tensors' device;
// else the stream's address.
void* stream(Call& c, PyObject* o)
{
    c.make_current();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(c.device()).stream();
    void* s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) raise_set();
    return s;
}

int64_t whole(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) raise_set();
    return v;
}

int32_t whole32(PyObject* o, const char* name)
{
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_OverflowError, "%s: more than 32 bits", name);
        raise_set();
    }
    return (int32_t)v;
}

int32_t flags(PyObject* o) { return whole32(o, "flags"); }

int32_t truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) raise_set();
    return v;
}

double real64(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) raise_set();
    return v;
}

float real(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) raise_set();
    return (float)v;
}

// A width that the entry point refuses, rather than one that wraps around.
int32_t width(int64_t d) { return d > INT32_MAX ? INT32_MAX : (int32_t)d; }

// Nothing but Python errors leaves a function.
template <Py_ssize_t N, typename F>
PyObject* guarded(Py_ssize_t n, bool bound, F&& f)
{
    try {
        if (n != N) {
            PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
            return nullptr;
        }
        if (!bound) {
            PyErr_SetString(PyExc_RuntimeError, "the library's entry points are not bound");
            return nullptr;
        }
        Call c;
        return PyLong_FromLong((long)f(c));
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// table, tokens, out, scale, dev_status, stream
PyObject* py_embed(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<6>(n, lib.embed, [&](Call& c) {
        int64_t V, D;
        sizes(a[0], V, D, "table");
        const Ids t = ids(c, a[1], "tokens");
        const Rows out = rows(c, a[2], t.n, D, "out");
        const auto* table = dense<uint16_t>(c, a[0], at::kBFloat16, V, D, "table");
        int32_t* word = status(c, a[4]);
        return lib.embed(table, V, width(D), t.p, t.bytes, t.n, real(a[3]), out.p, out.ld,
                         word, stream(c, a[5]));
    });
}

// dy, tokens, grad, scratch, scale, accumulate, dev_status, stream
PyObject* py_embed_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<8>(n, lib.embed_grad, [&](Call& c) {
        int64_t V, D;
        sizes(a[2], V, D, "grad");
        const Ids t = ids(c, a[1], "tokens");
        const Rows dy = rows(c, a[0], t.n, D, "dy");
        auto* grad = dense<uint16_t>(c, a[2], at::kBFloat16, V, D, "grad");
        const Scratch s = scratch(c, a[3]);
        int32_t* word = status(c, a[6]);
        const int add = PyObject_IsTrue(a[5]);
        if (add < 0) raise_set();
        return lib.embed_grad(dy.p, dy.ld, t.p, t.bytes, t.n, real(a[4]), V, width(D), grad, add,
                              s.p, s.bytes, word, stream(c, a[7]));
    });
}

int64_t blocks(int64_t D) { return (D + ZERO_NORM_BLOCK - 1) / ZERO_NORM_BLOCK; }

// x, weight, y, codes, scales, rstd, residual, sum_out, eps, stream
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<10>(n, lib.norm, [&](Call& c) {
        int64_t T, D;
        sizes(a[0], T, D, "x");
        const Rows x = rows(c, a[0], T, D, "x");
        const auto* w = dense<uint16_t>(c, a[1], at::kBFloat16, D, -1, "weight");
        const Rows y = rows(c, a[2], T, D, "y");
        auto* codes =
            a[3] == Py_None ? nullptr : dense<int8_t>(c, a[3], at::kChar, T, D, "codes");
        auto* scales = a[4] == Py_None
                           ? nullptr
                           : dense<float>(c, a[4], at::kFloat, T, blocks(D), "scales");
        auto* rstd = dense<float>(c, a[5], at::kFloat, T, -1, "rstd");
        const Rows res = rows_or_none(c, a[6], T, D, "residual");
        const Rows sum = rows_or_none(c, a[7], T, D, "sum_out");
        return lib.norm(x.p, x.ld, res.p, res.ld, w, T, width(D), real(a[8]), y.p, y.ld, sum.p,
                        sum.ld, codes, scales, rstd, stream(c, a[9]));
    });
}

struct Checkpoint {
    int64_t T, D;
    const int8_t* codes;
    const float* scales;
    const float* rstd;
    const uint16_t* w;
};

Checkpoint checkpoint(Call& c, PyObject* codes, PyObject* scales, PyObject* rstd, PyObject* weight)
{
    Checkpoint k;
    sizes(codes, k.T, k.D, "codes");
    k.codes = dense<int8_t>(c, codes, at::kChar, k.T, k.D, "codes");
    k.scales = dense<float>(c, scales, at::kFloat, k.T, blocks(k.D), "scales");
    k.rstd = dense<float>(c, rstd, at::kFloat, k.T, -1, "rstd");
    k.w = dense<uint16_t>(c, weight, at::kBFloat16, k.D, -1, "weight");
    return k;
}

// codes, scales, rstd, weight, y, stream
PyObject* py_norm_replay(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<6>(n, lib.norm_replay, [&](Call& c) {
        const Checkpoint k = checkpoint(c, a[0], a[1], a[2], a[3]);
        const Rows y = rows(c, a[4], k.T, k.D, "y");
        return lib.norm_replay(k.codes, k.scales, k.rstd, k.w, k.T, width(k.D), y.p, y.ld,
                               stream(c, a[5]));
    });
}

// dy, codes, scales, rstd, weight, dx, dweight, scratch, dsum, stream
PyObject* py_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<10>(n, lib.norm_grad, [&](Call& c) {
        const Checkpoint k = checkpoint(c, a[1], a[2], a[3], a[4]);
        const Rows dy = rows(c, a[0], k.T, k.D, "dy");
        const Rows dx = rows(c, a[5], k.T, k.D, "dx");
        auto* dw = dense<uint16_t>(c, a[6], at::kBFloat16, k.D, -1, "dweight");
        const Scratch s = scratch(c, a[7]);
        const Rows dsum = rows_or_none(c, a[8], k.T, k.D, "dsum");
        return lib.norm_grad(dy.p, dy.ld, dsum.p, dsum.ld, k.codes, k.scales, k.rstd, k.w, k.T,
                             width(k.D), dx.p, dx.ld, dw, s.p, s.bytes, stream(c, a[9]));
    });
}

// h, table, targets, loss, lse, scratch, flags, dev_status, stream
PyObject* py_xent(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<9>(n, lib.xent, [&](Call& c) {
        int64_t V, D;
        sizes(a[1], V, D, "table");
        const Ids t = ids(c, a[2], "targets");
        const Rows h = rows(c, a[0], t.n, D, "h");
        const auto* table = dense<uint16_t>(c, a[1], at::kBFloat16, V, D, "table");
        auto* loss = dense<float>(c, a[3], at::kFloat, t.n, -1, "loss");
        auto* lse = dense<float>(c, a[4], at::kFloat, t.n, -1, "lse");
        const Scratch s = scratch(c, a[5]);
        int32_t* word = status(c, a[7]);
        const int32_t f = flags(a[6]);
        return lib.xent(h.p, h.ld, table, V, width(D), t.p, t.bytes, t.n, loss, lse, s.p, s.bytes, f,
                        word, stream(c, a[8]));
    });
}

// h, table, targets, lse, dloss, dh, dtable, scratch, piece, flags, dev_status, stream
PyObject* py_xent_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<12>(n, lib.xent_grad, [&](Call& c) {
        int64_t V, D;
        sizes(a[1], V, D, "table");
        const Ids t = ids(c, a[2], "targets");
        const Rows h = rows(c, a[0], t.n, D, "h");
        const auto* table = dense<uint16_t>(c, a[1], at::kBFloat16, V, D, "table");
        const auto* lse = dense<float>(c, a[3], at::kFloat, t.n, -1, "lse");
        const auto* dloss = dense<float>(c, a[4], at::kFloat, t.n, -1, "dloss");
        const Rows dh = rows(c, a[5], t.n, D, "dh");
        auto* dtable = dense<uint16_t>(c, a[6], at::kBFloat16, V, D, "dtable");
        const Scratch s = scratch(c, a[7]);
        int32_t* word = status(c, a[10]);
        const int32_t f = flags(a[9]);
        return lib.xent_grad(h.p, h.ld, table, V, width(D), t.p, t.bytes, t.n, lse, dloss, dh.p,
                             dh.ld, dtable, whole(a[8]), s.p, s.bytes, f, word, stream(c, a[11]));
    });
}

// x, weight, bias, y, mean, rstd, residual, sum_out, eps, stream
PyObject* py_layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<10>(n, lib.layer_norm, [&](Call& c) {
        int64_t T, D;
        sizes(a[0], T, D, "x");
        const Rows x = rows(c, a[0], T, D, "x");
        const auto* w = dense_or_none<uint16_t>(c, a[1], at::kBFloat16, D, "weight");
        const auto* b = dense_or_none<uint16_t>(c, a[2], at::kBFloat16, D, "bias");
        const Rows y = rows(c, a[3], T, D, "y");
        auto* mean = dense<float>(c, a[4], at::kFloat, T, -1, "mean");
        auto* rstd = dense<float>(c, a[5], at::kFloat, T, -1, "rstd");
        const Rows res = rows_or_none(c, a[6], T, D, "residual");
        const Rows sum = rows_or_none(c, a[7], T, D, "sum_out");
        return lib.layer_norm(x.p, x.ld, res.p, res.ld, w, b, T, width(D), real(a[8]), y.p, y.ld,
                              sum.p, sum.ld, mean, rstd, stream(c, a[9]));
    });
}

// dy, x, mean, rstd, weight, dx, dweight, dbias, scratch, dsum, stream
PyObject* py_layer_norm_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<11>(n, lib.layer_norm_grad, [&](Call& c) {
        int64_t T, D;
        sizes(a[0], T, D, "dy");
        const Rows dy = rows(c, a[0], T, D, "dy");
        const Rows x = rows(c, a[1], T, D, "x");
        const auto* mean = dense<float>(c, a[2], at::kFloat, T, -1, "mean");
        const auto* rstd = dense<float>(c, a[3], at::kFloat, T, -1, "rstd");
        const auto* w = dense_or_none<uint16_t>(c, a[4], at::kBFloat16, D, "weight");
        const Rows dx = rows(c, a[5], T, D, "dx");
        auto* dw = dense_or_none<uint16_t>(c, a[6], at::kBFloat16, D, "dweight");
        auto* db = dense_or_none<uint16_t>(c, a[7], at::kBFloat16, D, "dbias");
        const Scratch s = scratch_or_none(c, a[8]);
        const Rows dsum = rows_or_none(c, a[9], T, D, "dsum");
        return lib.layer_norm_grad(dy.p, dy.ld, dsum.p, dsum.ld, x.p, x.ld, mean, rstd, w, T,
                                   width(D), dx.p, dx.ld, dw, db, s.p, s.bytes, stream(c, a[10]));
    });
}

// The S + 1 offsets of packed sequences.
Ids offsets(Call& c, PyObject* o)
{
    const Ids f = ids(c, o, "offsets");
    if (f.n < 1) {
        PyErr_SetString(PyExc_ValueError, "offsets: expected one more than there are sequences");
        raise_set();
    }
    return f;
}

int64_t pairs(const Ids& offsets)
{
    if (offsets.n % 2 == 0) {
        PyErr_SetString(PyExc_ValueError, "offsets: an odd number of sequences");
        raise_set();
    }
    return offsets.n / 2;
}

// nll, ref_nll, targets, offsets, loss, slope, ratios, counts, scratch, kind, beta,
// smoothing, margin, average, dev_status, stream
PyObject* py_preference(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<16>(n, lib.preference, [&](Call& c) {
        const Ids t = ids(c, a[2], "targets"), f = offsets(c, a[3]);
        const int64_t P = pairs(f);
        const auto* nll = dense<float>(c, a[0], at::kFloat, t.n, -1, "nll");
        const auto* ref = dense_or_none<float>(c, a[1], at::kFloat, t.n, "ref_nll");
        auto* loss = dense<float>(c, a[4], at::kFloat, P, -1, "loss");
        auto* slope = dense<float>(c, a[5], at::kFloat, P, -1, "slope");
        auto* ratios = dense<float>(c, a[6], at::kFloat, 2 * P, -1, "ratios");
        auto* counts = dense<int32_t>(c, a[7], at::kInt, 2 * P, -1, "counts");
        const Scratch s = scratch(c, a[8]);
        int32_t* word = status(c, a[14]);
        const int32_t kind = whole32(a[9], "kind"), average = truth(a[13]);
        return lib.preference(nll, ref, t.p, t.bytes, t.n, f.p, f.bytes, P, kind, real64(a[10]),
                              real64(a[11]), real64(a[12]), average, loss, slope, ratios, counts,
                              s.p, s.bytes, word, stream(c, a[15]));
    });
}

// targets, offsets, slope, counts, dloss, dnll, average, stream
PyObject* py_preference_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<8>(n, lib.preference_grad, [&](Call& c) {
        const Ids t = ids(c, a[0], "targets"), f = offsets(c, a[1]);
        const int64_t P = pairs(f);
        const auto* slope = dense<float>(c, a[2], at::kFloat, P, -1, "slope");
        const auto* counts = dense<int32_t>(c, a[3], at::kInt, 2 * P, -1, "counts");
        const auto* dloss = dense<float>(c, a[4], at::kFloat, P, -1, "dloss");
        auto* dnll = dense<float>(c, a[5], at::kFloat, t.n, -1, "dnll");
        const int32_t average = truth(a[6]);
        return lib.preference_grad(t.p, t.bytes, t.n, f.p, f.bytes, P, average, slope, counts,
                                   dloss, dnll, stream(c, a[7]));
    });
}

// What the two calls of the policy loss take: nll, old_nll, ref_nll, advantages, targets,
// offsets first; per_token and the others where they stand in the call.
struct Policy {
    Ids t, f;
    int64_t S;
    const float *nll, *old, *ref, *adv;
    int32_t per_token;
};

Policy policy(Call& c, PyObject* const* a, PyObject* per_token)
{
    Policy p;
    p.t = ids(c, a[4], "targets");
    p.f = offsets(c, a[5]);
    p.S = p.f.n - 1;
    p.per_token = truth(per_token);
    p.nll = dense<float>(c, a[0], at::kFloat, p.t.n, -1, "nll");
    p.old = dense_or_none<float>(c, a[1], at::kFloat, p.t.n, "old_nll");
    p.ref = dense_or_none<float>(c, a[2], at::kFloat, p.t.n, "ref_nll");
    p.adv = dense<float>(c, a[3], at::kFloat, p.per_token ? p.t.n : p.S, -1, "advantages");
    return p;
}

// nll, old_nll, ref_nll, advantages, targets, offsets, loss, kl, clipped, counts, scratch,
// per_token, clip_low, clip_high, kl_coef, average, dev_status, stream
PyObject* py_policy(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<18>(n, lib.policy, [&](Call& c) {
        const Policy p = policy(c, a, a[11]);
        auto* loss = dense<float>(c, a[6], at::kFloat, p.S, -1, "loss");
        auto* kl = dense<float>(c, a[7], at::kFloat, p.S, -1, "kl");
        auto* clipped = dense<int32_t>(c, a[8], at::kInt, p.S, -1, "clipped");
        auto* counts = dense<int32_t>(c, a[9], at::kInt, p.S, -1, "counts");
        const Scratch s = scratch(c, a[10]);
        int32_t* word = status(c, a[16]);
        const int32_t average = truth(a[15]);
        return lib.policy(p.nll, p.old, p.ref, p.adv, p.per_token, p.t.p, p.t.bytes, p.t.n, p.f.p,
                          p.f.bytes, p.S, real64(a[12]), real64(a[13]), real64(a[14]), average,
                          loss, kl, clipped, counts, s.p, s.bytes, word, stream(c, a[17]));
    });
}

// nll, old_nll, ref_nll, advantages, targets, offsets, counts, dloss, dnll, per_token,
// clip_low, clip_high, kl_coef, average, stream
PyObject* py_policy_grad(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<15>(n, lib.policy_grad, [&](Call& c) {
        const Policy p = policy(c, a, a[9]);
        const auto* counts = dense<int32_t>(c, a[6], at::kInt, p.S, -1, "counts");
        const auto* dloss = dense<float>(c, a[7], at::kFloat, p.S, -1, "dloss");
        auto* dnll = dense<float>(c, a[8], at::kFloat, p.t.n, -1, "dnll");
        const int32_t average = truth(a[13]);
        return lib.policy_grad(p.nll, p.old, p.ref, p.adv, p.per_token, p.t.p, p.t.bytes, p.t.n,
                               p.f.p, p.f.bytes, p.S, real64(a[10]), real64(a[11]), real64(a[12]),
                               average, counts, dloss, dnll, stream(c, a[14]));
    });
}

// A list or tuple of tensors, each held by the caller while this lives.
class List {
public:
    List(Call& c, PyObject* o, const char* name)
        : seq_(PySequence_Fast(o, "expected a sequence of tensors"))
    {
        if (!seq_) raise_set();
        const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq_);
        if (n > ZERO_MAX_TENSORS) {
            PyErr_Format(PyExc_ValueError, "%s: %zd tensors, at most %d", name, n,
                         ZERO_MAX_TENSORS);
            fail();
        }
        try {
            items.reserve((size_t)n);
            for (Py_ssize_t i = 0; i < n; ++i) add(c, at(i), name, i);
        } catch (...) {
            Py_DECREF(seq_);
            throw;
        }
    }
    ~List() { Py_DECREF(seq_); }
    List(const List&) = delete;
    List& operator=(const List&) = delete;

    // Element by element the same places in both: the same strides, or both contiguous.
    void matches(const List& other, const char* name) const
    {
        if (items.size() != other.items.size()) {
            PyErr_Format(PyExc_ValueError, "%s: %zd tensors for %zd", name,
                         (Py_ssize_t)items.size(), (Py_ssize_t)other.items.size());
            raise_set();
        }
        for (Py_ssize_t i = 0; i < (Py_ssize_t)items.size(); ++i) {
            const at::Tensor& x = THPVariable_Unpack(at(i));
            const at::Tensor& y = THPVariable_Unpack(other.at(i));
            const bool flat = x.is_contiguous() && y.is_contiguous() && x.numel() == y.numel();
            if (!flat && !(x.sizes() == y.sizes() && x.strides() == y.strides())) {
                PyErr_Format(PyExc_ValueError, "%s[%zd]: shape or strides do not match", name, i);
                raise_set();
            }
            if (items[i].type != other.items[i].type && items[i].type != ZERO_TYPE_BF16) {
                PyErr_Format(PyExc_TypeError, "%s[%zd]: expected the tensor's type or "
                             "torch.bfloat16", name, i);
                raise_set();
            }
        }
    }

    std::vector<zero_tensor> items;

private:
    PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq_, i); }
    [[noreturn]] void fail()
    {
        Py_DECREF(seq_);
        raise_set();
    }
    void add(Call& c, PyObject* o, const char* name, Py_ssize_t i)
    {
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s[%zd]: expected a tensor", name, i);
            raise_set();
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        int32_t type;
        switch (t.scalar_type()) {
        case at::kBFloat16: type = ZERO_TYPE_BF16; break;
        case at::kHalf: type = ZERO_TYPE_FP16; break;
        case at::kFloat: type = ZERO_TYPE_FP32; break;
        default:
            PyErr_Format(PyExc_TypeError,
                         "%s[%zd]: expected bfloat16, float16 or float32, got %s", name, i,
                         c10::toString(t.scalar_type()));
            raise_set();
        }
        c.on_device(t, name);
        if (t.layout() != at::kStrided || t.is_neg() || !t.is_non_overlapping_and_dense()) {
            PyErr_Format(PyExc_ValueError, "%s[%zd]: must fill its memory without gaps", name, i);
            raise_set();
        }
        items.push_back(zero_tensor{t.data_ptr(), t.numel(), type});
    }
    PyObject* seq_;
};

// grads, norm, scratch, norms, dev_status, stream
PyObject* py_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<6>(n, lib.grad_norm, [&](Call& c) {
        const List g(c, a[0], "grads");
        const int64_t count = (int64_t)g.items.size();
        auto* norm = dense<float>(c, a[1], at::kFloat, 1, -1, "norm");
        const Scratch s = scratch(c, a[2]);
        auto* norms = dense_or_none<float>(c, a[3], at::kFloat, count, "norms");
        int32_t* word = status(c, a[4]);
        return lib.grad_norm(g.items.data(), (int32_t)count, norm, norms, s.p, s.bytes, word,
                             stream(c, a[5]));
    });
}

// grads, norm, max_norm, outs, stream
PyObject* py_grad_clip(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded<5>(n, lib.grad_clip, [&](Call& c) {
        const List g(c, a[0], "grads");
        const auto* norm = dense<float>(c, a[1], at::kFloat, 1, -1, "norm");
        const float most = real(a[2]);
        const int32_t count = (int32_t)g.items.size();
        if (a[3] == Py_None)
            return lib.grad_clip(g.items.data(), nullptr, count, norm, most, stream(c, a[4]));
        const List o(c, a[3], "outs");
        o.matches(g, "outs");
        return lib.grad_clip(g.items.data(), o.items.data(), count, norm, most, stream(c, a[4]));
    });
}

// The addresses of the entry points, in the order of Entries.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    constexpr int kEntries = 15;
    if (n != kEntries) {
        PyErr_Format(PyExc_TypeError, "expected the addresses of %d entry points", kEntries);
        return nullptr;
    }
    void* p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    lib.embed = reinterpret_cast<decltype(lib.embed)>(p[0]);
    lib.embed_grad = reinterpret_cast<decltype(lib.embed_grad)>(p[1]);
    lib.norm = reinterpret_cast<decltype(lib.norm)>(p[2]);
    lib.norm_replay = reinterpret_cast<decltype(lib.norm_replay)>(p[3]);
    lib.norm_grad = reinterpret_cast<decltype(lib.norm_grad)>(p[4]);
    lib.xent = reinterpret_cast<decltype(lib.xent)>(p[5]);
    lib.xent_grad = reinterpret_cast<decltype(lib.xent_grad)>(p[6]);
    lib.layer_norm = reinterpret_cast<decltype(lib.layer_norm)>(p[7]);
    lib.layer_norm_grad = reinterpret_cast<decltype(lib.layer_norm_grad)>(p[8]);
    lib.preference = reinterpret_cast<decltype(lib.preference)>(p[9]);
    lib.preference_grad = reinterpret_cast<decltype(lib.preference_grad)>(p[10]);
    lib.policy = reinterpret_cast<decltype(lib.policy)>(p[11]);
    lib.policy_grad = reinterpret_cast<decltype(lib.policy_grad)>(p[12]);
    lib.grad_norm = reinterpret_cast<decltype(lib.grad_norm)>(p[13]);
    lib.grad_clip = reinterpret_cast<decltype(lib.grad_clip)>(p[14]);
    Py_RETURN_NONE;
}

#define LM_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LM_METHOD(bind),        LM_METHOD(embed),     LM_METHOD(embed_grad),
                         LM_METHOD(norm),        LM_METHOD(norm_replay), LM_METHOD(norm_grad),
                         LM_METHOD(xent),        LM_METHOD(xent_grad),
                         LM_METHOD(layer_norm),  LM_METHOD(layer_norm_grad),
                         LM_METHOD(preference),  LM_METHOD(preference_grad),
                         LM_METHOD(policy),      LM_METHOD(policy_grad),
                         LM_METHOD(grad_norm),   LM_METHOD(grad_clip), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm(void) { return PyModule_Create(&module); }
