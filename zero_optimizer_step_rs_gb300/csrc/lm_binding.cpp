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

int32_t flags(PyObject* o)
{
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "flags: more than 32 bits");
        raise_set();
    }
    return (int32_t)v;
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

// The addresses of the seven entry points, in the order of Entries.
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "expected the addresses of 7 entry points");
        return nullptr;
    }
    void* p[7];
    for (int i = 0; i < 7; ++i) {
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
    Py_RETURN_NONE;
}

#define LM_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LM_METHOD(bind),        LM_METHOD(embed),     LM_METHOD(embed_grad),
                         LM_METHOD(norm),        LM_METHOD(norm_replay), LM_METHOD(norm_grad),
                         LM_METHOD(xent),        LM_METHOD(xent_grad), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lm", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lm(void) { return PyModule_Create(&module); }
