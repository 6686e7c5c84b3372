// binding.cpp -- the short way from Python to the operators around a feed-forward
// block, whose calls on a few rows are bound by the host: a module of one function
// per operator for the plain call (tensors of one CUDA device, the current one,
// contiguous and of matching types and sizes; outputs made here; torch's current
// stream).  Each function checks that, makes the outputs, calls the C entry point
// and returns the outputs, or returns None where anything is not plain or the entry
// point refuses: the caller (gemm_f16.py) then goes the long way, which names the
// reason or knows better.  The entry points come as addresses (init), so that the
// library is loaded once, by ctypes.
//
// One token's RMS norm with a residual (1 x 4096) is 12 us of host time the long way.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>

#include "gemm_f16.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Entries {
    decltype(&::rms_norm_fwd) rms_norm_fwd = nullptr;
    decltype(&::rms_norm_fp8) rms_norm_fp8 = nullptr;
    decltype(&::rms_norm_bwd) rms_norm_bwd = nullptr;
    decltype(&::rms_norm_bwd_workspace) rms_norm_bwd_workspace = nullptr;
    decltype(&::fp8_quantize) fp8_quantize = nullptr;
    decltype(&::dropout_philox) dropout_philox = nullptr;
    decltype(&::linear_w4) linear_w4 = nullptr;
} entries;

// The enum gemm_f16_type of a tensor's type, or -1.
int type_code(ScalarType t)
{
    if (t == ScalarType::Half) return GEMM_TYPE_F16;
    if (t == ScalarType::BFloat16) return GEMM_TYPE_BF16;
    return t == ScalarType::Float ? GEMM_TYPE_F32 : -1;
}

// The current device, if the object is a CUDA tensor, else -1 (nothing is asked of CUDA).
int device_for(PyObject *o)
{
    if (!THPVariable_CheckExact(o)) return -1;
    const Tensor &t = THPVariable_Unpack(o);
    return t.defined() && t.is_cuda() ? c10::cuda::current_device() : -1;
}

// The tensor of a Python object that is a torch.Tensor itself, contiguous and on
// device `dev`; else NULL.
const Tensor *plain(PyObject *o, int dev)
{
    if (!THPVariable_CheckExact(o)) return nullptr;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) return nullptr;
    if (t.device().index() != dev) return nullptr;
    return &t;
}

bool like(const Tensor &a, const Tensor &b) { return a.scalar_type() == b.scalar_type() && a.sizes() == b.sizes(); }

// An optional vector of weights: None, or `dim` elements of X's type or float32.
bool weight(PyObject *o, int dev, const Tensor &x, int64_t dim, const Tensor **out)
{
    *out = nullptr;
    if (o == Py_None) return true;
    const Tensor *t = plain(o, dev);
    if (!t || t->dim() != 1 || t->size(0) != dim) return false;
    if (t->scalar_type() != x.scalar_type() && t->scalar_type() != ScalarType::Float) return false;
    *out = t;
    return true;
}

void *pointer(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

Tensor make(at::IntArrayRef size, ScalarType type, int dev)
{
    return Tensor(at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
}

// Rows and row length of a tensor that is neither a scalar nor empty.
bool rows_of(const Tensor &x, int64_t *rows, int64_t *dim)
{
    if (x.dim() < 1 || x.numel() == 0) return false;
    *dim = x.size(-1);
    *rows = x.numel() / *dim;
    return true;
}

PyObject *tuple(std::initializer_list<PyObject *> items)
{
    PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t i = 0;
    for (PyObject *o : items) {
        if (t && o) PyTuple_SET_ITEM(t, i++, o);
        else Py_XDECREF(o);
    }
    return t;
}

PyObject *share(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

void *stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

struct NoGil {
    PyThreadState *state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

// (X, gamma, residual, eps, stats)
PyObject *short_rms_norm_fwd(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const int dev = n == 5 ? device_for(args[0]) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const Tensor *x = plain(args[0], dev), *gamma = nullptr, *r = nullptr;
    int64_t rows = 0, dim = 0;
    if (!x || type_code(x->scalar_type()) < 0 || !rows_of(*x, &rows, &dim)) Py_RETURN_NONE;
    if (!weight(args[1], dev, *x, dim, &gamma)) Py_RETURN_NONE;
    if (args[2] != Py_None && (!(r = plain(args[2], dev)) || !like(*r, *x))) Py_RETURN_NONE;
    if (!PyFloat_CheckExact(args[3])) Py_RETURN_NONE;
    const double eps = PyFloat_AS_DOUBLE(args[3]);
    const int stats = PyObject_IsTrue(args[4]);
    if (stats < 0) return nullptr;
    const int xt = type_code(x->scalar_type()), wt = gamma ? type_code(gamma->scalar_type()) : xt;
    Tensor y, h, rstd;
    int st;
    {
        NoGil no_gil;
        y = make(x->sizes(), x->scalar_type(), dev);
        if (r) h = make(x->sizes(), x->scalar_type(), dev);
        if (stats) rstd = make(x->sizes().slice(0, x->dim() - 1), ScalarType::Float, dev);
        st = entries.rms_norm_fwd(x->data_ptr(), pointer(r), pointer(gamma), r ? h.data_ptr() : nullptr, y.data_ptr(),
                                  static_cast<float *>(stats ? rstd.data_ptr() : nullptr), rows, dim,
                                  static_cast<float>(eps), xt, wt, stream_of(dev));
    }
    if (st != GEMM_OK) Py_RETURN_NONE;
    return tuple({THPVariable_Wrap(std::move(y)), r ? THPVariable_Wrap(std::move(h)) : share(args[0]),
                  stats ? THPVariable_Wrap(std::move(rstd)) : share(Py_None)});
    END_HANDLE_TH_ERRORS
}

// (X, gamma, residual, eps, pow2)
PyObject *short_rms_norm_fp8(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const int dev = n == 5 ? device_for(args[0]) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const Tensor *x = plain(args[0], dev), *gamma = nullptr, *r = nullptr;
    int64_t rows = 0, dim = 0;
    if (!x || type_code(x->scalar_type()) < 0 || !rows_of(*x, &rows, &dim)) Py_RETURN_NONE;
    if (!weight(args[1], dev, *x, dim, &gamma)) Py_RETURN_NONE;
    if (args[2] != Py_None && (!(r = plain(args[2], dev)) || !like(*r, *x))) Py_RETURN_NONE;
    if (!PyFloat_CheckExact(args[3])) Py_RETURN_NONE;
    const double eps = PyFloat_AS_DOUBLE(args[3]);
    const int pow2 = PyObject_IsTrue(args[4]);
    if (pow2 < 0) return nullptr;
    const int xt = type_code(x->scalar_type()), wt = gamma ? type_code(gamma->scalar_type()) : xt;
    Tensor q, s, h;
    int st;
    {
        NoGil no_gil;
        q = make(x->sizes(), ScalarType::Float8_e4m3fn, dev);
        c10::SmallVector<int64_t, 5> lead(x->sizes().begin(), x->sizes().end());
        lead.back() = (dim + 127) / 128;
        s = make(lead, pow2 ? ScalarType::Byte : ScalarType::Float, dev);
        if (r) h = make(x->sizes(), x->scalar_type(), dev);
        st = entries.rms_norm_fp8(x->data_ptr(), pointer(r), pointer(gamma), r ? h.data_ptr() : nullptr, q.data_ptr(),
                                  s.data_ptr(), nullptr, rows, dim, static_cast<float>(eps), xt, wt, pow2,
                                  stream_of(dev));
    }
    if (st != GEMM_OK) Py_RETURN_NONE;
    return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s)),
                  r ? THPVariable_Wrap(std::move(h)) : share(args[0])});
    END_HANDLE_TH_ERRORS
}

// (dY, H, rstd, gamma, dH, weights)
PyObject *short_rms_norm_bwd(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const int dev = n == 6 ? device_for(args[1]) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const Tensor *h = plain(args[1], dev), *dy = plain(args[0], dev), *rstd = plain(args[2], dev), *gamma = nullptr,
                 *dh = nullptr;
    int64_t rows = 0, dim = 0;
    if (!h || !dy || !rstd || type_code(h->scalar_type()) < 0 || !rows_of(*h, &rows, &dim)) Py_RETURN_NONE;
    if (!like(*dy, *h) || rstd->scalar_type() != ScalarType::Float ||
        rstd->sizes() != h->sizes().slice(0, h->dim() - 1))
        Py_RETURN_NONE;
    if (!weight(args[3], dev, *h, dim, &gamma)) Py_RETURN_NONE;
    if (args[4] != Py_None && (!(dh = plain(args[4], dev)) || !like(*dh, *h))) Py_RETURN_NONE;
    const int weights = PyObject_IsTrue(args[5]);
    if (weights < 0) return nullptr;
    const ScalarType wtype = gamma ? gamma->scalar_type() : h->scalar_type();
    Tensor dx, dgamma, workspace;
    int st;
    {
        NoGil no_gil;
        dx = make(h->sizes(), h->scalar_type(), dev);
        int64_t need = 0;
        if (weights) {
            need = entries.rms_norm_bwd_workspace(rows, dim);
            if (need >= 0) {
                dgamma = make({dim}, wtype, dev);
                workspace = make({need / 4}, ScalarType::Float, dev);
            }
        }
        st = need < 0 ? static_cast<int>(need)
                      : entries.rms_norm_bwd(dy->data_ptr(), h->data_ptr(), pointer(gamma),
                                             static_cast<const float *>(rstd->data_ptr()), pointer(dh), dx.data_ptr(),
                                             weights ? dgamma.data_ptr() : nullptr, rows, dim, type_code(h->scalar_type()),
                                             type_code(wtype), weights ? workspace.data_ptr() : nullptr, need,
                                             stream_of(dev));
    }
    if (st != GEMM_OK) Py_RETURN_NONE;
    return tuple({THPVariable_Wrap(std::move(dx)), weights ? THPVariable_Wrap(std::move(dgamma)) : share(Py_None)});
    END_HANDLE_TH_ERRORS
}

// (X, block_rows, pow2)
PyObject *short_fp8_quantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const int dev = n == 3 && PyLong_CheckExact(args[1]) ? device_for(args[0]) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const Tensor *x = plain(args[0], dev);
    if (!x || x->dim() != 2 || x->numel() == 0 || type_code(x->scalar_type()) < 0) Py_RETURN_NONE;
    int overflow = 0;
    const long block_rows = PyLong_AsLongAndOverflow(args[1], &overflow);
    if (overflow || (block_rows != 1 && block_rows != 128)) Py_RETURN_NONE;
    const int pow2 = PyObject_IsTrue(args[2]);
    if (pow2 < 0) return nullptr;
    const int64_t rows = x->size(0), K = x->size(1);
    Tensor q, s;
    int st;
    {
        NoGil no_gil;
        q = make(x->sizes(), ScalarType::Float8_e4m3fn, dev);
        s = make({(rows + block_rows - 1) / block_rows, (K + 127) / 128}, pow2 ? ScalarType::Byte : ScalarType::Float, dev);
        st = entries.fp8_quantize(x->data_ptr(), type_code(x->scalar_type()), q.data_ptr(), s.data_ptr(), rows, K,
                                  static_cast<int>(block_rows), pow2, stream_of(dev));
    }
    if (st != GEMM_OK) Py_RETURN_NONE;
    return tuple({THPVariable_Wrap(std::move(q)), THPVariable_Wrap(std::move(s))});
    END_HANDLE_TH_ERRORS
}

// A whole number in 0 .. 2^64 - 1.
bool whole(PyObject *o, uint64_t *out)
{
    if (!PyLong_CheckExact(o)) return false;
    *out = PyLong_AsUnsignedLongLong(o);
    if (*out == std::numeric_limits<uint64_t>::max() && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    return true;
}

// (X, p, seed, offset, residual); offset: a number or a tensor
PyObject *short_dropout(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const int dev = n == 5 && PyFloat_CheckExact(args[1]) ? device_for(args[0]) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const Tensor *x = plain(args[0], dev), *r = nullptr, *off = nullptr;
    if (!x || x->numel() == 0 || type_code(x->scalar_type()) < 0) Py_RETURN_NONE;
    const double p = PyFloat_AS_DOUBLE(args[1]);
    uint64_t seed = 0, offset = 0;
    if (!whole(args[2], &seed)) Py_RETURN_NONE;
    if (!whole(args[3], &offset) &&
        (!(off = plain(args[3], dev)) || off->scalar_type() != ScalarType::Long || off->numel() != 1))
        Py_RETURN_NONE;
    if (args[4] != Py_None && (!(r = plain(args[4], dev)) || !like(*r, *x))) Py_RETURN_NONE;
    Tensor y;
    int st;
    {
        NoGil no_gil;
        y = make(x->sizes(), x->scalar_type(), dev);
        st = entries.dropout_philox(x->data_ptr(), pointer(r), y.data_ptr(), x->numel(), type_code(x->scalar_type()), p,
                                    seed, offset, pointer(off), stream_of(dev));
    }
    if (st != GEMM_OK) Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(y));
    END_HANDLE_TH_ERRORS
}

// (X, Q, S, Z, N, group, relu); N None: Q's rows
PyObject *short_linear_w4(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    const int dev = n == 7 && PyLong_CheckExact(args[5]) ? device_for(args[0]) : -1;
    if (dev < 0) Py_RETURN_NONE;
    const Tensor *x = plain(args[0], dev), *q = plain(args[1], dev), *s = plain(args[2], dev), *z = nullptr;
    if (!x || !q || !s || x->dim() != 2 || x->numel() == 0) Py_RETURN_NONE;
    const ScalarType type = x->scalar_type();
    if (type != ScalarType::Half && type != ScalarType::BFloat16) Py_RETURN_NONE;
    int overflow = 0;
    const int64_t group = PyLong_AsLongLongAndOverflow(args[5], &overflow);
    if (overflow || (group != 32 && group != 64 && group != 128)) Py_RETURN_NONE;
    if (q->dim() != 3 || s->dim() != 3 || q->size(0) > (std::numeric_limits<int32_t>::max() - 15) / 16) Py_RETURN_NONE;
    int64_t N = 16 * q->size(0);
    if (args[4] != Py_None) {
        if (!PyLong_CheckExact(args[4])) Py_RETURN_NONE;
        N = PyLong_AsLongLongAndOverflow(args[4], &overflow);
        if (overflow || N < 1) Py_RETURN_NONE;
    }
    const int64_t M = x->size(0), K = x->size(1), strips = (N + 15) / 16, groups = (K + group - 1) / group;
    if (M > GEMM_W4_MAX_ROWS || N < 1) Py_RETURN_NONE;
    if (q->scalar_type() != ScalarType::Byte || q->size(0) != strips || q->size(1) != (K + 63) / 64 || q->size(2) != 512)
        Py_RETURN_NONE;
    if (s->scalar_type() != type || s->size(0) != strips || s->size(1) != groups || s->size(2) != 16) Py_RETURN_NONE;
    if (args[3] != Py_None &&
        (!(z = plain(args[3], dev)) || z->scalar_type() != ScalarType::Byte || z->sizes() != s->sizes()))
        Py_RETURN_NONE;
    const int relu = PyObject_IsTrue(args[6]);
    if (relu < 0) return nullptr;
    Tensor c;
    int st;
    {
        NoGil no_gil;
        c = make({M, N}, type, dev);
        st = entries.linear_w4(x->data_ptr(), type_code(type), q->data_ptr(), s->data_ptr(),
                               static_cast<const uint8_t *>(pointer(z)), c.data_ptr(), M, N, K, static_cast<int>(group),
                               relu, stream_of(dev));
    }
    if (st != GEMM_OK) Py_RETURN_NONE;
    return THPVariable_Wrap(std::move(c));
    END_HANDLE_TH_ERRORS
}

// (addresses of the entry points, in the order of Entries)
PyObject *init(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    constexpr Py_ssize_t kEntries = sizeof(Entries) / sizeof(void *);
    if (n != kEntries) {
        PyErr_SetString(PyExc_TypeError, "init takes the address of every entry point");
        return nullptr;
    }
    void *at[kEntries];
    for (Py_ssize_t i = 0; i < kEntries; ++i) {
        at[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    entries.rms_norm_fwd = reinterpret_cast<decltype(entries.rms_norm_fwd)>(at[0]);
    entries.rms_norm_fp8 = reinterpret_cast<decltype(entries.rms_norm_fp8)>(at[1]);
    entries.rms_norm_bwd = reinterpret_cast<decltype(entries.rms_norm_bwd)>(at[2]);
    entries.rms_norm_bwd_workspace = reinterpret_cast<decltype(entries.rms_norm_bwd_workspace)>(at[3]);
    entries.fp8_quantize = reinterpret_cast<decltype(entries.fp8_quantize)>(at[4]);
    entries.dropout_philox = reinterpret_cast<decltype(entries.dropout_philox)>(at[5]);
    entries.linear_w4 = reinterpret_cast<decltype(entries.linear_w4)>(at[6]);
    Py_RETURN_NONE;
}

#define SHORT(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(short_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(init)), METH_FASTCALL, nullptr},
    SHORT(rms_norm_fwd), SHORT(rms_norm_fp8), SHORT(rms_norm_bwd), SHORT(fp8_quantize), SHORT(dropout), SHORT(linear_w4),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "The short way to the operators around a feed-forward block.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding()
{
    PyObject *m = PyModule_Create(&module);
    // The torch whose tensors this module knows.
    if (m && PyModule_AddStringConstant(m, "torch_version", BINDING_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
