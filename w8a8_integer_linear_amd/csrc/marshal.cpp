// The binding's argument checks, compiled: a call of few tokens takes the GPU
// less time than a dozen tensors' checks take the interpreter (the projection
// with adapters at seven tokens: 8.8 us of host time per call instead of 12.7 us);
// and the allocation of outputs, 0.8 us each instead of 2.2 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <utility>

#include "qlin.h"

namespace {

PyObject *refuse = nullptr;     // the binding's own check, which names the fault
constexpr Py_ssize_t kMostDims = 4;

// The address of a contiguous GPU tensor of this dtype and, if any sizes are
// given, of this shape; false if it is not one.
bool fits(PyObject *o, PyObject *dtype, PyObject *const *dims, Py_ssize_t n, const void *&address)
{
    if (!THPVariable_Check(o) || !THPDtype_Check(dtype))
        return false;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided ||
        t.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type || !t.is_contiguous())
        return false;
    if (n > 0) {
        if (t.dim() != n)
            return false;
        for (Py_ssize_t i = 0; i < n; i++) {
            const long long d = PyLong_AsLongLong(dims[i]);
            if (d != t.size(i)) {
                PyErr_Clear();
                return false;
            }
        }
    }
    address = t.const_data_ptr();
    return true;
}

// address(tensor, name, dtype, *sizes)
PyObject *address(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n < 3) {
        PyErr_SetString(PyExc_TypeError, "address(tensor, name, dtype, *sizes)");
        return nullptr;
    }
    try {
        const void *p = nullptr;
        if (fits(args[0], args[2], args + 3, n - 3, p))
            return PyLong_FromVoidPtr(const_cast<void *>(p));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    PyObject *shape = Py_None;
    Py_INCREF(shape);
    if (n > 3) {
        Py_DECREF(shape);
        shape = PyTuple_New(n - 3);
        if (!shape)
            return nullptr;
        for (Py_ssize_t i = 3; i < n; i++) {
            Py_INCREF(args[i]);
            PyTuple_SET_ITEM(shape, i - 3, args[i]);
        }
    }
    PyObject *r = PyObject_CallFunctionObjArgs(refuse, args[0], args[1], args[2], shape, nullptr);
    Py_DECREF(shape);
    if (r) {
        Py_DECREF(r);
        PyErr_SetString(PyExc_ValueError, "unsupported tensor");
    }
    return nullptr;
}

// empty(like, dtype, *sizes): a new tensor on like's device.
PyObject *empty(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n < 2 || n > 2 + kMostDims || !THPVariable_Check(args[0]) || !THPDtype_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "empty(tensor, dtype, *sizes)");
        return nullptr;
    }
    int64_t sizes[kMostDims];
    for (Py_ssize_t i = 2; i < n; i++) {
        sizes[i - 2] = PyLong_AsLongLong(args[i]);
        if (sizes[i - 2] == -1 && PyErr_Occurred())
            return nullptr;
    }
    HANDLE_TH_ERRORS        // (the allocator's errors keep their types)
    const at::TensorOptions options =
        THPVariable_Unpack(args[0]).options().dtype(reinterpret_cast<THPDtype *>(args[1])->scalar_type);
    return THPVariable_Wrap(at::empty(at::IntArrayRef(sizes, (size_t)(n - 2)), options));
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------ inside a feed-forward block
//
// Whole calls: a dozen tensors' checks, their addresses and the library's call with
// twenty arguments take longer through the interpreter and ctypes than a few tokens
// take the GPU (host time per call 7.6 -> 4.4 us forward, 10.4 -> 6.6 backward).

PyObject *failed = nullptr;     // failed(name, status): raises for a nonzero status

// A Python error is set.
struct Raised {
};

// Checks tensors against one another's device.
struct Args {
    at::Device device = at::kCPU;
    bool first = true;

    // The address of a contiguous GPU tensor of this type and shape; raises the
    // binding's own error for another one.
    void *operator()(PyObject *o, const char *name, at::ScalarType type, std::initializer_list<int64_t> shape)
    {
        if (THPVariable_Check(o)) {
            const at::Tensor &t = THPVariable_Unpack(o);
            if (t.is_cuda() && t.layout() == at::kStrided && t.scalar_type() == type && t.is_contiguous() &&
                t.sizes() == at::IntArrayRef(shape)) {
                if (!first && t.device() != device) {
                    PyErr_Format(PyExc_ValueError, "the tensors are on different devices (%s: %s, not %s)", name,
                                 t.device().str().c_str(), device.str().c_str());
                    throw Raised();
                }
                device = t.device();
                first = false;
                return const_cast<void *>(t.const_data_ptr());
            }
        }
        PyObject *dims = PyTuple_New((Py_ssize_t)shape.size());
        Py_ssize_t i = 0;
        for (const int64_t d : shape)
            PyTuple_SET_ITEM(dims, i++, PyLong_FromLongLong(d));
        PyObject *dtype = reinterpret_cast<PyObject *>(torch::getTHPDtype(type));
        PyObject *r = PyObject_CallFunction(refuse, "OsOO", o, name, dtype, dims);
        Py_DECREF(dims);
        if (r) {
            Py_DECREF(r);
            PyErr_Format(PyExc_ValueError, "%s: unsupported tensor", name);
        }
        throw Raised();
    }

    // Of a float tensor: its type as the library names it.
    void *operator()(PyObject *o, const char *name, int &code, std::initializer_list<int64_t> shape)
    {
        at::ScalarType type = at::kFloat;
        if (THPVariable_Check(o))
            type = THPVariable_Unpack(o).scalar_type();
        if (type != at::kFloat && type != at::kBFloat16) {
            PyErr_Format(PyExc_TypeError, "%s must be float32 or bfloat16, got %s", name, c10::toString(type));
            throw Raised();
        }
        code = type == at::kFloat ? QLIN_F32 : QLIN_BF16;
        return (*this)(o, name, type, shape);
    }
};

// The two sizes of a tensor whose other checks follow.
std::pair<int64_t, int64_t> two(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2) {
        PyErr_Format(PyExc_ValueError, "%s must be a tensor of two dimensions", name);
        throw Raised();
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    return {t.size(0), t.size(1)};
}

// An owned reference: o, or if that is None a new tensor beside like.
struct Out {
    PyObject *o;
    Out(PyObject *given, PyObject *like, at::ScalarType type, std::initializer_list<int64_t> shape)
    {
        if (given != Py_None)
            Py_INCREF(o = given);
        else
            o = THPVariable_Wrap(at::empty(at::IntArrayRef(shape), THPVariable_Unpack(like).options().dtype(type)));
        if (!o)
            throw Raised();
    }
    explicit Out(PyObject *none) : o(none) { Py_INCREF(o); }
    Out(const Out &) = delete;
    ~Out() { Py_XDECREF(o); }
};

at::ScalarType type_of(PyObject *dtype)
{
    if (!THPDtype_Check(dtype)) {
        PyErr_SetString(PyExc_TypeError, "dtype must be a torch dtype");
        throw Raised();
    }
    return reinterpret_cast<THPDtype *>(dtype)->scalar_type;
}

// The address and size of a workspace (None: none is needed).
void *workspace_of(Args &arg, PyObject *o, size_t &bytes)
{
    bytes = 0;
    if (o == Py_None)
        return nullptr;
    bytes = THPVariable_Check(o) ? (size_t)THPVariable_Unpack(o).numel() : 0;
    return arg(o, "workspace", at::kByte, {(int64_t)bytes});
}

void check(const char *name, int status)
{
    if (status == QLIN_OK)
        return;
    PyObject *r = PyObject_CallFunction(failed, "si", name, status);
    Py_XDECREF(r);
    if (r)
        PyErr_SetString(PyExc_RuntimeError, name);
    throw Raised();
}

template <typename F> F function_at(PyObject *address) { return reinterpret_cast<F>(PyLong_AsVoidPtr(address)); }

// forward(function, gated, qx, sx, qw, sw, bias, act, residual, y, dtype, ck, ck_s, save,
// workspace, stream) -> (y, ck, ck_s)
PyObject *forward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 16) {
        PyErr_SetString(PyExc_TypeError, "forward takes 16 arguments");
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        const bool gated = PyObject_IsTrue(a[1]);
        const char *name = gated ? "qlin_fwd_gated" : "qlin_fwd_act";
        PyObject *qx = a[2];
        const auto [M, K] = two(qx, "qx");
        const int64_t N = two(a[4], "qw").first;
        if (gated && N % 2) {
            PyErr_Format(PyExc_ValueError, "qw has the gate's rows and as many others, got %lld", (long long)N);
            throw Raised();
        }
        const int64_t F = gated ? N / 2 : N;
        Args arg;
        const auto *px = static_cast<const int8_t *>(arg(qx, "qx", at::kChar, {M, K}));
        const auto *psx = static_cast<const float *>(arg(a[3], "sx", at::kFloat, {M}));
        const auto *pw = static_cast<const int8_t *>(arg(a[4], "qw", at::kChar, {N, K}));
        const auto *psw = static_cast<const float *>(arg(a[5], "sw", at::kFloat, {N}));
        const float *pb =
            a[6] == Py_None ? nullptr : static_cast<const float *>(arg(a[6], "bias", at::kFloat, {N}));
        const int act = (int)PyLong_AsLong(a[7]);
        int y_code = 0, r_code = 0;
        const void *pr = a[8] == Py_None ? nullptr : arg(a[8], "residual", r_code, {M, F});
        const Out y(a[9], qx, type_of(a[10]), {M, F});
        void *py = arg(y.o, "y", y_code, {M, F});
        const bool keep = PyObject_IsTrue(a[13]) || a[11] != Py_None || a[12] != Py_None;
        const int64_t per = (F + QLIN_CK_BLOCK - 1) / QLIN_CK_BLOCK * (gated ? 2 : 1);
        // (Named, so that both are given back where the second cannot be made.)
        std::optional<Out> ck, ck_s;
        int8_t *pc = nullptr;
        float *pcs = nullptr;
        if (keep) {
            ck.emplace(a[11], qx, at::kChar, std::initializer_list<int64_t>{M, N});
            ck_s.emplace(a[12], qx, at::kFloat, std::initializer_list<int64_t>{M, per});
            pc = static_cast<int8_t *>(arg(ck->o, "ck", at::kChar, {M, N}));
            pcs = static_cast<float *>(arg(ck_s->o, "ck_s", at::kFloat, {M, per}));
        } else {
            ck.emplace(Py_None);
            ck_s.emplace(Py_None);
        }
        size_t bytes;
        void *ws = workspace_of(arg, a[14], bytes);
        void *stream = PyLong_AsVoidPtr(a[15]);
        if (PyErr_Occurred())
            throw Raised();
        check(name, gated ? function_at<decltype(&qlin_fwd_gated)>(a[0])(px, psx, pw, psw, pb, act, M, F, K, py,
                                                                         y_code, pc, pcs, ws, bytes, stream)
                          : function_at<decltype(&qlin_fwd_act)>(a[0])(px, psx, pw, psw, pb, act, pr, r_code, M, N,
                                                                       K, py, y_code, pc, pcs, ws, bytes, stream));
        return PyTuple_Pack(3, y.o, ck->o, ck_s->o);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// backward(function, dy, ck, ck_s, act, gated, sw, sx, dz, dtype, s1, s2, db, want_db,
// workspace, stream) -> (dz, s1, s2, db)
PyObject *backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 16) {
        PyErr_SetString(PyExc_TypeError, "backward takes 16 arguments");
        return nullptr;
    }
    HANDLE_TH_ERRORS
    try {
        PyObject *dy = a[1];
        const auto [M, F] = two(dy, "dy");
        const bool gated = PyObject_IsTrue(a[5]);
        const int64_t N = gated ? 2 * F : F, per = (F + QLIN_CK_BLOCK - 1) / QLIN_CK_BLOCK * (gated ? 2 : 1);
        Args arg;
        int dy_code = 0, dz_code = 0;
        const void *pdy = arg(dy, "dy", dy_code, {M, F});
        const auto *pc = static_cast<const int8_t *>(arg(a[2], "ck", at::kChar, {M, N}));
        const auto *pcs = static_cast<const float *>(arg(a[3], "ck_s", at::kFloat, {M, per}));
        const int act = (int)PyLong_AsLong(a[4]);
        const Out dz(a[8], dy, type_of(a[9]), {M, N});
        void *pz = arg(dz.o, "dz", dz_code, {M, N});
        // A scale and what it is the scale of: both or neither.
        std::optional<Out> s[3];
        const float *p[2] = {nullptr, nullptr};
        float *out[3] = {nullptr, nullptr, nullptr};
        const char *names[3] = {"s1", "s2", "db"}, *of[2] = {"sw", "sx"};
        for (int k = 0; k < 3; k++) {
            const int64_t size = k == 0 ? M : N;
            if (k < 2 ? a[6 + k] != Py_None : PyObject_IsTrue(a[13]) || a[12] != Py_None) {
                if (k < 2)
                    p[k] = static_cast<const float *>(arg(a[6 + k], of[k], at::kFloat, {k == 0 ? N : M}));
                s[k].emplace(a[10 + k], dy, at::kFloat, std::initializer_list<int64_t>{size});
                out[k] = static_cast<float *>(arg(s[k]->o, names[k], at::kFloat, {size}));
            } else if (a[10 + k] != Py_None) {
                PyErr_Format(PyExc_ValueError, "%s needs %s", names[k], of[k]);
                throw Raised();
            } else {
                s[k].emplace(Py_None);
            }
        }
        size_t bytes;
        void *ws = workspace_of(arg, a[14], bytes);
        void *stream = PyLong_AsVoidPtr(a[15]);
        if (PyErr_Occurred())
            throw Raised();
        check("qlin_act_bwd", function_at<decltype(&qlin_act_bwd)>(a[0])(pdy, dy_code, pc, pcs, act, gated, p[0], p[1],
                                                                         M, F, pz, dz_code, out[0], out[1], out[2],
                                                                         ws, bytes, stream));
        return PyTuple_Pack(4, dz.o, s[0]->o, s[1]->o, s[2]->o);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_failed(PyObject *, PyObject *f)
{
    Py_INCREF(f);
    Py_XSETREF(failed, f);
    Py_RETURN_NONE;
}

PyObject *set_refuse(PyObject *, PyObject *f)
{
    Py_INCREF(f);
    Py_XSETREF(refuse, f);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"address", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(address)), METH_FASTCALL,
     "address(tensor, name, dtype, *sizes)"},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty)), METH_FASTCALL,
     "empty(like, dtype, *sizes)"},
    {"set_refuse", set_refuse, METH_O, "set_refuse(function)"},
    {"set_failed", set_failed, METH_O, "set_failed(function)"},
    {"forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(forward)), METH_FASTCALL,
     "a forward call inside a feed-forward block"},
    {"backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(backward)), METH_FASTCALL,
     "qlin_act_bwd"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
