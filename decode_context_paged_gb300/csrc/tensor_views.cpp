// tensor_views.cpp -- the binding's questions to torch tensors, and its calls of the library, in C++.
//
// A call of the library names up to 25 tensors, and asking each for its type, device, shape and
// pointer from Python costs about half a microsecond a tensor: more than the call itself for a
// decode step's small operators.  These functions answer for tensors that are as the call wants
// them and return None otherwise; the binding then asks again in Python and raises the error, so
// what is accepted is said in one place.  An exception that torch throws (a tensor without storage, as
// inside torch.vmap) becomes the Python error that the same question gives there.  Outputs are allocated here too (1.3 us against torch.empty's
// 1.7), and the serving calls go to the library without ctypes, which takes 1.5 to 3 us to convert 15
// to 30 arguments: a call of append 16 -> 11.5 us, prompt attention 20 -> 11, decode 41 -> 30, scales
// 6.5 -> 5.  The module is optional.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>
#include <torch/version.h>

#include <dlfcn.h>

#include <cstdint>
#include <tuple>
#include <type_traits>
#include <utility>

#include "dcp.h"

namespace {

PyObject *none() { Py_RETURN_NONE; }

bool is_tensor(PyObject *o) { return THPVariable_Check(o); }

bool fits(const at::Tensor &t, at::ScalarType type, long dev) {
    return t.layout() == at::kStrided && t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.is_contiguous();
}

bool read_type(PyObject *o, at::ScalarType *type) {
    if (!THPDtype_Check(o)) return false;
    *type = reinterpret_cast<THPDtype *>(o)->scalar_type;
    return true;
}

// ptr(tensor, dtype, device) -> address of a contiguous tensor, or None
PyObject *ptr(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    at::ScalarType type;
    if (n != 3 || !is_tensor(args[0]) || !read_type(args[1], &type)) return none();
    const at::Tensor &t = THPVariable_Unpack(args[0]);
    if (!fits(t, type, PyLong_AsLong(args[2]))) return none();
    return PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t.data_ptr()));
    END_HANDLE_TH_ERRORS
}

// ptrs(list, like, dtype, device) -> bytes of the addresses of contiguous tensors of like's shape, or None
PyObject *ptrs(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    at::ScalarType type;
    if (n != 4 || !PyList_Check(args[0]) || !is_tensor(args[1]) || !read_type(args[2], &type)) return none();
    const long dev = PyLong_AsLong(args[3]);
    const at::IntArrayRef shape = THPVariable_Unpack(args[1]).sizes();
    const Py_ssize_t count = PyList_GET_SIZE(args[0]);
    THPObjectPtr out(PyBytes_FromStringAndSize(nullptr, count * 8));
    if (!out) return nullptr;
    uint64_t *p = reinterpret_cast<uint64_t *>(PyBytes_AS_STRING(out.get()));
    for (Py_ssize_t i = 0; i < count; ++i) {
        PyObject *o = PyList_GET_ITEM(args[0], i);
        if (!is_tensor(o) || !fits(THPVariable_Unpack(o), type, dev) || THPVariable_Unpack(o).sizes() != shape) return none();
        p[i] = reinterpret_cast<uintptr_t>(THPVariable_Unpack(o).data_ptr());
    }
    return out.release();
    END_HANDLE_TH_ERRORS
}

// rows(tensor, width, dims, multiple, device) -> (address, outer strides...) of BF16 rows, or None
PyObject *rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 5 || !is_tensor(args[0])) return none();
    const at::Tensor &t = THPVariable_Unpack(args[0]);
    const long width = PyLong_AsLong(args[1]), dims = PyLong_AsLong(args[2]), mult = PyLong_AsLong(args[3]);
    if (t.layout() != at::kStrided || t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != PyLong_AsLong(args[4]) ||
        t.dim() != dims || (dims != 2 && dims != 3) || t.size(dims - 1) != width || t.stride(dims - 1) != 1)
        return none();
    const int64_t s0 = t.size(0) > 1 ? t.stride(0) : width;
    const int64_t s1 = dims == 2 ? mult : t.size(1) > 1 ? t.stride(1) : width;
    const uintptr_t p = reinterpret_cast<uintptr_t>(t.data_ptr());
    if (s0 % mult || s1 % mult || p % (2 * mult)) return none();
    if (dims == 2) return Py_BuildValue("KL", (unsigned long long)p, (long long)s0);
    return Py_BuildValue("KLL", (unsigned long long)p, (long long)s0, (long long)s1);
    END_HANDLE_TH_ERRORS
}

// empty(shape, dtype, device) -> a new contiguous tensor on that GPU, or None
PyObject *empty(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    at::ScalarType type;
    if (n != 3 || !PyTuple_Check(args[0]) || !read_type(args[1], &type) || !PyLong_Check(args[2])) return none();
    const long dev = PyLong_AsLong(args[2]);
    const Py_ssize_t dims = PyTuple_GET_SIZE(args[0]);
    int64_t shape[8];
    if (dims > 8 || dev < 0 || dev > 127) return none();
    for (Py_ssize_t i = 0; i < dims; ++i) {
        PyObject *x = PyTuple_GET_ITEM(args[0], i);
        if (!PyLong_Check(x)) return none();
        shape[i] = PyLong_AsLongLong(x);
        if (PyErr_Occurred()) return nullptr;
    }
    return THPVariable_Wrap(at::empty(at::IntArrayRef(shape, dims),
                                      at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))));
    END_HANDLE_TH_ERRORS
}

// The library's entry points, called with Python values: integers and bools, floats, addresses as
// integers, bytes for host arrays, None for null.
template <typename T>
T value(PyObject *o) {
    if constexpr (std::is_pointer_v<T>) {
        if (o == Py_None) return nullptr;
        if (PyBytes_Check(o)) return reinterpret_cast<T>(PyBytes_AS_STRING(o));
        return reinterpret_cast<T>(PyLong_AsUnsignedLongLong(o));
    } else if constexpr (std::is_floating_point_v<T>) {
        return static_cast<T>(PyFloat_AsDouble(o));
    } else {
        return static_cast<T>(PyLong_AsLongLong(o));
    }
}

template <typename F>
struct Call;
template <typename R, typename... A>
struct Call<R (*)(A...)> {
    template <size_t... I>
    static PyObject *run(R (*fn)(A...), PyObject *const *args, std::index_sequence<I...>) {
        std::tuple<A...> v{value<A>(args[I])...};
        if (PyErr_Occurred()) return nullptr;
        R r;
        Py_BEGIN_ALLOW_THREADS
        r = fn(std::get<I>(v)...);
        Py_END_ALLOW_THREADS
        return PyLong_FromLongLong(static_cast<long long>(r));
    }
    static PyObject *run(R (*fn)(A...), PyObject *const *args, Py_ssize_t n) {
        if (!fn || n != static_cast<Py_ssize_t>(sizeof...(A))) {
            PyErr_SetString(PyExc_TypeError, fn ? "wrong number of arguments" : "the library is not open");
            return nullptr;
        }
        return run(fn, args, std::index_sequence_for<A...>{});
    }
};

// (declared types only: the functions come from the library that the binding loaded)
#define DCP_CALLS(X)                           \
    X(dcp_append_kv)                           \
    X(dcp_reshard_scales)                      \
    X(dcp_partial_decode_attn_workspace_size)  \
    X(dcp_partial_decode_attn_scaled)          \
    X(dcp_decode_attn_merged_scaled)           \
    X(dcp_prefill_attn_workspace_size)         \
    X(dcp_prefill_attn)
#define DCP_FORWARD(name)                                                                  \
    decltype(&::name) name##_fn = nullptr;                                                 \
    PyObject *name##_call(PyObject *, PyObject *const *args, Py_ssize_t n) {               \
        return Call<decltype(&::name)>::run(name##_fn, args, n);                           \
    }
DCP_CALLS(DCP_FORWARD)

// open(handle): the entry points above of a loaded library (its dlopen handle); False if one is missing
PyObject *open(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void *lib = n == 1 ? PyLong_AsVoidPtr(args[0]) : nullptr;
    if (PyErr_Occurred()) return nullptr;
    bool all = lib != nullptr;
#define DCP_FIND(name)                                                                     \
    if (lib) name##_fn = reinterpret_cast<decltype(&::name)>(dlsym(lib, #name));           \
    all = all && name##_fn;
    DCP_CALLS(DCP_FIND)
    return PyBool_FromLong(all);
}

#define DCP_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name##_call)), METH_FASTCALL, nullptr},

PyMethodDef methods[] = {
    {"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ptr)), METH_FASTCALL, nullptr},
    {"ptrs", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ptrs)), METH_FASTCALL, nullptr},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rows)), METH_FASTCALL, nullptr},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty)), METH_FASTCALL, nullptr},
    {"open", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(open)), METH_FASTCALL, nullptr},
    DCP_CALLS(DCP_METHOD)
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_views", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_views(void) {
    PyObject *m = PyModule_Create(&module);
    // what the layouts that this file was compiled with belong to: the binding uses no other
    if (m && (PyModule_AddStringConstant(m, "built_for_torch", TORCH_VERSION) < 0 ||
              PyModule_AddIntConstant(m, "built_for_python", PY_VERSION_HEX >> 16) < 0)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
