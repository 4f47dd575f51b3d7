// Python binding of the calls that a decode step makes (the paged appends with
// the rotary embedding and the attentions over 8-bit pages). Their kernels take
// 7 to 9 us, less than ctypes and per-tensor checks in Python need: here a
// tensor goes in as itself, is checked and read in tens of nanoseconds, and the
// C entry is called with the interpreter lock released. Arguments, statuses and
// errors are those of the C ABI; the package raises on a status as it does for
// every other call.
#include <ATen/ATen.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "loki.h"

namespace {

// one Python argument as a C one; false with an exception set
template <class T>
bool from_py(PyObject* o, T* out) {
    if constexpr (std::is_pointer_v<T>) {
        if (o == Py_None) {
            *out = nullptr;
            return true;
        }
        if (THPVariable_Check(o)) {
            *out = reinterpret_cast<T>(THPVariable_Unpack(o).data_ptr());
            return true;
        }
        *out = reinterpret_cast<T>(PyLong_AsVoidPtr(o));
        return !PyErr_Occurred();
    } else if constexpr (std::is_floating_point_v<T>) {
        *out = static_cast<T>(PyFloat_AsDouble(o));
        return !PyErr_Occurred();
    } else {
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) return false;
        if constexpr (sizeof(T) == 4) {
            if (v < INT32_MIN || v > INT32_MAX) {
                PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
                return false;
            }
        }
        *out = static_cast<T>(v);
        return true;
    }
}

template <auto F>
struct Call;

template <class R, class... A, R (*F)(A...)>
struct Call<F> {
    static PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t n) {
        return with(args, n, std::index_sequence_for<A...>());
    }
    template <size_t... I>
    static PyObject* with(PyObject* const* args, Py_ssize_t n, std::index_sequence<I...>) {
        HANDLE_TH_ERRORS
        if (n != (Py_ssize_t)sizeof...(A))
            return PyErr_Format(PyExc_TypeError, "%zd arguments expected (got %zd)", (Py_ssize_t)sizeof...(A), n);
        std::tuple<A...> a;
        if (!(from_py(args[I], &std::get<I>(a)) && ...)) return nullptr;
        R r;
        Py_BEGIN_ALLOW_THREADS;
        r = F(std::get<I>(a)...);
        Py_END_ALLOW_THREADS;
        if constexpr (std::is_same_v<R, size_t>) return PyLong_FromSize_t(r);
        else return PyLong_FromLong(static_cast<long>(r));
        END_HANDLE_TH_ERRORS
    }
};

// place(*tensors): the index of the CUDA device they share; None is skipped
PyObject* place(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int device = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (args[i] == Py_None) continue;
        if (!THPVariable_Check(args[i])) return PyErr_Format(PyExc_TypeError, "tensors expected");
        const at::Tensor& t = THPVariable_Unpack(args[i]);
        if (!t.is_cuda()) return PyErr_Format(PyExc_ValueError, "all tensors must be CUDA tensors");
        if (device >= 0 && t.get_device() != device)
            return PyErr_Format(PyExc_ValueError, "all tensors must be on the same device");
        if (!t.is_contiguous()) return PyErr_Format(PyExc_ValueError, "all tensors must be contiguous");
        device = t.get_device();
    }
    return PyLong_FromLong(device);
    END_HANDLE_TH_ERRORS
}

// fits(t, dtype, d0, d1, ...): whether t is a tensor of this type and shape
PyObject* fits(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n < 2 || !THPVariable_Check(args[0]) || !THPDtype_Check(args[1]))
        return PyErr_Format(PyExc_TypeError, "fits(tensor, dtype, *shape)");
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    bool ok = t.scalar_type() == reinterpret_cast<THPDtype*>(args[1])->scalar_type && t.dim() == n - 2;
    for (Py_ssize_t i = 2; ok && i < n; ++i) {
        const long long d = PyLong_AsLongLong(args[i]);
        if (d == -1 && PyErr_Occurred()) return nullptr;
        ok = t.size(i - 2) == d;
    }
    return PyBool_FromLong(ok);
    END_HANDLE_TH_ERRORS
}

// scratch(like, nbytes): uninitialised bytes on like's device
PyObject* scratch(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 2 || !THPVariable_Check(args[0])) return PyErr_Format(PyExc_TypeError, "scratch(like, nbytes)");
    const long long bytes = PyLong_AsLongLong(args[1]);
    if (bytes == -1 && PyErr_Occurred()) return nullptr;
    const at::Tensor& like = THPVariable_Unpack(args[0]);
    return THPVariable_Wrap(at::empty({bytes}, like.options().dtype(at::kByte)));
    END_HANDLE_TH_ERRORS
}

// empty_like(t[, dtype]): an uninitialised contiguous tensor of t's shape
PyObject* empty_like(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n < 1 || n > 2 || !THPVariable_Check(args[0]) || (n == 2 && !THPDtype_Check(args[1])))
        return PyErr_Format(PyExc_TypeError, "empty_like(tensor[, dtype])");
    const at::Tensor& like = THPVariable_Unpack(args[0]);
    at::TensorOptions o = like.options();
    if (n == 2) o = o.dtype(reinterpret_cast<THPDtype*>(args[1])->scalar_type);
    return THPVariable_Wrap(at::empty(like.sizes(), o));
    END_HANDLE_TH_ERRORS
}

#define LOKI_CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&Call<&f>::run)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"place", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&place)), METH_FASTCALL, nullptr},
    {"fits", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&fits)), METH_FASTCALL, nullptr},
    {"scratch", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&scratch)), METH_FASTCALL, nullptr},
    {"empty_like", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&empty_like)), METH_FASTCALL, nullptr},
    LOKI_CALL(loki_rope_table),
    LOKI_CALL(loki_append_keys_paged_rope),
    LOKI_CALL(loki_append_keys_paged_q8),
    LOKI_CALL(dense_decode_attention_paged_q8),
    LOKI_CALL(loki_sparse_attention_paged_q8),
    LOKI_CALL(loki_decode_attention_paged_q8),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
