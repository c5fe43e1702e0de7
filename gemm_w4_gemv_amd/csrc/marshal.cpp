// The tensor checks of the Python binding's small calls, compiled: a call of
// ten tensors spends longer asking for their types, shapes and addresses
// through Python than its kernel runs (tables of a step 7.6 us of host time
// with the checks in Python, 5.6 with these).
//
// Each function takes what the Python function of the same name in step.py (rows:
// in block.py) takes and gives what that gives; where a tensor is not as it should be it
// calls that function, which says what is wrong.  The module's ``built_for``
// names the torch (W4_BUILT_FOR, from the build) and the Python that it fits.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* slow_addresses = nullptr;
PyObject* slow_optional = nullptr;
PyObject* slow_heads = nullptr;
PyObject* slow_rows = nullptr;

// A dense tensor on GPU ``device``, or NULL.
const at::Tensor* tensor_on(PyObject* o, long device) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device) return nullptr;
    return &t;
}

// addresses(device, tensor, name, dtype, n, tensor, name, dtype, n, ...):
// the address of each contiguous tensor, n its length if it has to be a vector.
// optional_addresses: None for None.
template <bool kOptional>
PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t count) {
    const auto slow = [&] {
        return PyObject_Vectorcall(kOptional ? slow_optional : slow_addresses, args, (size_t)count, nullptr);
    };
    if (count < 1 || (count - 1) % 4) return slow();
    const long device = PyLong_AsLong(args[0]);
    if (device == -1 && PyErr_Occurred()) PyErr_Clear();
    const Py_ssize_t n = (count - 1) / 4;
    PyObject* out = PyTuple_New(n);
    if (!out) return nullptr;
    bool good = device >= 0;
    try {
        for (Py_ssize_t i = 0; good && i < n; ++i) {
            PyObject* const* a = args + 1 + 4 * i;
            if (kOptional && a[0] == Py_None) {
                Py_INCREF(Py_None);
                PyTuple_SET_ITEM(out, i, Py_None);
                continue;
            }
            const at::Tensor* t = tensor_on(a[0], device);
            good = t && THPDtype_Check(a[2]) && t->scalar_type() == reinterpret_cast<THPDtype*>(a[2])->scalar_type &&
                   t->is_contiguous();
            if (good && a[3] != Py_None) {
                const long long length = PyLong_AsLongLong(a[3]);
                if (length == -1 && PyErr_Occurred()) PyErr_Clear();
                good = t->dim() == 1 && t->size(0) == length;
            }
            if (good) {
                PyObject* address = PyLong_FromVoidPtr(t->data_ptr());
                good = address != nullptr;
                if (address) PyTuple_SET_ITEM(out, i, address);
            }
        }
    } catch (...) {
        good = false;
    }
    if (good) return out;
    Py_DECREF(out);
    PyErr_Clear();
    return slow();
}

// heads(t, name, device, rows, heads, dim): (address, row stride) of a BF16
// tensor [rows, heads, dim] whose heads lie together; None: any.
PyObject* heads(PyObject*, PyObject* const* args, Py_ssize_t count) {
    const auto slow = [&] { return PyObject_Vectorcall(slow_heads, args, (size_t)count, nullptr); };
    if (count < 3 || count > 6) return slow();
    const long device = PyLong_AsLong(args[2]);
    if (device == -1 && PyErr_Occurred()) PyErr_Clear();
    if (device < 0) return slow();
    try {
        const at::Tensor* t = tensor_on(args[0], device);
        if (!t || t->dim() != 3 || t->scalar_type() != at::kBFloat16) return slow();
        for (Py_ssize_t i = 3; i < count; ++i) {
            if (args[i] == Py_None) continue;
            const long long want = PyLong_AsLongLong(args[i]);
            if (want == -1 && PyErr_Occurred()) PyErr_Clear();
            if (t->size(i - 3) != want) return slow();
        }
        const int64_t n = t->size(0), h = t->size(1), d = t->size(2);
        if ((d > 1 && t->stride(2) != 1) || (h > 1 && t->stride(1) != d)) return slow();
        const int64_t step = n <= 1 ? std::max<int64_t>(h * d, 8) : t->stride(0);
        return Py_BuildValue("NL", PyLong_FromVoidPtr(t->data_ptr()), (long long)step);
    } catch (...) {
        return slow();
    }
}

// rows(device, n, wide, tensor, name, dtype, tensor, name, dtype, ...): address and row
// stride, one behind the other, of each tensor [n, wide] whose rows' values lie
// together; (None, 0) for None.
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t count) {
    const auto slow = [&] { return PyObject_Vectorcall(slow_rows, args, (size_t)count, nullptr); };
    if (count < 3 || count % 3) return slow();
    long long size[3];
    for (int i = 0; i < 3; ++i) {
        size[i] = PyLong_AsLongLong(args[i]);
        if (size[i] == -1 && PyErr_Occurred()) PyErr_Clear();
        if (size[i] < 0) return slow();
    }
    const int64_t n = size[1], wide = size[2];
    const Py_ssize_t tensors = count / 3 - 1;
    PyObject* out = PyTuple_New(2 * tensors);
    if (!out) return nullptr;
    bool good = true;
    try {
        for (Py_ssize_t i = 0; good && i < tensors; ++i) {
            PyObject* const* a = args + 3 + 3 * i;
            PyObject *address = nullptr, *stride = nullptr;
            if (a[0] == Py_None) {
                Py_INCREF(Py_None);
                address = Py_None;
                stride = PyLong_FromLong(0);
            } else {
                const at::Tensor* t = tensor_on(a[0], (long)size[0]);
                good = t && THPDtype_Check(a[2]) && t->scalar_type() == reinterpret_cast<THPDtype*>(a[2])->scalar_type &&
                       t->dim() == 2 && t->size(0) == n && t->size(1) == wide && (n == 0 || wide <= 1 || t->stride(1) == 1);
                if (!good) break;
                address = PyLong_FromVoidPtr(t->data_ptr());
                stride = PyLong_FromLongLong(n > 1 ? (long long)t->stride(0) : std::max<long long>(wide, 8));
            }
            good = address && stride;
            if (address) PyTuple_SET_ITEM(out, 2 * i, address);
            if (stride) PyTuple_SET_ITEM(out, 2 * i + 1, stride);
        }
    } catch (...) {
        good = false;
    }
    if (good) return out;
    Py_DECREF(out);
    PyErr_Clear();
    return slow();
}

// begin(addresses, optional_addresses, heads), begin_rows(rows): the Python
// functions to fall back on.
PyObject* begin(PyObject*, PyObject* const* args, Py_ssize_t count) {
    if (count != 3) {
        PyErr_SetString(PyExc_TypeError, "begin(addresses, optional_addresses, heads)");
        return nullptr;
    }
    PyObject** to[] = {&slow_addresses, &slow_optional, &slow_heads};
    for (int i = 0; i < 3; ++i) {
        PyObject* old = *to[i];
        Py_INCREF(args[i]);
        *to[i] = args[i];
        Py_XDECREF(old);
    }
    Py_RETURN_NONE;
}

PyObject* begin_rows(PyObject*, PyObject* const* args, Py_ssize_t count) {
    if (count != 1) {
        PyErr_SetString(PyExc_TypeError, "begin_rows(rows)");
        return nullptr;
    }
    PyObject* old = slow_rows;
    Py_INCREF(args[0]);
    slow_rows = args[0];
    Py_XDECREF(old);
    Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<addresses<false>>("addresses"), method<addresses<true>>("optional_addresses"),
                         method<heads>("heads"), method<begin>("begin"), method<rows>("rows"),
                         method<begin_rows>("begin_rows"), {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject* m = PyModule_Create(&module);
    PyObject* built_for = m ? Py_BuildValue("(si)", W4_BUILT_FOR, (int)(PY_VERSION_HEX >> 16)) : nullptr;
    if (!built_for || PyModule_AddObject(m, "built_for", built_for)) {
        Py_XDECREF(built_for);
        Py_XDECREF(m);
        return nullptr;
    }
    return m;
}
