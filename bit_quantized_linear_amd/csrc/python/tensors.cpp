// What the Python binding has to know of a call's tensors, looked at in one call: in
// Python each property of a tensor costs 50 to 100 ns, and an attention call has eleven
// tensors (5 of its 11 us on the host; with this 1). Nothing is decided here: a tensor
// that is not as the caller says gives None, and the binding then looks at each by
// itself and raises the error that fits.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// A plain tensor on GPU `device` with data of its own, or nullptr.
const at::Tensor *tensor_on(PyObject *o, long device) {
    if ((PyObject *)Py_TYPE(o) != THPVariableClass) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.defined() && t.layout() == at::kStrided && t.is_cuda() && t.get_device() == device ? &t : nullptr;
}

bool of_kind(const at::Tensor &t, PyObject *kind) {
    const unsigned long long mask = PyLong_AsUnsignedLongLong(kind);
    return mask >> static_cast<int>(t.scalar_type()) & 1;
}

// kind(*dtypes): the set of these types, for `pointers` and `heads`.
PyObject *kind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    unsigned long long mask = 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!THPDtype_Check(args[i])) {
            PyErr_SetString(PyExc_TypeError, "torch types are needed");
            return nullptr;
        }
        mask |= 1ull << static_cast<int>(reinterpret_cast<THPDtype *>(args[i])->scalar_type);
    }
    return PyLong_FromUnsignedLongLong(mask);
}

bool as_needed(const at::Tensor &t, PyObject *need) {
    if (PyLong_Check(need)) {
        const long long bytes = PyLong_AsLongLong(need);
        return !PyErr_Occurred() && (long long)t.nbytes() >= bytes;
    }
    if (!PyTuple_Check(need) || PyTuple_GET_SIZE(need) != t.dim()) return false;
    for (int64_t i = 0; i < t.dim(); ++i)
        if (PyLong_AsLongLong(PyTuple_GET_ITEM(need, i)) != t.size(i) || PyErr_Occurred()) return false;
    return true;
}

// pointers(device, t, kind, need, t, kind, need, ...): a tuple with each tensor's data
// pointer (None for None), or None if one is not a contiguous tensor on the device, of
// its kind, and of at least `need` bytes or of the shape `need`.
PyObject *pointers(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < 1 || n % 3 != 1) {
        PyErr_SetString(PyExc_TypeError, "pointers(device, tensor, kind, need, ...)");
        return nullptr;
    }
    const long device = PyLong_AsLong(args[0]);
    if (PyErr_Occurred()) return nullptr;
    PyObject *out = PyTuple_New(n / 3);
    if (!out) return nullptr;
    bool good = true;
    for (Py_ssize_t i = 0; good && i < n / 3; ++i) {
        PyObject *const *a = args + 1 + 3 * i;
        PyObject *item = nullptr;
        if (a[0] == Py_None) {
            Py_INCREF(Py_None);
            item = Py_None;
        } else {
            try {
                const at::Tensor *t = tensor_on(a[0], device);
                if (t && of_kind(*t, a[1]) && t->is_contiguous() && as_needed(*t, a[2]))
                    item = PyLong_FromVoidPtr(t->data_ptr());
            } catch (...) {  // the caller's own look says why
                item = nullptr;
            }
        }
        good = item != nullptr;
        if (good) PyTuple_SET_ITEM(out, i, item);
    }
    if (good) return out;
    Py_DECREF(out);
    PyErr_Clear();
    Py_RETURN_NONE;
}

// heads(device, kind, t): (data pointer, elements from row to row, T, H, D) of heads
// [T, H, D] whose rows are contiguous and at least a row apart; None if they are not.
PyObject *heads(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "heads(device, kind, tensor)");
        return nullptr;
    }
    const long device = PyLong_AsLong(args[0]);
    if (PyErr_Occurred()) return nullptr;
    try {
        const at::Tensor *t = tensor_on(args[2], device);
        if (t && of_kind(*t, args[1]) && t->dim() == 3) {
            const int64_t T = t->size(0), H = t->size(1), D = t->size(2), width = H * D;
            const int64_t row = T <= 1 || width == 0 ? (width + 7) / 8 * 8 : t->stride(0);  // there may be no next row
            if (row >= width && (t->stride(2) == 1 || D <= 1) && (t->stride(1) == D || H <= 1))
                return Py_BuildValue("NLLLL", PyLong_FromVoidPtr(t->data_ptr()), (long long)row, (long long)T, (long long)H,
                                     (long long)D);
        }
    } catch (...) {
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"kind", (PyCFunction)(void (*)(void))kind, METH_FASTCALL, "the set of some types"},
    {"pointers", (PyCFunction)(void (*)(void))pointers, METH_FASTCALL, "data pointers of tensors that are as they must be"},
    {"heads", (PyCFunction)(void (*)(void))heads, METH_FASTCALL, "data pointer, stride and shape of heads"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for names the Python and torch of the headers above: their structures may be
// others elsewhere, and the caller does without the module there.
PyMODINIT_FUNC PyInit__tensors() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
