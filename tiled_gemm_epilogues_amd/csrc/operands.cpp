// The checks of a run's tensors in one call (module _operands): Operands(specs) holds what a plan's operands
// must be, and calling it with the current device and the tensors gives their device pointers, or None where one of
// them does not fit (the caller then finds out which, and says so).  The checks are those of the
// binding's check(): type, device, contiguous, elements, the length of rows.  A run of the smallest sizes takes
// the GPU some 3 us; seven operands checked one by one from Python take as long.
#include <Python.h>

#include <vector>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

struct Spec {
    at::ScalarType type;
    int64_t need, row_len;       // elements; of a row (-1: any)
};

struct Operands {
    PyObject_HEAD
    vectorcallfunc call;
    std::vector<Spec> *specs;
};

// A new reference to the pointer of a tensor that fits (or what passes as it is), nullptr where it does not.
PyObject *pointer(const Spec &s, PyObject *t, int64_t device) {
    if (t == Py_None || PyLong_Check(t)) {
        Py_INCREF(t);
        return t;
    }
    if (!THPVariable_Check(t)) return nullptr;
    const at::Tensor &x = THPVariable_Unpack(t);
    if (x.scalar_type() != s.type || !x.is_cuda() || x.get_device() != device || !x.is_contiguous() || x.numel() < s.need) return nullptr;
    if (s.row_len >= 0 && x.dim() >= 2 && x.size(-1) != s.row_len) return nullptr;
    return PyLong_FromVoidPtr(x.data_ptr());
}

PyObject *call(PyObject *self, PyObject *const *args, size_t flags, PyObject *names) {
    const std::vector<Spec> &specs = *reinterpret_cast<Operands *>(self)->specs;
    const Py_ssize_t n = PyVectorcall_NARGS(flags);
    if (names || n != (Py_ssize_t)specs.size() + 1) {
        PyErr_SetString(PyExc_TypeError, "the device and one argument per operand");
        return nullptr;
    }
    const int64_t device = PyLong_AsLongLong(args[0]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    PyObject *out = PyTuple_New(n - 1);
    if (!out) return nullptr;
    for (Py_ssize_t i = 0; i + 1 < n; ++i) {
        PyObject *p = nullptr;
        try {
            p = pointer(specs[i], args[i + 1], device);
        } catch (...) {                              // (a tensor without storage or strides: not one that fits)
        }
        if (!p) {
            Py_DECREF(out);
            if (PyErr_Occurred()) return nullptr;
            Py_RETURN_NONE;
        }
        PyTuple_SET_ITEM(out, i, p);
    }
    return out;
}

PyObject *create(PyTypeObject *type, PyObject *args, PyObject *) {
    PyObject *list;
    if (!PyArg_ParseTuple(args, "O!", &PyTuple_Type, &list)) return nullptr;
    Operands *self = reinterpret_cast<Operands *>(type->tp_alloc(type, 0));   // (zeroed)
    if (!self) return nullptr;
    self->call = call;
    try {
        self->specs = new std::vector<Spec>();
        self->specs->reserve(PyTuple_GET_SIZE(list));    // (nothing below throws)
    } catch (...) {
        Py_DECREF(self);
        return PyErr_NoMemory();
    }
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(list); ++i) {
        PyObject *dtype, *row_len;
        long long need;
        if (!PyArg_ParseTuple(PyTuple_GET_ITEM(list, i), "OLO", &dtype, &need, &row_len) || !THPDtype_Check(dtype)) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "(dtype, elements, row length or None)");
            Py_DECREF(self);
            return nullptr;
        }
        const int64_t r = row_len == Py_None ? -1 : PyLong_AsLongLong(row_len);
        if (PyErr_Occurred()) {
            Py_DECREF(self);
            return nullptr;
        }
        self->specs->push_back({reinterpret_cast<THPDtype *>(dtype)->scalar_type, need, r});
    }
    return reinterpret_cast<PyObject *>(self);
}

void destroy(PyObject *self) {
    delete reinterpret_cast<Operands *>(self)->specs;
    Py_TYPE(self)->tp_free(self);
}

PyTypeObject operands_type = {PyVarObject_HEAD_INIT(nullptr, 0)};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operands", nullptr, -1, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operands() {
    operands_type.tp_name = "_operands.Operands";
    operands_type.tp_basicsize = sizeof(Operands);
    operands_type.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_VECTORCALL;
    operands_type.tp_vectorcall_offset = offsetof(Operands, call);
    operands_type.tp_call = PyVectorcall_Call;
    operands_type.tp_new = create;
    operands_type.tp_dealloc = destroy;
    if (PyType_Ready(&operands_type) < 0) return nullptr;
    PyObject *m = PyModule_Create(&module);
    if (!m) return nullptr;
    Py_INCREF(&operands_type);
    if (PyModule_AddObject(m, "Operands", reinterpret_cast<PyObject *>(&operands_type)) < 0) return nullptr;
    // (the binding uses the module with this torch only)
    if (PyModule_AddStringConstant(m, "torch_version", TGE_TORCH_VERSION) < 0) return nullptr;
    return m;
}
