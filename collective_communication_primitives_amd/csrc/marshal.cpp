// marshal.cpp -- the host side of the Python binding of the model-step
// operators: a list of tensors checked and turned into the array of device
// pointers that the C ABI takes, without a Python call per tensor and
// property.  It only looks at tensors; it touches no device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// A borrowed reference to item i of a list or tuple.
PyObject* item(PyObject* seq, Py_ssize_t i) { return PyList_Check(seq) ? PyList_GET_ITEM(seq, i) : PyTuple_GET_ITEM(seq, i); }
bool sequence(PyObject* o) { return PyList_Check(o) || PyTuple_Check(o); }

// buffers(tensors, sizes, dtype, device, stash) -> bytes of pointers, or None
// when a tensor is not a contiguous one of that dtype and size on that device
// (the caller then says which).  The tensors join the list `stash`.
PyObject* buffers(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 5 || !PyList_Check(args[1]) || !THPDtype_Check(args[2]) || !PyList_Check(args[4])) {
        PyErr_SetString(PyExc_TypeError, "buffers(tensors, sizes, dtype, device, stash)");
        return nullptr;
    }
    PyObject* tensors = args[0];
    if (!sequence(tensors)) Py_RETURN_NONE;
    const Py_ssize_t p = PyList_GET_SIZE(args[1]);
    if (Py_SIZE(tensors) != p) Py_RETURN_NONE;
    const at::ScalarType dtype = reinterpret_cast<THPDtype*>(args[2])->scalar_type;
    const long device = PyLong_AsLong(args[3]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    PyObject* out = PyBytes_FromStringAndSize(nullptr, p * Py_ssize_t(sizeof(void*)));
    if (out == nullptr) return nullptr;
    void** ptrs = reinterpret_cast<void**>(PyBytes_AS_STRING(out));
    try {
        for (Py_ssize_t i = 0; i < p; i++) {
            PyObject* o = item(tensors, i);
            const long long want = PyLong_AsLongLong(PyList_GET_ITEM(args[1], i));
            if (want == -1 && PyErr_Occurred()) {
                Py_DECREF(out);
                return nullptr;
            }
            bool ok = THPVariable_Check(o);
            if (ok) {
                const at::Tensor& t = THPVariable_Unpack(o);
                ok = t.scalar_type() == dtype && t.numel() == want && t.get_device() == device && t.is_contiguous();
                if (ok) ptrs[i] = t.data_ptr();
            }
            if (!ok) {
                Py_DECREF(out);
                Py_RETURN_NONE;
            }
        }
    } catch (const std::exception& e) {
        Py_DECREF(out);
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < p; i++)
        if (PyList_Append(args[4], item(tensors, i)) != 0) {
            Py_DECREF(out);
            return nullptr;
        }
    return out;
}

// counts(tensors, cols, times) -> (elements, rows, rows * times, bytes of rows),
// or None when a tensor does not hold whole rows of cols elements.
PyObject* counts(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 3 || !sequence(args[0])) Py_RETURN_NONE;
    const long long cols = PyLong_AsLongLong(args[1]), times = PyLong_AsLongLong(args[2]);
    if (PyErr_Occurred()) return nullptr;
    if (cols < 1) Py_RETURN_NONE;
    const Py_ssize_t p = Py_SIZE(args[0]);
    PyObject *sizes = PyList_New(p), *rows = PyList_New(p), *more = PyList_New(p);
    PyObject* packed = PyBytes_FromStringAndSize(nullptr, p * Py_ssize_t(sizeof(size_t)));
    bool ok = sizes != nullptr && rows != nullptr && more != nullptr && packed != nullptr;
    PyObject* out = nullptr;
    try {
        for (Py_ssize_t i = 0; ok && i < p; i++) {
            PyObject* o = item(args[0], i);
            ok = THPVariable_Check(o);
            if (!ok) break;
            const long long size = THPVariable_Unpack(o).numel();
            ok = size % cols == 0;
            if (!ok) break;
            PyObject *a = PyLong_FromLongLong(size), *b = PyLong_FromLongLong(size / cols), *c = PyLong_FromLongLong(size / cols * times);
            ok = a != nullptr && b != nullptr && c != nullptr;
            PyList_SET_ITEM(sizes, i, a);
            PyList_SET_ITEM(rows, i, b);
            PyList_SET_ITEM(more, i, c);
            reinterpret_cast<size_t*>(PyBytes_AS_STRING(packed))[i] = size_t(size / cols);
        }
        if (ok) out = PyTuple_Pack(4, sizes, rows, more, packed);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    Py_XDECREF(sizes);
    Py_XDECREF(rows);
    Py_XDECREF(more);
    Py_XDECREF(packed);
    if (out != nullptr || PyErr_Occurred()) return out;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"buffers", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(buffers)), METH_FASTCALL, "device pointers of a list of tensors"},
    {"counts", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(counts)), METH_FASTCALL, "row counts of a list of tensors"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the build that the tensors' layout was compiled against.
PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", DT_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
