// py_args.cpp -- argument checks of the Python binding in native code: one call
// looks at all tensors of a library call and returns their addresses, at some
// 30 ns a tensor instead of 350 ns for the same checks in Python (a small
// norm or decode call is otherwise bound by them).  It decides nothing by
// itself: where a check fails, the binding repeats the checks in Python, which
// name the argument and raise.  So does an exception of torch's (a tensor
// without storage, as under torch.vmap, has no address to give): none may
// leave this C entry.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// Bits of the types that the binding distinguishes.
long type_bit(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return 1;
    case at::kFloat: return 2;
    case at::kByte: return 4;
    case at::kFloat8_e4m3fn: return 8;
    case at::kInt: return 16;
    default: return 0;
    }
}

// addresses(device, t0, types0, shape0, t1, types1, shape1, ..): the data
// addresses of the tensors (None for None), each a dense tensor on the device,
// of one of its types (bits above) and of its shape; None as soon as one is not.
PyObject *addresses(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < 1 || (n - 1) % 3 != 0) {
        PyErr_SetString(PyExc_TypeError, "addresses(device, tensor, types, shape, ...)");
        return nullptr;
    }
    const long device = PyLong_AsLong(args[0]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    const Py_ssize_t count = (n - 1) / 3;
    PyObject *out = PyTuple_New(count);
    if (!out) return nullptr;
    for (Py_ssize_t k = 0; k < count; ++k) {
        PyObject *t = args[1 + 3 * k], *types = args[2 + 3 * k], *shape = args[3 + 3 * k];
        PyObject *value = nullptr;
        if (t == Py_None) {
            Py_INCREF(Py_None);
            value = Py_None;
        } else if (THPVariable_Check(t) && PyTuple_Check(shape)) {
            const at::Tensor &v = THPVariable_Unpack(t);
            const long mask = PyLong_AsLong(types);
            if (mask == -1 && PyErr_Occurred()) {
                Py_DECREF(out);
                return nullptr;
            }
            bool ok = false;
            void *data = nullptr;
            try {
                ok = v.defined() && v.layout() == at::kStrided && v.is_cuda() && v.get_device() == device &&
                     (type_bit(v.scalar_type()) & mask) != 0 && v.dim() == PyTuple_GET_SIZE(shape) && v.is_contiguous();
                for (Py_ssize_t d = 0; ok && d < v.dim(); ++d) {
                    const long want = PyLong_AsLong(PyTuple_GET_ITEM(shape, d));
                    if (want == -1 && PyErr_Occurred()) {
                        Py_DECREF(out);
                        return nullptr;
                    }
                    ok = v.size(d) == want;
                }
                // an empty tensor has no address: NULL, as the library takes it
                if (ok && v.numel()) data = v.data_ptr();
            } catch (...) {
                PyErr_Clear();
                ok = false;
            }
            if (ok) {
                value = PyLong_FromVoidPtr(data);
                if (!value) {
                    Py_DECREF(out);
                    return nullptr;
                }
            }
        }
        if (!value) {
            Py_DECREF(out);
            Py_RETURN_NONE;
        }
        PyTuple_SET_ITEM(out, k, value);
    }
    return out;
}

PyMethodDef methods[] = {
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(addresses)), METH_FASTCALL,
     "addresses(device, t0, types0, shape0, ...) -> addresses of dense device tensors, or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_args", "Argument checks of the binding.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__args(void) { return PyModule_Create(&module); }
