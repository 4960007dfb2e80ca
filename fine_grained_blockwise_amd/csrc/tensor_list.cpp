// tensor_list.cpp -- what the binding needs to know of a list of tensors, in one call.
//
// describe(list) -> (addresses, lengths, types, device): int64, int64 and int32 arrays as
// bytes objects, one entry a tensor, types as in fgb.h (FGB_F32, FGB_BF16), the GPU's index
// all tensors share.  Raises TypeError for what is no FP32 or BF16 tensor, ValueError for a
// tensor that is not on that GPU or not contiguous.  (Asked one by one in Python a tensor's
// properties cost 0.4 us, 100 us for the gradients and outputs of 122 tensors.)
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fgb.h"

static PyObject *describe(PyObject *, PyObject *arg)
{
    PyObject *seq = PySequence_Fast(arg, "expected a list of tensors");
    if (!seq)
        return nullptr;
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    PyObject *at = PyBytes_FromStringAndSize(nullptr, 8 * n), *len = PyBytes_FromStringAndSize(nullptr, 8 * n);
    PyObject *type = PyBytes_FromStringAndSize(nullptr, 4 * n), *result = nullptr;
    long device = -1;
    if (!at || !len || !type)
        goto done;
    for (Py_ssize_t i = 0; i < n; i++) {
        PyObject *item = PySequence_Fast_GET_ITEM(seq, i);
        if (!THPVariable_Check(item)) {
            PyErr_Format(PyExc_TypeError, "entry %zd is no tensor", i);
            goto done;
        }
        try { // (what torch throws must not cross into the interpreter)
            const at::Tensor &t = THPVariable_Unpack(item);
            if (!t.is_cuda()) {
                PyErr_SetString(PyExc_ValueError, "all tensors must be on the GPU");
                goto done;
            }
            const long on = t.get_device();
            if (device >= 0 && on != device) {
                PyErr_SetString(PyExc_ValueError, "all tensors must be on the same GPU");
                goto done;
            }
            device = on;
            const at::ScalarType s = t.scalar_type();
            if (s != at::kFloat && s != at::kBFloat16) {
                PyErr_Format(PyExc_TypeError, "entry %zd: expected float32 or bfloat16", i);
                goto done;
            }
            if (!t.is_contiguous()) {
                PyErr_Format(PyExc_ValueError, "entry %zd must be contiguous", i);
                goto done;
            }
            ((int64_t *)PyBytes_AS_STRING(at))[i] = (int64_t)t.data_ptr();
            ((int64_t *)PyBytes_AS_STRING(len))[i] = t.numel();
            ((int32_t *)PyBytes_AS_STRING(type))[i] = s == at::kFloat ? FGB_F32 : FGB_BF16;
        } catch (const std::exception &e) {
            PyErr_Format(PyExc_ValueError, "entry %zd: %s", i, e.what());
            goto done;
        }
    }
    result = Py_BuildValue("(OOOl)", at, len, type, device);
done:
    Py_XDECREF(at);
    Py_XDECREF(len);
    Py_XDECREF(type);
    Py_DECREF(seq);
    return result;
}

static PyMethodDef methods[] = {{"describe", describe, METH_O, "addresses, lengths, types and device of a list of tensors"},
                                {nullptr, nullptr, 0, nullptr}};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
