// tensor_list.cpp -- what the binding does with several tensors in one call.
//
// describe(list) -> (addresses, lengths, types, device): int64, int64 and int32 arrays as
// bytes objects, one entry a tensor, types as in fgb.h (FGB_F32, FGB_BF16), the GPU's index
// all tensors share.  Raises TypeError for what is no FP32 or BF16 tensor, ValueError for a
// tensor that is not on that GPU or not contiguous.  (Asked one by one in Python a tensor's
// properties cost 0.4 us, 100 us for the gradients and outputs of 122 tensors.)
//
// empties(tensor, (kind, sizes...), ...) -> uninitialised tensors on the given one's device, of
// kind 0 float32, 1 bfloat16, 2 uint8, 3 int32.  (torch.empty costs 1.3 us from Python, 0.5 us
// here.)
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "../../include/fgb.h"

static PyObject *describe(PyObject *, PyObject *arg)
{
    HANDLE_TH_ERRORS
    THPObjectPtr seq(PySequence_Fast(arg, "expected a list of tensors"));
    if (!seq)
        return nullptr;
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq.get());
    THPObjectPtr at(PyBytes_FromStringAndSize(nullptr, 8 * n)), len(PyBytes_FromStringAndSize(nullptr, 8 * n));
    THPObjectPtr type(PyBytes_FromStringAndSize(nullptr, 4 * n));
    if (!at || !len || !type)
        return nullptr;
    long device = -1;
    for (Py_ssize_t i = 0; i < n; i++) {
        PyObject *item = PySequence_Fast_GET_ITEM(seq.get(), i);
        if (!THPVariable_Check(item))
            return PyErr_Format(PyExc_TypeError, "entry %zd is no tensor", i);
        const at::Tensor &t = THPVariable_Unpack(item);
        if (!t.is_cuda())
            return PyErr_Format(PyExc_ValueError, "all tensors must be on the GPU");
        const long on = t.get_device();
        if (device >= 0 && on != device)
            return PyErr_Format(PyExc_ValueError, "all tensors must be on the same GPU");
        device = on;
        const at::ScalarType s = t.scalar_type();
        if (s != at::kFloat && s != at::kBFloat16)
            return PyErr_Format(PyExc_TypeError, "entry %zd: expected float32 or bfloat16", i);
        if (!t.is_contiguous())
            return PyErr_Format(PyExc_ValueError, "entry %zd must be contiguous", i);
        ((int64_t *)PyBytes_AS_STRING(at.get()))[i] = (int64_t)t.data_ptr();
        ((int64_t *)PyBytes_AS_STRING(len.get()))[i] = t.numel();
        ((int32_t *)PyBytes_AS_STRING(type.get()))[i] = s == at::kFloat ? FGB_F32 : FGB_BF16;
    }
    return Py_BuildValue("(OOOl)", at.get(), len.get(), type.get(), device);
    END_HANDLE_TH_ERRORS
}

static PyObject *empties(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    static const at::ScalarType kinds[] = {at::kFloat, at::kBFloat16, at::kByte, at::kInt};
    if (n < 1 || !THPVariable_Check(args[0]))
        return PyErr_Format(PyExc_TypeError, "empties: expected a tensor first");
    const at::Device device = THPVariable_Unpack(args[0]).device();
    THPObjectPtr out(PyTuple_New(n - 1));
    if (!out)
        return nullptr;
    for (Py_ssize_t i = 1; i < n; i++) {
        int64_t v[4];
        const Py_ssize_t m = PyTuple_Check(args[i]) ? PyTuple_GET_SIZE(args[i]) : 0;
        if (m < 1 || m > 4)
            return PyErr_Format(PyExc_TypeError, "empties: expected (kind, up to three sizes)");
        for (Py_ssize_t k = 0; k < m; k++) {
            v[k] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[i], k));
            if (v[k] < 0)
                return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "empties: negative size");
        }
        if (v[0] > 3)
            return PyErr_Format(PyExc_ValueError, "empties: unknown kind");
        PyObject *t = THPVariable_Wrap(at::empty(at::IntArrayRef(v + 1, (size_t)m - 1),
                                                 at::TensorOptions().dtype(kinds[v[0]]).device(device)));
        if (!t)
            return nullptr;
        PyTuple_SET_ITEM(out.get(), i - 1, t);
    }
    return out.release();
    END_HANDLE_TH_ERRORS
}

static PyMethodDef methods[] = {
    {"describe", describe, METH_O, "addresses, lengths, types and device of a list of tensors"},
    {"empties", (PyCFunction)(void (*)(void))empties, METH_FASTCALL, "uninitialised tensors on a tensor's device"},
    {nullptr, nullptr, 0, nullptr}};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
