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
//
// usual(matrix, vector, matrices...) -> (rows, cols, address and type of each, 0 and FGB_F32 for
// None) where all are as the calls mostly have them: FP32 or BF16, on one GPU, contiguous and
// 16-byte aligned, the matrices of one shape [rows, cols], the vector [cols].  None where
// anything is not: the caller then looks for what it is.  (3 us in Python, 0.3 us here.)
//
// torch_version: that of the torch which this was compiled against.  Another's tensors may be laid
// out differently, so the package does not go on with it.
#include <ATen/ops/empty.h>
#include <pybind11/pybind11.h>
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
    struct Spec {
        int64_t v[4]; // the kind, then the sizes
        size_t dims;
    };
    c10::SmallVector<Spec, 8> specs(n - 1);
    for (Py_ssize_t i = 1; i < n; i++) {
        int64_t *const v = specs[i - 1].v;
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
        specs[i - 1].dims = (size_t)m - 1;
    }
    c10::SmallVector<at::Tensor, 8> tensors;
    {
        pybind11::gil_scoped_release others_run; // (the allocator may wait for the GPU)
        for (const Spec &s : specs)
            tensors.push_back(at::empty(at::IntArrayRef(s.v + 1, s.dims),
                                        at::TensorOptions().dtype(kinds[s.v[0]]).device(device)));
    }
    THPObjectPtr out(PyTuple_New(n - 1));
    if (!out)
        return nullptr;
    for (Py_ssize_t i = 0; i < n - 1; i++) {
        PyObject *t = THPVariable_Wrap(std::move(tensors[i]));
        if (!t)
            return nullptr;
        PyTuple_SET_ITEM(out.get(), i, t);
    }
    return out.release();
    END_HANDLE_TH_ERRORS
}

// Whether t is an FP32 or BF16 tensor on GPU `device` (-1: any, which it then is), contiguous and
// 16-byte aligned.
static bool is_usual(const at::Tensor &t, long &device)
{
    if (!t.is_cuda() || t.layout() != at::kStrided || (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16))
        return false;
    const long on = t.get_device();
    if (device < 0)
        device = on;
    return on == device && t.is_contiguous() && ((uintptr_t)t.data_ptr() & 15) == 0;
}

static PyObject *usual(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n < 2)
        return PyErr_Format(PyExc_TypeError, "usual: expected a matrix and a vector");
    for (Py_ssize_t i = 0; i < n; i++)
        if (!THPVariable_Check(args[i]) && !(i > 1 && args[i] == Py_None))
            Py_RETURN_NONE;
    const at::Tensor &m = THPVariable_Unpack(args[0]), &v = THPVariable_Unpack(args[1]);
    long device = -1;
    if (!is_usual(m, device) || m.dim() != 2 || !is_usual(v, device) || v.dim() != 1 || v.size(0) != m.size(1))
        Py_RETURN_NONE;
    for (Py_ssize_t i = 2; i < n; i++)
        if (args[i] != Py_None) {
            const at::Tensor &t = THPVariable_Unpack(args[i]);
            if (!is_usual(t, device) || t.sizes() != m.sizes())
                Py_RETURN_NONE;
        }
    THPObjectPtr out(PyTuple_New(2 + 2 * n));
    if (!out)
        return nullptr;
    const auto put = [&](Py_ssize_t at, long long value) {
        PyObject *o = PyLong_FromLongLong(value);
        if (o)
            PyTuple_SET_ITEM(out.get(), at, o);
        return o != nullptr;
    };
    if (!put(0, m.size(0)) || !put(1, m.size(1)))
        return nullptr;
    for (Py_ssize_t i = 0; i < n; i++) {
        const bool none = args[i] == Py_None;
        if (!put(2 + 2 * i, none ? 0 : (long long)(uintptr_t)THPVariable_Unpack(args[i]).data_ptr()) ||
            !put(3 + 2 * i, none || THPVariable_Unpack(args[i]).scalar_type() == at::kFloat ? FGB_F32 : FGB_BF16))
            return nullptr;
    }
    return out.release();
    END_HANDLE_TH_ERRORS
}

static PyMethodDef methods[] = {
    {"describe", describe, METH_O, "addresses, lengths, types and device of a list of tensors"},
    {"empties", (PyCFunction)(void (*)(void))empties, METH_FASTCALL, "uninitialised tensors on a tensor's device"},
    {"usual", (PyCFunction)(void (*)(void))usual, METH_FASTCALL, "sizes, addresses and types of tensors laid out as usual"},
    {nullptr, nullptr, 0, nullptr}};
static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

PyMODINIT_FUNC PyInit__tensors(void)
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", FGB_TORCH) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
