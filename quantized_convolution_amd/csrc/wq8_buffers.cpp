// CPython module: the addresses of a call's tensors if all are what the plan
// says, in one step. What takes Python half a microsecond a tensor takes this
// some nanoseconds, in front of kernels that take three. It refuses nothing by
// itself: where anything is not as it should be, or is to be made, its answer is
// None, and the checks in Python name what is wrong.
#include <c10/core/GradMode.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

namespace {

struct Buffer {
    at::ScalarType dtype;
    std::vector<int64_t> shape, strides;  // no strides: contiguous
    bool required, workspace;
    int64_t bytes;                        // of a workspace
};

constexpr const char *kName = "wq8 buffers";

void destroy(PyObject *c) { delete (std::vector<Buffer> *)PyCapsule_GetPointer(c, kName); }

bool numbers(PyObject *t, std::vector<int64_t> &out) {
    if (!PyTuple_Check(t)) return false;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(t); ++i) {
        out.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(t, i)));
        if (PyErr_Occurred()) return false;
    }
    return true;
}

// form(entries): (dtype, shape, strides or None, required) for a tensor, a number
// of bytes for a workspace.
PyObject *form(PyObject *, PyObject *entries) {
    auto *v = new std::vector<Buffer>;
    bool ok = PyTuple_Check(entries);
    for (Py_ssize_t i = 0; ok && i < PyTuple_GET_SIZE(entries); ++i) {
        PyObject *e = PyTuple_GET_ITEM(entries, i);
        Buffer b = {};
        if (PyLong_Check(e)) {
            b.workspace = true;
            b.bytes = PyLong_AsLongLong(e);
        } else {
            ok = PyTuple_Check(e) && PyTuple_GET_SIZE(e) == 4 && THPDtype_Check(PyTuple_GET_ITEM(e, 0)) &&
                 numbers(PyTuple_GET_ITEM(e, 1), b.shape);
            if (!ok) break;
            b.dtype = ((THPDtype *)PyTuple_GET_ITEM(e, 0))->scalar_type;
            PyObject *s = PyTuple_GET_ITEM(e, 2);
            ok = s == Py_None || (numbers(s, b.strides) && b.strides.size() == b.shape.size());
            b.required = PyObject_IsTrue(PyTuple_GET_ITEM(e, 3)) == 1;
        }
        v->push_back(std::move(b));
    }
    if (!ok || PyErr_Occurred()) {
        delete v;
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "a buffer's form is (dtype, shape, strides or None, required)");
        return nullptr;
    }
    return PyCapsule_New(v, kName, destroy);
}

bool fits(const at::Tensor &t, const Buffer &b) {
    if (t.scalar_type() != b.dtype || t.layout() != at::kStrided || t.sizes() != at::IntArrayRef(b.shape)) return false;
    if (b.strides.empty()) return t.is_contiguous();
    for (size_t i = 0; i < b.shape.size(); ++i)
        if (b.shape[i] > 1 && t.stride(i) != b.strides[i]) return false;
    return true;
}

// addresses(form, tensor or None, ...): (device, address, ...), a workspace as
// its address and bytes; None where a tensor is not as its form says, asks for a
// gradient while graphs are recorded, carries a tangent, or is not on the same GPU
// as the others.
PyObject *addresses(PyObject *, PyObject *const *args, Py_ssize_t n) {
    auto *v = n > 0 ? (std::vector<Buffer> *)PyCapsule_GetPointer(args[0], kName) : nullptr;
    if (!v || (size_t)n != v->size() + 1) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "as many tensors as the form has");
        return nullptr;
    }
    int64_t out[40];
    size_t count = 1;
    int device = -1;
    try {
        for (size_t i = 0; i < v->size(); ++i) {
            const Buffer &b = (*v)[i];
            PyObject *o = args[i + 1];
            if (count + 2 > 40) Py_RETURN_NONE;
            if (o == Py_None || (b.workspace && b.bytes == 0)) {
                if (b.required || (b.workspace && b.bytes > 0)) Py_RETURN_NONE;
                out[count++] = 0;
                if (b.workspace) out[count++] = 0;
                continue;
            }
            if (!THPVariable_CheckExact(o)) Py_RETURN_NONE;
            const at::Tensor &t = THPVariable_Unpack(o);
            if (!t.is_cuda() || (t.requires_grad() && c10::GradMode::is_enabled()) || t._fw_grad(0).defined()) Py_RETURN_NONE;
            if (device < 0) device = t.get_device();
            if (t.get_device() != device) Py_RETURN_NONE;
            if (b.workspace) {
                const int64_t bytes = t.numel() * (int64_t)t.element_size();
                if (t.layout() != at::kStrided || !t.is_contiguous() || bytes < b.bytes) Py_RETURN_NONE;
                out[count++] = (int64_t)t.data_ptr();
                out[count++] = bytes;
            } else {
                if (!fits(t, b)) Py_RETURN_NONE;
                out[count++] = (int64_t)t.data_ptr();
            }
        }
    } catch (...) {  // a tensor without memory of its own
        Py_RETURN_NONE;
    }
    if (device < 0) Py_RETURN_NONE;
    out[0] = device;
    PyObject *r = PyTuple_New((Py_ssize_t)count);
    if (!r) return nullptr;
    for (size_t i = 0; i < count; ++i) {
        PyObject *p = PyLong_FromLongLong(out[i]);
        if (!p) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, (Py_ssize_t)i, p);
    }
    return r;
}

PyMethodDef kMethods[] = {{"form", form, METH_O, nullptr},
                          {"addresses", (PyCFunction)(void (*)(void))addresses, METH_FASTCALL, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_wq8_buffers", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wq8_buffers(void) { return PyModule_Create(&kModule); }
