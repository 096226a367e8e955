// Tensor marshalling for the Python binding of the training-step operators,
// as a CPython module (_armarshal): the addresses of a list of tensors after
// one check of each, the outputs that a call makes, one tensor per rank, and
// the version counters of what it wrote.  A call over 150 tensors spends 0.1 ms
// on this in Python, several times what its kernel takes.
//
// Every function returns None when anything is not as the call needs it; the
// Python code then goes through the same checks one by one and raises what is
// wrong.  No arithmetic, no launches, no state.

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ops/empty.h>

#include <cstdint>
#include <utility>
#include <vector>

namespace {

constexpr int64_t kStateBlock = 256;   // AR_STATE_BLOCK of include/ar.h

// A sequence's items, borrowed while it lives; ok() false leaves no error set.
struct Items {
    PyObject* fast;
    explicit Items(PyObject* o) : fast(PySequence_Fast(o, "")) {
        if (fast == nullptr) PyErr_Clear();
    }
    ~Items() { Py_XDECREF(fast); }
    Items(const Items&) = delete;
    Items& operator=(const Items&) = delete;
    bool ok() const { return fast != nullptr; }
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
    PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// A plain strided tensor of the type on the GPU, or null.
const at::Tensor* plain(PyObject* o, at::ScalarType type, int64_t index) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != index ||
        t.scalar_type() != type || t.is_neg())
        return nullptr;
    return &t;
}

bool scalar_type(PyObject* dtype, at::ScalarType* out) {
    if (!THPDtype_Check(dtype)) return false;
    *out = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    return true;
}

bool as_int(PyObject* o, int64_t* out) {
    *out = PyLong_AsLongLong(o);
    if (*out == -1 && PyErr_Occurred() != nullptr) {
        PyErr_Clear();
        return false;
    }
    return true;
}

PyObject* address_bytes(const std::vector<uintptr_t>& at) {
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(at.data()),
                                     static_cast<Py_ssize_t>(at.size() * sizeof(uintptr_t)));
}

// Runs body; a C++ exception (a tensor without storage, memory running out)
// ends as None, and the Python code finds out or tries by itself.
template <class Body>
PyObject* guarded(Body body) {
    try {
        PyObject* r = body();
        if (r != nullptr || PyErr_Occurred() != nullptr) return r;
    } catch (...) {
        PyErr_Clear();
    }
    Py_RETURN_NONE;
}

// pointers(tensors, dtype, index, counts or None): bytes of the addresses.
PyObject* pointers(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        at::ScalarType type;
        int64_t index;
        if (n_args != 4 || !scalar_type(args[1], &type) || !as_int(args[2], &index)) return nullptr;
        const Items items(args[0]);
        if (!items.ok()) return nullptr;
        std::vector<uintptr_t> at;
        at.reserve(static_cast<size_t>(items.size()));
        const bool counted = args[3] != Py_None;
        if (counted && (!PyList_Check(args[3]) || PyList_GET_SIZE(args[3]) != items.size())) return nullptr;
        for (Py_ssize_t i = 0; i < items.size(); ++i) {
            const at::Tensor* t = plain(items[i], type, index);
            if (t == nullptr || !t->is_contiguous()) return nullptr;
            int64_t count = 0;
            if (counted && (!as_int(PyList_GET_ITEM(args[3], i), &count) || t->numel() != count)) return nullptr;
            at.push_back(reinterpret_cast<uintptr_t>(t->data_ptr()));
        }
        return address_bytes(at);
    });
}

// states(pairs, index, counts): bytes of the codes' addresses, of the scales'.
PyObject* states(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        int64_t index;
        if (n_args != 3 || !as_int(args[1], &index) || !PyList_Check(args[2])) return nullptr;
        const Items items(args[0]);
        if (!items.ok() || PyList_GET_SIZE(args[2]) != items.size()) return nullptr;
        std::vector<uintptr_t> codes, scales;
        codes.reserve(static_cast<size_t>(items.size()));
        scales.reserve(static_cast<size_t>(items.size()));
        for (Py_ssize_t i = 0; i < items.size(); ++i) {
            int64_t count;
            if (!PyTuple_Check(items[i]) || PyTuple_GET_SIZE(items[i]) != 2 ||
                !as_int(PyList_GET_ITEM(args[2], i), &count))
                return nullptr;
            const at::Tensor* c = plain(PyTuple_GET_ITEM(items[i], 0), at::kByte, index);
            const at::Tensor* s = plain(PyTuple_GET_ITEM(items[i], 1), at::kByte, index);
            if (c == nullptr || s == nullptr || !c->is_contiguous() || !s->is_contiguous() || c->numel() != count ||
                s->numel() != (count + kStateBlock - 1) / kStateBlock)
                return nullptr;
            codes.push_back(reinterpret_cast<uintptr_t>(c->data_ptr()));
            scales.push_back(reinterpret_cast<uintptr_t>(s->data_ptr()));
        }
        PyObject* a = address_bytes(codes);
        PyObject* b = a == nullptr ? nullptr : address_bytes(scales);
        PyObject* r = b == nullptr ? nullptr : PyTuple_Pack(2, a, b);
        Py_XDECREF(a);
        Py_XDECREF(b);
        return r;
    });
}

// rows(tensors, dtype, index, rows, cols): bytes of the addresses and the
// common row stride, for [rows, cols] tensors with contiguous rows.
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        at::ScalarType type;
        int64_t index, n_rows, n_cols;
        if (n_args != 5 || !scalar_type(args[1], &type) || !as_int(args[2], &index) || !as_int(args[3], &n_rows) ||
            !as_int(args[4], &n_cols))
            return nullptr;
        const Items items(args[0]);
        if (!items.ok()) return nullptr;
        std::vector<uintptr_t> at;
        at.reserve(static_cast<size_t>(items.size()));
        int64_t stride = n_cols;
        for (Py_ssize_t i = 0; i < items.size(); ++i) {
            const at::Tensor* t = plain(items[i], type, index);
            if (t == nullptr || t->dim() != 2 || t->size(0) != n_rows || t->size(1) != n_cols) return nullptr;
            if (n_cols > 1 && t->stride(1) != 1) return nullptr;
            if (n_rows > 1) {
                if (i == 0) stride = t->stride(0);
                if (t->stride(0) != stride || stride < n_cols) return nullptr;
            }
            at.push_back(reinterpret_cast<uintptr_t>(t->data_ptr()));
        }
        PyObject* bytes = address_bytes(at);
        if (bytes == nullptr) return nullptr;
        PyObject* r = Py_BuildValue("(NL)", bytes, static_cast<long long>(stride));
        return r;
    });
}

// new_parts((n, ...), dtype, index): n new tensors that share one allocation
// of the current stream's, and bytes of their addresses.
PyObject* new_parts(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        at::ScalarType type;
        int64_t index;
        if (n_args != 3 || !PyTuple_Check(args[0]) || !scalar_type(args[1], &type) || !as_int(args[2], &index))
            return nullptr;
        std::vector<int64_t> shape(static_cast<size_t>(PyTuple_GET_SIZE(args[0])));
        if (shape.empty()) return nullptr;
        for (size_t i = 0; i < shape.size(); ++i) {
            if (!as_int(PyTuple_GET_ITEM(args[0], static_cast<Py_ssize_t>(i)), &shape[i])) return nullptr;
        }
        const at::Tensor whole = at::empty(
            shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<at::DeviceIndex>(index))));
        const size_t n = static_cast<size_t>(shape[0]);
        const at::IntArrayRef part = at::IntArrayRef(shape).slice(1);
        const int64_t numel = n == 0 ? 0 : whole.numel() / shape[0];
        std::vector<uintptr_t> at;
        at.reserve(n);
        THPObjectPtr list(PyList_New(static_cast<Py_ssize_t>(n)));
        if (!list) return nullptr;
        for (size_t i = 0; i < n; ++i) {
            // a tensor of its own in the shared storage: no view for autograd to track
            at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                                    whole.dtype());
            t.unsafeGetTensorImpl()->set_storage_offset(static_cast<int64_t>(i) * numel);
            t.unsafeGetTensorImpl()->set_sizes_contiguous(part);
            at.push_back(reinterpret_cast<uintptr_t>(t.data_ptr()));
            PyObject* o = THPVariable_Wrap(std::move(t));
            if (o == nullptr) return nullptr;
            PyList_SET_ITEM(list.get(), static_cast<Py_ssize_t>(i), o);
        }
        PyObject* bytes = address_bytes(at);
        if (bytes == nullptr) return nullptr;
        return Py_BuildValue("(ON)", list.get(), bytes);
    });
}

// Whether o is a tensor; if so, counts a write into it, as torch's in-place
// operations do.  A tensor made in inference mode has no counter outside it.
bool count_write(PyObject* o) {
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    return true;
}

// written(tensors, or pairs of tensors): counts a write into each; True.
PyObject* written(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        if (n_args != 1) return nullptr;
        const Items items(args[0]);
        if (!items.ok()) return nullptr;
        for (Py_ssize_t i = 0; i < items.size(); ++i) {
            if (count_write(items[i])) continue;
            const Items pair(items[i]);
            if (!pair.ok()) return nullptr;
            for (Py_ssize_t j = 0; j < pair.size(); ++j) {
                if (!count_write(pair[j])) return nullptr;
            }
        }
        Py_RETURN_TRUE;
    });
}

PyMethodDef kMethods[] = {
    {"pointers", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pointers)), METH_FASTCALL, nullptr},
    {"states", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(states)), METH_FASTCALL, nullptr},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rows)), METH_FASTCALL, nullptr},
    {"new_parts", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(new_parts)), METH_FASTCALL, nullptr},
    {"written", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(written)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_armarshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__armarshal() { return PyModule_Create(&kModule); }
