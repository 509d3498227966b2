// binding.cpp -- the quick half of the Python binding of the language-model
// operators (module _marshal): tests of tensor arguments, allocation, and the
// calls of the C ABI with tensors for pointers.  A decode step of 8 us of GPU
// time has a dozen arguments; checked and converted one by one in Python they
// took as long again.  What a refused argument is told, and everything else,
// is in lm.py and attn.py.
//
// The library itself stays the one that the package loaded: bind() is given
// the addresses of its entry points.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cstdint>
#include <cstring>
#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/msscan.h"

namespace {

const at::Tensor* tensor_of(PyObject* o) {
    return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// ---- checks ------------------------------------------------------------------

// io(x, dims): MS_F32 or MS_BF16 of a contiguous device tensor of so many
// dimensions, -1 of anything else.
PyObject* io(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    long code = -1;
    const at::Tensor* t = n == 2 ? tensor_of(a[0]) : nullptr;
    if (t && t->is_cuda() && t->dim() == PyLong_AsLong(a[1]) && t->is_contiguous())
        code = t->scalar_type() == at::kFloat      ? MS_F32
               : t->scalar_type() == at::kBFloat16 ? MS_BF16
                                                   : -1;
    return PyLong_FromLong(code);
    END_HANDLE_TH_ERRORS
}

// rows(x, dims, *ts): 2 ld + io code, where x is a device tensor of dims
// dimensions and MS_F32 or MS_BF16, whose rows (the last dimension) are
// contiguous and ld apart, in order, and each of ts is None or has the same
// dtype, sizes, device and ld; -1 of anything else.  A row that is alone has no
// ld: where one of them does not begin on 16 bytes it is a slice of a wider
// row, and has the ld of one.
int64_t row_pitch(const at::Tensor& t) {
    const int64_t dims = t.dim(), d = t.size(dims - 1);
    if (d > 1 && t.stride(dims - 1) != 1) return -1;
    if (t.numel() == 0) return d;
    int64_t ld = -1, want = 0;  // -1: no dimension before the rows' has told it yet
    for (int64_t k = dims - 2; k >= 0; --k) {
        if (t.size(k) == 1) continue;
        if (ld < 0) ld = want = t.stride(k);
        if (ld < d || t.stride(k) != want) return -1;  // overlapping (an expanded dimension's is 0)
        want *= t.size(k);
    }
    return ld < 0 ? d : ld;
}
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* x = n >= 2 ? tensor_of(a[0]) : nullptr;
    if (!x || !x->is_cuda() || x->layout() != at::kStrided || x->dim() != PyLong_AsLong(a[1]) ||
        (x->scalar_type() != at::kFloat && x->scalar_type() != at::kBFloat16))
        return PyLong_FromLong(-1);
    int64_t ld = row_pitch(*x);
    bool ok = ld >= 0;
    const bool alone = x->numel() && x->numel() == x->size(-1);
    auto off = [&](const at::Tensor& t) {
        return alone && (reinterpret_cast<uintptr_t>(t.const_data_ptr()) & 15u);
    };
    bool slice = off(*x);
    for (Py_ssize_t k = 2; ok && k < n; ++k) {
        if (a[k] == Py_None) continue;
        const at::Tensor* t = tensor_of(a[k]);
        ok = t && t->layout() == at::kStrided && t->scalar_type() == x->scalar_type() &&
             t->sizes() == x->sizes() && t->device() == x->device() && row_pitch(*t) == ld;
        slice = slice || (ok && off(*t));
    }
    ld += slice;
    const int64_t io = x->scalar_type() == at::kFloat ? MS_F32 : MS_BF16;
    return PyLong_FromLongLong(ok ? 2 * ld + io : -1);
    END_HANDLE_TH_ERRORS
}

// pitch(x, dims, inner): 2 ld + io code, where x is a device tensor of dims
// dimensions and MS_F32 or MS_BF16, whose last `inner` dimensions are one
// contiguous row, the rows ld apart and in order; -1 of anything else.
PyObject* pitch(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* x = n == 3 ? tensor_of(a[0]) : nullptr;
    if (!x || !x->is_cuda() || x->layout() != at::kStrided || x->dim() != PyLong_AsLong(a[1]) ||
        (x->scalar_type() != at::kFloat && x->scalar_type() != at::kBFloat16))
        return PyLong_FromLong(-1);
    const int64_t dims = x->dim(), inner = PyLong_AsLong(a[2]);
    const int64_t io = x->scalar_type() == at::kFloat ? MS_F32 : MS_BF16;
    int64_t d = 1;
    for (int64_t k = dims - 1; k >= dims - inner; --k) {
        if (x->numel() && x->size(k) > 1 && x->stride(k) != d) return PyLong_FromLong(-1);
        d *= x->size(k);
    }
    if (x->numel() == 0) return PyLong_FromLongLong(2 * d + io);
    int64_t ld = -1, want = 0;  // -1: every dimension so far has one entry
    for (int64_t k = dims - inner - 1; k >= 0; --k) {
        if (x->size(k) == 1) continue;
        if (ld < 0) ld = want = x->stride(k);
        if (ld < d || x->stride(k) != want) return PyLong_FromLong(-1);
        want *= x->size(k);
    }
    return PyLong_FromLongLong(2 * (ld < 0 ? d : ld) + io);
    END_HANDLE_TH_ERRORS
}

// fits(x, dtype, sizes, *ts): each of ts is None or a contiguous tensor of
// that dtype and those sizes on x's device.
PyObject* fits(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* x = n >= 3 ? tensor_of(a[0]) : nullptr;
    bool ok = x && THPDtype_Check(a[1]) && PyTuple_Check(a[2]);
    for (Py_ssize_t k = 3; ok && k < n; ++k) {
        if (a[k] == Py_None) continue;
        const at::Tensor* t = tensor_of(a[k]);
        ok = t && t->scalar_type() == reinterpret_cast<THPDtype*>(a[1])->scalar_type &&
             t->device() == x->device() && t->dim() == PyTuple_GET_SIZE(a[2]) &&
             t->is_contiguous();
        for (int64_t d = 0; ok && d < t->dim(); ++d)
            ok = t->size(d) == PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], d));
    }
    if (PyErr_Occurred()) return nullptr;
    return PyBool_FromLong(ok);
    END_HANDLE_TH_ERRORS
}

// empty(x, dtype, *sizes): an uninitialised tensor on x's device.
PyObject* empty(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const at::Tensor* x = n >= 2 ? tensor_of(a[0]) : nullptr;
    if (!x || !THPDtype_Check(a[1]) || n - 2 > 8) {
        PyErr_SetString(PyExc_TypeError, "empty(tensor, dtype, *sizes)");
        return nullptr;
    }
    int64_t size[8];
    for (Py_ssize_t k = 2; k < n; ++k) size[k - 2] = PyLong_AsLongLong(a[k]);
    if (PyErr_Occurred()) return nullptr;
    return THPVariable_Wrap(
        at::empty(at::IntArrayRef(size, n - 2),
                  at::TensorOptions()
                      .dtype(reinterpret_cast<THPDtype*>(a[1])->scalar_type)
                      .device(x->device())));
    END_HANDLE_TH_ERRORS
}

// together(x, dtype, sizes, dtype, sizes, ...): a tuple of uninitialised tensors
// on x's device, in one allocation (an allocation costs about a microsecond).
// None is a view of another: each has a version of its own.
PyObject* together(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    constexpr int kMost = 8, kMostDims = 4;
    const at::Tensor* x = n ? tensor_of(a[0]) : nullptr;
    const int count = (int)(n / 2);
    bool ok = x && n % 2 == 1 && count >= 1 && count <= kMost;
    int64_t size[kMost][kMostDims], at[kMost], total = 0;
    for (int k = 0; ok && k < count; ++k) {
        PyObject *dtype = a[1 + 2 * k], *sizes = a[2 + 2 * k];
        ok = THPDtype_Check(dtype) && PyTuple_Check(sizes) && PyTuple_GET_SIZE(sizes) <= kMostDims;
        if (!ok) break;
        int64_t bytes = c10::elementSize(reinterpret_cast<THPDtype*>(dtype)->scalar_type);
        for (Py_ssize_t d = 0; d < PyTuple_GET_SIZE(sizes); ++d) {
            size[k][d] = PyLong_AsLongLong(PyTuple_GET_ITEM(sizes, d));
            ok = ok && size[k][d] >= 0 && size[k][d] < (1LL << 40);
            bytes *= size[k][d];
        }
        at[k] = total;
        total += (bytes + 255) / 256 * 256;
    }
    if (PyErr_Occurred()) return nullptr;
    if (!ok) {
        PyErr_SetString(PyExc_TypeError, "together(tensor, dtype, sizes, ...)");
        return nullptr;
    }
    const at::Tensor buf =
        at::empty({total}, at::TensorOptions().dtype(at::kByte).device(x->device()));
    PyObject* out = PyTuple_New(count);
    for (int k = 0; out && k < count; ++k) {
        const at::ScalarType type = reinterpret_cast<THPDtype*>(a[1 + 2 * k])->scalar_type;
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            c10::Storage(buf.storage()), buf.key_set(), caffe2::TypeMeta::fromScalarType(type));
        t.unsafeGetTensorImpl()->set_storage_offset(at[k] / (int64_t)c10::elementSize(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(
            at::IntArrayRef(size[k], PyTuple_GET_SIZE(a[2 + 2 * k])));
        PyTuple_SET_ITEM(out, k, THPVariable_Wrap(std::move(t)));
    }
    return out;
    END_HANDLE_TH_ERRORS
}

// ---- calls -------------------------------------------------------------------

// A C argument from a Python one: pointers from tensors, addresses or None.
template <class T>
T convert(PyObject* o) {
    if (PyErr_Occurred()) return T{};  // an earlier argument's
    if constexpr (std::is_pointer<T>::value) {
        if (o == Py_None) return nullptr;
        if (const at::Tensor* t = tensor_of(o))
            return static_cast<T>(const_cast<void*>(static_cast<const void*>(t->data_ptr())));
        return static_cast<T>(PyLong_AsVoidPtr(o));
    } else if constexpr (std::is_floating_point<T>::value) {
        return static_cast<T>(PyFloat_AsDouble(o));
    } else if constexpr (sizeof(T) == 4) {
        const long long v = PyLong_AsLongLong(o);
        if (v != static_cast<T>(v) && !PyErr_Occurred())
            PyErr_SetString(PyExc_OverflowError, "argument does not fit in 32 bits");
        return static_cast<T>(v);
    } else {
        return static_cast<T>(PyLong_AsLongLong(o));
    }
}

template <class... A, size_t... I>
PyObject* call(ms_status (*f)(A...), PyObject* const* a, Py_ssize_t n,
               std::index_sequence<I...>) {
    HANDLE_TH_ERRORS
    if (!f || n != sizeof...(A)) {
        PyErr_Format(PyExc_TypeError, "%zd arguments given, %zu taken", n, sizeof...(A));
        return nullptr;
    }
    const std::tuple<A...> v{convert<A>(a[I])...};
    if (PyErr_Occurred()) return nullptr;
    ms_status rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f(std::get<I>(v)...);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}
template <class... A>
PyObject* call(ms_status (*f)(A...), PyObject* const* a, Py_ssize_t n) {
    return call(f, a, n, std::index_sequence_for<A...>{});
}

#define ENTRY_(name)                                                        \
    decltype(&ms_##name) p_##name;                                          \
    PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {           \
        return call(p_##name, a, n);                                        \
    }
#define ENTRIES_(do_)                                                       \
    do_(gated_scan_fwd) do_(gated_scan_bwd) do_(gated_step) do_(embed_fwd)  \
    do_(embed_bwd) do_(token_logprobs_fwd) do_(token_logprobs_bwd)          \
    do_(linear_attn_fwd) do_(linear_attn_bwd) do_(linear_attn_step)         \
    do_(group_norm_fwd) do_(group_norm_bwd) do_(verify_drafts)
ENTRIES_(ENTRY_)

// bind(name, address) of an entry point
PyObject* bind(PyObject*, PyObject* args) {
    const char* name;
    PyObject* address;
    if (!PyArg_ParseTuple(args, "sO", &name, &address)) return nullptr;
    void* p = PyLong_AsVoidPtr(address);
    if (PyErr_Occurred()) return nullptr;
#define BIND_(entry)                                                        \
    if (!strcmp(name, #entry)) {                                            \
        p_##entry = reinterpret_cast<decltype(p_##entry)>(p);               \
        Py_RETURN_NONE;                                                     \
    }
    ENTRIES_(BIND_)
    return PyErr_Format(PyExc_KeyError, "%s", name);
}

#define METHOD_(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr},
PyMethodDef methods[] = {METHOD_(io) METHOD_(rows) METHOD_(pitch) METHOD_(fits)
                         METHOD_(empty) METHOD_(together)
                         ENTRIES_(METHOD_)
                         {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
