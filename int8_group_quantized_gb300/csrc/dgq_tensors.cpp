// dgq_tensors.cpp -- the binding's checks on tensors, as one native call (type, shape, contiguity and device
// of every operand of an entry point, and their addresses), and the entry points of the smallest calls
// without ctypes' conversions.  In Python the checks take 0.35 us for each operand (3.2 us of the 9.6 us of a
// call with nine of them), here 1 us for ten; ctypes takes 1.4 to 1.9 us for 18 to 24 arguments, here 0.3.
// The smallest calls' kernels take 2 to 4 us.  __init__.py has the same checks, and ctypes, for a tree in
// which this module is not built.
#include <c10/util/SmallVector.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <tuple>
#include <type_traits>
#include <utility>

#include "dgq.h"

namespace {

// ---- entry points -----------------------------------------------------------------------------------

void *library = nullptr;  // libdgq.so, as the binding opened it

template <typename A>
A argument(PyObject *x)
{
    if constexpr (std::is_pointer_v<A>) {
        return static_cast<A>(PyLong_AsVoidPtr(x));
    } else if constexpr (std::is_unsigned_v<A>) {
        return static_cast<A>(PyLong_AsSize_t(x));
    } else {
        const long long v = PyLong_AsLongLong(x);
        if (!PyErr_Occurred() && v != static_cast<A>(v)) PyErr_SetString(PyExc_OverflowError, "argument out of range");
        return static_cast<A>(v);
    }
}

template <typename... A, size_t... I>
PyObject *invoke(dgq_status (*f)(A...), PyObject *const *args, Py_ssize_t n, std::index_sequence<I...>)
{
    if (!f || n != static_cast<Py_ssize_t>(sizeof...(A))) {
        PyErr_SetString(PyExc_TypeError, f ? "wrong number of arguments" : "the library is not loaded");
        return nullptr;
    }
    const std::tuple<A...> a{argument<A>(args[I])...};
    if (PyErr_Occurred()) return nullptr;
    dgq_status status;
    Py_BEGIN_ALLOW_THREADS
    status = f(std::get<I>(a)...);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

template <typename... A>
PyObject *invoke(dgq_status (*f)(A...), PyObject *const *args, Py_ssize_t n)
{
    return invoke(f, args, n, std::index_sequence_for<A...>{});
}

#define ENTRY(name)                                                                                            \
    PyObject *call_##name(PyObject *, PyObject *const *args, Py_ssize_t n)                                      \
    {                                                                                                          \
        static const auto f = reinterpret_cast<decltype(&name)>(library ? dlsym(library, #name) : nullptr);     \
        return invoke(f, args, n);                                                                             \
    }
ENTRY(dgq_extend_tables)
ENTRY(dgq_write_slots)
ENTRY(dgq_store_block8)
ENTRY(dgq_load_block8)
ENTRY(dgq_paged_decode_attn_block8)
#undef ENTRY

// load(path): opens the library (the one that ctypes has open already).
PyObject *load(PyObject *, PyObject *path)
{
    const char *p = PyUnicode_AsUTF8(path);
    if (!p) return nullptr;
    if (!library) library = dlopen(p, RTLD_NOW | RTLD_LOCAL);
    if (!library) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
    Py_RETURN_NONE;
}

// ---- checks -------------------------------------------------------------------------------------------

const at::Tensor *tensor_of(PyObject *x) { return THPVariable_Check(x) ? &THPVariable_Unpack(x) : nullptr; }

bool on_device(const at::Tensor &t, long device) { return t.is_cuda() && t.get_device() == device; }

// operands(device, workspace, (tensor, dtype, shape), ...): addresses of the tensors and of the workspace, or
// None: one of them is not what the raw pointers would be read as.
PyObject *operands(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n < 2) {
        PyErr_SetString(PyExc_TypeError, "operands(device, workspace, ...)");
        return nullptr;
    }
    const long device = PyLong_AsLong(args[0]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    const at::Tensor *ws = tensor_of(args[1]);
    if (!ws || !ws->is_contiguous() || !on_device(*ws, device)) Py_RETURN_NONE;
    c10::SmallVector<const void *, 16> found;  // (the list is made when nothing can throw any more)
    for (Py_ssize_t i = 2; i < n; ++i) {
        PyObject *spec = args[i];
        bool ok = PyTuple_Check(spec) && PyTuple_GET_SIZE(spec) == 3;
        const at::Tensor *t = ok ? tensor_of(PyTuple_GET_ITEM(spec, 0)) : nullptr;
        PyObject *dtype = ok ? PyTuple_GET_ITEM(spec, 1) : nullptr, *shape = ok ? PyTuple_GET_ITEM(spec, 2) : nullptr;
        ok = t && THPDtype_Check(dtype) && PyTuple_Check(shape) &&
             t->scalar_type() == reinterpret_cast<THPDtype *>(dtype)->scalar_type && t->dim() == PyTuple_GET_SIZE(shape) &&
             t->is_contiguous() && on_device(*t, device);
        for (Py_ssize_t d = 0; ok && d < t->dim(); ++d)
            ok = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, d)) == t->size(d);
        if (PyErr_Occurred()) return nullptr;
        if (!ok) Py_RETURN_NONE;
        found.push_back(t->mutable_data_ptr());  // (written by some calls: a lazy clone gets its own storage first)
    }
    found.push_back(ws->mutable_data_ptr());
    PyObject *out = PyList_New(n - 1);
    for (Py_ssize_t i = 0; out && i < n - 1; ++i) PyList_SET_ITEM(out, i, PyLong_FromVoidPtr(const_cast<void *>(found[i])));
    return out;
}

// token_rows(device, tensor, ...): address and token stride of bf16 rows [T, heads, D] of one shape whose heads
// lie side by side, or None.
PyObject *token_rows(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n < 2) {
        PyErr_SetString(PyExc_TypeError, "token_rows(device, rows, ...)");
        return nullptr;
    }
    const long device = PyLong_AsLong(args[0]);
    if (device == -1 && PyErr_Occurred()) return nullptr;
    const at::Tensor *first = tensor_of(args[1]);
    for (Py_ssize_t i = 1; i < n; ++i) {
        const at::Tensor *t = tensor_of(args[i]);
        if (!first || !t || t->dim() != 3 || t->scalar_type() != at::kBFloat16 || t->sizes() != first->sizes() ||
            t->stride(2) != 1 || (t->stride(1) != t->size(2) && t->size(1) > 1) || !on_device(*t, device))
            Py_RETURN_NONE;
    }
    c10::SmallVector<const void *, 4> found;
    for (Py_ssize_t i = 1; i < n; ++i) found.push_back(tensor_of(args[i])->const_data_ptr());
    PyObject *out = PyList_New(2 * (n - 1));
    for (Py_ssize_t i = 1; out && i < n; ++i) {
        PyList_SET_ITEM(out, 2 * (i - 1), PyLong_FromVoidPtr(const_cast<void *>(found[i - 1])));
        PyList_SET_ITEM(out, 2 * (i - 1) + 1, PyLong_FromLongLong(tensor_of(args[i])->stride(0)));
    }
    return out;
}

// No C++ exception reaches the interpreter: torch throws for what a tensor of another kind (sparse, without
// storage) cannot answer.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n)
{
    try {
        return F(self, args, n);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "an operand could not be looked at");
    }
    return nullptr;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(call_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    ENTRY(dgq_extend_tables),
    ENTRY(dgq_write_slots),
    ENTRY(dgq_store_block8),
    ENTRY(dgq_load_block8),
    ENTRY(dgq_paged_decode_attn_block8),
    {"load", load, METH_O, nullptr},
    {"operands", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded<operands>)), METH_FASTCALL, nullptr},
    {"token_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(guarded<token_rows>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
