// Python calls of the library's per-step entry points with plain numbers:
// pointers, sizes and strides as Python integers (None: a null pointer), scales
// as floats, in the order of the C declaration.  A ctypes call converts each
// argument through a Python-level descriptor, which takes longer than the
// launch for a call of twenty.  The module is not linked to the library: bind()
// gives it the functions of the one that the binding opened.  Nothing is
// computed here; each function returns what the C call returns.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <string.h>

#include <tuple>
#include <utility>

#include "pagedkv.h"

namespace {

// The arguments of one call, read in order; a bad one leaves a Python error.
class Args {
public:
    explicit Args(PyObject* const* a) : a_(a) {}

    // pointers, sizes, strides
    operator void*() { return pointer(); }
    operator const void*() { return pointer(); }
    operator const int32_t*() { return static_cast<const int32_t*>(pointer()); }
    operator const int64_t*() { return static_cast<const int64_t*>(pointer()); }
    operator const float*() { return static_cast<const float*>(pointer()); }
    operator int() {
        const long long v = whole();
        if (v != (int)v && !PyErr_Occurred()) PyErr_SetString(PyExc_OverflowError, "a size does not fit 32 bits");
        return (int)v;
    }
    operator pkv_dtype() { return static_cast<pkv_dtype>(static_cast<int>(*this)); }
    operator int64_t() { return whole(); }
    operator size_t() { return (size_t)whole(); }
    operator float() { return (float)PyFloat_AsDouble(*a_++); }

private:
    long long whole() { return PyLong_AsLongLong(*a_++); }
    void* pointer() {
        PyObject* o = *a_++;
        return o == Py_None ? nullptr : PyLong_AsVoidPtr(o);
    }
    PyObject* const* a_;
};

inline PyObject* result(pkv_status st) { return PyLong_FromLong(st); }
inline PyObject* result(size_t n) { return PyLong_FromSize_t(n); }

// One entry point of the library that bind() was given; Fn is its declaration.
template <typename Fn, int ID>
struct Entry;
template <typename R, typename... A, int ID>
struct Entry<R (*)(A...), ID> {
    static inline R (*fn)(A...) = nullptr;

    static PyObject* py(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(a, n, std::index_sequence_for<A...>{}); }

    template <size_t... I>
    static PyObject* call(PyObject* const* a, Py_ssize_t n, std::index_sequence<I...>) {
        if (!fn) return PyErr_Format(PyExc_RuntimeError, "bind() comes first");
        if (n != (Py_ssize_t)sizeof...(A))
            return PyErr_Format(PyExc_TypeError, "%zd arguments wanted, %zd given", (Py_ssize_t)sizeof...(A), n);
        Args args(a);
        std::tuple<A...> t{static_cast<A>(args)...};   // braces: read left to right
        if (PyErr_Occurred()) return nullptr;
        R r;
        Py_BEGIN_ALLOW_THREADS
        r = fn(std::get<I>(t)...);
        Py_END_ALLOW_THREADS
        return result(r);
    }
};

#define PKV_ENTRIES(X)                                                            \
    X(rotary_embedding) X(rotary_reshape_and_cache) X(rotary_reshape_and_cache_fp8row) \
    X(reshape_and_cache_fp8row) X(gather_cache) X(gather_cache_fp8kv) X(gather_cache_fp8row) \
    X(paged_attention_decode_fp8row) X(paged_attention_prefill_fp8row)            \
    X(paged_attention_prefill_fp8kv) X(paged_attention_workspace_size)

enum { // one id a name: entries of one signature stay apart
#define X(name) ID_##name,
    PKV_ENTRIES(X)
#undef X
};

// bind(name, address): where the opened library has that function
PyObject* bind(PyObject*, PyObject* args) {
    const char* name;
    PyObject* address;
    if (!PyArg_ParseTuple(args, "sO", &name, &address)) return nullptr;
    void* at = PyLong_AsVoidPtr(address);
    if (PyErr_Occurred()) return nullptr;
#define X(f)                                                                          \
    if (!strcmp(name, #f)) {                                                          \
        Entry<decltype(&f), ID_##f>::fn = reinterpret_cast<decltype(&f)>(at);         \
        Py_RETURN_NONE;                                                               \
    }
    PKV_ENTRIES(X)
#undef X
    return PyErr_Format(PyExc_ValueError, "no entry point %s", name);
}

PyMethodDef kMethods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
#define X(f)                                                                                            \
    {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&Entry<decltype(&f), ID_##f>::py)), \
     METH_FASTCALL, nullptr},
    PKV_ENTRIES(X)
#undef X
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", "libpagedkv entry points with plain numbers", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall(void) { return PyModule_Create(&kModule); }
