// Argument checks of the Python binding, in C++: one call looks over all of an
// entry point's tensors (type, dimensions, contiguity, one CUDA device) and
// returns their addresses and sizes.  Reading five attributes of each of ten
// tensors from Python takes 5 to 7 us, more than most of these operators run; here
// it is below one.  A CPython extension module (_pa_tensors) that uses
// torch's C++ headers for nothing but the tensors' fields.
//
//   make_spec(((name, type, ndim, kind), ...)) -> spec
//   take(spec, tensor, ...) -> (device, address, size, ..., address, size, ...)
//
// type: "bf16", "f32", "i32", "i64", "u8", "any", or "logits" (bf16 or fp32: its
// code, 0 or 1, precedes the address).  kind: "whole" (contiguous), "rows"
// (contiguous but for the stride of dimension 0, which follows the sizes),
// "optional" (whole, or None: address and sizes 0), "space" (optional, any
// dimensions: address and bytes).
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <new>
#include <string>
#include <vector>

namespace {

enum Kind { kWhole, kRows, kOptional, kSpace };

struct Arg {
    std::string name, type;
    c10::ScalarType scalar = c10::ScalarType::Undefined;  // Undefined: any, or logits
    int64_t ndim = 0;
    Kind kind = kWhole;
    bool logits = false;
};
using Spec = std::vector<Arg>;

constexpr const char *kCapsule = "_pa_tensors.spec";

void free_spec(PyObject *capsule) { delete static_cast<Spec *>(PyCapsule_GetPointer(capsule, kCapsule)); }

bool parse(PyObject *item, Arg *a) {
    const char *name, *type, *kind;
    long ndim;
    if (!PyArg_ParseTuple(item, "ssls", &name, &type, &ndim, &kind)) return false;
    a->name = name;
    a->type = type;
    a->ndim = ndim;
    const std::string t = type, k = kind;
    if (t == "bf16") a->scalar = c10::ScalarType::BFloat16;
    else if (t == "f32") a->scalar = c10::ScalarType::Float;
    else if (t == "i32") a->scalar = c10::ScalarType::Int;
    else if (t == "i64") a->scalar = c10::ScalarType::Long;
    else if (t == "u8") a->scalar = c10::ScalarType::Byte;
    else if (t == "logits") a->logits = true;
    else if (t != "any") return PyErr_Format(PyExc_ValueError, "unknown type %s", type), false;
    if (k == "whole") a->kind = kWhole;
    else if (k == "rows") a->kind = kRows;
    else if (k == "optional") a->kind = kOptional;
    else if (k == "space") a->kind = kSpace;
    else return PyErr_Format(PyExc_ValueError, "unknown kind %s", kind), false;
    return true;
}

PyObject *make_spec(PyObject *, PyObject *items) {
    PyObject *seq = PySequence_Fast(items, "make_spec takes a sequence");
    if (!seq) return nullptr;
    Spec *spec = new (std::nothrow) Spec;
    bool ok = spec != nullptr;
    if (!ok) PyErr_NoMemory();
    try {
        for (Py_ssize_t i = 0; ok && i < PySequence_Fast_GET_SIZE(seq); ++i) {
            Arg a;
            ok = parse(PySequence_Fast_GET_ITEM(seq, i), &a);
            if (ok) spec->push_back(a);
        }
    } catch (const std::exception &e) {
        ok = false;
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    Py_DECREF(seq);
    PyObject *capsule = ok ? PyCapsule_New(spec, kCapsule, free_spec) : nullptr;
    if (!capsule) delete spec;
    return capsule;
}

// Whether the tensor fits; the fields it is asked for go to `out`.
bool take_one(const Arg &a, PyObject *obj, int64_t *device, std::vector<int64_t> *out) {
    const bool may_be_none = a.kind == kOptional || a.kind == kSpace;
    if (may_be_none && obj == Py_None) {
        out->insert(out->end(), a.kind == kSpace ? 2 : 1 + a.ndim, 0);
        return true;
    }
    if (!THPVariable_Check(obj)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", a.name.c_str());
        return false;
    }
    const at::Tensor &t = THPVariable_Unpack(obj);
    const c10::ScalarType got = t.scalar_type();
    const bool type_ok = a.logits ? got == c10::ScalarType::BFloat16 || got == c10::ScalarType::Float
                                  : a.scalar == c10::ScalarType::Undefined || got == a.scalar;
    if (!type_ok) {
        PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", a.name.c_str(),
                     a.logits ? "torch.bfloat16 or torch.float32" : a.type.c_str(), c10::toString(got));
        return false;
    }
    if (!t.is_cuda()) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", a.name.c_str());
        return false;
    }
    if (*device < 0) *device = t.get_device();
    if (t.get_device() != *device) {
        PyErr_Format(PyExc_ValueError, "tensors on several devices (%s is on cuda:%d, others on cuda:%d)", a.name.c_str(),
                     static_cast<int>(t.get_device()), static_cast<int>(*device));
        return false;
    }
    if (a.kind == kSpace) {
        if (!t.is_contiguous()) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous", a.name.c_str());
            return false;
        }
        out->push_back(reinterpret_cast<int64_t>(t.data_ptr()));
        out->push_back(static_cast<int64_t>(t.nbytes()));
        return true;
    }
    if (t.dim() != a.ndim) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dims, got %d", a.name.c_str(), static_cast<int>(a.ndim),
                     static_cast<int>(t.dim()));
        return false;
    }
    if (a.kind == kRows) {
        int64_t want = 1;
        for (int64_t d = a.ndim - 1; d >= 1; --d) {
            if (t.size(d) > 1 && t.stride(d) != want) {
                PyErr_Format(PyExc_ValueError, "%s: every row (all but dimension 0) must be contiguous", a.name.c_str());
                return false;
            }
            want *= t.size(d);
        }
        if (a.logits) out->push_back(got == c10::ScalarType::Float);
        out->push_back(reinterpret_cast<int64_t>(t.data_ptr()));
        for (int64_t d = 0; d < a.ndim; ++d) out->push_back(t.size(d));
        out->push_back(t.size(0) > 1 ? t.stride(0) : want);  // (a single row's stride says nothing)
        return true;
    }
    if (!t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", a.name.c_str());
        return false;
    }
    out->push_back(reinterpret_cast<int64_t>(t.data_ptr()));
    for (int64_t d = 0; d < a.ndim; ++d) out->push_back(t.size(d));
    return true;
}

PyObject *take(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < 1) {
        PyErr_SetString(PyExc_TypeError, "take(spec, tensor, ...)");
        return nullptr;
    }
    const Spec *spec = static_cast<const Spec *>(PyCapsule_GetPointer(args[0], kCapsule));
    if (!spec) return nullptr;
    if (static_cast<size_t>(n - 1) != spec->size()) {
        PyErr_Format(PyExc_TypeError, "take: %d tensors expected, got %d", static_cast<int>(spec->size()),
                     static_cast<int>(n - 1));
        return nullptr;
    }
    static thread_local std::vector<int64_t> out;
    int64_t device = -1;
    try {
        out.clear();
        for (size_t i = 0; i < spec->size(); ++i)
            if (!take_one((*spec)[i], args[i + 1], &device, &out)) return nullptr;
    } catch (const std::exception &e) {  // (a tensor without storage, for instance)
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(out.size()) + 1);
    if (!r) return nullptr;
    for (size_t i = 0; i <= out.size(); ++i) {
        PyObject *v = PyLong_FromLongLong(i ? out[i - 1] : device);
        if (!v) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, static_cast<Py_ssize_t>(i), v);
    }
    return r;
}

PyMethodDef kMethods[] = {
    {"make_spec", make_spec, METH_O, "A spec of tensors for take()."},
    {"take", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(take)), METH_FASTCALL,
     "Check tensors against a spec; their device, addresses and sizes."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pa_tensors", "Tensor checks of the paged-attention binding.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_tensors(void) { return PyModule_Create(&kModule); }
