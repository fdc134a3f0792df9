// The Python binding's calls of the operators around a decode step, in C++: each
// takes the wrapper's arguments, checks its tensors (type, dimensions,
// contiguity, one CUDA device, shapes that fit), and calls the C entry point on the
// current stream.  From Python, ten tensors' fields and a foreign call of twenty
// arguments take 9 us or more on the Arm host, longer than most of these operators run;
// here a call takes 3 to 4, the launch included.  A CPython extension module
// (_pa_binding) that uses torch's C++ headers for nothing but the tensors' fields,
// and reaches libpagedattn.so by its C ABI.
#include <Python.h>
#include <dlfcn.h>

#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <new>
#include <vector>

#include "../../include/pa.h"

namespace {

// ---- the library and what is asked of Python ------------------------------------------

PyObject *g_error = nullptr;           // PAError(name, code, text)
PyObject *g_raw_stream = nullptr;      // device -> cudaStream_t of its current stream
PyObject *g_current_device = nullptr;  // () -> device
PyObject *g_set_device = nullptr;      // device ->
struct Library {
    decltype(&::pa_rope_write) rope_write;
    decltype(&::pa_rope_write_fp8) rope_write_fp8;
    decltype(&::pa_decode_scored) decode_scored;
    decltype(&::pa_decode_scored_fp8) decode_scored_fp8;
    decltype(&::pa_beam_select) beam_select;
    decltype(&::pa_sequences_fork) sequences_fork;
    decltype(&::pa_blocks_compact_slots) blocks_compact_slots;
    decltype(&::pa_blocks_copy) blocks_copy;
    decltype(&::pa_strerror) strerror;
} g_lib;

template <typename F>
bool find(void *handle, const char *name, F *f) {
    *f = reinterpret_cast<F>(dlsym(handle, name));
    if (!*f) PyErr_Format(PyExc_RuntimeError, "%s is missing from the library", name);
    return *f != nullptr;
}

// init(path of libpagedattn.so, PAError, raw_stream, current_device, set_device)
PyObject *init(PyObject *, PyObject *args) {
    const char *path;
    PyObject *error, *raw_stream, *current_device, *set_device;
    if (!PyArg_ParseTuple(args, "sOOOO", &path, &error, &raw_stream, &current_device, &set_device)) return nullptr;
    void *h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
    if (!find(h, "pa_rope_write", &g_lib.rope_write) || !find(h, "pa_rope_write_fp8", &g_lib.rope_write_fp8) ||
        !find(h, "pa_decode_scored", &g_lib.decode_scored) ||
        !find(h, "pa_decode_scored_fp8", &g_lib.decode_scored_fp8) ||
        !find(h, "pa_beam_select", &g_lib.beam_select) || !find(h, "pa_sequences_fork", &g_lib.sequences_fork) ||
        !find(h, "pa_blocks_compact_slots", &g_lib.blocks_compact_slots) || !find(h, "pa_blocks_copy", &g_lib.blocks_copy) ||
        !find(h, "pa_strerror", &g_lib.strerror))
        return nullptr;
    for (PyObject *o : {error, raw_stream, current_device, set_device}) Py_INCREF(o);
    g_error = error, g_raw_stream = raw_stream, g_current_device = current_device, g_set_device = set_device;
    Py_RETURN_NONE;
}

// ---- arguments ---------------------------------------------------------------------------

// A call's arguments: the first failure sets the Python exception and `ok` to
// false; what is taken after it is not looked at.
struct Call {
    const char *name;
    int device = -1;
    bool ok = true;

    bool fail(PyObject *type, const char *format, ...) {
        if (ok) {
            va_list v;
            va_start(v, format);
            PyErr_FormatV(type, format, v);
            va_end(v);
        }
        return ok = false;
    }
    bool need(bool fits, const char *what) { return fits || fail(PyExc_ValueError, "%s: %s", name, what); }
};

enum Type { kBf16, kF32, kI32, kI64, kU8 };
constexpr c10::ScalarType kScalar[] = {c10::ScalarType::BFloat16, c10::ScalarType::Float, c10::ScalarType::Int,
                                       c10::ScalarType::Long, c10::ScalarType::Byte};
constexpr const char *kTypeName[] = {"torch.bfloat16", "torch.float32", "torch.int32", "torch.int64", "torch.uint8"};

struct Tensor {
    void *at = nullptr;
    int64_t size[4] = {0, 0, 0, 0};
    int64_t row = 0;   // elements between rows of dimension 0 (kRows)
    int ndim = 0;
    bool f32 = false;  // logits: fp32 rather than bf16

    bool is(std::initializer_list<int64_t> shape) const {
        int d = 0;
        for (const int64_t n : shape)
            if (d >= ndim || size[d++] != n) return false;
        return d == ndim;
    }
};

enum Layout { kWhole, kRows };  // contiguous, or contiguous but for the stride of dimension 0

const at::Tensor *cuda_tensor(Call &c, PyObject *o, const char *what) {
    if (!c.ok) return nullptr;
    if (!THPVariable_Check(o)) return c.fail(PyExc_TypeError, "%s must be a torch.Tensor", what), nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) return c.fail(PyExc_ValueError, "%s must be a CUDA tensor", what), nullptr;
    const int dev = static_cast<int>(t.get_device());
    if (c.device < 0) c.device = dev;
    if (dev != c.device)
        return c.fail(PyExc_ValueError, "%s: tensors on several devices (%s on cuda:%d, others on cuda:%d)", c.name, what,
                      dev, c.device),
               nullptr;
    return &t;
}

// `type` < 0: logits, bf16 or fp32.
Tensor take(Call &c, PyObject *o, const char *what, int type, int ndim, Layout layout = kWhole) {
    Tensor r;
    if (c.ok && THPVariable_Check(o)) {  // (the type first: it says most)
        const c10::ScalarType got = THPVariable_Unpack(o).scalar_type();
        r.f32 = got == c10::ScalarType::Float;
        if (type < 0 ? got != c10::ScalarType::BFloat16 && !r.f32 : got != kScalar[type]) {
            c.fail(PyExc_TypeError, "%s must be %s, got %s", what,
                   type < 0 ? "torch.bfloat16 or torch.float32" : kTypeName[type], c10::toString(got));
            return r;
        }
    }
    const at::Tensor *t = cuda_tensor(c, o, what);
    if (!t) return r;
    if (t->dim() != ndim) {
        c.fail(PyExc_ValueError, "%s must have %d dims, got %d", what, ndim, static_cast<int>(t->dim()));
        return r;
    }
    r.ndim = ndim;
    for (int d = 0; d < ndim; ++d) r.size[d] = t->size(d);
    if (layout == kRows) {
        int64_t want = 1;
        for (int d = ndim - 1; d >= 1; --d) {
            if (r.size[d] > 1 && t->stride(d) != want) {
                c.fail(PyExc_ValueError, "%s: every row (all but dimension 0) must be contiguous", what);
                return r;
            }
            want *= r.size[d];
        }
        r.row = r.size[0] > 1 ? t->stride(0) : want;  // (a single row's stride says nothing)
    } else if (!t->is_contiguous()) {
        c.fail(PyExc_ValueError, "%s must be contiguous", what);
        return r;
    }
    r.at = t->data_ptr();
    return r;
}

Tensor take_optional(Call &c, PyObject *o, const char *what, int type, int ndim) {
    return o == Py_None ? Tensor() : take(c, o, what, type, ndim);
}

int32_t *take_status(Call &c, PyObject *o) {
    return static_cast<int32_t *>(take_optional(c, o, "status", kI32, 1).at);
}

// A workspace of any type: its address and bytes.
void *take_space(Call &c, PyObject *o, size_t *bytes) {
    *bytes = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor *t = cuda_tensor(c, o, "workspace");
    if (!t || !c.need(t->is_contiguous(), "workspace must be contiguous")) return nullptr;
    *bytes = t->nbytes();
    return t->data_ptr();
}

int32_t take_int(Call &c, PyObject *o, const char *what) {
    if (!c.ok) return 0;
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    if (v == -1 && !overflow && PyErr_Occurred()) return c.ok = false, 0;
    if (overflow || v < INT32_MIN || v > INT32_MAX) c.fail(PyExc_ValueError, "%s: %s is out of range", c.name, what);
    return static_cast<int32_t>(v);
}

float take_float(Call &c, PyObject *o) {
    if (!c.ok) return 0.f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) c.ok = false;
    return static_cast<float>(v);
}

// ---- the call itself -----------------------------------------------------------------------

long ask(PyObject *callable, PyObject *arg, bool *ok) {
    PyObject *r = arg ? PyObject_CallOneArg(callable, arg) : PyObject_CallNoArgs(callable);
    const long v = r ? PyLong_AsLong(r) : -1;
    Py_XDECREF(r);
    if (v == -1 && PyErr_Occurred()) *ok = false;
    return v;
}

bool set_device(int device) {
    PyObject *d = PyLong_FromLong(device);
    PyObject *r = d ? PyObject_CallOneArg(g_set_device, d) : nullptr;
    Py_XDECREF(d);
    Py_XDECREF(r);
    return r != nullptr;
}

// f(stream) on the tensors' device, on `stream` (a torch.cuda.Stream) or the
// device's current stream; None, or PAError from its return code.
template <typename F>
PyObject *run(Call &c, PyObject *stream, F &&f) {
    if (!c.ok) return nullptr;
    pa_stream_t s = nullptr;
    if (stream == Py_None) {
        PyObject *d = PyLong_FromLong(c.device);
        PyObject *r = d ? PyObject_CallOneArg(g_raw_stream, d) : nullptr;
        Py_XDECREF(d);
        if (!r) return nullptr;
        s = static_cast<pa_stream_t>(PyLong_AsVoidPtr(r));
        Py_DECREF(r);
    } else {
        PyObject *dev = PyObject_GetAttrString(stream, "device_index");
        const long index = dev ? PyLong_AsLong(dev) : -1;
        Py_XDECREF(dev);
        if (PyErr_Occurred()) return nullptr;
        if (index != c.device) {
            c.fail(PyExc_ValueError, "%s: stream on cuda:%d, tensors on cuda:%d", c.name, static_cast<int>(index), c.device);
            return nullptr;
        }
        PyObject *r = PyObject_GetAttrString(stream, "cuda_stream");
        if (!r) return nullptr;
        s = static_cast<pa_stream_t>(PyLong_AsVoidPtr(r));
        Py_DECREF(r);
    }
    if (PyErr_Occurred()) return nullptr;
    bool ok = true;
    const long current = ask(g_current_device, nullptr, &ok);
    if (!ok) return nullptr;
    if (current != c.device && !set_device(c.device)) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;  // (a launch waits while the device's queue is full)
    rc = f(s);
    Py_END_ALLOW_THREADS;
    if (current != c.device && !set_device(static_cast<int>(current))) return nullptr;
    if (rc == PA_OK) Py_RETURN_NONE;
    PyObject *e = PyObject_CallFunction(g_error, "sis", c.name, rc, g_lib.strerror(rc));
    if (e) PyErr_SetObject(g_error, e);
    Py_XDECREF(e);
    return nullptr;
}

bool count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", static_cast<int>(want), static_cast<int>(n));
    return n == want;
}

pa_cache_desc desc_of(const Tensor &pool) {
    return pa_cache_desc{static_cast<int32_t>(pool.size[0]), static_cast<int32_t>(pool.size[1]),
                         static_cast<int32_t>(pool.size[2]), static_cast<int32_t>(pool.size[3])};
}

// Sizes that a C argument of 32 bits takes.
bool fits_int(std::initializer_list<int64_t> sizes) {
    for (const int64_t n : sizes)
        if (n > INT32_MAX) return false;
    return true;
}

// rope_write(fp8, q_out, q, k_new, v_new, positions, slot_mapping, k_cache, v_cache, k_scale, v_scale,
//            rope (a buffer), status, stream)
PyObject *rope_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 14)) return nullptr;
    const bool fp8 = a[0] == Py_True;
    Call c{fp8 ? "pa_rope_write_fp8" : "pa_rope_write"};
    const Tensor qo = take(c, a[1], "q_out", kBf16, 3, kRows), q = take(c, a[2], "q", kBf16, 3, kRows);
    const Tensor k = take(c, a[3], "k_new", kBf16, 3, kRows), v = take(c, a[4], "v_new", kBf16, 3, kRows);
    const Tensor pos = take(c, a[5], "positions", kI32, 1), slots = take(c, a[6], "slot_mapping", kI64, 1);
    const Tensor kc = take(c, a[7], "k_cache", fp8 ? kU8 : kBf16, 4), vc = take(c, a[8], "v_cache", fp8 ? kU8 : kBf16, 4);
    const float ks = fp8 ? take_float(c, a[9]) : 1.f, vs = fp8 ? take_float(c, a[10]) : 1.f;
    int32_t *status = take_status(c, a[12]);
    if (!c.ok) return nullptr;
    const int64_t tokens = q.size[0], hq = q.size[1], d = q.size[2], hkv = kc.size[2];
    c.need(qo.is({tokens, hq, d}), "q_out and q must be [N, Hq, D]") &&
        c.need(k.is({tokens, hkv, d}) && v.is({tokens, hkv, d}) && kc.size[3] == d &&
                   vc.is({kc.size[0], kc.size[1], hkv, d}),
               "k_new and v_new must be [N, Hkv, D] matching q and the pools") &&
        c.need(pos.is({tokens}) && slots.is({tokens}), "positions and slot_mapping must be [N]") &&
        c.need(fits_int({hq, kc.size[0], kc.size[1], hkv}), "a size is out of range");
    if (!c.ok) return nullptr;
    Py_buffer plan;
    if (PyObject_GetBuffer(a[11], &plan, PyBUF_SIMPLE) < 0) return nullptr;
    PyObject *r = nullptr;
    if (plan.len != static_cast<Py_ssize_t>(sizeof(pa_rope))) {
        PyErr_SetString(PyExc_TypeError, "rope must be a plan made by pa_rope_init");
    } else {
        const pa_rope *rope = static_cast<const pa_rope *>(plan.buf);
        const int64_t *sl = static_cast<const int64_t *>(slots.at);
        const int32_t *ps = static_cast<const int32_t *>(pos.at), heads = static_cast<int32_t>(hq);
        r = run(c, a[13], [&](pa_stream_t s) {
            return fp8 ? g_lib.rope_write_fp8(qo.at, qo.row, q.at, q.row, k.at, k.row, v.at, v.row, ps, sl, tokens, heads,
                                              kc.at, vc.at, desc_of(kc), ks, vs, rope, status, s)
                       : g_lib.rope_write(qo.at, qo.row, q.at, q.row, k.at, k.row, v.at, v.row, ps, sl, tokens, heads,
                                          kc.at, vc.at, desc_of(kc), rope, status, s);
        });
    }
    PyBuffer_Release(&plan);
    return r;
}

// decode_scored(fp8, out, lse, q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens, scale, softcap,
//               alibi_slopes, window, prefix_lens, max_prefix, num_splits, workspace, status, stream)
PyObject *decode_scored(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 20)) return nullptr;
    const bool fp8 = a[0] == Py_True;
    Call c{fp8 ? "pa_decode_scored_fp8" : "pa_decode_scored"};
    // q and out: [B, Hq, D], or [B, q_len, Hq, D]
    const int nd = THPVariable_Check(a[3]) && THPVariable_Unpack(a[3]).dim() == 4 ? 4 : 3;
    const Tensor q = take(c, a[3], "q", kBf16, nd), out = take(c, a[1], "out", kBf16, nd);
    const Tensor lse = take_optional(c, a[2], "lse", kF32, nd - 1);
    const Tensor kc = take(c, a[4], "k_cache", fp8 ? kU8 : kBf16, 4), vc = take(c, a[5], "v_cache", fp8 ? kU8 : kBf16, 4);
    const float ks = fp8 ? take_float(c, a[6]) : 1.f, vs = fp8 ? take_float(c, a[7]) : 1.f;
    const Tensor bt = take(c, a[8], "block_tables", kI32, 2), sl = take(c, a[9], "seq_lens", kI32, 1);
    const float scale = take_float(c, a[10]);
    const Tensor slopes = take_optional(c, a[12], "alibi_slopes", kF32, 1);
    const Tensor prefix = take_optional(c, a[14], "prefix_lens", kI32, 1);
    pa_score_rules rules{};
    rules.softcap = take_float(c, a[11]);
    rules.alibi_slopes = static_cast<const float *>(slopes.at);
    rules.window = take_int(c, a[13], "window");
    rules.prefix_lens = static_cast<const int32_t *>(prefix.at);
    const int32_t splits = take_int(c, a[16], "num_splits");
    size_t bytes = 0;
    void *space = take_space(c, a[17], &bytes);
    int32_t *status = take_status(c, a[18]);
    if (!c.ok) return nullptr;
    const int64_t B = q.size[0], q_len = nd == 4 ? q.size[1] : 1, hq = q.size[nd - 2], d = q.size[nd - 1];
    bool same = true, lse_ok = true;
    for (int i = 0; i < nd; ++i) same &= out.size[i] == q.size[i];
    for (int i = 0; i < nd - 1; ++i) lse_ok &= lse.ndim == 0 || lse.size[i] == q.size[i];
    c.need(same && kc.size[3] == d && vc.is({kc.size[0], kc.size[1], kc.size[2], d}) && bt.size[0] == B && sl.is({B}),
           "inconsistent out / q / cache / table shapes") &&
        c.need(lse_ok, "lse must have q's shape without its last dimension") &&
        c.need(slopes.ndim == 0 || slopes.is({hq}), "alibi_slopes must be [Hq]") &&
        c.need(prefix.ndim == 0 || prefix.is({B}), "prefix_lens must be [B]") &&
        c.need(fits_int({B, q_len, hq, bt.size[1], kc.size[0], kc.size[1], kc.size[2]}), "a size is out of range");
    if (!c.ok) return nullptr;
    if (prefix.ndim) {  // (the default bound: the table's tokens)
        const int64_t all = bt.size[1] * kc.size[1];
        rules.max_prefix = a[15] == Py_None ? static_cast<int32_t>(all < INT32_MAX ? all : INT32_MAX)
                                            : take_int(c, a[15], "max_prefix");
    }
    const int32_t *tables = static_cast<const int32_t *>(bt.at), *lens = static_cast<const int32_t *>(sl.at);
    const int32_t mb = static_cast<int32_t>(bt.size[1]), b = static_cast<int32_t>(B), h = static_cast<int32_t>(hq);
    const int32_t ql = static_cast<int32_t>(q_len);
    float *l = static_cast<float *>(lse.at);
    return run(c, a[19], [&](pa_stream_t s) {
        return fp8 ? g_lib.decode_scored_fp8(out.at, l, q.at, ql, kc.at, vc.at, desc_of(kc), ks, vs, tables, mb, lens, b, h,
                                             scale, &rules, splits, space, bytes, status, s)
                   : g_lib.decode_scored(out.at, l, q.at, ql, kc.at, vc.at, desc_of(kc), tables, mb, lens, b, h, scale,
                                         &rules, splits, space, bytes, status, s);
    });
}

// beam_select(scores, tokens, parents, logits, cum, finished, eos, workspace, stream)
PyObject *beam_select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 9)) return nullptr;
    Call c{"pa_beam_select"};
    const Tensor logits = take(c, a[3], "logits", -1, 2, kRows);
    const Tensor scores = take(c, a[0], "scores", kF32, 2), tokens = take(c, a[1], "tokens", kI32, 2);
    const Tensor parents = take(c, a[2], "parents", kI32, 2), cum = take(c, a[4], "cum", kF32, 2);
    const Tensor finished = take_optional(c, a[5], "finished", kU8, 2);
    const int32_t eos = take_int(c, a[6], "eos");
    size_t bytes = 0;
    void *space = take_space(c, a[7], &bytes);
    if (!c.ok) return nullptr;
    const int64_t groups = cum.size[0], beams = cum.size[1], K = scores.size[1];
    c.need(logits.size[0] == groups * beams && scores.is({groups, K}) && tokens.is({groups, K}) && parents.is({groups, K}),
           "logits must be [groups * beams, vocab]; scores, tokens and parents [groups, K]") &&
        c.need(finished.ndim == 0 || finished.is({groups, beams}), "finished must be [groups, beams]") &&
        c.need(fits_int({groups, beams, K, logits.size[1]}), "a size is out of range");
    return run(c, a[8], [&](pa_stream_t s) {
        return g_lib.beam_select(static_cast<float *>(scores.at), static_cast<int32_t *>(tokens.at),
                                 static_cast<int32_t *>(parents.at), logits.at, logits.f32 ? PA_LOGITS_F32 : PA_LOGITS_BF16,
                                 logits.row, static_cast<const float *>(cum.at), static_cast<const uint8_t *>(finished.at),
                                 eos, static_cast<int32_t>(groups), static_cast<int32_t>(beams),
                                 static_cast<int32_t>(logits.size[1]), static_cast<int32_t>(K), space, bytes, s);
    });
}

// ---- pools that share tables ------------------------------------------------------------------

// The tensors, not their addresses: what a tensor's memory is may change (set_, .data =,
// resize_), and every call takes it anew.
struct Pools {
    std::vector<at::Tensor> tensors;
    pa_cache_desc desc;
    int32_t elem_bytes;
    int device;
};
// A call's view of them (the library takes at most 256).
constexpr size_t kMostPools = 256;
struct PoolsNow {
    void *at[kMostPools];
    int32_t n;
    pa_cache_desc desc;
    int32_t elem_bytes;
};
constexpr const char *kPools = "_pa_binding.pools";

void free_pools(PyObject *capsule) { delete static_cast<Pools *>(PyCapsule_GetPointer(capsule, kPools)); }

// pools(tensor, ...) -> a handle that holds the tensors, alike in every respect
PyObject *pools(PyObject *, PyObject *const *a, Py_ssize_t n) {
    Call c{"PoolSet"};
    if (n < 1) return c.fail(PyExc_ValueError, "a PoolSet needs at least one pool"), nullptr;
    Pools *p = new (std::nothrow) Pools;
    if (!p) return PyErr_NoMemory();
    try {
        const bool u8 = THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).scalar_type() == c10::ScalarType::Byte;
        Tensor first;
        for (Py_ssize_t i = 0; i < n && c.ok; ++i) {
            const Tensor t = take(c, a[i], "every pool", u8 ? kU8 : kBf16, 4);
            if (i == 0) first = t;
            c.ok && c.need(t.is({first.size[0], first.size[1], first.size[2], first.size[3]}), "the pools differ in shape") &&
                c.need(fits_int({t.size[0], t.size[1], t.size[2], t.size[3]}), "a size is out of range");
            if (c.ok) p->tensors.push_back(THPVariable_Unpack(a[i]));
        }
        p->desc = desc_of(first);
        p->elem_bytes = u8 ? 1 : 2;
        p->device = c.device;
    } catch (const std::exception &e) {
        c.fail(PyExc_RuntimeError, "%s", e.what());
    }
    PyObject *capsule = c.ok ? PyCapsule_New(p, kPools, free_pools) : nullptr;
    if (!capsule) delete p;
    return capsule;
}

void pools_of(Call &c, PyObject *o, PoolsNow *now) {
    const Pools *p = static_cast<const Pools *>(PyCapsule_GetPointer(o, kPools));
    if (!p) {
        c.ok = false;
        return;
    }
    c.device = p->device;
    now->desc = p->desc;
    now->elem_bytes = p->elem_bytes;
    now->n = static_cast<int32_t>(p->tensors.size());
    const int64_t size[4] = {p->desc.num_blocks, p->desc.block_size, p->desc.num_kv_heads, p->desc.head_dim};
    const c10::ScalarType type = p->elem_bytes == 1 ? c10::ScalarType::Byte : c10::ScalarType::BFloat16;
    const size_t bytes = static_cast<size_t>(size[0]) * size[1] * size[2] * size[3] * p->elem_bytes;
    for (size_t i = 0; i < p->tensors.size(); ++i) {
        const at::Tensor &t = p->tensors[i];
        const c10::IntArrayRef now_size = t.sizes();
        const c10::Device device = t.device();
        const bool same = now_size.size() == 4 && now_size[0] == size[0] && now_size[1] == size[1] && now_size[2] == size[2] &&
                          now_size[3] == size[3] && t.scalar_type() == type && t.is_contiguous() && device.is_cuda() &&
                          device.index() == p->device && t.has_storage() &&
                          t.storage().nbytes() >= static_cast<size_t>(t.storage_offset()) * p->elem_bytes + bytes;
        if (!c.need(same, "a pool is not the tensor any more (shape, type, device or size of its memory) that the "
                          "PoolSet was made of"))
            return;
        if (i < kMostPools) now->at[i] = t.data_ptr();
    }
}

int32_t *i32(const Tensor &t) { return static_cast<int32_t *>(t.at); }

// sequences_fork(new_tables, new_lens, new_refs, slot_mapping, tables, lens, refs, parents, pools, workspace,
//                status, stream)
PyObject *sequences_fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 12)) return nullptr;
    Call c{"pa_sequences_fork"};
    PoolsNow p;
    pools_of(c, a[8], &p);
    const Tensor nt = take(c, a[0], "new_tables", kI32, 2), nl = take(c, a[1], "new_lens", kI32, 1);
    const Tensor nr = take(c, a[2], "new_refs", kI32, 1), slots = take(c, a[3], "slot_mapping", kI64, 1);
    const Tensor tables = take(c, a[4], "tables", kI32, 2), lens = take(c, a[5], "lens", kI32, 1);
    const Tensor refs = take(c, a[6], "refs", kI32, 1), parents = take(c, a[7], "parents", kI32, 1);
    size_t bytes = 0;
    void *space = take_space(c, a[9], &bytes);
    int32_t *status = take_status(c, a[10]);
    if (!c.ok) return nullptr;
    const int64_t rows = parents.size[0], old = tables.size[0], mb = tables.size[1], nb = p.desc.num_blocks;
    c.need(lens.is({old}) && refs.is({nb}) && nr.is({nb}), "tables, lens and refs must be [B, max_blocks], [B] and [num_blocks]") &&
        c.need(nt.is({rows, mb}) && nl.is({rows}) && slots.is({rows}),
               "the new tables, lens and slots must have a row for every parent") &&
        c.need(fits_int({rows, old, mb}), "a size is out of range");
    return run(c, a[11], [&](pa_stream_t s) {
        return g_lib.sequences_fork(i32(nt), i32(nl), i32(nr), static_cast<int64_t *>(slots.at), i32(tables), i32(lens),
                                    i32(refs), i32(parents), static_cast<int32_t>(old), static_cast<int32_t>(rows),
                                    static_cast<int32_t>(mb), p.at, p.n,
                                    p.elem_bytes, p.desc, space, bytes, status, s);
    });
}

// blocks_compact(new_tables, new_refs, remap, n_live, tables, lens, refs, pools, workspace, status, stream,
//                new_slots, slots)
PyObject *blocks_compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 13)) return nullptr;
    Call c{"pa_blocks_compact"};
    PoolsNow p;
    pools_of(c, a[7], &p);
    const Tensor nt = take(c, a[0], "new_tables", kI32, 2), nr = take(c, a[1], "new_refs", kI32, 1);
    const Tensor remap = take(c, a[2], "remap", kI32, 1), live = take(c, a[3], "n_live", kI32, 1);
    const Tensor tables = take(c, a[4], "tables", kI32, 2), lens = take(c, a[5], "lens", kI32, 1);
    const Tensor refs = take(c, a[6], "refs", kI32, 1);
    size_t bytes = 0;
    void *space = take_space(c, a[8], &bytes);
    int32_t *status = take_status(c, a[9]);
    const Tensor ns = take_optional(c, a[11], "new_slots", kI64, 1), slots = take_optional(c, a[12], "slots", kI64, 1);
    if (!c.ok) return nullptr;
    const int64_t B = tables.size[0], mb = tables.size[1], nb = p.desc.num_blocks;
    c.need(nt.is({B, mb}) && lens.is({B}) && refs.is({nb}) && nr.is({nb}) && remap.is({nb}) && live.is({1}),
           "tables [B, max_blocks], lens [B], counts and remap [num_blocks], n_live [1]") &&
        c.need(ns.ndim == slots.ndim && (slots.ndim == 0 || (slots.is({B}) && ns.is({B}))),
               "slots and new_slots must both be [B], or both be left out") &&
        c.need(fits_int({B, mb}), "a size is out of range");
    return run(c, a[10], [&](pa_stream_t s) {
        return g_lib.blocks_compact_slots(i32(nt), i32(nr), i32(remap), i32(live), static_cast<int64_t *>(ns.at),
                                          i32(tables), i32(lens), i32(refs), static_cast<const int64_t *>(slots.at),
                                          static_cast<int32_t>(B), static_cast<int32_t>(mb), p.at, p.n, p.elem_bytes, p.desc, space, bytes,
                                          status, s);
    });
}

// blocks_copy(pools, pairs, status, stream)
PyObject *blocks_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (!count_is(n, 4)) return nullptr;
    Call c{"pa_blocks_copy"};
    PoolsNow p;
    pools_of(c, a[0], &p);
    const Tensor pairs = take(c, a[1], "pairs", kI32, 2);
    int32_t *status = take_status(c, a[2]);
    if (!c.ok) return nullptr;
    c.need(pairs.size[1] == 2 && fits_int({pairs.size[0]}), "pairs must be [n, 2]");
    return run(c, a[3], [&](pa_stream_t s) {
        return g_lib.blocks_copy(p.at, p.n, p.elem_bytes, p.desc, i32(pairs),
                                 static_cast<int32_t>(pairs.size[0]), status, s);
    });
}

// A C++ exception (a tensor without storage, for instance) as a Python one.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {{"init", init, METH_VARARGS, nullptr},
                          method<rope_write>("rope_write"),
                          method<decode_scored>("decode_scored"),
                          method<beam_select>("beam_select"),
                          method<pools>("pools"),
                          method<sequences_fork>("sequences_fork"),
                          method<blocks_compact>("blocks_compact"),
                          method<blocks_copy>("blocks_copy"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pa_binding", "Calls of libpagedattn with torch tensors.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_binding(void) { return PyModule_Create(&kModule); }
