// The serving step's calls from Python without ctypes: a step of small batches
// takes its GPU 3 to 8 us a call, and one check per tensor and one conversion per
// argument in Python took longer than that (pa_append_q8b for 64 single tokens:
// 9.2 us a call, 2.4 of them on the GPU).
//
// Each function takes its tensors as they are, checks their types, shapes,
// layouts and device (ValueError), calls the C entry point of its name and
// returns its status.
#include <Python.h>

#include <climits>
#include <exception>
#include <sstream>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

struct Raised {};  // the Python exception is set

[[noreturn]] void raise(PyObject *kind, const std::string &text) {
    PyErr_SetString(kind, text.c_str());
    throw Raised{};
}

const at::Tensor &tensor(PyObject *o) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string("expected a tensor, got ") + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int number(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT_MIN || v > INT_MAX) raise(PyExc_OverflowError, "a number past 32 bits");
    return (int)v;
}

int size_of(const at::Tensor &t, int dim) {
    const int64_t n = t.size(dim);
    if (n > INT_MAX) raise(PyExc_ValueError, "a size past 32 bits");
    return (int)n;
}

void expect(bool ok, const char *what) {
    if (!ok) raise(PyExc_ValueError, what);
}

bool shaped(const at::Tensor &t, std::initializer_list<int64_t> sizes) {
    return t.sizes() == at::IntArrayRef(sizes);
}

pa_dtype dtype_of(const at::Tensor &t) {
    switch (t.scalar_type()) {
        case at::kFloat: return PA_F32;
        case at::kHalf: return PA_F16;
        case at::kBFloat16: return PA_BF16;
        default: raise(PyExc_ValueError, std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
    }
}

// The call's device is the current one, and its stream that one's current stream
// unless the caller gives one (a torch stream or a handle).
struct Call {
    int device = c10::cuda::current_device();
    cudaStream_t stream;

    explicit Call(PyObject *given) {
        if (given == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
            return;
        }
        PyObject *handle = PyLong_Check(given) ? Py_NewRef(given) : PyObject_GetAttrString(given, "cuda_stream");
        if (!handle) throw Raised{};
        stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
        Py_DECREF(handle);
        if (PyErr_Occurred()) throw Raised{};
    }

    // Address of a contiguous tensor of the type on the device.
    void *address(const at::Tensor &t, at::ScalarType type) const {
        if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != device || !t.is_contiguous()) {
            std::ostringstream s;
            s << "expected a contiguous " << c10::toString(type) << " tensor on cuda:" << device << ", got "
              << c10::toString(t.scalar_type()) << " on " << t.device() << " of shape " << t.sizes() << " and strides "
              << t.strides();
            raise(PyExc_ValueError, s.str());
        }
        return t.data_ptr();
    }
    void *address(const at::Tensor &t) const { return address(t, t.scalar_type()); }
    template <typename T> T *i32(const at::Tensor &t) const { return static_cast<T *>(address(t, at::kInt)); }
    int32_t *i32(const at::Tensor &t) const { return i32<int32_t>(t); }
};

// An int8 cache with a scale per (block, head).
struct Cache {
    const at::Tensor &k, &v, &ks, &vs;
    int nb, heads, bs, dim;

    explicit Cache(PyObject *const *a) : k(tensor(a[0])), v(tensor(a[1])), ks(tensor(a[2])), vs(tensor(a[3])) {
        const char *want = "expected k_cache and v_cache [NB, Hkv, bs, D] with k_scale and v_scale [NB, Hkv]";
        expect(k.dim() == 4 && v.sizes() == k.sizes(), want);
        nb = size_of(k, 0);
        heads = size_of(k, 1);
        bs = size_of(k, 2);
        dim = size_of(k, 3);
        expect(shaped(ks, {nb, heads}) && shaped(vs, {nb, heads}), want);
    }
    int8_t *codes(const Call &c, const at::Tensor &t) const { return static_cast<int8_t *>(c.address(t, at::kChar)); }
    float *scales(const Call &c, const at::Tensor &t) const { return static_cast<float *>(c.address(t, at::kFloat)); }
};

// The C call without the interpreter's lock: a launch waits while the stream's queue is full.
template <typename F> int unlocked(F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

// `f(args)` as a Python function of `count` positional arguments.
template <typename F> PyObject *enter(Py_ssize_t n, Py_ssize_t count, F f) {
    if (n != count) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", count, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// state, num_blocks, block_size, block_tables, context_lens, new_lens, q_start, slot_mapping, cow_pairs, num_cow, stream
PyObject *dpool_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return enter(n, 11, [&]() -> int {
        const Call c(a[10]);
        const at::Tensor &tables = tensor(a[3]), &ctx = tensor(a[4]), &lens = tensor(a[5]), &q_start = tensor(a[6]),
                         &slots = tensor(a[7]), &pairs = tensor(a[8]), &num = tensor(a[9]);
        const char *want = "pa_dpool_append: one row, length and pair per sequence, and one more q_start";
        expect(tables.dim() == 2 && slots.dim() == 1, want);
        const int S = size_of(tables, 0), MB = size_of(tables, 1), T = size_of(slots, 0);
        expect(shaped(ctx, {S}) && shaped(lens, {S}) && shaped(q_start, {S + 1ll}) && shaped(pairs, {S, 2}), want);
        expect(num.numel() > 0, "pa_dpool_append: num_cow is one number");
        int32_t *state = c.i32(tensor(a[0])), *t = c.i32(tables), *l = c.i32(ctx), *nl = c.i32(lens), *q = c.i32(q_start),
                *sl = c.i32(slots), *nc = c.i32(num);
        int64_t *pr = static_cast<int64_t *>(c.address(pairs, at::kLong));
        const int nb = number(a[1]), bs = number(a[2]);
        return unlocked([&] { return pa_dpool_append(state, nb, bs, t, MB, l, nl, S, q, sl, T, pr, nc, c.stream); });
    });
}

// state, num_blocks, block_size, block_tables, context_lens, finished, stream
PyObject *dpool_release(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return enter(n, 7, [&]() -> int {
        const Call c(a[6]);
        const at::Tensor &tables = tensor(a[3]), &ctx = tensor(a[4]), &fin = tensor(a[5]);
        const char *want = "pa_dpool_release: one row, length and mark per sequence";
        expect(tables.dim() == 2, want);
        const int S = size_of(tables, 0), MB = size_of(tables, 1);
        expect(shaped(ctx, {S}) && shaped(fin, {S}), want);
        int32_t *state = c.i32(tensor(a[0])), *t = c.i32(tables), *l = c.i32(ctx), *f = c.i32(fin);
        const int nb = number(a[1]), bs = number(a[2]);
        return unlocked([&] { return pa_dpool_release(state, nb, bs, t, MB, l, f, S, c.stream); });
    });
}

// key, value, q_start, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, stream
PyObject *append_q8b(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return enter(n, 10, [&]() -> int {
        const Call c(a[9]);
        const at::Tensor &key = tensor(a[0]), &value = tensor(a[1]), &q_start = tensor(a[2]), &tables = tensor(a[7]),
                         &ctx = tensor(a[8]);
        const Cache m(a + 3);
        expect(key.dim() == 3 && key.size(1) == m.heads && key.size(2) == m.dim && value.sizes() == key.sizes(),
               "pa_append_q8b: key and value are [T, Hkv, D]");
        const int T = size_of(key, 0);
        const char *want = "pa_append_q8b: one table row and length per sequence, and one more q_start";
        expect(tables.dim() == 2, want);
        const int S = size_of(tables, 0), MB = size_of(tables, 1);
        expect(shaped(q_start, {S + 1ll}) && shaped(ctx, {S}), want);
        const pa_dtype dt = dtype_of(key);
        const void *k = c.address(key), *v = c.address(value, key.scalar_type());
        const int32_t *q = c.i32(q_start), *t = c.i32(tables), *l = c.i32(ctx);
        int8_t *kc = m.codes(c, m.k), *vc = m.codes(c, m.v);
        float *ks = m.scales(c, m.ks), *vs = m.scales(c, m.vs);
        return unlocked([&] {
            return pa_append_q8b(k, v, dt, q, T, kc, vc, ks, vs, t, MB, l, S, m.nb, m.heads, m.dim, m.bs, c.stream);
        });
    });
}

// out, query, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens, scale, max_context_len, workspace or None,
// seq_order or None, stream
PyObject *decode_q8b(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return enter(n, 13, [&]() -> int {
        const Call c(a[12]);
        const at::Tensor &out = tensor(a[0]), &query = tensor(a[1]), &tables = tensor(a[6]), &ctx = tensor(a[7]);
        const Cache m(a + 2);
        const char *want = "pa_decode_q8b: query and out [S, Hq, D], one table row and length per sequence";
        expect(query.dim() == 3 && query.size(2) == m.dim && out.sizes() == query.sizes() && tables.dim() == 2, want);
        const int S = size_of(query, 0), heads = size_of(query, 1), MB = size_of(tables, 1);
        expect(shaped(ctx, {S}) && tables.size(0) == S, want);
        void *ws = nullptr;
        size_t ws_bytes = 0;
        if (a[10] != Py_None) {
            const at::Tensor &w = tensor(a[10]);
            ws = c.address(w);
            ws_bytes = w.nbytes();
            if (ws_bytes == 0) return PA_ERR_WORKSPACE;  // an empty tensor has no address: not "no workspace"
        }
        const int32_t *order = nullptr;
        if (a[11] != Py_None) {
            expect(shaped(tensor(a[11]), {S}), "pa_decode_q8b: seq_order has one entry per sequence");
            order = c.i32(tensor(a[11]));
        }
        const double scale = PyFloat_AsDouble(a[8]);
        if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
        const int max_ctx = number(a[9]);
        const pa_dtype qt = dtype_of(query), ot = dtype_of(out);
        void *o = c.address(out);
        const void *q = c.address(query);
        const int32_t *t = c.i32(tables), *l = c.i32(ctx);
        const int8_t *kc = m.codes(c, m.k), *vc = m.codes(c, m.v);
        const float *ks = m.scales(c, m.ks), *vs = m.scales(c, m.vs);
        return unlocked([&] {
            return pa_decode_q8b(o, q, qt, kc, vc, ks, vs, t, MB, l, S, heads, m.heads, m.dim, (float)scale, m.bs, m.nb,
                                 max_ctx, ot, order, ws, ws_bytes, c.stream);
        });
    });
}

// k_cache, v_cache, k_scale, v_scale, src_dst_pairs, num_pairs or None, stream
PyObject *copy_blocks_q8b(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return enter(n, 7, [&]() -> int {
        const Call c(a[6]);
        const Cache m(a);
        const at::Tensor &pairs = tensor(a[4]);
        expect(pairs.dim() == 2 && pairs.size(1) == 2, "pa_copy_blocks_q8b: src_dst_pairs is [n, 2]");
        const int count = size_of(pairs, 0);
        int8_t *kc = m.codes(c, m.k), *vc = m.codes(c, m.v);
        float *ks = m.scales(c, m.ks), *vs = m.scales(c, m.vs);
        const int64_t *pr = static_cast<const int64_t *>(c.address(pairs, at::kLong));
        const int32_t *num = nullptr;
        if (a[5] != Py_None) {
            expect(tensor(a[5]).numel() > 0, "pa_copy_blocks_q8b: num_pairs is one number");
            num = c.i32(tensor(a[5]));
        }
        return unlocked([&] {
            return pa_copy_blocks_q8b(kc, vc, ks, vs, pr, num, count, m.nb, m.heads, m.dim, m.bs, c.stream);
        });
    });
}

#define PA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD(dpool_append), PA_METHOD(dpool_release), PA_METHOD(append_q8b), PA_METHOD(decode_q8b),
                         PA_METHOD(copy_blocks_q8b), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_call() { return PyModule_Create(&module); }
