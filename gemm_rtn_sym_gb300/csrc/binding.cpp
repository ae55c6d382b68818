// The calls on shared pages of the cache, from Python with little on the way.
//
// A call's kernels last a few microseconds, and looking at a dozen tensors from
// Python takes longer than that: 18 µs of host time for an append with norms
// (4 here), 13 for a fork (6), 21 for attention over shared prefixes (9).  Each
// function here takes its Python counterpart's arguments, in its order, and
// handles the usual case: the tensors are what they should be, on the current
// device.  Anything else, and any call that the library refuses, it leaves
// alone (NotImplemented) to the Python function, which says what is wrong.  Any
// other status (an int) is the end of the call: some of its kernels may run
// already, and a second call would change pages and holders once more.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "w4.h"

namespace {

using at::Tensor;
constexpr auto kInt = at::kInt;
constexpr auto kLong = at::kLong;

// A call's arguments, as far as they are what they should be.
struct Call {
    PyObject* const* args;
    bool ok = true;
    int index = -1;
    void* stream = nullptr;

    Call(PyObject* const* a, Py_ssize_t given, Py_ssize_t wanted) : args(a), ok(given == wanted) {}

    bool none(int i) const { return args[i] == Py_None; }
    bool flag(int i) {
        const int v = PyObject_IsTrue(args[i]);
        if (v < 0) PyErr_Clear(), ok = false;
        return v > 0;
    }
    long long number(int i) {
        const long long v = PyLong_AsLongLong(args[i]);
        if (v == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
        return v;
    }
    double real(int i) {
        const double v = PyFloat_AsDouble(args[i]);
        if (v == -1.0 && PyErr_Occurred()) PyErr_Clear(), ok = false;
        return v;
    }
    // The tensor of an argument; its device has to be the first one's, and that the current one.
    const Tensor* tensor(int i) {
        if (!ok || !THPVariable_CheckExact(args[i])) return ok = false, nullptr;
        const Tensor& t = THPVariable_Unpack(args[i]);
        if (!t.is_cuda()) return ok = false, nullptr;
        if (index < 0) {
            index = t.get_device();
            if (c10::cuda::current_device() != index) return ok = false, nullptr;
            stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
        } else if (t.get_device() != index) {
            return ok = false, nullptr;
        }
        return &t;
    }
    const Tensor* typed(int i, at::ScalarType type, int dims) {
        const Tensor* t = tensor(i);
        if (!t || t->scalar_type() != type || t->dim() != dims) return ok = false, nullptr;
        return t;
    }
    // Address of a contiguous tensor of n values.
    template <class V = void>
    V* vector(int i, at::ScalarType type, int64_t n) {
        const Tensor* t = typed(i, type, 1);
        if (!t || t->size(0) != n || !t->is_contiguous()) return ok = false, nullptr;
        return static_cast<V*>(t->data_ptr());
    }
    // A tensor with unit stride in its last dimension.
    const Tensor* strided(int i, at::ScalarType type, int dims) {
        const Tensor* t = typed(i, type, dims);
        if (!t || (t->stride(-1) != 1 && t->size(-1) > 1 && t->numel() > 0)) return ok = false, nullptr;
        return t;
    }
    w4_rows rows(int i, int64_t T, int64_t heads, int64_t dim) {
        const Tensor* t = strided(i, at::kBFloat16, 3);
        if (!t || t->size(0) != T || t->size(1) != heads || t->size(2) != dim) return ok = false, w4_rows{};
        return {t->data_ptr(), t->stride(0), t->stride(1)};
    }
    w4_kv_cache cache(int k, int v, int k_scales, int v_scales) {
        w4_kv_cache c = {};
        const Tensor* t = tensor(k);
        if (!t) return c;
        const bool q8 = t->scalar_type() == at::kChar;
        const at::ScalarType type = q8 ? at::kChar : at::kBFloat16;
        const Tensor *kt = strided(k, type, 4), *vt = strided(v, type, 4);
        if (!kt || !vt || kt->sizes() != vt->sizes() || kt->strides() != vt->strides()) return ok = false, c;
        c = {kt->data_ptr(), vt->data_ptr(), nullptr, nullptr, kt->size(0), kt->stride(0), kt->stride(1), kt->stride(2),
             static_cast<int32_t>(kt->size(1)), static_cast<int32_t>(kt->size(2)), static_cast<int32_t>(kt->size(3)), q8 ? 8 : 16};
        if (q8) {
            void** const to[2] = {&c.k_scales, &c.v_scales};
            for (int j = 0; j < 2; ++j) {
                const Tensor* s = typed(j ? v_scales : k_scales, at::kBFloat16, 3);
                if (!s || s->size(0) != kt->size(0) || s->size(1) != kt->size(2) || s->size(2) != kt->size(1) || !s->is_contiguous())
                    return ok = false, c;
                *to[j] = s->data_ptr();
            }
        } else if (!none(k_scales) || !none(v_scales)) {
            ok = false;
        }
        return c;
    }
};

// What a call that did not work out returns.
PyObject* failed(int status) {
    if (status == W4_ERR_INVALID_ARG || status == W4_ERR_MISALIGNED || status == W4_ERR_UNSUPPORTED) Py_RETURN_NOTIMPLEMENTED;  // before any launch
    return PyLong_FromLong(status);
}

// Outputs, in their order: the caller's, or new ones.
struct Outputs {
    Call& call;
    PyObject* tuple;
    int count = 0;
    Outputs(Call& c, int n) : call(c), tuple(c.ok ? PyTuple_New(n) : nullptr) {
        if (!tuple) call.ok = false;
    }
    ~Outputs() { Py_XDECREF(tuple); }
    template <class V>
    V* next(int i, at::ScalarType type, at::IntArrayRef shape) {
        if (!call.ok) return nullptr;
        if (call.none(i)) {
            Tensor t = at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(call.index)));
            V* const p = static_cast<V*>(t.data_ptr());
            PyObject* const o = THPVariable_Wrap(std::move(t));
            if (!o) return PyErr_Clear(), call.ok = false, nullptr;
            PyTuple_SET_ITEM(tuple, count++, o);
            return p;
        }
        const Tensor* t = call.typed(i, type, static_cast<int>(shape.size()));
        if (!t || t->sizes() != shape || !t->is_contiguous()) return call.ok = false, nullptr;
        PyTuple_SET_ITEM(tuple, count++, Py_NewRef(call.args[i]));
        return static_cast<V*>(t->data_ptr());
    }
    PyObject* done(int status) {
        if (status != W4_OK) return failed(status);
        PyObject* const t = tuple;
        tuple = nullptr;
        return t;
    }
};

// Memory for the time of a call: the stream's next allocations may have it afterwards.
struct Scratch {
    size_t size;
    void* p;
    Scratch(size_t bytes, void* stream)
        : size(bytes), p(bytes ? c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, static_cast<cudaStream_t>(stream)) : nullptr) {}
    Scratch(const Scratch&) = delete;
    ~Scratch() {
        if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
};

// Runs a library call without the interpreter's lock.
template <class F>
int run(F f) {
    int status;
    Py_BEGIN_ALLOW_THREADS status = f();
    Py_END_ALLOW_THREADS return status;
}

// What a C++ exception on the way (an allocation that fails) leaves to the Python function.
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NOTIMPLEMENTED;
    }
}

// q, k, v, q_weight, k_weight, positions, cos, sin, k_cache, v_cache, slots, eps, unit_offset, sections, cycled, paired,
// k_scales, v_scales, q_out
PyObject* kv_append_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 19);
        if (!c.ok || c.none(0) || c.none(6)) Py_RETURN_NOTIMPLEMENTED;
        const Tensor* const k = c.typed(1, at::kBFloat16, 3);
        const w4_kv_cache cache = c.cache(8, 9, 16, 17);
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        const int64_t T = k->size(0), dim = cache.head_dim;
        const Tensor *const q = c.typed(0, at::kBFloat16, 3), *const cos = c.typed(6, at::kFloat, 2), *const sin = c.typed(7, at::kFloat, 2);
        const Tensor *const positions = c.tensor(5), *const weight = c.tensor(4);
        if (!c.ok || cos->sizes() != sin->sizes() || !cos->is_contiguous() || !sin->is_contiguous() || positions->scalar_type() != kInt) Py_RETURN_NOTIMPLEMENTED;
        const int64_t heads = q->size(1);
        w4_rope rope = {};
        rope.axes = 1;
        rope.sections[0] = static_cast<int32_t>(cos->size(1));
        if (!c.none(13)) {
            if (!PyTuple_CheckExact(args[13]) || PyTuple_GET_SIZE(args[13]) < 1 || PyTuple_GET_SIZE(args[13]) > 4) Py_RETURN_NOTIMPLEMENTED;
            rope.axes = static_cast<int32_t>(PyTuple_GET_SIZE(args[13]));
            for (int i = 0; i < rope.axes; ++i) {
                const long v = PyLong_AsLong(PyTuple_GET_ITEM(args[13], i));
                if ((v == -1 && PyErr_Occurred()) || v < 0 || v > 256) return PyErr_Clear(), Py_NewRef(Py_NotImplemented);
                rope.sections[i] = static_cast<int32_t>(v);
            }
        }
        const bool each = positions->dim() == 2;
        if ((each ? positions->size(0) != rope.axes || positions->size(1) != T : positions->dim() != 1 || positions->size(0) != T) ||
            (positions->stride(-1) != 1 && T > 1))
            Py_RETURN_NOTIMPLEMENTED;
        rope.positions = positions->const_data_ptr<int32_t>();
        rope.axis_stride = each ? positions->stride(0) : 0;
        rope.cos = cos->const_data_ptr<float>();
        rope.sin = sin->const_data_ptr<float>();
        rope.rows = cos->size(0);
        rope.rotary = static_cast<int32_t>(2 * cos->size(1));
        rope.cycled = c.flag(14);
        rope.paired = c.flag(15);
        const at::ScalarType type = weight->scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat) Py_RETURN_NOTIMPLEMENTED;
        w4_norm norm = {};
        norm.q_weight = c.vector(3, type, dim);
        norm.k_weight = c.vector(4, type, dim);
        norm.format = type == at::kFloat ? 32 : 16;
        norm.eps = static_cast<float>(c.real(11));
        norm.unit_offset = c.flag(12);
        Outputs out(c, 1);
        const int64_t shape[] = {T, heads, dim};
        w4_rows q_rows = c.rows(0, T, heads, dim), k_rows = c.rows(1, T, cache.kv_heads, dim), v_rows = c.rows(2, T, cache.kv_heads, dim), out_rows = {};
        const int64_t* const slots = c.vector<int64_t>(10, kLong, T);
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        if (c.none(18)) {
            out_rows = {out.next<void>(18, at::kBFloat16, shape), heads * dim, dim};
        } else {
            out_rows = c.rows(18, T, heads, dim);
            if (c.ok) PyTuple_SET_ITEM(out.tuple, 0, Py_NewRef(args[18]));
        }
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        return out.done(run([&] { return w4_kv_append_norm(&cache, &rope, &norm, T, static_cast<int32_t>(heads), &q_rows, &out_rows, &k_rows, &v_rows, slots, c.stream); }));
    });
}

// lens, target, block_table, free_pages, free_range, page_size, tokens, holders, new_lens, starts, slots, positions,
// free_range_out
PyObject* kv_pages_held(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 13);
        const Tensor* const table = c.ok ? c.strided(2, kInt, 2) : nullptr;
        const Tensor* const ring = c.ok ? c.typed(3, kInt, 1) : nullptr;
        if (!c.ok || !ring->is_contiguous()) Py_RETURN_NOTIMPLEMENTED;
        const int64_t B = table->size(0), width = table->size(1), pages = ring->size(0);
        const long long page_size = c.number(5), T = c.number(6);
        const int32_t *const lens = c.vector<int32_t>(0, kInt, B), *const target = c.vector<int32_t>(1, kInt, B);
        const int64_t* const range = c.vector<int64_t>(4, kLong, 2);
        int32_t* const holders = c.vector<int32_t>(7, kInt, pages);
        if (!c.ok || B > INT32_MAX || width > INT32_MAX || page_size < 1 || page_size > INT32_MAX || T < 0) Py_RETURN_NOTIMPLEMENTED;
        Outputs out(c, 5);
        int32_t* const new_lens = out.next<int32_t>(8, kInt, {B});
        int32_t* const starts = out.next<int32_t>(9, kInt, {B + 1});
        int64_t* const slots = out.next<int64_t>(10, kLong, {T});
        int32_t* const positions = out.next<int32_t>(11, kInt, {T});
        int64_t* const left = out.next<int64_t>(12, kLong, {2});
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        const Scratch scratch(w4_kv_pages_held_workspace_bytes(static_cast<int32_t>(B), static_cast<int32_t>(width), pages), c.stream);
        return out.done(run([&] {
            return w4_kv_pages_held(lens, target, static_cast<int32_t>(B), static_cast<int32_t>(page_size), static_cast<int32_t*>(ring->data_ptr()), pages, range,
                                    static_cast<int32_t*>(table->data_ptr()), table->stride(0), static_cast<int32_t>(width), T, holders, new_lens, starts, slots,
                                    positions, left, scratch.p, scratch.size, c.stream);
        }));
    });
}

// lens, source, keep, block_table, holders, free_pages, free_range, page_size, new_lens, copies, free_range_out
PyObject* kv_fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 11);
        const Tensor* const table = c.ok ? c.strided(3, kInt, 2) : nullptr;
        const Tensor* const ring = c.ok ? c.typed(5, kInt, 1) : nullptr;
        if (!c.ok || !ring->is_contiguous()) Py_RETURN_NOTIMPLEMENTED;
        const int64_t B = table->size(0), width = table->size(1), pages = ring->size(0);
        const long long page_size = c.number(7);
        const int32_t *const lens = c.vector<int32_t>(0, kInt, B), *const source = c.vector<int32_t>(1, kInt, B), *const keep = c.vector<int32_t>(2, kInt, B);
        int32_t* const holders = c.vector<int32_t>(4, kInt, pages);
        const int64_t* const range = c.vector<int64_t>(6, kLong, 2);
        if (!c.ok || B > INT32_MAX || width > INT32_MAX || page_size < 1 || page_size > INT32_MAX) Py_RETURN_NOTIMPLEMENTED;
        Outputs out(c, 3);
        int32_t* const new_lens = out.next<int32_t>(8, kInt, {B});
        int32_t* const copies = out.next<int32_t>(9, kInt, {3, B});
        int64_t* const left = out.next<int64_t>(10, kLong, {2});
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        return out.done(run([&] {
            return w4_kv_fork(lens, source, keep, static_cast<int32_t>(B), static_cast<int32_t>(page_size), static_cast<int32_t*>(table->data_ptr()), table->stride(0),
                              static_cast<int32_t>(width), holders, static_cast<const int32_t*>(ring->data_ptr()), pages, range, new_lens, copies, left, c.stream);
        }));
    });
}

// lens, block_table, holders, free_range, page_size, new_table, new_holders, free_pages, free_range_out, copies
PyObject* kv_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 10);
        const Tensor* const table = c.ok ? c.strided(1, kInt, 2) : nullptr;
        const Tensor* const held = c.ok ? c.typed(2, kInt, 1) : nullptr;
        if (!c.ok || !held->is_contiguous()) Py_RETURN_NOTIMPLEMENTED;
        const int64_t B = table->size(0), width = table->size(1), pages = held->size(0);
        const long long page_size = c.number(4);
        const int32_t* const lens = c.vector<int32_t>(0, kInt, B);
        const int64_t* const range = c.vector<int64_t>(3, kLong, 2);
        if (!c.ok || B > INT32_MAX || width > INT32_MAX || page_size < 1 || page_size > INT32_MAX) Py_RETURN_NOTIMPLEMENTED;
        Outputs out(c, 5);
        int32_t* const new_table = out.next<int32_t>(5, kInt, {B, width});
        int32_t* const new_holders = out.next<int32_t>(6, kInt, {pages});
        int32_t* const ring = out.next<int32_t>(7, kInt, {pages});
        int64_t* const left = out.next<int64_t>(8, kLong, {2});
        int32_t* const copies = out.next<int32_t>(9, kInt, {3, pages / 2});
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        return out.done(run([&] {
            return w4_kv_compact(lens, static_cast<int32_t>(B), static_cast<int32_t>(page_size), static_cast<const int32_t*>(table->data_ptr()), table->stride(0),
                                 static_cast<int32_t>(width), static_cast<const int32_t*>(held->data_ptr()), pages, range, new_table, width, new_holders, ring, left, copies,
                                 c.stream);
        }));
    });
}

// k_cache, v_cache, copies, k_scales, v_scales
PyObject* kv_copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 5);
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        const w4_kv_cache cache = c.cache(0, 1, 3, 4);
        const Tensor* const copies = c.typed(2, kInt, 2);
        if (!c.ok || copies->size(0) != 3 || !copies->is_contiguous() || copies->size(1) > INT32_MAX) Py_RETURN_NOTIMPLEMENTED;
        const int status = run([&] { return w4_kv_copy(&cache, copies->const_data_ptr<int32_t>(), static_cast<int32_t>(copies->size(1)), c.stream); });
        if (status != W4_OK) return failed(status);
        Py_RETURN_NONE;
    });
}

// q, k_cache, v_cache, block_table, lens, group_starts, prefix_table, prefix_lens, starts, k_scales, v_scales, scale, out
PyObject* attn_decode_shared(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c(args, n, 13);
        const Tensor* const q = c.ok ? c.typed(0, at::kBFloat16, 3) : nullptr;
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        const w4_kv_cache cache = c.cache(1, 2, 9, 10);
        const Tensor *const table = c.strided(3, kInt, 2), *const prefix = c.strided(6, kInt, 2);
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        const int64_t B = table->size(0), width = table->size(1), groups = prefix->size(0), prefix_width = prefix->size(1);
        const int64_t T = q->size(0), heads = q->size(1), dim = cache.head_dim;
        if (B > INT32_MAX || width > INT32_MAX || groups > INT32_MAX || prefix_width > INT32_MAX || heads > INT32_MAX) Py_RETURN_NOTIMPLEMENTED;
        const int32_t *const lens = c.vector<int32_t>(4, kInt, B), *const starts = c.none(8) ? nullptr : c.vector<int32_t>(8, kInt, B + 1);
        const int32_t *const group_starts = c.vector<int32_t>(5, kInt, groups + 1), *const prefix_lens = c.vector<int32_t>(7, kInt, groups);
        const double scale = c.none(11) ? 1.0 / std::sqrt(static_cast<double>(dim)) : c.real(11);
        const w4_rows q_rows = c.rows(0, T, heads, dim);
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        Outputs out(c, 1);
        w4_rows out_rows = {};
        if (c.none(12)) {
            const int64_t shape[] = {T, heads, dim};
            out_rows = {out.next<void>(12, at::kBFloat16, shape), heads * dim, dim};
        } else {
            out_rows = c.rows(12, T, heads, dim);
            if (c.ok) PyTuple_SET_ITEM(out.tuple, 0, Py_NewRef(args[12]));
        }
        if (!c.ok) Py_RETURN_NOTIMPLEMENTED;
        const size_t size = w4_attn_decode_shared_workspace_bytes(&cache, static_cast<int32_t>(B), T, static_cast<int32_t>(heads), static_cast<int32_t>(groups));
        if (size == 0) Py_RETURN_NOTIMPLEMENTED;
        const Scratch scratch(size, c.stream);
        return out.done(run([&] {
            return w4_attn_decode_shared(&cache, static_cast<int32_t>(B), T, static_cast<int32_t>(heads), &q_rows, &out_rows, static_cast<const int32_t*>(table->data_ptr()),
                                         table->stride(0), static_cast<int32_t>(width), lens, starts, static_cast<int32_t>(groups), group_starts,
                                         static_cast<const int32_t*>(prefix->data_ptr()), prefix->stride(0), static_cast<int32_t>(prefix_width), prefix_lens,
                                         static_cast<float>(scale), scratch.p, size, c.stream);
        }));
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(kv_append_norm), FAST(kv_pages_held), FAST(kv_fork), FAST(kv_compact), FAST(kv_copy), FAST(attn_decode_shared), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
