// tensor_calls.cpp -- the index calls and attention behind a shared prompt
// straight from tensors: a CPython module that looks the arguments over and
// calls the C ABI.
//
// A small call is bound by the host.  From Python an attribute of a tensor costs
// 0.07 to 0.11 us, some 45 of them a call, and ctypes another 1.5 to 2 us; here
// they are a few loads.  Each function returns True once the call is enqueued and
// False where an argument is not what a right call has (or the tensors' GPU is
// not the current one, or the library refuses): then the checks in Python say
// what is wrong, or make the call.  No exception leaves a function.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <limits>

#include "topkidx.h"

namespace {

using at::Tensor;

decltype(&topk_index_append) index_append_fn;
decltype(&topk_index_scores) index_scores_fn;
decltype(&topk_attend_shared) attend_shared_fn;
decltype(&topk_attend_shared_workspace_bytes) shared_bytes_fn;

// A tensor, or null for None and for what is no tensor.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool small(int64_t n) { return n >= 0 && n <= std::numeric_limits<int32_t>::max(); }

struct Call {
    bool right = true;
    bool grad = c10::GradMode::is_enabled();
    c10::Device device{c10::DeviceType::CUDA, 0};
    c10::ScalarType type = c10::ScalarType::Undefined;
    topk_dtype_t code = TOPK_BF16;

    void need(bool x) { right = right && x; }
    // The tensor that the others go by: its GPU and its type.
    void begin(const Tensor* t) {
        need(t && t->is_cuda());
        if (!right) return;
        device = t->device();
        type = t->scalar_type();
        need(device.index() == c10::cuda::current_device() && (type == at::kBFloat16 || type == at::kHalf));
        code = type == at::kHalf ? TOPK_FP16 : TOPK_BF16;
    }
    void is(const Tensor* t, c10::ScalarType as) {
        need(t && t->scalar_type() == as && t->device() == device && t->layout() == c10::kStrided);
        if (right && grad) need(!t->requires_grad());
    }
    // Rows of `width` values, next to one another.
    void rows(const Tensor* t, c10::ScalarType as, int64_t dims, int64_t width) {
        is(t, as);
        need(right && t->dim() == dims && t->size(dims - 1) == width && (width <= 1 || t->stride(dims - 1) == 1));
    }
    // Contiguous, of this shape.
    void whole(const Tensor* t, c10::ScalarType as, at::IntArrayRef shape) {
        is(t, as);
        need(right && t->sizes() == shape && t->is_contiguous());
    }
    void line(const Tensor* t, int64_t n) { whole(t, at::kInt, {n}); }

    topk_stream_t stream(PyObject* handle) const {
        if (handle == Py_None)
            return reinterpret_cast<topk_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
        return reinterpret_cast<topk_stream_t>(PyLong_AsVoidPtr(handle));
    }
};

// The stride of a dimension of one entry means nothing.
int64_t step(const Tensor& t, int64_t dim, int64_t any) { return t.size(dim) > 1 ? t.stride(dim) : any; }
void* at_of(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
int32_t* ints(const Tensor* t) { return static_cast<int32_t*>(at_of(t)); }
float* floats(const Tensor* t) { return static_cast<float*>(at_of(t)); }

// Whether it is None or a tensor (anything else is not right).
bool optional(PyObject* o) { return o == Py_None || THPVariable_Check(o); }

template <typename Run>
PyObject* guarded(Run run) {
    bool done = false;
    try {
        done = run();
    } catch (...) {
        done = false;
    }
    if (PyErr_Occurred()) PyErr_Clear();
    return PyBool_FromLong(done);
}

// rows, slots, cache, norm_weight, norm_bias, eps, cos_sin, positions, interleaved, rope_last, stream
PyObject* index_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        if (n != 11 || !optional(a[3]) || !optional(a[4]) || !optional(a[6]) || !optional(a[7])) return false;
        const Tensor *rows = tensor(a[0]), *slots = tensor(a[1]), *cache = tensor(a[2]), *weight = tensor(a[3]),
                     *bias = tensor(a[4]), *turns = tensor(a[6]), *positions = tensor(a[7]);
        Call c;
        c.begin(cache);
        c.rows(cache, c.type, 2, TOPK_INDEX_DIM);
        c.rows(rows, c.type, 2, TOPK_INDEX_DIM);
        if (!c.right) return false;
        const int64_t tokens = rows->size(0);
        c.line(slots, tokens);
        if (weight) c.whole(weight, c.type, {TOPK_INDEX_DIM});
        if (bias) c.whole(bias, c.type, {TOPK_INDEX_DIM});
        if (positions) c.line(positions, tokens);
        int64_t angles = 0;
        if (turns) {
            c.rows(turns, at::kFloat, 2, TOPK_ROPE_DIM);
            c.need(c.right && turns->is_contiguous());
            if (c.right) angles = turns->size(0);
            c.need(angles > 0);  // (an empty table has no address)
        }
        const double eps = PyFloat_AsDouble(a[5]);
        const int interleaved = PyObject_IsTrue(a[8]), rope_last = PyObject_IsTrue(a[9]);
        const topk_stream_t stream = c.right ? c.stream(a[10]) : nullptr;
        if (!c.right || PyErr_Occurred() || !small(tokens) || !small(cache->size(0)) || !small(angles)) return false;
        void *const rows_at = at_of(rows), *const weight_at = at_of(weight), *const bias_at = at_of(bias),
                    *const cache_at = at_of(cache);
        const float* turns_at = floats(turns);
        const int32_t *positions_at = ints(positions), *slots_at = ints(slots);
        topk_status_t status;
        Py_BEGIN_ALLOW_THREADS
        status = index_append_fn(rows_at, step(*rows, 0, TOPK_INDEX_DIM), static_cast<int32_t>(tokens), weight_at, bias_at,
                                 static_cast<float>(eps), turns_at, static_cast<int32_t>(angles), positions_at, interleaved,
                                 rope_last, slots_at, cache_at, step(*cache, 0, TOPK_INDEX_DIM),
                                 static_cast<int32_t>(cache->size(0)), c.code, stream);
        Py_END_ALLOW_THREADS
        return status == TOPK_OK;
    });
}

// q, weights, cache, seq_lens, page_table, page_size, cu_q, max_seq_len, out, stream
PyObject* index_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        if (n != 10 || !optional(a[6])) return false;
        const Tensor *q = tensor(a[0]), *weights = tensor(a[1]), *cache = tensor(a[2]), *lens = tensor(a[3]),
                     *table = tensor(a[4]), *cu = tensor(a[6]), *out = tensor(a[8]);
        Call c;
        c.begin(q);
        c.rows(q, c.type, 3, TOPK_INDEX_DIM);
        c.rows(cache, c.type, 2, TOPK_INDEX_DIM);
        if (!c.right) return false;
        const int64_t total = q->size(0), heads = q->size(1);
        c.rows(weights, at::kFloat, 2, heads);
        c.is(table, at::kInt);
        c.is(out, at::kFloat);
        c.need(c.right && weights->size(0) == total && table->dim() == 2 && out->dim() == 2 && out->size(0) == total &&
               (table->size(1) <= 1 || table->stride(1) == 1) && (out->size(1) <= 1 || out->stride(1) == 1));
        if (!c.right) return false;
        const int64_t batch = table->size(0), pages = table->size(1);
        c.line(lens, batch);
        if (cu)
            c.line(cu, batch + 1);
        else
            c.need(batch > 0 && total % batch == 0);
        const int64_t page = PyLong_AsLongLong(a[5]);
        const int64_t limit = small(page) && small(pages) ? page * pages : -1;
        const int64_t most = a[7] != Py_None ? PyLong_AsLongLong(a[7])
                                             : std::min<int64_t>(limit, std::numeric_limits<int32_t>::max());
        const topk_stream_t stream = c.right ? c.stream(a[9]) : nullptr;
        if (!c.right || PyErr_Occurred() || most < 0 || most > limit || !small(most) || out->size(1) < most || !small(total) ||
            !small(heads) || !small(batch) || !small(cache->size(0)))
            return false;
        void *const q_at = at_of(q), *const cache_at = at_of(cache);
        const float* weights_at = floats(weights);
        const int32_t *lens_at = ints(lens), *table_at = ints(table), *cu_at = ints(cu);
        float* out_at = floats(out);
        topk_status_t status;
        Py_BEGIN_ALLOW_THREADS
        status = index_scores_fn(q_at, step(*q, 0, TOPK_INDEX_DIM), step(*q, 1, TOPK_INDEX_DIM), weights_at,
                                 step(*weights, 0, heads), cache_at, step(*cache, 0, TOPK_INDEX_DIM),
                                 static_cast<int32_t>(cache->size(0)), lens_at, table_at, step(*table, 0, pages),
                                 static_cast<int32_t>(page), static_cast<int32_t>(most), cu_at, static_cast<int32_t>(batch),
                                 static_cast<int32_t>(total), static_cast<int32_t>(heads), c.code, out_at,
                                 step(*out, 0, out->size(1)), stream);
        Py_END_ALLOW_THREADS
        return status == TOPK_OK;
    });
}

// q, cache, seq_lens, page_table, shared_pages, shared_len, page_size, scale, max_seq_len, out, lse, workspace, stream
PyObject* attend_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        if (n != 13) return false;
        constexpr int64_t kWidth = TOPK_LATENT_DIM + TOPK_ROPE_DIM;
        const Tensor *q = tensor(a[0]), *cache = tensor(a[1]), *lens = tensor(a[2]), *table = tensor(a[3]),
                     *common = tensor(a[4]), *length = tensor(a[5]), *out = tensor(a[9]), *lse = tensor(a[10]),
                     *room = tensor(a[11]);
        Call c;
        c.begin(q);
        c.rows(q, c.type, 4, kWidth);
        c.rows(cache, c.type, 2, kWidth);
        c.is(table, at::kInt);
        if (!c.right) return false;
        const int64_t batch = q->size(0), queries = q->size(1), heads = q->size(2);
        c.need(table->dim() == 2 && table->size(0) == batch && (table->size(1) <= 1 || table->stride(1) == 1));
        c.line(lens, batch);
        c.is(common, at::kInt);
        c.need(c.right && common->is_contiguous());
        c.is(length, at::kInt);
        c.need(c.right && length->numel() == 1);
        c.whole(out, c.type, {batch, queries, heads, TOPK_LATENT_DIM});
        c.whole(lse, at::kFloat, {batch, queries, heads});
        c.need(room && room->device() == c.device && room->layout() == c10::kStrided && room->is_contiguous());
        if (!c.right) return false;
        const int64_t pages = table->size(1), listed = common->numel(), page = PyLong_AsLongLong(a[6]);
        const int64_t limit = small(page) && small(pages) ? page * pages : -1;
        const int64_t most = a[8] != Py_None ? PyLong_AsLongLong(a[8])
                                             : std::min<int64_t>(limit, std::numeric_limits<int32_t>::max());
        const double scale = PyFloat_AsDouble(a[7]);
        const topk_stream_t stream = c.stream(a[12]);
        if (PyErr_Occurred() || most < 0 || most > limit || !small(most) || !small(batch) || !small(queries) || !small(heads) ||
            !small(listed) || !small(cache->size(0)))
            return false;
        const size_t bytes = room->nbytes();
        if (bytes < shared_bytes_fn(static_cast<int32_t>(batch), static_cast<int32_t>(queries), static_cast<int32_t>(heads)))
            return false;
        void *const q_at = at_of(q), *const cache_at = at_of(cache), *const out_at = at_of(out), *const room_at = at_of(room);
        const int32_t *lens_at = ints(lens), *table_at = ints(table), *common_at = ints(common), *length_at = ints(length);
        float* lse_at = floats(lse);
        topk_status_t status;
        Py_BEGIN_ALLOW_THREADS
        status = attend_shared_fn(q_at, step(*q, 0, kWidth), step(*q, 1, kWidth), step(*q, 2, kWidth), cache_at,
                                  step(*cache, 0, kWidth), static_cast<int32_t>(cache->size(0)), lens_at, table_at,
                                  step(*table, 0, pages), common_at, static_cast<int32_t>(listed), length_at,
                                  static_cast<int32_t>(page), static_cast<int32_t>(most), static_cast<int32_t>(batch),
                                  static_cast<int32_t>(queries), static_cast<int32_t>(heads), static_cast<float>(scale), c.code,
                                  out_at, lse_at, room_at, bytes, stream);
        Py_END_ALLOW_THREADS
        return status == TOPK_OK;
    });
}

// Addresses of the library's functions, in the order of their declaration above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* at[4];
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
        return nullptr;
    }
    for (int i = 0; i < 4; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    index_append_fn = reinterpret_cast<decltype(index_append_fn)>(at[0]);
    index_scores_fn = reinterpret_cast<decltype(index_scores_fn)>(at[1]);
    attend_shared_fn = reinterpret_cast<decltype(attend_shared_fn)>(at[2]);
    shared_bytes_fn = reinterpret_cast<decltype(shared_bytes_fn)>(at[3]);
    Py_RETURN_NONE;
}

template <PyObject* (*kFn)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(kFn));
}

PyMethodDef methods[] = {{"bind", fast<bind>(), METH_FASTCALL, nullptr},
                         {"index_append", fast<index_append>(), METH_FASTCALL, nullptr},
                         {"index_scores", fast<index_scores>(), METH_FASTCALL, nullptr},
                         {"attend_shared", fast<attend_shared>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&module); }
