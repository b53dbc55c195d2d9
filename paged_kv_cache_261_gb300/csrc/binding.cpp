// The short way of the Python calls of a serving step into the C ABI: a CPython module that reads
// the tensors directly. Every function takes what the Python function of its name takes, by
// position, and answers with the status of the C call, or with None where anything is not as the
// plain call has it (a tensor of another type, shape or device, a foreign device current, numbers
// that are none): then nothing was done, and the Python function, which knows how to refuse or
// adapt, goes its own way. So this file raises nothing and checks everything. (interface() alone is another thing.)
//
// (On a GB300's host, us of host time with the checks in Python and here: the two layout calls of a
// step 13.2 and 4.5, a rotary call 8.4 and 2.7, a write and its read-back 12.3 and 4.6, one decode
// 11.1 and 4.6. A launch alone is 1.6.)
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <algorithm>
#include <climits>
#include <map>
#include <utility>

#include "../../include/pagedattn.h"

extern "C" uint64_t pa_internal_interface(void);   // the library's PA_INTERFACE

namespace {

using at::Tensor;

// Arguments of one call. Each getter notes what does not fit in `ok`; what it returns then is
// not used.
struct Args {
    PyObject *const *v;
    bool ok;
    int device = -1;
    cudaStream_t stream = nullptr;

    Args(PyObject *const *args, Py_ssize_t n, Py_ssize_t want) : v(args), ok(n == want) {}

    const Tensor *tensor(int i) {
        if (!ok || !THPVariable_Check(v[i])) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(v[i]);
    }
    // The tensor whose device is the call's, which has to be the current one.
    const Tensor *first(int i) {
        const Tensor *t = tensor(i);
        if (!t || !t->is_cuda()) {
            ok = false;
            return nullptr;
        }
        device = t->device().index();
        ok = c10::cuda::current_device() == device;
        return t;
    }
    bool here(const Tensor *t, at::ScalarType type, int dims) {
        ok = ok && t && t->is_cuda() && t->device().index() == device && t->scalar_type() == type && t->dim() == dims;
        return ok;
    }
    const Tensor *dense(int i, at::ScalarType type, int dims) {
        const Tensor *t = tensor(i);
        if (here(t, type, dims)) ok = t->is_contiguous();
        return t;
    }
    const Tensor *vector(int i, at::ScalarType type, int64_t n) {
        const Tensor *t = dense(i, type, 1);
        ok = ok && t->size(0) == n;
        return t;
    }
    // A single number, in any shape.
    const Tensor *scalar(int i) {
        const Tensor *t = tensor(i);
        ok = ok && t->is_cuda() && t->device().index() == device && t->scalar_type() == at::kInt && t->numel() == 1;
        return t;
    }
    // Rows [T, heads, d] whose heads are contiguous; their stride.
    const Tensor *rows(int i, at::ScalarType type, int64_t T, int64_t heads, int64_t d, int64_t &stride) {
        const Tensor *t = tensor(i);
        if (!here(t, type, 3)) return t;
        const auto size = t->sizes(), step = t->strides();
        ok = size[0] == T && size[1] == heads && size[2] == d && step[2] == 1 && (heads <= 1 || step[1] == d) && step[0] >= 0;
        stride = T > 1 ? step[0] : heads * d;
        return t;
    }
    int64_t integer(int i) {
        if (!ok) return 0;
        const long long x = PyLong_Check(v[i]) ? PyLong_AsLongLong(v[i]) : -1;
        if (!PyLong_Check(v[i]) || (x == -1 && PyErr_Occurred())) {
            PyErr_Clear();
            ok = false;
        }
        return x;
    }
    int small(int i) {
        const int64_t x = integer(i);
        ok = ok && x >= INT_MIN && x <= INT_MAX;
        return (int)x;
    }
    double real(int i) {
        if (!ok) return 0;
        const double x = PyFloat_AsDouble(v[i]);
        if (x == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return x;
    }
    bool none(int i) const { return v[i] == Py_None; }
    // The stream given, or the current one; last of the getters.
    void on_stream(int i) {
        if (!ok) return;
        if (none(i)) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
            return;
        }
        PyObject *s = PyObject_GetAttrString(v[i], "cuda_stream");
        const long long p = s && PyLong_Check(s) ? PyLong_AsLongLong(s) : -1;
        if (!s || !PyLong_Check(s) || PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        Py_XDECREF(s);
        stream = reinterpret_cast<cudaStream_t>(p);
    }
};

int element_code(at::ScalarType t) {
    return t == at::kFloat ? PA_DTYPE_F32 : (t == at::kHalf ? PA_DTYPE_F16 : (t == at::kBFloat16 ? PA_DTYPE_BF16 : -1));
}

template <typename T = void> T *ptr(const Tensor *t) { return static_cast<T *>(t->data_ptr()); }

PyObject *status(int rc) { return PyLong_FromLong(rc); }

// block_tables, context_lens, query_lens, free_blocks, num_free, query_start_loc, slot_mapping,
// positions, block_size, num_blocks, new_context_lens, new_num_free, stream
PyObject *blocks_append(PyObject *, PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 13);
    const Tensor *table = a.first(0);
    if (!a.ok || table->dim() != 2) Py_RETURN_NONE;
    a.dense(0, at::kInt, 2);
    const int64_t B = table->size(0), width = table->size(1);
    const Tensor *lens = a.vector(1, at::kInt, B), *query = a.vector(2, at::kInt, B), *free = a.dense(3, at::kInt, 1);
    const Tensor *height = a.scalar(4), *start = a.vector(5, at::kInt, B + 1), *slots = a.dense(6, at::kInt, 1);
    if (!a.ok) Py_RETURN_NONE;
    const Tensor *pos = a.vector(7, at::kInt, slots->size(0));
    const int bs = a.small(8);
    const int64_t blocks = a.integer(9);
    const Tensor *new_lens = a.none(10) ? lens : a.vector(10, at::kInt, B), *new_height = a.none(11) ? height : a.scalar(11);
    a.on_stream(12);
    if (!a.ok || width > INT_MAX || B > INT_MAX) Py_RETURN_NONE;
    return status(pa_paged_blocks_append(ptr<int32_t>(table), (int)width, ptr<int32_t>(lens), ptr<int32_t>(new_lens),
                                         ptr<int32_t>(query), (int)B, ptr<int32_t>(free), free->size(0),
                                         ptr<int32_t>(height), ptr<int32_t>(new_height), ptr<int32_t>(start),
                                         ptr<int32_t>(slots), ptr<int32_t>(pos), slots->size(0), bs, blocks, a.stream));
}

// block_tables, context_lens, finished, free_blocks, num_free, block_size, new_context_lens,
// new_num_free, num_blocks, stream
PyObject *blocks_release(PyObject *, PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 10);
    const Tensor *table = a.first(0);
    if (!a.ok || table->dim() != 2) Py_RETURN_NONE;
    a.dense(0, at::kInt, 2);
    const int64_t B = table->size(0), width = table->size(1);
    const Tensor *lens = a.vector(1, at::kInt, B), *done = a.tensor(2);
    if (!a.ok) Py_RETURN_NONE;
    done = a.vector(2, done->scalar_type() == at::kByte ? at::kByte : at::kBool, B);
    const Tensor *free = a.dense(3, at::kInt, 1), *height = a.scalar(4);
    const int bs = a.small(5);
    const Tensor *new_lens = a.none(6) ? lens : a.vector(6, at::kInt, B), *new_height = a.none(7) ? height : a.scalar(7);
    if (!a.ok) Py_RETURN_NONE;
    const int64_t blocks = a.none(8) ? INT_MAX / std::max(bs, 1) : a.integer(8);
    a.on_stream(9);
    if (!a.ok || width > INT_MAX || B > INT_MAX) Py_RETURN_NONE;
    return status(pa_paged_blocks_release(ptr<int32_t>(table), (int)width, ptr<int32_t>(lens), ptr<int32_t>(new_lens),
                                          ptr<uint8_t>(done), (int)B, ptr<int32_t>(free), free->size(0),
                                          ptr<int32_t>(height), ptr<int32_t>(new_height), bs, blocks, a.stream));
}

// What both rotary calls take: the queries and their shape, positions and frequencies.
struct Rotary {
    const Tensor *q, *q_out, *k, *pos, *freq;
    at::ScalarType type;
    int64_t T = 0, H = 0, Hk = 0, D = 0, half = 0, q_stride = 0, q_out_stride = 0, k_stride = 0;

    Rotary(Args &a, int i_q_out, int i_q, int i_k, int i_pos, int i_freq) {
        q = a.first(i_q);
        a.ok = a.ok && q->dim() == 3;
        if (!a.ok) return;
        type = q->scalar_type();
        T = q->size(0), H = q->size(1), D = q->size(2);
        a.rows(i_q, type, T, H, D, q_stride);
        q_out = a.rows(i_q_out, type, T, H, D, q_out_stride);
        k = nullptr;
        if (!a.none(i_k)) {
            k = a.tensor(i_k);
            a.ok = a.ok && k->dim() == 3;
            if (!a.ok) return;
            Hk = k->size(1);
            a.rows(i_k, type, T, Hk, D, k_stride);
        }
        pos = a.vector(i_pos, at::kInt, T);
        freq = a.dense(i_freq, at::kDouble, 1);
        if (a.ok) half = freq->size(0);
        a.ok = a.ok && element_code(type) >= 0 && std::max({H, Hk, D, 2 * half}) <= INT_MAX;
    }
};

// q_out, k_out, q, k, positions, inv_freq, factor, interleaved, stream
PyObject *rotary_embedding(PyObject *, PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 9);
    if (!a.ok || a.none(1) != a.none(3)) Py_RETURN_NONE;
    const Rotary r(a, 0, 2, 3, 4, 5);
    int64_t k_out_stride = 0;
    const Tensor *k_out = a.ok && r.k ? a.rows(1, r.type, r.T, r.Hk, r.D, k_out_stride) : nullptr;
    const double factor = a.real(6);
    const int inter = a.ok ? PyObject_IsTrue(args[7]) : 0;
    a.on_stream(8);
    if (!a.ok || inter < 0) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return status(pa_rotary_embedding(ptr(r.q_out), r.q_out_stride, k_out ? ptr(k_out) : nullptr, k_out_stride, ptr(r.q),
                                      r.q_stride, r.k ? ptr(r.k) : nullptr, r.k_stride, ptr<int32_t>(r.pos),
                                      ptr<double>(r.freq), (float)factor, inter, r.T, (int)r.H, (int)r.Hk, (int)r.D,
                                      (int)(2 * r.half), element_code(r.type), a.stream));
}

// q_out, q, k, v, positions, inv_freq, slot_mapping, key_cache, value_cache, factor, interleaved, stream
PyObject *kv_write_rotary(PyObject *, PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 12);
    if (!a.ok || a.none(2)) Py_RETURN_NONE;
    const Rotary r(a, 0, 1, 2, 4, 5);
    if (!a.ok) Py_RETURN_NONE;
    int64_t v_stride = 0;
    const Tensor *v = a.rows(3, r.type, r.T, r.Hk, r.D, v_stride), *slots = a.vector(6, at::kInt, r.T);
    const Tensor *kc = a.dense(7, r.type, 4), *vc = a.dense(8, r.type, 4);
    a.ok = a.ok && kc->sizes() == vc->sizes() && kc->size(2) == r.Hk && kc->size(3) == r.D && kc->size(1) <= INT_MAX;
    const double factor = a.real(9);
    const int inter = a.ok ? PyObject_IsTrue(args[10]) : 0;
    a.on_stream(11);
    if (!a.ok || inter < 0) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    return status(pa_paged_kv_write_rotary(ptr(r.q_out), r.q_out_stride, ptr(r.q), r.q_stride, ptr(r.k), r.k_stride, ptr(v),
                                           v_stride, ptr<int32_t>(r.pos), ptr<double>(r.freq), (float)factor, inter,
                                           ptr<int32_t>(slots), r.T, ptr(kc), ptr(vc), kc->size(0), (int)kc->size(1),
                                           (int)r.H, (int)r.Hk, (int)r.D, (int)(2 * r.half), element_code(r.type),
                                           a.stream));
}

// A block-scaled 8-bit cache at arguments i, i + 1 and i + 2.
struct Cache {
    const Tensor *k, *v, *scales;
    int64_t NB = 0, Hk = 0, bs = 0, D = 0;

    Cache(Args &a, int i) {
        k = a.first(i);
        a.ok = a.ok && k->dim() == 4 && (k->scalar_type() == at::kByte || k->scalar_type() == at::kFloat8_e4m3fn);
        if (!a.ok) return;
        a.dense(i, k->scalar_type(), 4);
        v = a.dense(i + 1, k->scalar_type(), 4);
        scales = a.dense(i + 2, at::kFloat, 3);
        if (!a.ok) return;
        NB = k->size(0), Hk = k->size(1), bs = k->size(2), D = k->size(3);
        a.ok = v->sizes() == k->sizes() && scales->size(0) == NB && scales->size(1) == Hk && scales->size(2) == 2 &&
               std::max({Hk, bs, D}) <= INT_MAX;
    }
};

// k, v, slot_mapping, key_cache, value_cache, kv_scales, stream
PyObject *move_fp8_block(PyObject *const *args, Py_ssize_t n, bool write) {
    Args a(args, n, 7);
    if (!a.ok) Py_RETURN_NONE;
    const Cache c(a, 3);
    const Tensor *slots = a.ok ? a.dense(2, at::kInt, 1) : nullptr, *k = a.tensor(0);
    if (!a.ok) Py_RETURN_NONE;
    const at::ScalarType type = k->scalar_type();
    const int64_t T = slots->size(0);
    int64_t k_stride = 0, v_stride = 0;
    a.rows(0, type, T, c.Hk, c.D, k_stride);
    const Tensor *v = a.rows(1, type, T, c.Hk, c.D, v_stride);
    a.ok = a.ok && element_code(type) >= 0 && (write || (k->is_contiguous() && v->is_contiguous()));
    a.on_stream(6);
    if (!a.ok) Py_RETURN_NONE;
    if (write)
        return status(pa_paged_kv_write_fp8_block(ptr(k), k_stride, ptr(v), v_stride, ptr<int32_t>(slots), T, ptr(c.k),
                                                  ptr(c.v), ptr<float>(c.scales), c.NB, (int)c.bs, (int)c.Hk, (int)c.D,
                                                  element_code(type), a.stream));
    return status(pa_paged_kv_read_fp8_block(ptr(k), ptr(v), ptr<int32_t>(slots), T, ptr(c.k), ptr(c.v),
                                             ptr<float>(c.scales), c.NB, (int)c.bs, (int)c.Hk, (int)c.D,
                                             element_code(type), a.stream));
}
PyObject *kv_write_fp8_block(PyObject *, PyObject *const *args, Py_ssize_t n) { return move_fp8_block(args, n, true); }
PyObject *kv_read_fp8_block(PyObject *, PyObject *const *args, Py_ssize_t n) { return move_fp8_block(args, n, false); }

// A workspace buffer of the current stream, as the Python binding's: cached and grown on demand, or
// the call's own, from the graph's memory, while the stream is captured.
Tensor workspace(int device, cudaStream_t stream, int64_t bytes) {
    static auto *cache = new std::map<std::pair<int, cudaStream_t>, Tensor>;   // never destroyed: CUDA may be gone first
    const auto options = at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)device);
    if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None)
        return at::empty({std::max<int64_t>(bytes, 16)}, options);
    Tensor &t = (*cache)[{device, stream}];
    if (!t.defined() || t.numel() < bytes) t = at::empty({std::max<int64_t>(bytes, 1 << 20)}, options);
    return t;
}

// out, q, key_cache, value_cache, kv_scales, block_tables, context_lens, scale, max_context_len,
// workspace, stream
PyObject *attention_decode_fp8_block(PyObject *, PyObject *const *args, Py_ssize_t n) {
    Args a(args, n, 11);
    if (!a.ok) Py_RETURN_NONE;
    const Cache c(a, 2);
    const Tensor *q = a.tensor(1);
    if (!a.ok || q->dim() != 3) Py_RETURN_NONE;
    const at::ScalarType type = q->scalar_type();
    const int64_t B = q->size(0), H = q->size(1);
    a.dense(1, type, 3);
    const Tensor *out = a.dense(0, type, 3), *table = a.dense(5, at::kInt, 2), *lens = a.vector(6, at::kInt, B);
    a.ok = a.ok && q->size(2) == c.D && out->sizes() == q->sizes() && table->size(0) == B && element_code(type) >= 0 &&
           std::max({B, H, table->size(1)}) <= INT_MAX;
    const double scale = a.real(7);
    const int bound = a.small(8);
    a.on_stream(10);
    if (!a.ok || bound < 0) Py_RETURN_NONE;
    const int64_t longest = bound ? bound : table->size(1) * c.bs;
    if (longest > INT_MAX) Py_RETURN_NONE;
    Tensor ws;
    if (a.none(9)) {
        // on another stream than the current one the buffer would have to be allocated there
        if (!a.none(10) && a.stream != c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)a.device).stream()) Py_RETURN_NONE;
        const size_t need = pa_decode_fp8_block_workspace_bytes((int)B, (int)H, (int)c.Hk, (int)c.D, (int)longest);
        ws = workspace(a.device, a.stream, (int64_t)need);
    } else {
        const Tensor *given = a.dense(9, at::kByte, 1);
        if (!a.ok) Py_RETURN_NONE;
        ws = *given;
    }
    return status(pa_paged_attention_decode_fp8_block(
        ptr(out), ptr(q), ptr(c.k), ptr(c.v), ptr<float>(c.scales), ptr<int32_t>(table), (int)table->size(1),
        ptr<int32_t>(lens), (int)B, (int)H, (int)c.Hk, (int)c.D, (int)c.bs, c.NB, (float)scale, bound, ws.data_ptr(),
        (size_t)ws.numel(), element_code(type), a.stream));
}

// torch reports failures (a CUDA error left by earlier work, no memory) as exceptions, which must not pass
// through Python's frames: the Python code meets them again, in its own way.
template <PyObject *(*kFunction)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    try {
        return kFunction(self, args, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// The header that this module was built with, that of the library which it calls, and where that library is: the
// package takes the module only if the two are one and the library is its own.
PyObject *interface(PyObject *, PyObject *) {
    return Py_BuildValue("KKK", (unsigned long long)PA_INTERFACE, (unsigned long long)pa_internal_interface(),
                         (unsigned long long)reinterpret_cast<uintptr_t>(&pa_version));
}

#define PA_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD(blocks_append),      PA_METHOD(blocks_release),    PA_METHOD(rotary_embedding),
                         PA_METHOD(kv_write_rotary),    PA_METHOD(kv_write_fp8_block), PA_METHOD(kv_read_fp8_block),
                         PA_METHOD(attention_decode_fp8_block), {"interface", interface, METH_NOARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pagedattn_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__pagedattn_binding() { return PyModule_Create(&module); }
