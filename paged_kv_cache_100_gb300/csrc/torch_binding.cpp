// The step operators' way from tensors to the C ABI, compiled: what the ctypes
// functions of the package do in Python (addresses, sizes, checks, the output's
// allocation) takes 18 to 46 us of host time a call for operators that run in 3 to 10
// us on the GPU; a call through here takes 4.8 to 6.1, the launch among it.
// Arguments are positional and checked as in
// Python: shapes and types first, then the device.  A library status other than
// PA_OK is returned as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <memory>
#include <optional>
#include <string>

#include "pagedkv.h"

namespace {

decltype(&pa_plan_step) f_plan;
decltype(&pa_rope_cache_write) f_rope;
decltype(&pa_decode_block_fp8_rows) f_decode;
decltype(&pa_decode_block_fp8_workspace_bytes) f_decode_bytes;
decltype(&pa_prefill_block_fp8) f_prefill;
decltype(&pa_prefill_block_fp8_workspace_bytes) f_prefill_bytes;

constexpr int64_t kBlock = 16;

struct Bad {
    PyObject *type;
    std::string what;
};
[[noreturn]] void bad_value(std::string what) { throw Bad{PyExc_ValueError, std::move(what)}; }
[[noreturn]] void bad_type(std::string what) { throw Bad{PyExc_TypeError, std::move(what)}; }
struct PyFailed {};                  // a Python error is set

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor *optional_tensor(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyFailed{};
    return v;
}
// what the C ABI takes as int: a size beyond it must not wrap round
int int_of(int64_t v, const char *name) {
    if (v < INT32_MIN || v > INT32_MAX) bad_value(std::string(name) + " is too large");
    return (int)v;
}
double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyFailed{};
    return v;
}
bool is_codes(const at::Tensor &t) { return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn; }

int device_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
    return t.get_device();
}
void on_device(const at::Tensor &t, const char *name, int dev) {
    if (!t.is_cuda() || t.get_device() != dev)
        bad_value(std::string(name) + " must be a CUDA tensor on device " + std::to_string(dev));
}
void *address(const at::Tensor &t, const char *name, int dev) {
    on_device(t, name, dev);
    if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
template <typename T = void>
T *address(const at::Tensor &t, const char *name, int dev, at::ScalarType type) {
    if (t.scalar_type() != type)
        bad_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    return static_cast<T *>(address(t, name, dev));
}
int32_t *status_of(const at::Tensor *t, int dev) {
    if (t == nullptr) return nullptr;
    if (t->numel() < 1) bad_value("status must hold an int32");
    return address<int32_t>(*t, "status", dev, at::kInt);
}

// Makes the tensors' device current and a given stream (its address, None for
// the current one) the current stream, so that what the call allocates belongs
// to the stream that uses it.
struct Place {
    std::optional<c10::cuda::CUDAGuard> device;
    std::optional<c10::cuda::CUDAStreamGuard> stream;
    cudaStream_t at;
    Place(int dev, PyObject *given) {
        if (given != Py_None) {
            void *p = PyLong_AsVoidPtr(given);
            if (p == nullptr && PyErr_Occurred()) throw PyFailed{};
            stream.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), (c10::DeviceIndex)dev));
        } else if (c10::cuda::current_device() != dev) {
            device.emplace((c10::DeviceIndex)dev);
        }
        at = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    }
};

template <typename F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t want, F &&f) {
    HANDLE_TH_ERRORS
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return f();
    } catch (const Bad &e) {
        PyErr_SetString(e.type, e.what.c_str());
        return nullptr;
    } catch (const PyFailed &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// Calls the library with the interpreter released (a full launch queue waits).
template <typename F, typename... A>
pa_status call(F f, A... args) {
    pa_status rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f(args...);
    Py_END_ALLOW_THREADS;
    return rc;
}

PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 6, [&]() -> PyObject * {
        void *p[6];
        for (int i = 0; i < 6; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (p[i] == nullptr) bad_value("missing function");
        }
        f_plan = reinterpret_cast<decltype(f_plan)>(p[0]);
        f_rope = reinterpret_cast<decltype(f_rope)>(p[1]);
        f_decode = reinterpret_cast<decltype(f_decode)>(p[2]);
        f_decode_bytes = reinterpret_cast<decltype(f_decode_bytes)>(p[3]);
        f_prefill = reinterpret_cast<decltype(f_prefill)>(p[4]);
        f_prefill_bytes = reinterpret_cast<decltype(f_prefill_bytes)>(p[5]);
        Py_RETURN_NONE;
    });
}

// `count` elements of `type` that begin at byte `at` of a byte tensor, sharing its
// storage (one allocation for several outputs).
at::Tensor part_of(const at::Tensor &whole, int64_t at, int64_t count, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)c10::elementSize(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous({count});
    return t;
}

// plan_step(block_tables, context_lens, new_lens, free_blocks, num_free, token_capacity, num_blocks,
//           out (five tensors or None), status, stream) -> tuple of five tensors
PyObject *plan_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const at::Tensor &tables = tensor(a[0], "block_tables"), &lens = tensor(a[1], "context_lens"),
                         &add = tensor(a[2], "new_lens"), &free = tensor(a[3], "free_blocks"),
                         &num_free = tensor(a[4], "num_free");
        const int64_t capacity = integer(a[5]);
        const int num_blocks = int_of(integer(a[6]), "num_blocks");
        if (tables.dim() != 2) bad_value("block_tables must be [num_seqs][max_blocks]");
        const int64_t B = tables.size(0);
        if (lens.sizes() != at::IntArrayRef{B} || add.sizes() != at::IntArrayRef{B})
            bad_value("context_lens and new_lens must be [num_seqs]");
        if (num_free.numel() != 1 || free.dim() != 1) bad_value("free_blocks must be [capacity], num_free [1]");
        if (capacity < 0) bad_value("token_capacity must not be negative");
        const at::Tensor *status = optional_tensor(a[8], "status");
        const int dev = device_of(tables, "block_tables");
        int32_t *p_tables = address<int32_t>(tables, "block_tables", dev, at::kInt);
        const int32_t *p_lens = address<int32_t>(lens, "context_lens", dev, at::kInt),
                      *p_add = address<int32_t>(add, "new_lens", dev, at::kInt),
                      *p_free = address<int32_t>(free, "free_blocks", dev, at::kInt),
                      *p_num = address<int32_t>(num_free, "num_free", dev, at::kInt);
        int32_t *p_status = status_of(status, dev);
        Place place(dev, a[9]);
        at::Tensor out[5];
        static const char *names[5] = {"out.context_lens", "out.query_start", "out.slot_mapping", "out.positions", "out.num_free"};
        const int64_t sizes[5] = {B, B + 1, capacity, capacity, 1};
        void *p[5];
        if (a[7] != Py_None) {
            PyObject *seq = PySequence_Fast(a[7], "out must be a StepPlan");
            if (seq == nullptr) throw PyFailed{};
            std::unique_ptr<PyObject, void (*)(PyObject *)> hold(seq, [](PyObject *o) { Py_DECREF(o); });
            if (PySequence_Fast_GET_SIZE(seq) != 5) bad_value("out must be a StepPlan");
            for (int i = 0; i < 5; ++i) out[i] = tensor(PySequence_Fast_GET_ITEM(seq, i), names[i]);
        }
        at::Tensor whole;
        int64_t at = 0;                  // in bytes, every part on 16
        if (a[7] == Py_None) whole = at::empty({8 * capacity + 4 * (capacity + 2 * B + 2) + 64}, tables.options().dtype(at::kByte));
        static const int order[5] = {2, 3, 1, 0, 4};
        for (int i : order) {
            const at::ScalarType type = i == 2 ? at::kLong : at::kInt;
            const int64_t size = i == 2 ? 8 : 4;
            if (a[7] == Py_None) {
                out[i] = part_of(whole, at, sizes[i], type);
                at = (at + sizes[i] * size + 15) & ~int64_t(15);
            } else if (i == 4 ? out[i].numel() != 1 : out[i].sizes() != at::IntArrayRef{sizes[i]})
                {
                bad_value("out does not fit num_seqs and token_capacity");
            }
            p[i] = address<void>(out[i], names[i], dev, type);
        }
        const pa_status rc =
            call(f_plan, p_tables, p_lens, p_add, p_free, p_num, (int32_t *)p[0], (int32_t *)p[1], (int64_t *)p[2],
                 (int32_t *)p[3], (int32_t *)p[4], int_of(B, "num_seqs"), int_of(tables.size(1), "max_blocks"), (int)kBlock,
                 num_blocks, int_of(free.size(0), "free_blocks"), int_of(capacity, "token_capacity"), p_status, (void *)place.at);
        if (rc != PA_OK) return PyLong_FromLong(rc);
        PyObject *t = PyTuple_New(5);
        if (t == nullptr) throw PyFailed{};
        for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(out[i]));
        return t;
    });
}

struct Rows {
    void *at;
    int64_t stride;
};
// Address and token stride of [tokens][heads][head_dim] rows, whose tokens may lie apart.
Rows rows_of(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType type) {
    if (t.sizes() != shape)
        bad_value(std::string(name) + " must be [" + std::to_string(shape[0]) + "][" + std::to_string(shape[1]) + "][" +
                  std::to_string(shape[2]) + "]");
    if (t.scalar_type() != type)
        bad_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if ((shape[2] > 1 && t.stride(2) != 1) || (shape[1] > 1 && t.stride(1) != shape[2]))
        bad_value(std::string(name) + ": the heads of a token must be contiguous");
    return {t.data_ptr(), shape[0] > 1 ? t.stride(0) : shape[1] * shape[2]};
}

// rope_cache_write(query or None, key, value, positions or None, turns or None, factor, rotary_dim,
//                  interleaved, key_cache, value_cache, slot_mapping, k_scales or None, v_scales or None,
//                  query_out or None, status, stream) -> query_out
PyObject *rope_cache_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 16, [&]() -> PyObject * {
        const at::Tensor *query = optional_tensor(a[0], "query"), *positions = optional_tensor(a[3], "positions"),
                         *turns = optional_tensor(a[4], "turns"), *ks = optional_tensor(a[11], "k_scales"),
                         *vs = optional_tensor(a[12], "v_scales"), *given = optional_tensor(a[13], "query_out"),
                         *status = optional_tensor(a[14], "status");
        const at::Tensor &key = tensor(a[1], "key"), &value = tensor(a[2], "value"), &kc = tensor(a[8], "key_cache"),
                         &vc = tensor(a[9], "value_cache"), &slots = tensor(a[10], "slot_mapping");
        const double factor = number(a[5]);
        const int64_t rot = integer(a[6]);
        const int interleaved = (int)integer(a[7]);
        if (kc.dim() != 4 || kc.size(2) != kBlock || vc.sizes() != kc.sizes())
            bad_value("pools must be [num_blocks][num_kv_heads][16][head_dim]");
        if (slots.dim() != 1) bad_value("slot_mapping must be [num_tokens]");
        const int64_t NB = kc.size(0), Hkv = kc.size(1), D = kc.size(3), T = slots.size(0);
        const at::ScalarType type = key.scalar_type();
        if (type != at::kFloat && type != at::kBFloat16) bad_type("rows must be float32 or bfloat16");
        const bool codes = is_codes(kc);
        if (codes) {
            if (!ks || !vs || ks->sizes() != at::IntArrayRef{NB, Hkv} || vs->sizes() != at::IntArrayRef{NB, Hkv})
                bad_value("E4M3 pools need k_scales and v_scales [num_blocks][num_kv_heads]");
            if (!is_codes(vc)) bad_type("both pools must hold E4M3 codes");
        } else if (kc.scalar_type() != type || vc.scalar_type() != type) {
            bad_type("pools must have the rows' element type, or hold E4M3 codes");
        }
        const Rows k = rows_of(key, "key", {T, Hkv, D}, type), v = rows_of(value, "value", {T, Hkv, D}, type);
        if (rot > 0) {
            if (!positions || positions->sizes() != at::IntArrayRef{T}) bad_value("positions must be [num_tokens]");
            if (!turns || turns->numel() * 2 != rot) bad_value("rope: turns must be [rotary_dim / 2]");
        }
        int64_t Hq = 0;
        if (query) {
            if (query->dim() != 3) bad_value("query must be [num_tokens][num_q_heads][head_dim]");
            Hq = query->size(1);
        }
        const int dev = device_of(kc, "key_cache");
        on_device(key, "key", dev);
        on_device(value, "value", dev);
        void *p_kc = address(kc, "key_cache", dev), *p_vc = address(vc, "value_cache", dev);
        const int64_t *p_slots = address<int64_t>(slots, "slot_mapping", dev, at::kLong);
        const int32_t *p_pos = rot > 0 ? address<int32_t>(*positions, "positions", dev, at::kInt) : nullptr;
        const uint64_t *p_turns =
            rot > 0 ? reinterpret_cast<const uint64_t *>(address<int64_t>(*turns, "turns", dev, at::kLong)) : nullptr;
        float *p_ks = codes ? address<float>(*ks, "k_scales", dev, at::kFloat) : nullptr;
        float *p_vs = codes ? address<float>(*vs, "v_scales", dev, at::kFloat) : nullptr;
        int32_t *p_status = status_of(status, dev);
        Place place(dev, a[15]);
        Rows q{nullptr, 0}, o{nullptr, 0};
        at::Tensor out;
        if (query) {
            on_device(*query, "query", dev);
            q = rows_of(*query, "query", {T, Hq, D}, type);
            out = given ? *given : at::empty({T, Hq, D}, query->options());
            on_device(out, "query_out", dev);
            o = rows_of(out, "query_out", {T, Hq, D}, type);
        }
        const pa_dtype dtype = type == at::kFloat ? PA_DTYPE_F32 : PA_DTYPE_BF16;
        const pa_status rc =
            call(f_rope, o.at, (const void *)q.at, (const void *)k.at, (const void *)v.at, p_pos, p_turns, factor,
                 int_of(rot, "rotary_dim"), interleaved, p_kc, p_vc, p_ks, p_vs, p_slots, int_of(T, "num_tokens"),
                 int_of(Hq, "num_q_heads"), int_of(Hkv, "num_kv_heads"), int_of(D, "head_dim"), o.stride, q.stride, k.stride,
                 v.stride, (int)kBlock, int_of(NB, "num_blocks"), dtype, codes ? PA_DTYPE_FP8_E4M3 : dtype, p_status,
                 (void *)place.at);
        if (rc != PA_OK) return PyLong_FromLong(rc);
        if (!query) Py_RETURN_NONE;
        return THPVariable_Wrap(out);
    });
}

// What decode and prefill check of their pools.
struct Pools {
    int dev, num_blocks, hq, hkv, head_dim, num_seqs, max_blocks;
    void *query, *kc, *vc, *workspace;
    const float *ks, *vs;
    const int32_t *tables, *lens;
    size_t workspace_bytes;
    int32_t *status;
};
Pools pools_of(PyObject *const *a, PyObject *status) {
    const at::Tensor &q = tensor(a[0], "query"), &kc = tensor(a[1], "key_cache"), &vc = tensor(a[2], "value_cache"),
                     &ks = tensor(a[3], "k_scales"), &vs = tensor(a[4], "v_scales"), &tables = tensor(a[5], "block_tables"),
                     &lens = tensor(a[6], "context_lens");
    if (q.dim() != 3) bad_value("query must be [rows][num_q_heads][head_dim]");
    if (kc.dim() != 4 || kc.size(2) != kBlock || kc.size(3) != q.size(2) || vc.sizes() != kc.sizes())
        bad_value("pools must be [num_blocks][num_kv_heads][16][head_dim] like query");
    if (!is_codes(kc) || !is_codes(vc) || q.scalar_type() != at::kBFloat16)
        bad_type("E4M3 pools and a bfloat16 query are expected");
    const int64_t NB = kc.size(0), Hkv = kc.size(1);
    if (ks.sizes() != at::IntArrayRef{NB, Hkv} || vs.sizes() != at::IntArrayRef{NB, Hkv})
        bad_value("k_scales / v_scales must be [num_blocks][num_kv_heads]");
    if (lens.dim() != 1) bad_value("context_lens must be [num_seqs]");
    if (tables.dim() != 2 || tables.size(0) != lens.size(0)) bad_value("block_tables must be [num_seqs][max_blocks]");
    Pools p;
    p.dev = device_of(q, "query");
    p.num_blocks = int_of(NB, "num_blocks");
    p.hq = int_of(q.size(1), "num_q_heads");
    p.hkv = int_of(Hkv, "num_kv_heads");
    p.head_dim = int_of(q.size(2), "head_dim");
    p.num_seqs = int_of(lens.size(0), "num_seqs");
    p.max_blocks = int_of(tables.size(1), "max_blocks");
    p.query = address(q, "query", p.dev);
    p.kc = address(kc, "key_cache", p.dev);
    p.vc = address(vc, "value_cache", p.dev);
    p.ks = address<float>(ks, "k_scales", p.dev, at::kFloat);
    p.vs = address<float>(vs, "v_scales", p.dev, at::kFloat);
    p.tables = address<int32_t>(tables, "block_tables", p.dev, at::kInt);
    p.lens = address<int32_t>(lens, "context_lens", p.dev, at::kInt);
    p.status = status_of(optional_tensor(status, "status"), p.dev);
    p.workspace = nullptr;
    p.workspace_bytes = 0;
    return p;
}
at::Tensor output_of(PyObject *given, const at::Tensor &q, int dev) {
    if (given == Py_None) return at::empty(q.sizes(), q.options());
    const at::Tensor &out = tensor(given, "out");
    if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type()) bad_value("out must match query");
    address(out, "out", dev);
    return out;
}
at::Tensor workspace_of(PyObject *given, size_t need, const at::Tensor &q, Pools &p) {
    at::Tensor w;
    if (given != Py_None) w = tensor(given, "workspace");
    else if (need > 0 && need < (size_t)1 << 62)       // invalid sizes are the call's to refuse
        w = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    if (w.defined()) {
        p.workspace = address(w, "workspace", p.dev);
        p.workspace_bytes = w.nbytes();
    }
    return w;
}

// decode_block_fp8(query, key_cache, value_cache, k_scales, v_scales, block_tables, context_lens, scale or
//                  None, window, out, partition_size, workspace, status, stream, query_start or None) -> out
PyObject *decode_block_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const int window = int_of(integer(a[8]), "window"), partition = int_of(integer(a[10]), "partition_size");
        const at::Tensor &q = tensor(a[0], "query"), &lens = tensor(a[6], "context_lens");
        const at::Tensor *start = optional_tensor(a[14], "query_start");
        if (!start && q.dim() == 3 && lens.sizes() != at::IntArrayRef{q.size(0)}) bad_value("context_lens must be [num_seqs]");
        if (start && (lens.dim() != 1 || start->sizes() != at::IntArrayRef{lens.size(0) + 1}))
            bad_value("query_start must be [num_seqs + 1]");
        Pools p = pools_of(a, a[12]);
        const int32_t *p_start = start ? address<int32_t>(*start, "query_start", p.dev, at::kInt) : nullptr;
        const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)p.head_dim)) : (float)number(a[7]);
        Place place(p.dev, a[13]);
        at::Tensor out = output_of(a[9], q, p.dev);
        const size_t need = a[11] != Py_None ? 0
                                             : f_decode_bytes(p.num_seqs, p.hq, p.hkv, p.head_dim, p.max_blocks,
                                                              (int)kBlock, window, partition);
        at::Tensor w = workspace_of(a[11], need, q, p);
        const pa_status rc = call(f_decode, out.data_ptr(), (const void *)p.query, (const void *)p.kc, (const void *)p.vc, p.ks,
                                  p.vs, p.tables, p.lens, p_start, p.num_seqs, int_of(q.size(0), "query"), p.hq, p.hkv,
                                  p.head_dim, (int)kBlock, p.max_blocks, p.num_blocks, scale, window, partition, p.workspace,
                                  p.workspace_bytes, p.status, (void *)place.at);
        if (rc != PA_OK) return PyLong_FromLong(rc);
        return THPVariable_Wrap(out);
    });
}

// prefill_block_fp8(query, key_cache, value_cache, k_scales, v_scales, block_tables, context_lens, query_start,
//                   max_query_len, scale or None, window, out, workspace, status, stream) -> out
PyObject *prefill_block_fp8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject * {
        const int longest = int_of(integer(a[8]), "max_query_len"), window = int_of(integer(a[10]), "window");
        Pools p = pools_of(a, a[13]);
        const at::Tensor &q = tensor(a[0], "query"), &start = tensor(a[7], "query_start");
        if (start.sizes() != at::IntArrayRef{p.num_seqs + 1}) bad_value("query_start must be [num_seqs + 1]");
        const int32_t *p_start = address<int32_t>(start, "query_start", p.dev, at::kInt);
        const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)p.head_dim)) : (float)number(a[9]);
        Place place(p.dev, a[14]);
        at::Tensor out = output_of(a[11], q, p.dev);
        const int tokens = int_of(q.size(0), "query");
        const size_t need = a[12] != Py_None ? 0
                                             : f_prefill_bytes(p.num_seqs, p.hq, p.hkv, p.head_dim, p.max_blocks, tokens,
                                                               longest, window);
        at::Tensor w = workspace_of(a[12], need, q, p);
        const pa_status rc = call(f_prefill, out.data_ptr(), (const void *)p.query, (const void *)p.kc, (const void *)p.vc,
                                  p.ks, p.vs, p.tables, p.lens, p_start, p.num_seqs, p.hq, p.hkv, p.head_dim, (int)kBlock,
                                  p.max_blocks, p.num_blocks, tokens, longest, scale, window, p.workspace,
                                  p.workspace_bytes, p.status, (void *)place.at);
        if (rc != PA_OK) return PyLong_FromLong(rc);
        return THPVariable_Wrap(out);
    });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"plan_step", (PyCFunction)(void (*)(void))plan_step, METH_FASTCALL, nullptr},
    {"rope_cache_write", (PyCFunction)(void (*)(void))rope_cache_write, METH_FASTCALL, nullptr},
    {"decode_block_fp8", (PyCFunction)(void (*)(void))decode_block_fp8, METH_FASTCALL, nullptr},
    {"prefill_block_fp8", (PyCFunction)(void (*)(void))prefill_block_fp8, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pagedkv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pagedkv_torch(void) { return PyModule_Create(&module); }
