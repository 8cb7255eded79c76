// Native marshalling of the attention path's tensor-level calls.
//
// A decode step's launches take 2 to 10 us on the GPU; reading a dozen tensors'
// shapes, strides and pointers from Python and converting two dozen arguments
// takes longer than that.  These functions make the same checks as attn.py and
// step.py and call the same C ABI (include/rmsnorm_attn.h) on the current stream.  What
// they do not take (a tensor on another device than the current one, a wrong
// shape, a refused call) they leave: they return None before anything is
// launched, and attn.py (or step.py) makes the call, or raises the error, itself.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "rmsnorm_attn.h"

namespace {

using at::Tensor;

PyObject* leave() { Py_RETURN_NONE; }

const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on_device(const Tensor& t, int64_t index) {
    return t.layout() == at::kStrided && t.is_cuda() && t.get_device() == index;
}

int dtype_flag(at::ScalarType t) {
    return t == at::kBFloat16 ? RMSN_IN_BF16 : (t == at::kHalf ? RMSN_IN_F16 : (t == at::kFloat ? RMSN_IN_F32 : -1));
}

// Whether the program looks at what is called (a TorchDispatchMode): it then sees new tensors, too.
bool watched() { return c10::impl::TorchDispatchModeTLS::any_modes_set(); }

// (at::empty by way of the dispatcher takes 0.4 us more: fused_block_norms of 8 x 4096, with
// two results, 6.1 us a call and 7.0)
Tensor make(at::IntArrayRef sizes, at::ScalarType type, int64_t index) {
    const c10::Device device(c10::kCUDA, (c10::DeviceIndex)index);
    if (watched()) return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
    return at::detail::empty_cuda(sizes, type, device, std::nullopt);
}

// [size] of a type, at a byte of another tensor's memory.
Tensor part(const Tensor& whole, int64_t at, int64_t size, at::ScalarType type) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(whole.storage()),
                                                     c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                     c10::scalarTypeToTypeMeta(type));
    impl->set_storage_offset(at / (int64_t)c10::elementSize(type));
    impl->set_sizes_contiguous({size});
    return Tensor(std::move(impl));
}

cudaStream_t stream_of(int64_t index) {
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
}

// Heads and token stride of [T, H * D] or [T, H, D], a token's heads back to back.
bool heads(const Tensor& t, int64_t D, int64_t* H, int64_t* stride) {
    int64_t width;
    if (t.dim() == 2) {
        width = t.size(1);
        if (width % D || (t.stride(1) != 1 && width != 1)) return false;
    } else if (t.dim() == 3) {
        if (t.size(2) != D || (t.stride(2) != 1 && D != 1) || (t.stride(1) != D && t.size(1) > 1)) return false;
        width = t.size(1) * D;
    } else {
        return false;
    }
    *H = width / D;
    *stride = t.size(0) > 1 ? t.stride(0) : width;
    return true;
}

// A block table and its lengths, as the kernels read them.
bool sequences(const Tensor& table, const Tensor& lengths, int64_t n, int64_t index, int64_t* stride) {
    if (table.dim() != 2 || table.size(0) != n || table.scalar_type() != at::kInt || !on_device(table, index) ||
        (table.size(1) > 1 && table.stride(1) != 1))
        return false;
    if (lengths.dim() != 1 || lengths.size(0) != n || lengths.scalar_type() != at::kInt ||
        !on_device(lengths, index) || (n > 1 && lengths.stride(0) != 1))
        return false;
    *stride = n > 1 ? table.stride(0) : table.size(1);
    return true;
}

// n contiguous int32, on the device, and their address (NULL: None).
bool ints(PyObject* o, int64_t n, int64_t index) {
    const Tensor* t = tensor(o);
    return t && t->dim() == 1 && t->size(0) == n && t->scalar_type() == at::kInt && on_device(*t, index) &&
           t->is_contiguous();
}
const int32_t* words(PyObject* o) {
    const Tensor* t = tensor(o);
    return t ? static_cast<const int32_t*>(t->const_data_ptr()) : nullptr;
}

// Tokens of [B, n, H, D] (or [B, H, D], n = 1): evenly spaced, heads back to back.
bool token_stride(const Tensor& t, int64_t n, int64_t* step) {
    const int64_t d = t.dim(), H = t.size(d - 2), D = t.size(d - 1), B = t.size(0);
    if (t.stride(d - 1) != 1 || (H > 1 && t.stride(d - 2) != D)) return false;
    if (n > 1) {
        if (B > 1 && t.stride(0) != n * t.stride(1)) return false;
        *step = t.stride(1);
    } else {
        *step = B > 1 ? t.stride(0) : H * D;
    }
    return true;
}

// The cache described at `address`, if its four tensors still lie where the
// description says (one may have been given other memory since).
const rmsattn_cache* cache_at(PyObject* address, PyObject* tensors) {
    const rmsattn_cache* c = static_cast<const rmsattn_cache*>(PyLong_AsVoidPtr(address));
    if (!c || !PyTuple_Check(tensors) || PyTuple_GET_SIZE(tensors) != 4) return nullptr;
    const void* const at[4] = {c->k, c->v, c->k_scale, c->v_scale};
    for (int i = 0; i < 4; ++i) {
        const Tensor* t = tensor(PyTuple_GET_ITEM(tensors, i));
        if (!t || t->const_data_ptr() != at[i]) return nullptr;
    }
    return c;
}

// (q, cache, tensors, index, block_table, lengths, scale, window, sinks, out, pdl) -> out
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t count) {
    try {
        const Tensor *q = count == 11 ? tensor(a[0]) : nullptr, *table = q ? tensor(a[4]) : nullptr,
                     *lengths = table ? tensor(a[5]) : nullptr;
        if (!lengths || !PyLong_Check(a[7]) || !PyLong_Check(a[8]) || !PyBool_Check(a[10]) || (a[6] != Py_None && !PyFloat_Check(a[6])))
            return leave();
        const rmsattn_cache* cache = cache_at(a[1], a[2]);
        const int64_t index = PyLong_AsLongLong(a[3]), window = PyLong_AsLongLong(a[7]),
                      sinks = PyLong_AsLongLong(a[8]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return leave();
        }
        if (!cache || index < 0 || index != c10::cuda::current_device() || !on_device(*q, index)) return leave();
        const int64_t d = q->dim();
        if (d != 3 && d != 4) return leave();
        const int64_t B = q->size(0), n = d == 4 ? q->size(1) : 1, H = q->size(d - 2), D = q->size(d - 1);
        const at::ScalarType type = q->scalar_type();
        if ((type != at::kBFloat16 && type != at::kHalf) || D != cache->head_dim || H < 1 ||
            H % cache->n_kv_heads || n < 1 || n > RMSATTN_MAX_QUERIES || window < 0 || sinks < 0)
            return leave();
        int64_t stride, qs, os = H * D;
        if (!sequences(*table, *lengths, B, index, &stride) || !token_stride(*q, n, &qs)) return leave();
        Tensor out;
        if (a[9] != Py_None) {
            const Tensor* o = tensor(a[9]);
            if (!o || !on_device(*o, index) || o->scalar_type() != type || o->sizes() != q->sizes() ||
                !token_stride(*o, n, &os))
                return leave();
            out = *o;
        }
        const int64_t width = table->size(1);
        const int64_t need = rmsattn_kv_attention_workspace(B, n, H, cache->n_kv_heads, D,
                                                            width * cache->page_size, window, sinks);
        if (need < 0) return leave();
        if (!out.defined()) out = make(q->sizes(), type, index);
        // freed when this returns: the allocator hands it to later work of the
        // same stream only, which runs behind the kernels
        Tensor ws;
        if (need > 0) ws = make({need}, at::kByte, index);
        const double scale = a[6] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AS_DOUBLE(a[6]);
        const int st = rmsattn_kv_attention(
            q->const_data_ptr(), cache, static_cast<const int32_t*>(table->const_data_ptr()), stride, width,
            static_cast<const int32_t*>(lengths->const_data_ptr()), out.mutable_data_ptr(), qs, os, B, n, H,
            (float)scale, window, sinks, need > 0 ? ws.mutable_data_ptr() : nullptr, need,
            (uint32_t)dtype_flag(type) | (a[10] == Py_True ? RMSN_PDL : 0u), stream_of(index));
        if (st != RMSN_OK) return leave();
        if (a[9] != Py_None) {
            Py_INCREF(a[9]);
            return a[9];
        }
        return THPVariable_Wrap(out);
    } catch (...) {
        PyErr_Clear();
        return leave();
    }
}

// (k, v, cache, tensors, index, block_table, lengths, cu_seqlens, pdl) -> True
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t count) {
    try {
        const Tensor *k = count == 9 ? tensor(a[0]) : nullptr, *v = k ? tensor(a[1]) : nullptr,
                     *table = v ? tensor(a[5]) : nullptr, *lengths = table ? tensor(a[6]) : nullptr;
        if (!lengths || !PyBool_Check(a[8])) return leave();
        const rmsattn_cache* cache = cache_at(a[2], a[3]);
        const int64_t index = PyLong_AsLongLong(a[4]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return leave();
        }
        if (!cache || index < 0 || index != c10::cuda::current_device() || !on_device(*k, index) || !on_device(*v, index))
            return leave();
        const int type = dtype_flag(k->scalar_type());
        int64_t hk, ks, hv, vs, stride;
        if (type < 0 || v->scalar_type() != k->scalar_type() || !heads(*k, cache->head_dim, &hk, &ks) ||
            !heads(*v, cache->head_dim, &hv, &vs) || hk != cache->n_kv_heads || hv != hk ||
            v->size(0) != k->size(0) || lengths->dim() != 1)
            return leave();
        const int64_t T = k->size(0), n = lengths->size(0);
        if (!sequences(*table, *lengths, n, index, &stride)) return leave();
        const int32_t* cu = nullptr;
        if (a[7] != Py_None) {
            const Tensor* c = tensor(a[7]);
            if (!c || c->dim() != 1 || c->size(0) != n + 1 || c->scalar_type() != at::kInt ||
                !on_device(*c, index) || (n && c->stride(0) != 1))
                return leave();
            cu = static_cast<const int32_t*>(c->const_data_ptr());
        } else if (T != n) {
            return leave();
        }
        const int st = rmsattn_kv_append(
            cache, k->const_data_ptr(), v->const_data_ptr(), ks, vs,
            static_cast<const int32_t*>(table->const_data_ptr()), stride, table->size(1),
            static_cast<const int32_t*>(lengths->const_data_ptr()), cu, T, n,
            (uint32_t)type | (a[8] == Py_True ? RMSN_PDL : 0u), stream_of(index));
        if (st != RMSN_OK) return leave();
        Py_RETURN_TRUE;
    } catch (...) {
        PyErr_Clear();
        return leave();
    }
}

// One side of qk_rope: the input's heads and strides, the output (made where
// `given` is None).
struct Side {
    const Tensor* x = nullptr;
    Tensor out;
    int64_t H = 0, stride = 0, out_stride = 0;
    bool of(PyObject* in, PyObject* given, int64_t D, at::ScalarType type, int64_t T, int64_t index) {
        if (in == Py_None) return true;
        x = tensor(in);
        if (!x || !on_device(*x, index) || x->scalar_type() != type || x->dim() < 1 || x->size(0) != T ||
            !heads(*x, D, &H, &stride))
            return false;
        if (given == Py_None) return true;
        const Tensor* o = tensor(given);
        int64_t h;
        if (!o || !on_device(*o, index) || o->scalar_type() != type || o->sizes() != x->sizes() ||
            !heads(*o, D, &h, &out_stride))
            return false;
        out = *o;
        return true;
    }
    void allocate(int64_t D, at::ScalarType type, int64_t index) {
        if (!x || out.defined()) return;
        out = make(x->sizes(), type, index);
        out_stride = H * D;
    }
    PyObject* result(PyObject* given) const {
        if (x && given == Py_None) return THPVariable_Wrap(out);
        Py_INCREF(given);
        return given;
    }
};

bool weight_ok(PyObject* o, int64_t D, at::ScalarType type, int64_t index, const void** p) {
    *p = nullptr;
    if (o == Py_None) return true;
    const Tensor* w = tensor(o);
    if (!w || !on_device(*w, index) || w->dim() != 1 || w->size(0) != D || w->scalar_type() != type ||
        (D > 1 && w->stride(0) != 1))
        return false;
    *p = w->const_data_ptr();
    return true;
}

// (q, k, positions, turns, axis, n_axes, q_weight, k_weight, head_dim, eps,
//  weight_offset, interleaved, q_out, k_out, pdl) -> (q_out, k_out)
PyObject* qk_rope(PyObject*, PyObject* const* a, Py_ssize_t count) {
    try {
        if (count != 15) return leave();
        const Tensor *pos = tensor(a[2]), *turns = tensor(a[3]), *axis = tensor(a[4]);
        const Tensor* ref = a[0] != Py_None ? tensor(a[0]) : tensor(a[1]);
        if (!pos || !turns || !axis || !ref || ref->dim() < 1 || !PyLong_Check(a[8]) ||
            (a[9] != Py_None && !PyFloat_Check(a[9])) || !PyFloat_Check(a[10]) || !PyBool_Check(a[11]) ||
            !PyBool_Check(a[14]))
            return leave();
        const int64_t n_axes = PyLong_AsLongLong(a[5]), D = PyLong_AsLongLong(a[8]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return leave();
        }
        if (!ref->is_cuda() || D < 1) return leave();
        const int64_t index = ref->get_device(), T = ref->size(0), R = turns->dim() == 1 ? 2 * turns->size(0) : D + 1;
        const at::ScalarType type = ref->scalar_type();
        int flags = dtype_flag(type);
        if (flags < 0 || index != c10::cuda::current_device() || R > D || !on_device(*turns, index) ||
            !on_device(*axis, index) || !on_device(*pos, index))
            return leave();
        // the table is as it was made
        if (turns->scalar_type() != at::kLong || axis->scalar_type() != at::kInt || axis->dim() != 1 ||
            axis->size(0) * 2 != R || !turns->is_contiguous() || !axis->is_contiguous())
            return leave();
        Side q, k;
        if (!q.of(a[0], a[12], D, type, T, index) || !k.of(a[1], a[13], D, type, T, index)) return leave();
        const int64_t pd = pos->dim();
        if (pd == 2 ? (pos->size(0) != n_axes || pos->size(1) != T) : (pd != 1 || n_axes != 1 || pos->size(0) != T))
            return leave();
        if (T > 1 && pos->stride(pd - 1) != 1) return leave();
        if (pos->scalar_type() == at::kLong) flags |= RMSATTN_POS_I64;
        else if (pos->scalar_type() != at::kInt) return leave();
        const void *qw = nullptr, *kw = nullptr;
        if (a[9] != Py_None) {
            flags |= RMSATTN_NORM;
            if (!weight_ok(a[6], D, type, index, &qw) || !weight_ok(a[7], D, type, index, &kw)) return leave();
        } else if (a[6] != Py_None || a[7] != Py_None) {
            return leave();
        }
        if (a[11] == Py_True) flags |= RMSATTN_INTERLEAVED;
        if (a[14] == Py_True) flags |= RMSN_PDL;
        q.allocate(D, type, index);
        k.allocate(D, type, index);
        const int st = rmsattn_qk_rope_fwd(
            q.x ? q.x->const_data_ptr() : nullptr, k.x ? k.x->const_data_ptr() : nullptr, qw, kw,
            q.x ? q.out.mutable_data_ptr() : nullptr, k.x ? k.out.mutable_data_ptr() : nullptr,
            pos->const_data_ptr(), n_axes > 1 ? pos->stride(0) : T,
            static_cast<const uint64_t*>(turns->const_data_ptr()),
            static_cast<const int32_t*>(axis->const_data_ptr()), T, q.H, k.H, D, R, n_axes, q.stride, k.stride,
            q.out_stride, k.out_stride, a[9] == Py_None ? 0.f : (float)PyFloat_AS_DOUBLE(a[9]),
            (float)PyFloat_AS_DOUBLE(a[10]), (uint32_t)flags, stream_of(index));
        if (st != RMSN_OK) return leave();
        PyObject *qo = q.result(a[12]), *ko = k.result(a[13]);
        PyObject* both = qo && ko ? PyTuple_Pack(2, qo, ko) : nullptr;
        Py_XDECREF(qo);
        Py_XDECREF(ko);
        return both;
    } catch (...) {
        PyErr_Clear();
        return leave();
    }
}

// (q, cache, tensors, index, block_table, lengths, prefix_lengths, groups, scale, out, pdl) -> out
PyObject* kv_prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t count) {
    try {
        const Tensor *q = count == 11 ? tensor(a[0]) : nullptr, *table = q ? tensor(a[4]) : nullptr,
                     *lengths = table ? tensor(a[5]) : nullptr, *shared = lengths ? tensor(a[6]) : nullptr;
        if (!shared || !PyBool_Check(a[10]) || (a[8] != Py_None && !PyFloat_Check(a[8]))) return leave();
        const rmsattn_cache* cache = cache_at(a[1], a[2]);
        const int64_t index = PyLong_AsLongLong(a[3]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return leave();
        }
        if (!cache || index < 0 || index != c10::cuda::current_device() || !on_device(*q, index)) return leave();
        const int64_t d = q->dim();
        if (d != 3 && d != 4) return leave();
        const int64_t B = q->size(0), n = d == 4 ? q->size(1) : 1, H = q->size(d - 2), D = q->size(d - 1);
        const at::ScalarType type = q->scalar_type();
        if ((type != at::kBFloat16 && type != at::kHalf) || D != cache->head_dim || H < 1 ||
            H % cache->n_kv_heads || n < 1 || n > RMSATTN_MAX_QUERIES)
            return leave();
        int64_t stride, qs, os = H * D;
        if (!sequences(*table, *lengths, B, index, &stride) || !token_stride(*q, n, &qs)) return leave();
        if (!ints(a[6], shared->dim() == 1 ? shared->size(0) : -1, index)) return leave();
        const int64_t n_groups = shared->size(0);
        if (a[7] == Py_None ? n_groups != 1 : !ints(a[7], n_groups + 1, index)) return leave();
        Tensor out;
        if (a[9] != Py_None) {
            const Tensor* o = tensor(a[9]);
            if (!o || !on_device(*o, index) || o->scalar_type() != type || o->sizes() != q->sizes() ||
                !token_stride(*o, n, &os))
                return leave();
            out = *o;
        }
        const int64_t width = table->size(1);
        const int64_t need = rmsattn_kv_prefix_attention_workspace(B, n, H, cache->n_kv_heads, D,
                                                                   width * cache->page_size, n_groups);
        if (need < 0) return leave();
        if (!out.defined()) out = make(q->sizes(), type, index);
        // freed when this returns, as above
        Tensor ws = make({need}, at::kByte, index);
        const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)D) : PyFloat_AS_DOUBLE(a[8]);
        const int st = rmsattn_kv_prefix_attention(
            q->const_data_ptr(), cache, static_cast<const int32_t*>(table->const_data_ptr()), stride, width,
            static_cast<const int32_t*>(lengths->const_data_ptr()), words(a[6]), words(a[7]), n_groups,
            out.mutable_data_ptr(), qs, os, B, n, H, (float)scale, ws.mutable_data_ptr(), need,
            (uint32_t)dtype_flag(type) | (a[10] == Py_True ? RMSN_PDL : 0u), stream_of(index));
        if (st != RMSN_OK) return leave();
        if (a[9] != Py_None) {
            Py_INCREF(a[9]);
            return a[9];
        }
        return THPVariable_Wrap(out);
    } catch (...) {
        PyErr_Clear();
        return leave();
    }
}

// (free_pages, n_free, block_table, lengths, new_tokens, shared_pages, page_size, n_rows, pdl)
//   -> (cu_seqlens, positions, slots, rows, before, after, n_free)
PyObject* pages_step(PyObject*, PyObject* const* a, Py_ssize_t count) {
    try {
        const Tensor *free_pages = count == 9 ? tensor(a[0]) : nullptr, *table = free_pages ? tensor(a[2]) : nullptr,
                     *lengths = table ? tensor(a[3]) : nullptr;
        // (a mode sees seven results)
        if (!lengths || watched() || !PyLong_Check(a[6]) || !PyLong_Check(a[7]) || !PyBool_Check(a[8])) return leave();
        const int64_t page = PyLong_AsLongLong(a[6]), T = PyLong_AsLongLong(a[7]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return leave();
        }
        if (!free_pages->is_cuda() || free_pages->dim() != 1 || lengths->dim() != 1) return leave();
        const int64_t index = free_pages->get_device(), n = lengths->size(0), pages = free_pages->size(0);
        int64_t stride;
        if (index != c10::cuda::current_device() || !sequences(*table, *lengths, n, index, &stride) ||
            !ints(a[0], pages, index) || !ints(a[1], 1, index) || !ints(a[4], n, index) ||
            (a[5] != Py_None && !ints(a[5], n, index)) || T < 0 || page < RMSATTN_BLOCK)
            return leave();
        const int64_t need = rmsattn_pages_workspace(n);
        // (a size that the library refuses is not allocated for)
        if (need < 0 || T > (int64_t(1) << 29)) return leave();
        // the results lie in one allocation, each at a multiple of 16 bytes: with seven of their
        // own a step of 8 sequences took 12.5 us, not 8 (its kernel 4.6)
        const int64_t size[7] = {n + 1, T, T, T, n, n, 1};
        const at::ScalarType type[7] = {at::kInt, at::kInt, at::kLong, at::kInt, at::kInt, at::kInt, at::kInt};
        int64_t at[8] = {0};
        for (int i = 0; i < 7; ++i) at[i + 1] = (at[i] + size[i] * (int64_t)c10::elementSize(type[i]) + 15) / 16 * 16;
        const Tensor whole = make({at[7]}, at::kByte, index);
        Tensor out[7], ws;
        for (int i = 0; i < 7; ++i) out[i] = part(whole, at[i], size[i], type[i]);
        if (need > 0) ws = make({need}, at::kByte, index);
        auto to = [&](int i) { return static_cast<int32_t*>(out[i].mutable_data_ptr()); };
        const int st = rmsattn_pages_step(
            static_cast<int32_t*>(free_pages->mutable_data_ptr()), pages, words(a[1]),
            static_cast<int32_t*>(table->mutable_data_ptr()), stride, table->size(1), words(a[3]), words(a[4]),
            words(a[5]), n, page, T, to(0), to(1), static_cast<int64_t*>(out[2].mutable_data_ptr()), to(3), to(4),
            to(5), to(6), need > 0 ? ws.mutable_data_ptr() : nullptr, need, a[8] == Py_True ? RMSN_PDL : 0u,
            stream_of(index));
        if (st != RMSN_OK) return leave();
        PyObject* all = PyTuple_New(7);
        for (int i = 0; all && i < 7; ++i) {
            PyObject* o = THPVariable_Wrap(out[i]);
            if (!o) {
                Py_DECREF(all);
                return nullptr;
            }
            PyTuple_SET_ITEM(all, i, o);
        }
        return all;
    } catch (...) {
        PyErr_Clear();
        return leave();
    }
}

// [rows, cols] of a type, contiguous, on the device
bool matrix(const Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, int64_t index) {
    return t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && t.scalar_type() == type &&
           on_device(t, index) && t.is_contiguous();
}

// (x, residual, post_weight, weight, eps, gate, gate_index, residual_scale, weight_offset, out_dtype, out,
//  residual_out, out_scale, pdl) -> (out, residual_out, out_scale)
PyObject* block_norms(PyObject*, PyObject* const* a, Py_ssize_t count) {
    try {
        const Tensor *x = count == 14 ? tensor(a[0]) : nullptr, *residual = x ? tensor(a[1]) : nullptr;
        if (!residual || !PyFloat_Check(a[4]) || !PyFloat_Check(a[7]) || !PyFloat_Check(a[8]) || !PyBool_Check(a[13]))
            return leave();
        if (!x->is_cuda() || x->dim() != 2) return leave();
        const int64_t index = x->get_device(), T = x->size(0), H = x->size(1);
        const at::ScalarType type = x->scalar_type(), rtype = residual->scalar_type();
        int flags = dtype_flag(type);
        if (flags < 0 || index != c10::cuda::current_device() || !matrix(*x, T, H, type, index) ||
            (rtype != type && rtype != at::kFloat) || !matrix(*residual, T, H, rtype, index))
            return leave();
        bool fp8 = false;
        if (a[9] != Py_None) {  // (x's own type is the other way's)
            if (!PyUnicode_Check(a[9]) || PyUnicode_CompareWithASCIIString(a[9], "fp8") != 0) return leave();
            fp8 = true;
        }
        const at::ScalarType otype = fp8 ? at::kByte : type;
        const void *post = nullptr, *weight = nullptr, *gates = nullptr;
        if (!weight_ok(a[2], H, type, index, &post) || !weight_ok(a[3], H, type, index, &weight)) return leave();
        int64_t n_gates = 0, stride = 0;
        if (a[5] == Py_None) {
            if (a[6] != Py_None) return leave();
        } else {
            const Tensor* g = tensor(a[5]);
            if (!g) return leave();
            if (g->dim() == 1 && a[6] == Py_None) {
                if (!weight_ok(a[5], H, type, index, &gates)) return leave();
                n_gates = 1;
            } else {
                if (g->dim() != 2 || g->size(1) != H || g->scalar_type() != type || !on_device(*g, index) ||
                    (H > 1 && g->stride(1) != 1))
                    return leave();
                n_gates = g->size(0);
                stride = n_gates > 1 ? g->stride(0) : H;
                if (stride < H || (a[6] == Py_None ? n_gates != T : !ints(a[6], T, index))) return leave();
                gates = g->const_data_ptr();
            }
        }
        Tensor out[3];
        for (int i = 0; i < 3; ++i) {
            if (a[10 + i] == Py_None) continue;
            const Tensor* o = tensor(a[10 + i]);
            if (!o || (i == 2 ? !fp8 || o->dim() != 1 || o->size(0) != T || o->scalar_type() != at::kFloat ||
                                    !on_device(*o, index) || !o->is_contiguous()
                              : !matrix(*o, T, H, i == 0 ? otype : rtype, index)))
                return leave();
            out[i] = *o;
        }
        if (rtype != type) flags |= RMSN_RESIDUAL_F32;
        if (fp8) flags |= RMSATTN_OUT_FP8;
        if (a[13] == Py_True) flags |= RMSN_PDL;
        if (a[6] != Py_None) {  // rows that are left out of new outputs
            if (!out[0].defined()) flags |= RMSATTN_ZERO_OUT;
            if (!out[1].defined()) flags |= RMSATTN_ZERO_RESIDUAL;
            if (fp8 && !out[2].defined()) flags |= RMSATTN_ZERO_SCALE;
        }
        if (!out[0].defined()) out[0] = make({T, H}, otype, index);
        if (!out[1].defined()) out[1] = make({T, H}, rtype, index);
        if (fp8 && !out[2].defined()) out[2] = make({T}, at::kFloat, index);
        const int st = rmsattn_block_norms(
            x->const_data_ptr(), residual->const_data_ptr(), post, weight, gates, stride, words(a[6]), n_gates,
            out[0].mutable_data_ptr(), out[1].mutable_data_ptr(),
            fp8 ? static_cast<float*>(out[2].mutable_data_ptr()) : nullptr, T, H, (float)PyFloat_AS_DOUBLE(a[4]),
            (float)PyFloat_AS_DOUBLE(a[7]), (float)PyFloat_AS_DOUBLE(a[8]), (uint32_t)flags, stream_of(index));
        if (st != RMSN_OK) return leave();
        PyObject* all = PyTuple_New(3);
        for (int i = 0; all && i < 3; ++i) {
            PyObject* o = a[10 + i];
            if (o != Py_None || !out[i].defined()) Py_INCREF(o);
            else o = THPVariable_Wrap(out[i]);
            if (!o) {
                Py_DECREF(all);
                return nullptr;
            }
            PyTuple_SET_ITEM(all, i, o);
        }
        return all;
    } catch (...) {
        PyErr_Clear();
        return leave();
    }
}

PyMethodDef methods[] = {
    {"qk_rope", (PyCFunction)(void (*)(void))qk_rope, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, nullptr},
    {"kv_prefix_attention", (PyCFunction)(void (*)(void))kv_prefix_attention, METH_FASTCALL, nullptr},
    {"pages_step", (PyCFunction)(void (*)(void))pages_step, METH_FASTCALL, nullptr},
    {"block_norms", (PyCFunction)(void (*)(void))block_norms, METH_FASTCALL, nullptr},
    {"kv_attention", (PyCFunction)(void (*)(void))kv_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "rmsattn_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rmsattn_fast() { return PyModule_Create(&module); }
