// Native marshalling of the attention path's tensor-level calls.
//
// A decode step's launches take 2 to 10 us on the GPU; reading a dozen tensors'
// shapes, strides and pointers from Python and converting two dozen arguments
// takes longer than that.  These functions make the same checks as attn.py and
// call the same C ABI (include/rmsnorm_attn.h) on the current stream.  What
// they do not take (a tensor on another device than the current one, a wrong
// shape, a refused call) they leave: they return None before anything is
// launched, and attn.py makes the call, or raises the error, itself.
#include <Python.h>

#include <ATen/ATen.h>
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

Tensor make(at::IntArrayRef sizes, at::ScalarType type, int64_t index) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)index));
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

PyMethodDef methods[] = {
    {"qk_rope", (PyCFunction)(void (*)(void))qk_rope, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, nullptr},
    {"kv_attention", (PyCFunction)(void (*)(void))kv_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "rmsattn_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rmsattn_fast() { return PyModule_Create(&module); }
