// The binding's short way: the calls on the rotating append, the 4-bit cache and drafted tokens
// with their operands read from torch's tensors in C++.
//
// A call of a small step is bound by the host: of 16.9 us for a rotating append of eight tokens 9 were checks
// and allocations in Python and 8 ctypes with the launch; this way it takes 4.1 (verification of drafts 11.6 and 4.3,
// attention, with two launches and three allocations, 22.7 and 8.2).  Each function here takes the Python function's arguments in its order
// and makes the call where they are in the common form (CUDA tensors of the current device, the current stream, the
// documented types and layouts).  For anything else it returns NotImplemented and has done nothing: the Python function
// then goes through its own checks, which name what is wrong, or make the call's rarer forms.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "pkv.h"

namespace {

using at::Tensor;

constexpr int64_t kInt = INT_MAX;

// Not the common form.
struct Rare {};
void need(bool ok) {
    if (!ok) throw Rare{};
}

// The call's operands so far: all on the device of the first, which is the current one.
struct Call {
    int device = -1;

    const Tensor &tensor(PyObject *o) {
        need(THPVariable_CheckExact(o));
        const Tensor &t = THPVariable_Unpack(o);
        need(t.is_cuda() && t.layout() == at::kStrided);
        if (device < 0) {
            device = t.get_device();
            need(c10::cuda::current_device() == device);
        }
        need(t.get_device() == device);
        return t;
    }
    const Tensor &tensor(PyObject *o, at::ScalarType type) {
        const Tensor &t = tensor(o);
        need(t.scalar_type() == type && t.is_contiguous());
        return t;
    }
    void *pointer(PyObject *o, at::ScalarType type) { return tensor(o, type).data_ptr(); }
    Tensor make(at::IntArrayRef sizes, at::ScalarType type) const {
        return at::empty(sizes, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
    }
    pkv_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
};

int32_t int32_of(PyObject *o) {
    need(PyLong_CheckExact(o));
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    need(!overflow && x >= INT_MIN && x <= INT_MAX);
    return static_cast<int32_t>(x);
}
float float_of(PyObject *o) {
    need(PyFloat_CheckExact(o));
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
}
int32_t *error_word(PyObject *o) {
    if (o == Py_None) return nullptr;
    need(PyLong_CheckExact(o));
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
    need(!overflow && x >= 0);
    return reinterpret_cast<int32_t *>(x);
}
// The common form has no stream of its own, and raises errors.
void plain(PyObject *stream, PyObject *check) { need(stream == Py_None && check == Py_True); }

int32_t kind_of(at::ScalarType t) {
    need(t == at::kBFloat16 || t == at::kHalf);
    return t == at::kHalf ? PKV_FP16 : PKV_BF16;
}

// Bytes between the rows of [tokens, heads, dim] of a 16-bit type, each contiguous.
int64_t rows_of(const Tensor &x) {
    need(x.dim() == 3 && x.stride(2) == 1 && x.stride(1) == x.size(2) && x.size(1) <= kInt && x.size(2) <= kInt);
    return 2 * (x.size(0) > 1 ? x.stride(0) : x.size(1) * x.size(2));
}

template <typename F>
int without_lock(F f) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f();
    Py_END_ALLOW_THREADS
    return rc;
}

// f's result (a new reference), or NotImplemented where the call is not of the common form or fails.
template <typename F>
PyObject *call(F f) {
    try {
        return f();
    } catch (...) {                                   // Rare, or torch's own errors (out of memory)
        PyErr_Clear();
        Py_RETURN_NOTIMPLEMENTED;
    }
}

// A step's rows: k, v, q and what its queries are rotated into.
struct Rows {
    int32_t tokens, kind, q_heads = 0;
    int64_t k_stride, v_stride, q_stride = 0, out_stride = 0;
    const void *k, *v, *q = nullptr;
    void *out = nullptr;
    const int64_t *slots;
    Tensor made;

    Rows(Call &c, PyObject *k_, PyObject *v_, PyObject *q_, PyObject *out_, PyObject *slots_, int64_t heads, int64_t dim) {
        const Tensor &a = c.tensor(k_), &b = c.tensor(v_), &s = c.tensor(slots_, at::kLong);
        need(s.numel() <= kInt && a.scalar_type() == b.scalar_type() && a.sizes() == b.sizes());
        tokens = static_cast<int32_t>(s.numel());
        kind = kind_of(a.scalar_type());
        k_stride = rows_of(a);
        v_stride = rows_of(b);
        need(a.size(0) >= tokens && a.size(1) == heads && a.size(2) == dim);
        k = a.data_ptr();
        v = b.data_ptr();
        slots = static_cast<const int64_t *>(s.data_ptr());
        if (q_ == Py_None) {
            need(out_ == Py_None);
            return;
        }
        const Tensor &x = c.tensor(q_);
        need(x.scalar_type() == a.scalar_type());
        q_stride = rows_of(x);
        need(x.size(0) >= tokens && x.size(2) == dim);
        q_heads = static_cast<int32_t>(x.size(1));
        q = x.data_ptr();
        if (out_ == Py_None) {
            made = c.make({tokens, x.size(1), dim}, x.scalar_type());
        } else {
            made = c.tensor(out_);
            need(made.scalar_type() == x.scalar_type() && made.sizes() == x.sizes());
        }
        out_stride = rows_of(made);
        out = made.data_ptr();
    }
    PyObject *result() const {
        if (!made.defined()) Py_RETURN_NONE;        // no queries
        return THPVariable_Wrap(made);
    }
};

struct Rope : pkv_rope {
    uint8_t axes[128];

    Rope(Call &c, PyObject *positions_, PyObject *table_, PyObject *axes_, PyObject *interleaved_, int64_t tokens) {
        const Tensor &at_ = c.tensor(positions_), &t = c.tensor(table_, at::kFloat);
        const int64_t d = at_.dim();
        need(at_.scalar_type() == at::kInt && (d == 1 || d == 2) && at_.size(d - 1) >= tokens &&
             (at_.size(d - 1) <= 1 || at_.stride(d - 1) == 1));
        need(t.dim() == 2 && t.size(0) <= kInt && t.size(1) <= 256);
        const int64_t count = d == 2 ? at_.size(0) : 1, pairs = t.size(1) / 2;
        need(count <= kInt && (interleaved_ == Py_True || interleaved_ == Py_False));
        table = static_cast<const float *>(t.data_ptr());
        positions = static_cast<const int32_t *>(at_.data_ptr());
        pair_axes = nullptr;
        if (axes_ != Py_None) {
            const bool list = PyList_CheckExact(axes_);
            need(list || PyBytes_CheckExact(axes_));
            need((list ? PyList_GET_SIZE(axes_) : PyBytes_GET_SIZE(axes_)) == pairs);
            for (int64_t i = 0; i < pairs; i++) {
                const int32_t a = list ? int32_of(PyList_GET_ITEM(axes_, i)) : static_cast<uint8_t>(PyBytes_AS_STRING(axes_)[i]);
                need(a >= 0 && a <= 255);
                axes[i] = static_cast<uint8_t>(a);
            }
            pair_axes = axes;
        }
        axis_stride = count > 1 ? at_.stride(0) : 0;
        max_position = static_cast<int32_t>(t.size(0));
        rot_dim = static_cast<int32_t>(t.size(1));
        num_axes = static_cast<int32_t>(count);
        interleaved = interleaved_ == Py_True;
    }
};

struct Cache : pkv_kv4_cache {
    Cache(Call &c, PyObject *const *a, PyObject *k_unit_, PyObject *v_unit_) {
        const Tensor &k = c.tensor(a[0]), &v = c.tensor(a[1]), &ks = c.tensor(a[2]), &vs = c.tensor(a[3]);
        need(k.dim() == 4 && ks.dim() == 4 && v.sizes() == k.sizes() && vs.sizes() == ks.sizes());
        for (int i = 0; i < 3; i++) need(k.size(i) == ks.size(i));
        need(8 * ks.size(3) == k.size(3) && k.size(1) <= kInt && k.size(2) <= kInt && k.size(3) <= 256);
        for (const Tensor *t : {&k, &v, &ks, &vs}) need(t->itemsize() == 1 && t->is_contiguous());
        k_cache = k.data_ptr();
        v_cache = v.data_ptr();
        k_scale = ks.data_ptr();
        v_scale = vs.data_ptr();
        num_blocks = k.size(0);
        num_heads = static_cast<int32_t>(k.size(1));
        block_size = static_cast<int32_t>(k.size(2));
        head_dim = static_cast<int32_t>(2 * k.size(3));
        k_unit = float_of(k_unit_);
        v_unit = float_of(v_unit_);
    }
};

// k, v, k_cache, v_cache, slot_mapping, positions, table, axes, interleaved, q, q_out, d_error, stream, check
PyObject *rope_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call([&] {
        need(n == 14);
        plain(a[12], a[13]);
        Call c;
        const Tensor &k = c.tensor(a[0]), &kc = c.tensor(a[2], k.scalar_type()), &vc = c.tensor(a[3], k.scalar_type());
        need(k.dim() == 3 && kc.dim() >= 1 && kc.sizes() == vc.sizes());
        const int64_t heads = k.size(1), dim = k.size(2), lines = kc.size(0);
        need(heads <= kInt && dim <= kInt && kc.numel() == lines * heads * dim);
        const Rows r(c, a[0], a[1], a[9], a[10], a[4], heads, dim);
        const Rope rope(c, a[5], a[6], a[7], a[8], r.tokens);
        int32_t *const word = error_word(a[11]);
        const pkv_stream_t s = c.stream();
        void *const kp = kc.data_ptr(), *const vp = vc.data_ptr();
        need(without_lock([&] {
                 return pkv_rope_store(&rope, r.k, r.v, r.k_stride, r.v_stride, static_cast<int32_t>(heads), static_cast<int32_t>(dim),
                                       r.kind, r.q, r.q_stride, r.q_heads, r.out, r.out_stride, kp, vp, lines, r.slots, r.tokens,
                                       word, s);
             }) == PKV_OK);
        return r.result();
    });
}

// k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, positions, table, axes, interleaved, q, q_out, k_unit, v_unit,
// d_error, stream, check
PyObject *kv4_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call([&]() -> PyObject * {
        need(n == 18);
        plain(a[16], a[17]);
        Call c;
        const Cache cache(c, a + 2, a[13], a[14]);
        const bool turned = a[7] != Py_None;
        need(turned == (a[8] != Py_None) && (turned || (a[9] == Py_None && a[11] == Py_None)));
        const Rows r(c, a[0], a[1], a[11], a[12], a[6], cache.num_heads, cache.head_dim);
        int32_t *const word = error_word(a[15]);
        const pkv_stream_t s = c.stream();
        auto store = [&](const pkv_rope *rope) {
            need(without_lock([&] {
                     return pkv_kv4_store(&cache, rope, r.k, r.v, r.k_stride, r.v_stride, r.kind, r.q, r.q_stride, r.q_heads, r.out,
                                          r.out_stride, r.slots, r.tokens, word, s);
                 }) == PKV_OK);
        };
        if (turned) {
            const Rope rope(c, a[7], a[8], a[9], a[10], r.tokens);
            store(&rope);
        } else {
            store(nullptr);
        }
        return r.result();
    });
}

// k_cache, v_cache, k_scale, v_scale, slots, dtype, k, v, k_unit, v_unit, d_error, stream, check
PyObject *kv4_load(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call([&] {
        need(n == 13 && a[6] == Py_None && a[7] == Py_None);
        plain(a[11], a[12]);
        Call c;
        const Cache cache(c, a, a[8], a[9]);
        const Tensor &slots = c.tensor(a[4], at::kLong);
        need(slots.numel() <= kInt && (a[5] == Py_None || THPDtype_Check(a[5])));
        const at::ScalarType type = a[5] == Py_None ? at::kBFloat16 : reinterpret_cast<THPDtype *>(a[5])->scalar_type;
        const int32_t kind = kind_of(type), count = static_cast<int32_t>(slots.numel());
        int32_t *const word = error_word(a[10]);
        const Tensor k = c.make({count, cache.num_heads, cache.head_dim}, type), v = c.make(k.sizes(), type);
        const int64_t *const from = static_cast<const int64_t *>(slots.data_ptr());
        const pkv_stream_t s = c.stream();
        void *const kp = k.data_ptr(), *const vp = v.data_ptr();
        need(without_lock([&] { return pkv_kv4_load(&cache, from, count, kind, kp, vp, word, s); }) == PKV_OK);
        return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
    });
}

// q, k_cache, v_cache, k_scale, v_scale, block_tables, query_start_loc, seq_lens, softmax_scale, window, k_unit, v_unit, out,
// lse, workspace, d_error, stream, check
PyObject *kv4_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call([&] {
        need(n == 18);
        plain(a[16], a[17]);
        Call c;
        const Cache cache(c, a + 1, a[10], a[11]);
        const Tensor &q = c.tensor(a[0]), &tables = c.tensor(a[5], at::kInt), &starts = c.tensor(a[6], at::kInt);
        const Tensor &lens = c.tensor(a[7], at::kInt);
        const int32_t kind = kind_of(q.scalar_type());
        const int64_t stride = rows_of(q), T = q.size(0), heads = q.size(1), requests = lens.numel();
        need(q.size(2) == cache.head_dim && T <= kInt && requests < kInt && starts.numel() >= requests + 1 &&
             tables.dim() == 2 && tables.size(0) >= requests && tables.size(1) <= kInt);
        const float scale = a[8] == Py_None ? static_cast<float>(std::pow(static_cast<double>(cache.head_dim), -0.5)) : float_of(a[8]);
        const int32_t window = int32_of(a[9]);
        int32_t *const word = error_word(a[15]);
        Tensor out, lse, workspace;
        if (a[12] == Py_None) {
            out = c.make(q.sizes(), q.scalar_type());
        } else {
            out = c.tensor(a[12]);
            need(out.scalar_type() == q.scalar_type() && out.sizes() == q.sizes());
        }
        if (a[13] == Py_None) {
            lse = c.make({T, heads}, at::kFloat);
        } else {
            lse = c.tensor(a[13], at::kFloat);
            need(lse.dim() == 2 && lse.size(0) == T && lse.size(1) == heads);
        }
        if (a[14] == Py_None) {
            int64_t bytes = 0;
            need(pkv_kv4_attention_workspace(cache.head_dim, &bytes) == PKV_OK);
            workspace = c.make({bytes}, at::kByte);
        } else {
            workspace = c.tensor(a[14]);
            need(workspace.is_contiguous());
        }
        const int64_t out_stride = rows_of(out), bytes = static_cast<int64_t>(workspace.nbytes());
        const pkv_stream_t s = c.stream();
        const void *const qp = q.data_ptr();
        const int32_t *const tp = static_cast<const int32_t *>(tables.data_ptr()), *const sp = static_cast<const int32_t *>(starts.data_ptr());
        const int32_t *const lp = static_cast<const int32_t *>(lens.data_ptr());
        void *const op = out.data_ptr(), *const wp = workspace.data_ptr();
        float *const ep = static_cast<float *>(lse.data_ptr());
        const int32_t width = static_cast<int32_t>(tables.size(1));
        need(without_lock([&] {
                 return pkv_kv4_attention(&cache, qp, stride, kind, static_cast<int32_t>(heads), tp, width, sp, lp,
                                          static_cast<int32_t>(requests), static_cast<int32_t>(T), scale, window, op, out_stride, ep,
                                          wp, bytes, word, s);
             }) == PKV_OK);
        return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
    });
}

// target_probs, draft_ids, query_start_loc, uniforms, max_drafts, draft_probs, tokens, accepted, d_error, stream, check
PyObject *verify_drafts(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return call([&] {
        need(n == 11);
        plain(a[9], a[10]);
        Call c;
        const Tensor &p = c.tensor(a[0]), &ids = c.tensor(a[1], at::kInt), &starts = c.tensor(a[2], at::kInt);
        const Tensor &u = c.tensor(a[3], at::kFloat);
        const int32_t kind = p.scalar_type() == at::kFloat ? PKV_FP32 : kind_of(p.scalar_type());
        need(p.dim() == 2 && p.size(0) <= kInt && p.size(1) <= kInt && starts.numel() >= 1 && starts.numel() <= kInt);
        const int64_t rows = p.size(0), vocab = p.size(1), requests = starts.numel() - 1;
        auto stride_of = [&](const Tensor &t) {
            need(t.stride(1) == 1 || vocab == 1);
            return rows > 1 ? t.stride(0) : vocab;
        };
        const int32_t drafts = int32_of(a[4]);
        need(drafts >= 0 && drafts < kInt && ids.numel() >= rows - 1 && u.numel() >= rows);
        const int64_t p_stride = stride_of(p);
        int64_t q_stride = 0;
        const void *pp = p.data_ptr(), *qp = nullptr;
        if (a[5] != Py_None) {
            const Tensor &q = c.tensor(a[5]);
            need(q.scalar_type() == p.scalar_type() && q.sizes() == p.sizes());
            q_stride = stride_of(q);
            qp = q.data_ptr();
        }
        int32_t *const word = error_word(a[8]);
        Tensor tokens, accepted;
        if (a[6] == Py_None) {
            tokens = c.make({requests, drafts + 1LL}, at::kInt);
        } else {
            tokens = c.tensor(a[6], at::kInt);
            need(tokens.dim() == 2 && tokens.size(0) == requests && tokens.size(1) == drafts + 1LL);
        }
        if (a[7] == Py_None) {
            accepted = c.make({requests}, at::kInt);
        } else {
            accepted = c.tensor(a[7], at::kInt);
            need(accepted.dim() == 1 && accepted.size(0) == requests);
        }
        const pkv_stream_t s = c.stream();
        const int32_t *const ip = static_cast<const int32_t *>(ids.data_ptr()), *const sp = static_cast<const int32_t *>(starts.data_ptr());
        const float *const up = static_cast<const float *>(u.data_ptr());
        int32_t *const tp = static_cast<int32_t *>(tokens.data_ptr()), *const ap = static_cast<int32_t *>(accepted.data_ptr());
        need(without_lock([&] {
                 return pkv_verify_drafts(pp, p_stride, qp, q_stride, kind, static_cast<int32_t>(vocab), static_cast<int32_t>(rows), ip, sp,
                                          static_cast<int32_t>(requests), up, drafts, tp, ap, word, s);
             }) == PKV_OK);
        return Py_BuildValue("NN", THPVariable_Wrap(tokens), THPVariable_Wrap(accepted));
    });
}

#define PKV_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PKV_METHOD(rope_store), PKV_METHOD(kv4_store), PKV_METHOD(kv4_load), PKV_METHOD(kv4_attention),
                         PKV_METHOD(verify_drafts), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
