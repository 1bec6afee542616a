// The short way from torch tensors to the attention entry points.
//
// These calls are a few microseconds of GPU work at decode sizes, and the
// checks, allocations and marshalling cost 10 us a call in Python (an append
// of 8 tokens 16 us a call there and 5 us here, 3.5 us of it the kernel).  Each
// function here takes the arguments of the binding's function of the same
// name (without `stream`), recognises the plain valid call -- tensors of the
// right type and layout on the current device -- and makes it on the current
// stream.  It returns None for anything else, with nothing done: the Python
// function then goes through the checks that say what is wrong, or handles
// the case.  An int is the entry point's bl_status.  No arithmetic, no device
// code.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cmath>
#include <cstring>

#include "bitlinear_attn.h"

namespace {

// Addresses of the library's entry points (bind()).
struct Entry {
    decltype(&bl_rope_append) rope_append;
    decltype(&bl_attn_decode_workspace_bytes) decode_bytes;
    decltype(&bl_attn_decode) attn_decode;
    decltype(&bl_kv_extend) kv_extend;
    decltype(&bl_kv_free) kv_free;
    decltype(&bl_kv_fork_workspace_bytes) fork_bytes;
    decltype(&bl_kv_fork) kv_fork;
    decltype(&bl_kv_compact_workspace_bytes) compact_bytes;
    decltype(&bl_kv_compact) kv_compact;
    decltype(&bl_attn_forward) attn_forward;
    decltype(&bl_attn_backward_workspace_bytes) backward_bytes;
    decltype(&bl_attn_backward) attn_backward;
} g;
bool g_bound = false;

using at::Tensor;
using c10::ScalarType;

// Allocations and launches may wait for the GPU, and what the GPU waits for may
// be a host function that needs the interpreter.
struct NoGil {
    PyThreadState *state = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(state); }
};

template <typename F, typename... A>
bl_status launch(F fn, A... args) {
    NoGil nogil;
    return fn(args...);
}

// One call's arguments: everything that is not plain and valid sets bad.
struct Args {
    PyObject *const *a;
    int dev = -1;  // the current device, looked up for the first CUDA tensor
    bool bad = false;

    explicit Args(PyObject *const *args) : a(args) {}
    bool none(int i) const { return a[i] == Py_None; }

    const Tensor *tensor(int i) {
        if (!THPVariable_CheckExact(a[i])) {
            bad = true;
            return nullptr;
        }
        const Tensor &t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda()) {
            bad = true;
            return &t;
        }
        if (dev < 0) dev = c10::cuda::current_device();
        if (t.get_device() != dev) bad = true;
        return &t;
    }
    // A contiguous buffer of the type and at least (exactly, if `exact`) n elements; null for None.
    void *buffer(int i, ScalarType type, int64_t n, bool exact = false) {
        if (none(i)) return nullptr;
        const Tensor *t = tensor(i);
        if (bad || t->scalar_type() != type || !t->is_contiguous() || (exact ? t->numel() != n : t->numel() < n)) {
            bad = true;
            return nullptr;
        }
        return t->data_ptr();
    }
    int32_t *ints(int i, int64_t n, bool exact = true) {
        return static_cast<int32_t *>(buffer(i, ScalarType::Int, n, exact));
    }
    // Rows of contiguous heads [T, H, D], float32 or bfloat16.
    const Tensor *rows(int i, int64_t *stride) {
        const Tensor *t = tensor(i);
        if (bad) return nullptr;
        if (t->dim() != 3 || (t->scalar_type() != ScalarType::Float && t->scalar_type() != ScalarType::BFloat16)) {
            bad = true;
            return nullptr;
        }
        const auto s = t->sizes();
        const auto st = t->strides();
        *stride = s[0] == 1 ? s[1] * s[2] : st[0];
        if (st[2] != 1 || (st[1] != s[2] && s[1] != 1) || *stride < s[1] * s[2]) bad = true;
        return t;
    }
    int64_t integer(int i) {
        if (!PyLong_CheckExact(a[i])) {
            bad = true;
            return 0;
        }
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            bad = true;
        }
        return v;
    }
    float real(int i, double otherwise) {
        if (none(i)) return (float)otherwise;
        if (!PyFloat_CheckExact(a[i])) {
            bad = true;
            return 0.f;
        }
        return (float)PyFloat_AS_DOUBLE(a[i]);
    }
    bool flag(int i) {
        if (a[i] != Py_True && a[i] != Py_False) bad = true;
        return a[i] == Py_True;
    }
    bl_stream_t stream() const {
        return reinterpret_cast<bl_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    }
};

bl_dtype code(ScalarType t) { return t == ScalarType::BFloat16 ? BL_BF16 : BL_F32; }

Tensor make(const Tensor &like, at::IntArrayRef shape, ScalarType type) {
    NoGil nogil;
    return at::empty(shape, like.options().dtype(type));
}

// The tensor at argument i, or a new one for None.
struct Out {
    Tensor made;
    PyObject *given = nullptr;
    void *ptr = nullptr;
    void take(Args &c, int i, const Tensor &like, at::IntArrayRef shape, ScalarType type) {
        int64_t n = 1;
        for (int64_t s : shape) n *= s;
        if (c.none(i)) {
            if (c.bad) return;
            made = make(like, shape, type);
            ptr = made.data_ptr();
        } else {
            ptr = c.buffer(i, type, n);
            given = c.a[i];
        }
    }
    PyObject *object() const {  // a new reference
        if (given != nullptr) return Py_NewRef(given);
        if (made.defined()) return THPVariable_Wrap(made);
        Py_RETURN_NONE;
    }
};

PyObject *answer(bl_status rc) { return PyLong_FromLong((long)rc); }

// k_pages, v_pages, tables, lengths at arguments i .. i + 3.
struct Cache {
    bl_kv_cache c;
    int64_t heads = 0, D = 0;
    bool read(Args &x, int i) {
        const Tensor *k = x.tensor(i), *v = x.tensor(i + 1), *t = x.tensor(i + 2);
        if (x.bad) return false;
        const ScalarType type = k->scalar_type();
        if ((type != ScalarType::Float && type != ScalarType::BFloat16) || v->scalar_type() != type || k->dim() != 4 ||
            v->sizes() != k->sizes() || !k->is_contiguous() || !v->is_contiguous() || t->dim() != 2 ||
            t->scalar_type() != ScalarType::Int || !t->is_contiguous()) {
            x.bad = true;
            return false;
        }
        c.k_pages = k->data_ptr();
        c.v_pages = v->data_ptr();
        c.tables = static_cast<int32_t *>(t->data_ptr());
        c.lengths = x.ints(i + 3, t->size(0));
        if (x.bad || c.lengths == nullptr) {
            x.bad = true;
            return false;
        }
        c.num_pages = k->size(0);
        heads = k->size(1);
        c.page_size = k->size(2);
        D = k->size(3);
        c.max_seqs = t->size(0);
        c.max_pages = t->size(1);
        c.dtype = code(type);
        return true;
    }
};

#define FAST(name, count)                                                                   \
    PyObject *name(PyObject *, PyObject *const *args, Py_ssize_t nargs) {                    \
        HANDLE_TH_ERRORS                                                                     \
        if (!g_bound || nargs != (count)) Py_RETURN_NONE;                                     \
        Args x(args);
#define FAST_END           \
        END_HANDLE_TH_ERRORS \
    }

// q, k, v, rope, cu_seqlens, lengths, seq_ids, k_pages, v_pages, tables, out_dtype, q_out, k_out, v_out, keep_kv, inverse
FAST(rope_append, 16)
    const int first = x.none(0) ? 1 : 0;
    if (x.none(first)) Py_RETURN_NONE;
    int64_t qs = 0, ks = 0, vs = 0;
    const Tensor *q = nullptr, *k = nullptr, *v = nullptr;
    if (!x.none(0)) q = x.rows(0, &qs);
    if (x.none(1) != x.none(2)) Py_RETURN_NONE;
    if (!x.none(1)) {
        k = x.rows(1, &ks);
        if (!x.bad) v = x.rows(2, &vs);
    }
    if (x.bad) Py_RETURN_NONE;
    const Tensor &f = q ? *q : *k;
    const int64_t T = f.size(0), D = f.size(2), Hq = f.size(1), Hkv = k ? k->size(1) : Hq;
    const ScalarType type = f.scalar_type();
    if (k && (k->size(0) != T || v->size(0) != T || k->size(2) != D || v->size(2) != D || v->size(1) != Hkv ||
              k->scalar_type() != type || v->scalar_type() != type))
        Py_RETURN_NONE;
    ScalarType out = type;
    if (!x.none(10)) {
        if (!THPDtype_Check(args[10])) Py_RETURN_NONE;
        out = reinterpret_cast<THPDtype *>(args[10])->scalar_type;
        if (out != ScalarType::Float && out != ScalarType::BFloat16) Py_RETURN_NONE;
    }
    int64_t B = T, rope_len = 0, max_seqs = 0;
    int32_t *cu = nullptr;
    if (!x.none(4)) {
        cu = x.ints(4, 2, false);
        if (x.bad) Py_RETURN_NONE;
        B = THPVariable_Unpack(args[4]).numel() - 1;
    }
    int32_t *ids = x.ints(6, B);
    float *rope = nullptr;
    if (!x.none(3)) {
        rope = static_cast<float *>(x.buffer(3, ScalarType::Float, 0));
        if (x.bad) Py_RETURN_NONE;
        const Tensor &r = THPVariable_Unpack(args[3]);
        if (r.dim() != 2 || r.size(1) != D) Py_RETURN_NONE;
        rope_len = r.size(0);
    }
    const bool keep = x.none(14) ? x.none(7) : x.flag(14);
    const bool inverse = x.flag(15);
    Cache cache;
    bool paged = false;
    int32_t *lengths = nullptr;
    if (!x.none(7)) {
        // (the cache's arguments stand at 7, 8, 9 and 5)
        PyObject *const four[4] = {args[7], args[8], args[9], args[5]};
        Args y(four);
        if (!k || x.bad || !cache.read(y, 0) || cache.heads != Hkv || cache.D != D) Py_RETURN_NONE;
        paged = true;
        max_seqs = cache.c.max_seqs;
    } else {
        if (!x.none(8)) Py_RETURN_NONE;
        if (!x.none(5)) {
            lengths = x.ints(5, 1, false);
            if (x.bad) Py_RETURN_NONE;
            max_seqs = THPVariable_Unpack(args[5]).numel();
        }
    }
    if (x.bad || ((paged || lengths) && !ids && B > max_seqs)) Py_RETURN_NONE;
    if ((!q && !x.none(11)) || (!k && (!x.none(12) || !x.none(13)))) Py_RETURN_NONE;
    Out qo, ko, vo;
    // (outputs that are given are looked at before any is made)
    for (int i = 11; i < 14; ++i)
        if (!x.none(i)) x.buffer(i, out, T * (i == 11 ? Hq : Hkv) * D);
    if (x.bad) Py_RETURN_NONE;
    if (q) qo.take(x, 11, *q, {T, Hq, D}, out);
    if (k && (keep || !x.none(12))) ko.take(x, 12, *k, {T, Hkv, D}, out);
    if (k && (keep || !x.none(13))) vo.take(x, 13, *k, {T, Hkv, D}, out);
    const bl_status rc = launch(g.rope_append, q ? q->data_ptr() : nullptr, k ? k->data_ptr() : nullptr, k ? v->data_ptr() : nullptr,
                                       code(type), qs, ks, vs, T, Hq, Hkv, D, rope, rope_len, inverse, cu, B, ids, lengths,
                                       max_seqs, paged ? &cache.c : nullptr, qo.ptr, ko.ptr, vo.ptr, code(out), x.stream());
    if (rc) return answer(rc);
    return Py_BuildValue("(NNN)", qo.object(), ko.object(), vo.object());
FAST_END

// q, k_pages, v_pages, tables, lengths, seq_ids, window, sinks, scale, out, lse, return_lse, workspace
FAST(attn_decode, 13)
    int64_t qs;
    const Tensor *q = x.rows(0, &qs);
    Cache cache;
    if (x.bad || !cache.read(x, 1) || cache.D != q->size(2)) Py_RETURN_NONE;
    const int64_t B = q->size(0), Hq = q->size(1), D = q->size(2), Hkv = cache.heads;
    int32_t *ids = x.ints(5, B);
    if (!ids && B > cache.c.max_seqs) Py_RETURN_NONE;
    const int64_t window = x.integer(6), sinks = x.integer(7);
    const float scale = x.real(8, 1.0 / std::sqrt((double)D));
    const bool want_lse = x.flag(11);
    const ScalarType type = q->scalar_type();
    if (!x.none(9)) x.buffer(9, type, B * Hq * D);
    if (!x.none(10)) x.buffer(10, ScalarType::Float, B * Hq);
    uint8_t *ws = static_cast<uint8_t *>(x.buffer(12, ScalarType::Byte, 1));
    if (x.bad) Py_RETURN_NONE;
    const size_t need = g.decode_bytes(B, Hq, Hkv, D);
    if (need == 0) Py_RETURN_NONE;
    Out out, lse, work;
    out.take(x, 9, *q, {B, Hq, D}, type);
    if (want_lse || !x.none(10)) lse.take(x, 10, *q, {B, Hq}, ScalarType::Float);
    size_t bytes = need;
    if (ws == nullptr) {
        work.made = make(*q, {(int64_t)need}, ScalarType::Byte);
        ws = static_cast<uint8_t *>(work.made.data_ptr());
    } else {
        bytes = (size_t)THPVariable_Unpack(args[12]).numel();
    }
    const bl_status rc = launch(g.attn_decode, q->data_ptr(), code(type), qs, B, Hq, Hkv, D, &cache.c, ids, window, sinks, scale, ws,
                                       bytes, out.ptr, static_cast<float *>(lse.ptr), x.stream());
    if (rc) return answer(rc);
    if (!want_lse) return out.object();
    return Py_BuildValue("(NN)", out.object(), lse.object());
FAST_END

// The tables, lengths (may be None) and refs at arguments i, j, k.
struct Tables {
    int32_t *tables = nullptr, *lengths = nullptr, *refs = nullptr;
    int64_t seqs = 0, cols = 0, pages = 0;
    const Tensor *like = nullptr;
    bool read(Args &x, int i, int j, int k) {
        like = x.tensor(i);
        if (x.bad || like->dim() != 2) return false;
        seqs = like->size(0);
        cols = like->size(1);
        tables = x.ints(i, seqs * cols);
        if (j >= 0) lengths = x.ints(j, seqs);
        refs = x.ints(k, 0, false);
        if (x.bad || refs == nullptr || (j >= 0 && lengths == nullptr)) return false;
        const Tensor &r = THPVariable_Unpack(x.a[k]);
        if (r.dim() != 1) return false;
        pages = r.numel();
        return true;
    }
};

// tables, lengths, refs, seq_ids, counts, page_size, status, active
FAST(kv_extend, 8)
    Tables t;
    if (!t.read(x, 0, 1, 2) || x.none(3)) Py_RETURN_NONE;
    int32_t *ids = x.ints(3, 1, false);
    if (x.bad) Py_RETURN_NONE;
    const int64_t n = THPVariable_Unpack(args[3]).numel();
    int32_t *counts = x.ints(4, n);
    const int64_t ps = x.integer(5);
    if (!x.none(6)) x.ints(6, 1, false);
    int32_t *active = x.ints(7, n);
    if (x.bad || counts == nullptr) Py_RETURN_NONE;
    Out status;
    status.take(x, 6, *t.like, {1}, ScalarType::Int);
    const bl_status rc = launch(g.kv_extend, t.tables, t.lengths, t.refs, t.pages, ps, t.seqs, t.cols, ids, counts, n,
                                     static_cast<int32_t *>(status.ptr), active, x.stream());
    return rc ? answer(rc) : status.object();
FAST_END

// tables, lengths, refs, seq_ids, page_size
FAST(kv_free, 5)
    Tables t;
    if (!t.read(x, 0, 1, 2) || x.none(3)) Py_RETURN_NONE;
    int32_t *ids = x.ints(3, 1, false);
    const int64_t ps = x.integer(4);
    if (x.bad) Py_RETURN_NONE;
    return answer(launch(g.kv_free, t.tables, t.lengths, t.refs, t.pages, ps, t.seqs, t.cols, ids,
                            THPVariable_Unpack(args[3]).numel(), x.stream()));
FAST_END

// A pool [..., num_pages, Hkv, page_size, D].
struct Pool {
    void *ptr = nullptr;
    int64_t planes = 1, page_bytes = 0, page_size = 0;
    bool read(Args &x, int i, int64_t pages) {
        const Tensor *p = x.tensor(i);
        if (x.bad) return false;
        const int d = (int)p->dim();
        if (d < 4 || !p->is_contiguous() || p->size(d - 4) != pages ||
            (p->scalar_type() != ScalarType::Float && p->scalar_type() != ScalarType::BFloat16))
            return false;
        for (int j = 0; j < d - 4; ++j) planes *= p->size(j);
        page_bytes = p->size(d - 3) * p->size(d - 2) * p->size(d - 1) * p->element_size();
        page_size = p->size(d - 2);
        ptr = p->data_ptr();
        return true;
    }
};

// The workspace at argument i (at least 1 byte of uint8), or a new one of `need` bytes.
struct Work {
    Tensor made;
    void *ptr = nullptr;
    size_t bytes = 0;
    void take(Args &x, int i, const Tensor &like, size_t need) {
        if (x.none(i)) {
            if (x.bad) return;
            made = make(like, {(int64_t)(need ? need : 16)}, ScalarType::Byte);
            ptr = made.data_ptr();
            bytes = (size_t)made.numel();
        } else {
            ptr = x.buffer(i, ScalarType::Byte, 1);
            if (!x.bad) bytes = (size_t)THPVariable_Unpack(x.a[i]).numel();
        }
    }
};

// pool, tables, lengths, refs, src, dst, status, workspace
FAST(kv_fork, 8)
    Tables t;
    Pool pool;
    if (!t.read(x, 1, 2, 3) || !pool.read(x, 0, t.pages) || x.none(4)) Py_RETURN_NONE;
    int32_t *src = x.ints(4, 1, false);
    if (x.bad) Py_RETURN_NONE;
    const int64_t n = THPVariable_Unpack(args[4]).numel();
    int32_t *dst = x.ints(5, n);
    if (!x.none(6)) x.ints(6, 1, false);
    if (!x.none(7)) x.buffer(7, ScalarType::Byte, 1);
    if (x.bad || dst == nullptr) Py_RETURN_NONE;
    Out status;
    Work work;
    status.take(x, 6, *t.like, {1}, ScalarType::Int);
    work.take(x, 7, *t.like, g.fork_bytes(n));
    const bl_status rc = launch(g.kv_fork, pool.ptr, pool.planes, pool.page_bytes, t.tables, t.lengths, t.refs, t.pages,
                                   pool.page_size, t.seqs, t.cols, src, dst, n, work.ptr, work.bytes,
                                   static_cast<int32_t *>(status.ptr), x.stream());
    return rc ? answer(rc) : status.object();
FAST_END

// pool, tables, refs, n_live, workspace
FAST(kv_compact, 5)
    Tables t;
    Pool pool;
    if (!t.read(x, 1, -1, 2) || !pool.read(x, 0, t.pages)) Py_RETURN_NONE;
    if (!x.none(3)) x.ints(3, 1, false);
    if (!x.none(4)) x.buffer(4, ScalarType::Byte, 1);
    if (x.bad) Py_RETURN_NONE;
    Out live;
    Work work;
    live.take(x, 3, *t.like, {1}, ScalarType::Int);
    work.take(x, 4, *t.like, g.compact_bytes(t.pages));
    const bl_status rc = launch(g.kv_compact, pool.ptr, pool.planes, pool.page_bytes, t.tables, t.refs, t.pages, t.seqs, t.cols,
                                      work.ptr, work.bytes, static_cast<int32_t *>(live.ptr), x.stream());
    return rc ? answer(rc) : live.object();
FAST_END

// q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale at arguments i ..
struct Ragged {
    const Tensor *q, *k, *v;
    int64_t qs, ks, vs, Tq, Tk, Hq, Hkv, D, B, max_q, max_k, window, sinks;
    int32_t *cu_q, *cu_k;
    float scale;
    bool read(Args &x, int q_at, int cu_at) {
        q = x.rows(q_at, &qs);
        if (x.bad) return false;
        k = x.rows(q_at + 1, &ks);
        if (x.bad) return false;
        v = x.rows(q_at + 2, &vs);
        if (x.bad || x.none(cu_at) || x.none(cu_at + 1)) return false;
        Tq = q->size(0), Hq = q->size(1), D = q->size(2);
        Tk = k->size(0), Hkv = k->size(1);
        for (const Tensor *t : {q, k, v})
            if (t->scalar_type() != ScalarType::BFloat16) return false;
        if (k->size(2) != D || v->size(2) != D || v->size(0) != Tk || v->size(1) != Hkv) return false;
        cu_q = x.ints(cu_at, 2, false);
        if (x.bad) return false;
        B = THPVariable_Unpack(x.a[cu_at]).numel() - 1;
        cu_k = x.ints(cu_at + 1, B + 1);
        max_q = x.integer(cu_at + 2);
        max_k = x.integer(cu_at + 3);
        window = x.integer(cu_at + 4);
        sinks = x.integer(cu_at + 5);
        scale = x.real(cu_at + 6, 1.0 / std::sqrt((double)D));
        return !x.bad;
    }
};

// q, k, v, cu_q, cu_k, max_q, max_k, window, sinks, scale, o, lse
FAST(attn_forward, 12)
    Ragged r;
    if (!r.read(x, 0, 3)) Py_RETURN_NONE;
    if (!x.none(10)) x.buffer(10, ScalarType::BFloat16, r.Tq * r.Hq * r.D);
    if (!x.none(11)) x.buffer(11, ScalarType::Float, r.Hq * r.Tq);
    if (x.bad) Py_RETURN_NONE;
    Out o, lse;
    o.take(x, 10, *r.q, {r.Tq, r.Hq, r.D}, ScalarType::BFloat16);
    lse.take(x, 11, *r.q, {r.Hq, r.Tq}, ScalarType::Float);
    const bl_status rc = launch(g.attn_forward, r.q->data_ptr(), r.k->data_ptr(), r.v->data_ptr(), r.qs, r.ks, r.vs, r.Tq, r.Tk, r.Hq,
                                        r.Hkv, r.D, r.cu_q, r.cu_k, r.B, r.max_q, r.max_k, r.window, r.sinks, r.scale, o.ptr,
                                        static_cast<float *>(lse.ptr), x.stream());
    if (rc) return answer(rc);
    return Py_BuildValue("(NN)", o.object(), lse.object());
FAST_END

// do, q, k, v, o, lse, cu_q, cu_k, max_q, max_k, window, sinks, scale, dq, dk, dv, workspace
FAST(attn_backward, 17)
    Ragged r;
    int64_t dos;
    const Tensor *grad = x.rows(0, &dos);
    if (x.bad || !r.read(x, 1, 6)) Py_RETURN_NONE;
    if (grad->scalar_type() != ScalarType::BFloat16 || grad->size(0) != r.Tq || grad->size(1) != r.Hq || grad->size(2) != r.D)
        Py_RETURN_NONE;
    void *o = x.buffer(4, ScalarType::BFloat16, r.Tq * r.Hq * r.D);
    void *lse = x.buffer(5, ScalarType::Float, r.Hq * r.Tq);
    if (!x.none(13)) x.buffer(13, ScalarType::BFloat16, r.Tq * r.Hq * r.D);
    for (int i = 14; i < 16; ++i)
        if (!x.none(i)) x.buffer(i, ScalarType::BFloat16, r.Tk * r.Hkv * r.D);
    if (!x.none(16)) x.buffer(16, ScalarType::Byte, 1);
    if (x.bad || o == nullptr || lse == nullptr) Py_RETURN_NONE;
    Out dq, dk, dv;
    Work work;
    dq.take(x, 13, *r.q, {r.Tq, r.Hq, r.D}, ScalarType::BFloat16);
    dk.take(x, 14, *r.k, {r.Tk, r.Hkv, r.D}, ScalarType::BFloat16);
    dv.take(x, 15, *r.k, {r.Tk, r.Hkv, r.D}, ScalarType::BFloat16);
    work.take(x, 16, *r.q, g.backward_bytes(r.Tq, r.Tk, r.Hq, r.Hkv, r.D, r.B, r.max_q, r.max_k, r.window, r.sinks));
    const bl_status rc = launch(g.attn_backward, grad->data_ptr(), r.q->data_ptr(), r.k->data_ptr(), r.v->data_ptr(), o,
                                         static_cast<float *>(lse), dos, r.qs, r.ks, r.vs, r.Tq, r.Tk, r.Hq, r.Hkv, r.D,
                                         r.cu_q, r.cu_k, r.B, r.max_q, r.max_k, r.window, r.sinks, r.scale, work.ptr,
                                         work.bytes, dq.ptr, dk.ptr, dv.ptr, x.stream());
    if (rc) return answer(rc);
    return Py_BuildValue("(NNN)", dq.object(), dk.object(), dv.object());
FAST_END

// bind(addresses): the library's entry points, in the order of Entry.
PyObject *bind(PyObject *, PyObject *list) {
    constexpr Py_ssize_t n = sizeof(Entry) / sizeof(void *);
    if (!PyTuple_Check(list) || PyTuple_GET_SIZE(list) != n) {
        PyErr_SetString(PyExc_ValueError, "bind: a tuple of the library's entry points");
        return nullptr;
    }
    void *at[n];
    for (Py_ssize_t i = 0; i < n; ++i) {
        at[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(list, i));
        if (at[i] == nullptr) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null entry point");
            return nullptr;
        }
    }
    std::memcpy(&g, at, sizeof(g));
    g_bound = true;
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(rope_append),  METHOD(attn_decode),  METHOD(kv_extend),
                         METHOD(kv_free),      METHOD(kv_fork),      METHOD(kv_compact),
                         METHOD(attn_forward), METHOD(attn_backward), {"bind", bind, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was built with (its classes' layouts are compiled in).
PyMODINIT_FUNC PyInit_attn_binding(void) {
    PyObject *m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", BL_TORCH_VERSION) != 0) Py_CLEAR(m);
    return m;
}
