// The quick way from Python to the rotary calls and those of the paged 4-bit cache.  A serving loop makes
// them a few times per layer and step, on kernels of a few microseconds, where checking some ten tensors
// and handing some thirty numbers over one by one takes Python longer (append of 64 tokens 11.9 us, of which 4.3 are
// the C call; 0.4 us per tensor).  Each function here takes the arguments of the Python function of its name, in order,
// and makes the C call, whose status it returns, if they fit it.  If anything does not, or is unusual
// (another device than the current one, a tensor of a derived class, a workspace to be allocated), it returns
// None and has done nothing: the Python function then goes its own way, which refuses or does it.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "csa2.h"

namespace {

PyObject *current_stream, *current_device;       // functions: (device) -> raw stream, () -> device
decltype(&csa2_rope_table) c_rope_table;
decltype(&csa2_rope) c_rope;
decltype(&csa2_quantize_kv_fp4_paged) c_quantize;
decltype(&csa2_dequantize_kv_fp4_paged) c_dequantize;
decltype(&csa2_paged_attn_fp4) c_attn;

// Reads arguments; `ok` falls, for good, at the first that does not fit.
struct Args {
    PyObject *const *at;
    bool ok;
    int dev = 0;

    Args(PyObject *const *a, Py_ssize_t n, Py_ssize_t want) : at(a), ok(n == want) {}

    const at::Tensor *tensor(PyObject *o) {
        if (!ok || !(ok = THPVariable_CheckExact(o))) return nullptr;
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.layout() == at::kStrided && !t.is_conj() && !t.is_neg() && (t.is_cuda() || t.is_cpu());     // of the CPU: device -1, never the current one
        return ok ? &t : nullptr;
    }
    const at::Tensor *tensor(PyObject *o, int dims) {
        const at::Tensor *t = tensor(o);
        if (t && !(ok = t->dim() == dims && t->get_device() == dev)) return nullptr;
        return t;
    }
    // A tensor whose device the others must be on, the current one.
    const at::Tensor *first(PyObject *o, int dims) {
        const at::Tensor *t = tensor(o);
        if (!t || !(ok = t->dim() == dims)) return nullptr;
        dev = t->get_device();
        PyObject *d = PyObject_CallNoArgs(current_device);
        ok = d && PyLong_Check(d) && PyLong_AsLong(d) == dev;
        Py_XDECREF(d);
        return ok ? t : nullptr;
    }
    void *dense(const at::Tensor *t, at::ScalarType type, std::initializer_list<int64_t> sizes) {
        if (!ok || !(ok = t && t->scalar_type() == type && t->sizes() == at::IntArrayRef(sizes) && t->is_contiguous())) return nullptr;
        return t->mutable_data_ptr();
    }
    void *dense(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> sizes) {
        return dense(tensor(o, (int)sizes.size()), type, sizes);
    }
    void *dense_or_none(PyObject *o, at::ScalarType type, std::initializer_list<int64_t> sizes) {
        return o == Py_None ? nullptr : dense(o, type, sizes);
    }
    // Rows [T, H, D] with contiguous channels; the stride of an extent of one says nothing.
    void *rows(const at::Tensor *t, at::ScalarType type, int64_t T, int64_t H, int64_t D, int64_t &token, int64_t &head) {
        if (!ok || !(ok = t && t->scalar_type() == type && t->size(0) == T && t->size(1) == H && t->size(2) == D && t->stride(2) == 1)) return nullptr;
        token = T > 1 ? t->stride(0) : H * D;
        head = H > 1 ? t->stride(1) : D;
        return t->mutable_data_ptr();
    }
    csa2_dtype row_type(const at::Tensor *t) {
        if (!ok) return CSA2_BF16;
        const at::ScalarType s = t->scalar_type();
        ok = s == at::kBFloat16 || s == at::kShort || s == at::kHalf;
        return s == at::kHalf ? CSA2_FP16 : CSA2_BF16;
    }
    const float *table(PyObject *o, int64_t &n_pos, int &rope_dim) {
        const at::Tensor *t = tensor(o, 3);
        if (!t || !(ok = t->size(2) == 2 && t->scalar_type() == at::kFloat && t->is_contiguous() && t->size(1) <= 1 << 20)) return nullptr;
        n_pos = t->size(0), rope_dim = 2 * (int)t->size(1);
        return (const float *)t->mutable_data_ptr();
    }
    uint32_t *flag(PyObject *o) {
        if (!ok || o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o);
        if (!t || !(ok = (t->scalar_type() == at::kInt || t->scalar_type() == at::kUInt32) && t->numel() >= 1 && t->get_device() == dev)) return nullptr;
        return (uint32_t *)t->mutable_data_ptr();
    }
    int64_t integer(PyObject *o, int64_t least, int64_t most) {
        if (!ok || !(ok = PyLong_CheckExact(o))) return 0;
        int over = 0;
        const int64_t v = PyLong_AsLongLongAndOverflow(o, &over);
        ok = !over && v >= least && v <= most;
        return v;
    }
    int int32(PyObject *o) { return (int)integer(o, INT32_MIN, INT32_MAX); }
    float real(PyObject *o) {
        if (!ok || !(ok = PyFloat_CheckExact(o))) return 0.0f;
        return (float)PyFloat_AS_DOUBLE(o);
    }
    // The last argument: None (the current stream), a stream or its handle.
    csa2_stream_t stream(PyObject *o) {
        if (!ok) return nullptr;
        PyObject *s;
        if (o == Py_None) {
            PyObject *d = PyLong_FromLong(dev);
            s = d ? PyObject_CallOneArg(current_stream, d) : nullptr;
            Py_XDECREF(d);
        } else {
            s = PyLong_CheckExact(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        }
        void *p = nullptr;
        ok = s && PyLong_Check(s);
        if (ok) p = PyLong_AsVoidPtr(s), ok = !PyErr_Occurred();
        Py_XDECREF(s);
        return (csa2_stream_t)p;
    }
};

// Code and scale planes [n, H, S, D/2] and [n, H, S, D/16] of a cache in 4 bits.
struct Planes {
    uint8_t *kc = nullptr, *vc = nullptr, *ks = nullptr, *vs = nullptr;
    int64_t n = 0;
    int H = 0, S = 0, D = 0;
    Planes(Args &a, PyObject *const *o) {
        const at::Tensor *k = a.tensor(o[0], 4), *s = a.tensor(o[2], 4);
        if (!k || !s) return;
        const int64_t h = k->size(1), t = k->size(2), half = k->size(3);
        n = k->size(0);
        a.ok = h <= 1 << 20 && t <= 1 << 20 && half <= 1 << 20;
        const at::ScalarType e = s->scalar_type();
        a.ok = a.ok && (e == at::kByte || e == at::kFloat8_e4m3fn);
        kc = (uint8_t *)a.dense(k, at::kByte, {n, h, t, half});
        vc = (uint8_t *)a.dense(o[1], at::kByte, {n, h, t, half});
        ks = (uint8_t *)a.dense(s, e, {n, h, t, half / 8});
        vs = (uint8_t *)a.dense(o[3], e, {n, h, t, half / 8});
        H = (int)h, S = (int)t, D = 2 * (int)half;
    }
};

template <typename Call>
PyObject *answer(const Args &a, Call call) {
    if (!a.ok) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    csa2_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong((long)st);
}

// C++ exceptions (of a tensor without memory, say) end here.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *o, Py_ssize_t n) {
    try {
        return F(o, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyObject *rope_table(PyObject *const *o, Py_ssize_t n) {
    Args a(o, n, 5);
    const at::Tensor *out = a.ok ? a.first(o[1], 3) : nullptr;
    if (!a.ok) return answer(a, [] { return CSA2_OK; });
    const int64_t rows = out->size(0), half = out->size(1);
    a.ok = half <= 1 << 20;
    float *table = (float *)a.dense(out, at::kFloat, {rows, half, 2});
    const double *freq = (const double *)a.dense(o[0], at::kDouble, {half});
    const int64_t start = a.integer(o[2], INT64_MIN, INT64_MAX);
    const float amplitude = a.real(o[3]);
    const csa2_stream_t s = a.stream(o[4]);
    return answer(a, [&] { return c_rope_table(freq, (int)half, start, rows, amplitude, table, s); });
}

PyObject *rope(PyObject *const *o, Py_ssize_t n) {
    enum { Q, POS, TABLE, K, Q_OUT, K_OUT, FIRST, LAYOUT, FLAG, STREAM, N };
    Args a(o, n, N);
    const at::Tensor *q = a.ok ? a.first(o[Q], 3) : nullptr;
    if (!a.ok) return answer(a, [] { return CSA2_OK; });
    const int64_t T = q->size(0), Hq = q->size(1), D = q->size(2);
    a.ok = Hq <= 1 << 20 && D <= 1 << 20;
    const csa2_dtype dt = a.row_type(q);
    const at::ScalarType type = q->scalar_type();
    int64_t s[8] = {}, n_pos = 0, Hk = 0;
    int rope_dim = 0;
    const void *qp = a.rows(q, type, T, Hq, D, s[0], s[1]), *kp = nullptr;
    void *qo = const_cast<void *>(qp), *ko = nullptr;
    s[2] = s[0], s[3] = s[1];
    if (o[Q_OUT] != Py_None) qo = a.rows(a.tensor(o[Q_OUT], 3), type, T, Hq, D, s[2], s[3]);
    if (o[K] != Py_None) {
        const at::Tensor *k = a.tensor(o[K], 3);
        if (k) Hk = k->size(1), a.ok = Hk <= 1 << 20;
        kp = a.rows(k, type, T, Hk, D, s[4], s[5]);
        ko = const_cast<void *>(kp);
        s[6] = s[4], s[7] = s[5];
        if (o[K_OUT] != Py_None) ko = a.rows(a.tensor(o[K_OUT], 3), type, T, Hk, D, s[6], s[7]);
    } else if (o[K_OUT] != Py_None) {
        a.ok = false;
    }
    const float *table = a.table(o[TABLE], n_pos, rope_dim);
    const int32_t *pos = (const int32_t *)a.dense(o[POS], at::kInt, {T});
    const int first = a.int32(o[FIRST]), layout = a.int32(o[LAYOUT]);
    uint32_t *flag = a.flag(o[FLAG]);
    const csa2_stream_t st = a.stream(o[STREAM]);
    return answer(a, [&] {
        return c_rope(qp, qo, (int)Hq, s[0], s[1], s[2], s[3], kp, ko, (int)Hk, s[4], s[5], s[6], s[7], dt, T, (int)D, pos, table, n_pos,
                      rope_dim, first, (csa2_rope_layout)layout, flag, st);
    });
}

PyObject *quantize(PyObject *const *o, Py_ssize_t n) {
    enum { K, V, SLOTS, PLANES, POS = PLANES + 4, TABLE, FIRST, LAYOUT, K_VALUES, V_VALUES, FLAG, STREAM, N };
    Args a(o, n, N);
    const at::Tensor *k = a.ok ? a.first(o[K], 3) : nullptr, *slots = a.ok ? a.tensor(o[SLOTS], 1) : nullptr;
    if (!a.ok) return answer(a, [] { return CSA2_OK; });
    const Planes p(a, o + PLANES);
    const int64_t T = slots->size(0);
    const csa2_dtype dt = a.row_type(k);
    const at::ScalarType type = k->scalar_type();
    int64_t s[4] = {}, n_pos = 0;
    int rope_dim = 0;
    const void *kp = a.rows(k, type, T, p.H, p.D, s[0], s[1]), *vp = a.rows(a.tensor(o[V], 3), type, T, p.H, p.D, s[2], s[3]);
    if ((o[POS] == Py_None) != (o[TABLE] == Py_None)) a.ok = false;
    const float *table = o[TABLE] == Py_None ? nullptr : a.table(o[TABLE], n_pos, rope_dim);
    const int32_t *pos = (const int32_t *)a.dense_or_none(o[POS], at::kInt, {T});
    const int64_t *at = (const int64_t *)a.dense(slots, at::kLong, {T});
    const int first = a.int32(o[FIRST]), layout = a.int32(o[LAYOUT]);
    void *kv = a.dense_or_none(o[K_VALUES], type, {T, p.H, p.D}), *vv = a.dense_or_none(o[V_VALUES], type, {T, p.H, p.D});
    uint32_t *flag = a.flag(o[FLAG]);
    const csa2_stream_t st = a.stream(o[STREAM]);
    return answer(a, [&] {
        return c_quantize(kp, vp, dt, T, p.H, p.D, s[0], s[1], s[2], s[3], at, p.n, p.S, p.kc, p.vc, p.ks, p.vs, pos, table, n_pos, rope_dim,
                          first, (csa2_rope_layout)layout, kv, vv, flag, st);
    });
}

PyObject *dequantize(PyObject *const *o, Py_ssize_t n) {
    enum { SLOTS, PLANES, K = PLANES + 4, V, FLAG, STREAM, N };
    Args a(o, n, N);
    const at::Tensor *k = a.ok ? a.first(o[K], 3) : nullptr, *slots = a.ok ? a.tensor(o[SLOTS], 1) : nullptr;
    if (!a.ok) return answer(a, [] { return CSA2_OK; });
    const Planes p(a, o + PLANES);
    const int64_t T = slots->size(0);
    const csa2_dtype dt = a.row_type(k);
    int64_t s[4] = {};
    void *kp = a.rows(k, k->scalar_type(), T, p.H, p.D, s[0], s[1]), *vp = a.rows(a.tensor(o[V], 3), k->scalar_type(), T, p.H, p.D, s[2], s[3]);
    const int64_t *at = (const int64_t *)a.dense(slots, at::kLong, {T});
    uint32_t *flag = a.flag(o[FLAG]);
    const csa2_stream_t st = a.stream(o[STREAM]);
    return answer(a, [&] {
        return c_dequantize(at, T, p.n, p.H, p.S, p.D, p.kc, p.vc, p.ks, p.vs, dt, kp, vp, s[0], s[1], s[2], s[3], flag, st);
    });
}

PyObject *attn(PyObject *const *o, Py_ssize_t n) {
    enum { Q, PLANES, TABLE = PLANES + 4, KV_LEN, CU_LEN, OUT, SCALE, MAX_NEW, WINDOW, LSE, FLAG, WORKSPACE, STREAM, N };
    Args a(o, n, N);
    const at::Tensor *q = a.ok ? a.first(o[Q], 3) : nullptr, *bt = a.ok ? a.tensor(o[TABLE], 2) : nullptr;
    if (!a.ok) return answer(a, [] { return CSA2_OK; });
    const Planes p(a, o + PLANES);
    const int64_t T = q->size(0), Hq = q->size(1), B = bt->size(0), M = bt->size(1);
    a.ok = a.ok && p.H >= 1 && Hq <= 1 << 20 && Hq % p.H == 0 && B <= INT32_MAX && M <= INT32_MAX && bt->scalar_type() == at::kInt &&
           (M <= 1 || bt->stride(1) == 1);
    const csa2_dtype dt = a.row_type(q);
    const at::ScalarType type = q->scalar_type();
    int64_t token = 0, head = 0;
    const void *qp = a.rows(q, type, T, Hq, p.D, token, head);
    const int32_t *table = a.ok ? (const int32_t *)bt->mutable_data_ptr() : nullptr;
    const int32_t *kv = (const int32_t *)a.dense(o[KV_LEN], at::kInt, {B}), *cu = (const int32_t *)a.dense(o[CU_LEN], at::kInt, {B + 1});
    void *out = a.dense(o[OUT], type, {T, Hq, p.D});
    const float scale = a.real(o[SCALE]);
    const int max_new = a.int32(o[MAX_NEW]), window = a.int32(o[WINDOW]);
    float *lse = (float *)a.dense_or_none(o[LSE], at::kFloat, {T, Hq});
    uint32_t *flag = a.flag(o[FLAG]);
    const at::Tensor *ws = a.tensor(o[WORKSPACE]);
    void *wp = nullptr;
    if (ws && (a.ok = ws->is_contiguous() && ws->get_device() == a.dev)) wp = ws->mutable_data_ptr();
    const csa2_stream_t st = a.stream(o[STREAM]);
    return answer(a, [&] {
        return c_attn((int)B, T, (int)Hq, p.H, p.D, dt, qp, token, head, p.kc, p.vc, p.ks, p.vs, p.n, p.S, table, (int)M,
                      B > 1 ? bt->stride(0) : M, kv, cu, max_new, window, scale, out, lse, flag, wp, ws->nbytes(), st);
    });
}

// bind(addresses of the five C functions, in the order below, then the two Python functions)
PyObject *bind(PyObject *, PyObject *const *o, Py_ssize_t n) {
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "bind takes 7 arguments");
        return nullptr;
    }
    void *p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(o[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    c_rope_table = (decltype(c_rope_table))p[0];
    c_rope = (decltype(c_rope))p[1];
    c_quantize = (decltype(c_quantize))p[2];
    c_dequantize = (decltype(c_dequantize))p[3];
    c_attn = (decltype(c_attn))p[4];
    Py_XSETREF(current_stream, Py_NewRef(o[5]));
    Py_XSETREF(current_device, Py_NewRef(o[6]));
    Py_RETURN_NONE;
}

#define FN(name, f) {name, (PyCFunction)(void (*)(void))(f), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN("bind", bind),
                         FN("csa2_rope_table", entry<rope_table>),
                         FN("csa2_rope", entry<rope>),
                         FN("csa2_quantize_kv_fp4_paged", entry<quantize>),
                         FN("csa2_dequantize_kv_fp4_paged", entry<dequantize>),
                         FN("csa2_paged_attn_fp4", entry<attn>),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_csa2_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and Python whose objects the functions read; the package uses them with no other.
PyMODINIT_FUNC PyInit__csa2_bind() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", CSA2_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
