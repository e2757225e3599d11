// tensor_args.cpp -- reading tensor arguments for the binding without Python's
// attribute calls.  A launch of a small decode call takes about 3 us of host
// time; checking and reading its dozen tensors in Python took three times that.
// Only the ordinary case is answered here: at() and rows() hand anything else
// to the Python function of the same name, append() and attend() return None
// without having called anything, and the binding goes through its own checks,
// which raise (or cope).
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dsa.h"

namespace {

// A call's tensors, all on one device: each is read once, and `good` stays true
// while every one is as the call wants it.
struct Reader {
    long device;
    bool good = true;
    const at::Tensor *tensor(PyObject *o) {
        if (!THPVariable_Check(o)) {
            good = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.get_device() != device) good = false;
        return &t;
    }
    // a contiguous tensor of one of two types and of `numel` elements (-1: any number)
    void *flat(PyObject *o, at::ScalarType type, long long numel = -1, at::ScalarType other = at::ScalarType::Undefined) {
        const at::Tensor *t = tensor(o);
        if (!good) return nullptr;
        if ((t->scalar_type() != type && t->scalar_type() != other) || !t->is_contiguous() ||
            (numel >= 0 && t->numel() != numel)) {
            good = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void *flat_or_null(PyObject *o, at::ScalarType type, long long numel, at::ScalarType other = at::ScalarType::Undefined) {
        return o == Py_None ? nullptr : flat(o, type, numel, other);
    }
    // int32 [axes][tokens] positions
    int32_t *positions(PyObject *o, long long axes, long long tokens) {
        void *p = flat_or_null(o, at::kInt, axes * tokens);
        if (good && p && THPVariable_Unpack(o).size(-1) != tokens) good = false;
        return static_cast<int32_t *>(p);
    }
    // a contiguous tensor of the sizes of another's first `dims` dimensions
    void *like(PyObject *o, at::ScalarType type, PyObject *other, int dims) {
        void *p = flat(o, type);
        if (good && THPVariable_Unpack(o).sizes() != THPVariable_Unpack(other).sizes().slice(0, dims)) good = false;
        return p;
    }
    // bf16 [tokens][heads][128] rows, only the tokens apart
    void *rows(PyObject *o, long long &tokens, long long &heads, int64_t &stride) {
        const at::Tensor *t = tensor(o);
        if (!good) return nullptr;
        if (t->scalar_type() != at::kBFloat16 || t->dim() != 3 || t->size(2) != 128 || t->stride(2) != 1 ||
            (t->stride(1) != 128 && t->size(1) > 1)) {
            good = false;
            return nullptr;
        }
        tokens = t->size(0);
        heads = t->size(1);
        stride = tokens > 1 ? t->stride(0) : heads * 128;
        return t->data_ptr();
    }
};

// k_pool, v_pool, kc_pool and, with fp8, k_scale, v_scale.  The caller names the
// form, the one that its entry point takes: it does not follow from the tensors.
bool read_cache(Reader &r, bool fp8, PyObject *const *o, dsa_kv_cache &c, dsa_kv_cache_fp8 &c8) {
    const at::ScalarType type = fp8 ? at::kByte : at::kBFloat16;
    const at::ScalarType other = fp8 ? at::kFloat8_e4m3fn : at::ScalarType::Undefined;
    const at::Tensor *k = r.tensor(o[0]), *kc = r.tensor(o[2]);
    if (!r.good || k->dim() != 4 || kc->dim() != 2 || kc->size(0) != k->size(0)) return false;
    const long long n = k->size(0), bs = k->size(1), hkv = k->size(2), d = k->size(3);
    if (n > INT32_MAX || bs > INT32_MAX || hkv > INT32_MAX) return false;
    void *kp = r.flat(o[0], type, -1, other), *vp = r.flat(o[1], type, -1, other);
    if (r.good && THPVariable_Unpack(o[1]).sizes() != k->sizes()) return false;
    void *kcp = r.flat(o[2], at::kChar, -1, at::kByte);
    if (!r.good) return false;
    c = dsa_kv_cache{kp, vp, static_cast<int8_t *>(kcp), (int32_t)n, (int32_t)bs, (int32_t)hkv, (int32_t)d,
                     (int32_t)kc->size(1)};
    if (fp8) {
        const long long tiles = n * (bs / 64) * hkv;
        c8 = dsa_kv_cache_fp8{kp, vp, static_cast<int8_t *>(kcp),
                              static_cast<float *>(r.flat(o[3], at::kFloat, tiles)),
                              static_cast<float *>(r.flat(o[4], at::kFloat, tiles)),
                              (int32_t)n, (int32_t)bs, (int32_t)hkv, (int32_t)d, (int32_t)kc->size(1)};
    }
    return r.good;
}

bool read_seqs(Reader &r, PyObject *table, PyObject *lens, dsa_seqs &s) {
    const at::Tensor *t = r.tensor(table);
    if (!r.good || t->dim() != 2) return false;
    s.block_table = static_cast<int32_t *>(r.flat(table, at::kInt));
    s.max_blocks = (int32_t)t->size(1);
    s.num_seqs = (int32_t)t->size(0);
    s.seq_lens = static_cast<int32_t *>(r.flat(lens, at::kInt, t->size(0)));
    return r.good;
}

bool read_queries(Reader &r, PyObject *cu_q, PyObject *q_pos, dsa_queries &q) {
    q.cu_q = static_cast<int32_t *>(r.flat(cu_q, at::kInt));
    q.q_pos = static_cast<int32_t *>(r.flat(q_pos, at::kInt));
    if (r.good) q.total_q = (int32_t)THPVariable_Unpack(q_pos).numel();
    return r.good;
}

// append(call, device, stream, fp8, k_pool, v_pool, kc_pool, k_scale, v_scale, block_table, seq_lens, cu_new, k_new,
//        v_new, kc_new, pos_new, inv_freq, pair_axis, interleaved, num_axes, scale, cu_q, q_pos, q, pos_q, q_out, dev_err)
// -> status of dsa_kv_append_rope (fp8 False) / dsa_kv_append_fp8 (True) at address `call`, or None
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    int status = -1;
    if (n == 27) try {
        Reader r{PyLong_AsLong(a[1])};
        dsa_kv_cache c;
        dsa_kv_cache_fp8 c8;
        dsa_seqs s;
        dsa_new_tokens f{};
        dsa_rope rope{};
        dsa_queries q{};
        dsa_query_rows w{};
        const bool fp8 = a[3] == Py_True;
        if (!read_cache(r, fp8, a + 4, c, c8) || !read_seqs(r, a[9], a[10], s)) Py_RETURN_NONE;
        const long long axes = PyLong_AsLong(a[19]);
        if (axes < 1 || axes > 4) Py_RETURN_NONE;
        if (a[12] != Py_None) {
            long long total, heads, v_total, v_heads;
            f.k = r.rows(a[12], total, heads, f.k_stride);
            f.v = r.rows(a[13], v_total, v_heads, f.v_stride);
            if (!r.good || total < 1 || total > INT32_MAX || v_total != total || heads != c.num_kv_heads ||
                v_heads != heads)
                Py_RETURN_NONE;
            f.total_new = (int32_t)total;
            f.cu_new = static_cast<int32_t *>(r.flat(a[11], at::kInt, s.num_seqs + 1ll));
            f.kc = static_cast<int8_t *>(r.flat_or_null(a[14], at::kChar, total * 64, at::kByte));
            f.pos = r.positions(a[15], axes, total);
        }
        const bool turns = a[16] != Py_None;
        if (turns) {
            rope.inv_freq = static_cast<float *>(r.flat(a[16], at::kFloat));
            if (!r.good) Py_RETURN_NONE;
            const long long half = THPVariable_Unpack(a[16]).numel();
            if (half < 1 || half > 64 || (axes > 1 && a[17] == Py_None)) Py_RETURN_NONE;
            rope.pair_axis = axes > 1 ? static_cast<int32_t *>(r.flat(a[17], at::kInt, half)) : nullptr;
            rope.rotary_dim = (int32_t)(2 * half);
            rope.layout = PyObject_IsTrue(a[18]) == 1 ? DSA_ROPE_PAIRS : DSA_ROPE_HALVES;
            rope.num_axes = (int32_t)axes;
            rope.scale = (float)PyFloat_AsDouble(a[20]);
        }
        const bool has_q = a[23] != Py_None;
        if (has_q) {
            long long tokens, heads;
            if (!turns || !read_queries(r, a[21], a[22], q)) Py_RETURN_NONE;
            w.q = r.rows(a[23], tokens, heads, w.q_stride);
            if (!r.good || tokens != q.total_q || heads > INT32_MAX) Py_RETURN_NONE;
            w.num_heads = (int32_t)heads;
            w.pos = r.positions(a[24], axes, tokens);
            w.out = r.like(a[25], at::kBFloat16, a[23], 3);
        }
        int32_t *err = static_cast<int32_t *>(r.flat_or_null(a[26], at::kInt, -1));
        if (!r.good || PyErr_Occurred()) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        void *call = PyLong_AsVoidPtr(a[0]);
        dsa_stream_t stream = static_cast<dsa_stream_t>(PyLong_AsVoidPtr(a[2]));
        Py_BEGIN_ALLOW_THREADS
        if (fp8)
            status = reinterpret_cast<decltype(&dsa_kv_append_fp8)>(call)(&c8, &s, &f, turns ? &rope : nullptr, &q,
                                                                          has_q ? &w : nullptr, err, stream);
        else
            status = reinterpret_cast<decltype(&dsa_kv_append_rope)>(call)(&c, &s, &f, turns ? &rope : nullptr, &q,
                                                                           has_q ? &w : nullptr, err, stream);
        Py_END_ALLOW_THREADS
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (status < 0) Py_RETURN_NONE;
    return PyLong_FromLong(status);
}

// attend(call, device, stream, k_pool, v_pool, kc_pool, k_scale, v_scale, block_table, seq_lens, cu_q, q_pos, q, sel,
//        cnt, sm_scale, out, lse, workspace, dev_err)
// -> status of the attention call over the 8-bit cache at address `call` (workspace None: the prefill call), or None
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    int status = -1;
    if (n == 20) try {
        Reader r{PyLong_AsLong(a[1])};
        dsa_kv_cache c;
        dsa_kv_cache_fp8 c8;
        dsa_seqs s;
        dsa_queries q;
        if (!read_cache(r, true, a + 3, c, c8) || !read_seqs(r, a[8], a[9], s) || !read_queries(r, a[10], a[11], q))
            Py_RETURN_NONE;
        if (THPVariable_Unpack(a[10]).numel() != s.num_seqs + 1ll) Py_RETURN_NONE;
        long long tokens, heads;
        int64_t stride;
        const void *qp = r.rows(a[12], tokens, heads, stride);
        const at::Tensor *sel = r.tensor(a[13]);
        if (!r.good || tokens != q.total_q || heads > INT32_MAX || (tokens > 1 && stride != heads * 128) ||
            sel->dim() != 2 || sel->size(0) != tokens || sel->size(1) > INT32_MAX)
            Py_RETURN_NONE;
        const int32_t *sp = static_cast<int32_t *>(r.flat(a[13], at::kInt));
        const int32_t *cp = static_cast<int32_t *>(r.flat(a[14], at::kInt, tokens));
        const float scale = (float)PyFloat_AsDouble(a[15]);
        void *out = r.like(a[16], at::kBFloat16, a[12], 3);
        float *lse = static_cast<float *>(r.like(a[17], at::kFloat, a[12], 2));
        void *ws = nullptr;
        size_t bytes = 0;
        if (a[18] != Py_None) {
            ws = r.flat(a[18], at::kByte);
            if (r.good) bytes = (size_t)THPVariable_Unpack(a[18]).numel();
        }
        int32_t *err = static_cast<int32_t *>(r.flat_or_null(a[19], at::kInt, -1));
        if (!r.good || PyErr_Occurred()) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        void *call = PyLong_AsVoidPtr(a[0]);
        dsa_stream_t stream = static_cast<dsa_stream_t>(PyLong_AsVoidPtr(a[2]));
        const int k_max = (int)sel->size(1);
        Py_BEGIN_ALLOW_THREADS
        if (a[18] != Py_None)
            status = reinterpret_cast<decltype(&dsa_sparse_attn_decode_fp8)>(call)(
                &c8, &s, &q, qp, (int32_t)heads, sp, cp, k_max, scale, out, lse, ws, bytes, err, stream);
        else
            status = reinterpret_cast<decltype(&dsa_sparse_attn_prefill_fp8)>(call)(
                &c8, &s, &q, qp, (int32_t)heads, sp, cp, k_max, scale, out, lse, err, stream);
        Py_END_ALLOW_THREADS
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    if (status < 0) Py_RETURN_NONE;
    return PyLong_FromLong(status);
}

PyObject *g_slow_at = nullptr, *g_slow_rows = nullptr;

// at(tensor, dtype, device, name) -> address of a contiguous tensor
PyObject *at(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n == 4 && THPVariable_Check(args[0]) && THPDtype_Check(args[1]) && PyLong_Check(args[2])) {
        try {
            const at::Tensor &t = THPVariable_Unpack(args[0]);
            if (t.scalar_type() == reinterpret_cast<THPDtype *>(args[1])->scalar_type &&
                t.get_device() == PyLong_AsLong(args[2]) && t.is_contiguous())
                return PyLong_FromVoidPtr(t.data_ptr());
        } catch (...) {
        }
        PyErr_Clear();
    }
    return PyObject_Vectorcall(g_slow_at, args, n, nullptr);
}

// rows(tensor, device, name) -> (address, tokens, heads, token stride) of bf16 [tokens][heads][128] rows
PyObject *rows(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n == 3 && THPVariable_Check(args[0]) && PyLong_Check(args[1])) {
        try {
            const at::Tensor &t = THPVariable_Unpack(args[0]);
            if (t.scalar_type() == at::kBFloat16 && t.get_device() == PyLong_AsLong(args[1]) && t.dim() == 3 &&
                t.size(2) == 128 && t.stride(2) == 1 && (t.stride(1) == 128 || t.size(1) <= 1)) {
                const long long stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * 128;
                return Py_BuildValue("(NLLL)", PyLong_FromVoidPtr(t.data_ptr()), (long long)t.size(0),
                                     (long long)t.size(1), stride);
            }
        } catch (...) {
        }
        PyErr_Clear();
    }
    return PyObject_Vectorcall(g_slow_rows, args, n, nullptr);
}

// use(at, rows): the Python functions for everything else
PyObject *use(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "use(at, rows)");
        return nullptr;
    }
    Py_INCREF(args[0]);
    Py_INCREF(args[1]);
    Py_XDECREF(g_slow_at);
    Py_XDECREF(g_slow_rows);
    g_slow_at = args[0];
    g_slow_rows = args[1];
    Py_RETURN_NONE;
}

#define DSA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DSA_METHOD(at),  DSA_METHOD(rows), DSA_METHOD(append), DSA_METHOD(attend),
                           DSA_METHOD(use), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) {
    PyObject *m = PyModule_Create(&g_module);
    // what it was built from (build.py): the binding uses it only beside that
    if (m) PyModule_AddStringConstant(m, "built_from", DSA_ARGS_KEY);
    return m;
}
