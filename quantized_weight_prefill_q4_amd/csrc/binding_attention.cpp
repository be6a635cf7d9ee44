// The torch side of the attention operators (attention.py): as binding.cpp, one
// native call per operator that checks its tensors, allocates outputs and
// workspace and calls the C entry point.

#include "binding.h"

#include <cmath>

namespace {

decltype(&mq_rope) p_rope;
decltype(&mq_kv_store_q4) p_store;
decltype(&mq_kv_load_q4) p_load;
decltype(&mq_attention_q4) p_attention;
decltype(&mq_attention_q4_workspace_bytes) p_attention_ws;

bool g_bound = false;

// A contiguous vector of at least n (exactly n where exact) elements of a type.
const void *plain_vector(const at::Tensor &t, int dev, at::ScalarType type, int64_t n, bool exact,
                         const char *name) {
    if (t.scalar_type() != type)
        refuse("%s must be %s, got %s", name, c10::toString(type), type_name(t));
    if (t.dim() != 1 || !t.is_contiguous() || t.size(0) < n || (exact && t.size(0) != n))
        refuse("%s must be a contiguous vector of %lld elements", name, (long long)n);
    same_device(t, dev, name);
    return t.const_data_ptr();
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
}

// The cache and batch of a call with M rows.
mq_kv_q4 batch(const at::Tensor &cache, PyObject *table_o, PyObject *lens_o, PyObject *cu_o, int dev,
               bool written) {
    if (cache.scalar_type() != at::kByte)
        refuse("cache must be torch.uint8, got %s", type_name(cache));
    const int64_t bytes = cache.dim() == 4 ? cache.size(3) : 0;
    if (cache.dim() != 4 || cache.size(3) % 36 || cache.stride(3) != 1 ||
        (cache.size(2) > 1 && cache.stride(2) != bytes) ||
        (cache.size(1) > 1 && cache.stride(1) != bytes * cache.size(2)))
        refuse("%s", "cache must be [pages, heads, page / 32, 36 * head_dim] with contiguous pages");
    same_device(cache, dev, "cache");
    mq_kv_q4 kv{};
    kv.cache = written ? cache.data_ptr() : const_cast<void *>(cache.const_data_ptr());
    kv.pages = to_int(cache.size(0));
    kv.heads = to_int(cache.size(1));
    kv.page = to_int(cache.size(2) < INT32_MAX / 32 ? 32 * cache.size(2) : INT32_MAX);
    kv.head_dim = to_int(bytes / 36);
    kv.page_bytes =
        cache.size(0) > 1 ? cache.stride(0) : cache.size(1) * cache.size(2) * bytes;
    const at::Tensor &table = tensor(table_o, "table");
    if (table.scalar_type() != at::kInt) refuse("table must be torch.int32, got %s", type_name(table));
    matrix_form(table, "table");
    const int64_t B = table.size(0);
    kv.batch = to_int(B);
    kv.table_width = to_int(table.size(1));
    kv.table_ld = matrix(table, dev, B, table.size(1), "table");
    kv.table = (const int32_t *)table.const_data_ptr();
    kv.lens = (const int32_t *)plain_vector(tensor(lens_o, "lens"), dev, at::kInt, B, true, "lens");
    if (const at::Tensor *cu = optional(cu_o, "cu_rows"))
        kv.cu_rows = (const int32_t *)plain_vector(*cu, dev, at::kInt, B + 1, true, "cu_rows");
    return kv;
}

// Heads of head_dim in a row of `width` elements.
int row_heads(int64_t width, int64_t head_dim, const char *name) {
    if (head_dim <= 0 || width % head_dim)
        refuse("the width of %s, %lld, must be a multiple of head_dim = %lld", name,
               (long long)width, (long long)head_dim);
    return to_int(width / head_dim);
}

struct Rotation {
    const double *freqs = nullptr;
    int n_rot = 0;
};
Rotation rotation(const at::Tensor &t, int dev) {
    Rotation r;
    r.freqs = (const double *)plain_vector(t, dev, at::kDouble, t.dim() == 1 ? t.size(0) : 0, true,
                                           "freqs");
    r.n_rot = to_int(2 * t.size(0));
    return r;
}

PyObject *give(PyObject *given, const at::Tensor *t, at::Tensor &made) {
    if (t || !made.defined()) {   // the caller's own tensor, or None
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(std::move(made));
}

void *stream_of(PyObject *o) {
    void *stream = PyLong_AsVoidPtr(o);
    if (!stream && PyErr_Occurred()) throw Refused{};
    return stream;
}

// rope(stream, x, positions, freqs, head_dim, layout, mscale, y_type, out): y_type
// -1: x's.
PyObject *rope_checked(PyObject *const *a, Py_ssize_t n) {
    need_bound(g_bound, n, 9, "rope");
    void *stream = stream_of(a[0]);
    const at::Tensor &x = tensor(a[1], "x");
    matrix_form(x, "x");
    const int dev = device_of(x, "x"), xt = element_type(x, "x");
    const int64_t M = x.size(0), width = x.size(1), head_dim = integer(a[4]);
    const int heads = row_heads(width, head_dim, "x");
    const int ldx = matrix(x, dev, M, width, "x");
    if (M == 0 || width == 0) return status_object(MQ_ERR_SHAPE);
    const void *pos = plain_vector(tensor(a[2], "positions"), dev, at::kInt, M, true, "positions");
    const Rotation rot = rotation(tensor(a[3], "freqs"), dev);
    const int layout = to_int(integer(a[5]));
    const float mscale = real(a[6]);
    int yt = to_int(integer(a[7])), ldy = to_int(width);
    if (yt < 0) yt = xt;
    const at::Tensor *out_t = optional(a[8], "out");
    at::Tensor out;
    if (out_t) {
        yt = element_type(*out_t, "out");
        ldy = matrix(*out_t, dev, M, width, "out");
    } else {
        out = make(x, {M, width}, scalar(yt));
    }
    const void *xp = x.const_data_ptr();
    void *yp = out_t ? out_t->data_ptr() : out.data_ptr();
    const int iM = to_int(M), iD = to_int(head_dim);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = p_rope(xt, xp, ldx, (const int32_t *)pos, rot.freqs, rot.n_rot, layout, mscale, heads, iD,
                yt, yp, ldy, iM, stream);
    Py_END_ALLOW_THREADS
    return rc < 0 ? status_object(rc) : give(a[8], out_t, out);
}

// kv_store(stream, k, v, cache, table, lens, cu_rows, freqs, layout, mscale,
// positions, q, q_type, q_out): q_out, or None without q.
PyObject *kv_store_checked(PyObject *const *a, Py_ssize_t n) {
    need_bound(g_bound, n, 14, "kv_store");
    void *stream = stream_of(a[0]);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    matrix_form(k, "k");
    const int dev = device_of(k, "k"), xt = element_type(k, "k");
    const at::Tensor &cache = tensor(a[3], "cache");
    const mq_kv_q4 kv = batch(cache, a[4], a[5], a[6], dev, true);
    const int64_t M = k.size(0), width = cache.size(1) * (cache.size(3) / 36);
    if (v.scalar_type() != k.scalar_type())
        refuse("v must be %s, got %s", type_name(k), type_name(v));
    if (k.size(1) != width || v.dim() != 2 || v.size(1) != width || v.size(0) != M)
        refuse("k and v must both be M x %lld, the width of the cache's heads", (long long)width);
    const int ldk = matrix(k, dev, M, width, "k"), ldv = matrix(v, dev, M, width, "v");
    if (M == 0 || width == 0) return status_object(MQ_ERR_SHAPE);
    Rotation rot;
    if (const at::Tensor *f = optional(a[7], "freqs")) {
        rot = rotation(*f, dev);
        if (rot.n_rot == 0) return status_object(MQ_ERR_SHAPE);
    }
    const int layout = to_int(integer(a[8]));
    const float mscale = real(a[9]);
    const void *pos = nullptr;
    if (const at::Tensor *t = optional(a[10], "positions"))
        pos = plain_vector(*t, dev, at::kInt, M, true, "positions");
    const at::Tensor *q = optional(a[11], "q"), *qo_t = optional(a[13], "q_out");
    if (!q && qo_t) refuse("%s", "q_out needs q");
    int qt = to_int(integer(a[12])), ldq = 0, ldqo = 0, q_heads = 0;
    at::Tensor qo;
    const void *qp = nullptr;
    void *qop = nullptr;
    if (q) {
        matrix_form(*q, "q");
        if (q->scalar_type() != k.scalar_type())
            refuse("q must be %s, as k and v, got %s", type_name(k), type_name(*q));
        if (q->size(0) != M) refuse("q must have %lld rows", (long long)M);
        q_heads = row_heads(q->size(1), kv.head_dim, "q");
        if (q_heads == 0) return status_object(MQ_ERR_SHAPE);
        ldq = matrix(*q, dev, M, q->size(1), "q");
        ldqo = to_int(q->size(1));
        if (qo_t) {
            qt = element_type(*qo_t, "q_out");
            ldqo = matrix(*qo_t, dev, M, q->size(1), "q_out");
            qop = qo_t->data_ptr();
        } else {
            qo = make(*q, {M, q->size(1)}, scalar(qt));
            qop = qo.data_ptr();
        }
        qp = q->const_data_ptr();
    }
    const void *kp = k.const_data_ptr(), *vp = v.const_data_ptr();
    const int iM = to_int(M);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = p_store(&kv, xt, kp, ldk, vp, ldv, rot.freqs, rot.n_rot, layout, mscale,
                 (const int32_t *)pos, qp, ldq, q_heads, qt, qop, ldqo, iM, stream);
    Py_END_ALLOW_THREADS
    return rc < 0 ? status_object(rc) : give(a[13], qo_t, qo);
}

// kv_load(stream, cache, table, lens, rows, cu_rows, y_type, k_out, v_out): (k, v).
PyObject *kv_load_checked(PyObject *const *a, Py_ssize_t n) {
    need_bound(g_bound, n, 9, "kv_load");
    void *stream = stream_of(a[0]);
    const at::Tensor &cache = tensor(a[1], "cache");
    const int dev = device_of(cache, "cache");
    const mq_kv_q4 kv = batch(cache, a[2], a[3], a[5], dev, false);
    const int64_t M = integer(a[4]), width = cache.size(1) * (cache.size(3) / 36);
    if (M <= 0 || M > MQ_MAX_DIM || width == 0 || width > MQ_MAX_K)
        return status_object(MQ_ERR_SHAPE);
    int yt = to_int(integer(a[6]));
    const at::Tensor *given[2] = {optional(a[7], "k_out"), optional(a[8], "v_out")};
    const char *names[2] = {"k_out", "v_out"};
    if (given[0] || given[1])
        yt = given[0] ? element_type(*given[0], names[0]) : element_type(*given[1], names[1]);
    at::Tensor made[2];
    void *p[2];
    int ld[2];
    for (int i = 0; i < 2; ++i) {
        if (given[i]) {
            if (element_type(*given[i], names[i]) != yt)
                refuse("%s", "k_out and v_out must be of one type");
            ld[i] = matrix(*given[i], dev, M, width, names[i]);
            p[i] = given[i]->data_ptr();
        } else {
            made[i] = make(cache, {M, width}, scalar(yt));
            ld[i] = to_int(width);
            p[i] = made[i].data_ptr();
        }
    }
    const int iM = to_int(M);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = p_load(&kv, yt, p[0], ld[0], p[1], ld[1], iM, stream);
    Py_END_ALLOW_THREADS
    if (rc < 0) return status_object(rc);
    PyObject *k = give(a[7], given[0], made[0]);
    PyObject *v = k ? give(a[8], given[1], made[1]) : nullptr;
    PyObject *pair = v ? PyTuple_New(2) : nullptr;
    if (!pair) {
        Py_XDECREF(k);
        Py_XDECREF(v);
        return nullptr;
    }
    PyTuple_SET_ITEM(pair, 0, k);
    PyTuple_SET_ITEM(pair, 1, v);
    return pair;
}

// attend(stream, q, cache, table, lens, cu_rows, scale, causal, window, cap, slopes,
// prefix, max_len, out, ws): scale None: 1 / sqrt(head_dim); max_len None: what the
// table can hold.
PyObject *attend_checked(PyObject *const *a, Py_ssize_t n) {
    need_bound(g_bound, n, 15, "attend");
    void *stream = stream_of(a[0]);
    const at::Tensor &q = tensor(a[1], "q");
    matrix_form(q, "q");
    const int dev = device_of(q, "q"), xt = element_type(q, "q");
    const mq_kv_q4 kv = batch(tensor(a[2], "cache"), a[3], a[4], a[5], dev, false);
    const int64_t M = q.size(0), width = q.size(1);
    const int q_heads = row_heads(width, kv.head_dim, "q");
    const int ldq = matrix(q, dev, M, width, "q");
    if (M == 0 || width == 0) return status_object(MQ_ERR_SHAPE);
    const float scale =
        a[6] == Py_None ? (float)(1.0 / std::sqrt((double)kv.head_dim)) : real(a[6]);
    const int causal = PyObject_IsTrue(a[7]);
    if (causal < 0) throw Refused{};
    const int window = to_int(integer(a[8]));
    const float cap = real(a[9]);
    const float *slopes = nullptr;
    if (const at::Tensor *t = optional(a[10], "slopes")) slopes = vector(*t, dev, q_heads, "slopes");
    const int32_t *prefix = nullptr;
    if (const at::Tensor *t = optional(a[11], "prefix"))
        prefix = (const int32_t *)plain_vector(*t, dev, at::kInt, kv.batch, true, "prefix");
    const int64_t max_len =
        a[12] == Py_None ? (int64_t)kv.table_width * kv.page : integer(a[12]);
    const int iM = to_int(M);
    const int64_t need = p_attention_ws(&kv, q_heads, iM, max_len);
    if (need < 0) return status_object((int)need);
    const at::Tensor *out_t = optional(a[13], "out");
    at::Tensor out;
    int ldy = to_int(width);
    if (out_t) {
        if (out_t->scalar_type() != at::kHalf)
            refuse("out must be torch.float16, got %s", type_name(*out_t));
        ldy = matrix(*out_t, dev, M, width, "out");
    } else {
        out = make(q, {M, width}, at::kHalf);
    }
    at::Tensor own_ws;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (const at::Tensor *ws_t = optional(a[14], "ws")) {
        if (!ws_t->is_contiguous() || !ws_t->is_cuda() || ws_t->get_device() != dev)
            refuse("%s", "ws must be contiguous, on the same GPU as the activations");
        ws = ws_t->data_ptr();
        ws_bytes = ws_t->nbytes();
    } else if (need > 0) {
        own_ws = make(q, {need}, at::kByte);
        ws = own_ws.data_ptr();
        ws_bytes = (size_t)need;
    }
    const void *qp = q.const_data_ptr();
    uint16_t *yp = (uint16_t *)(out_t ? out_t->data_ptr() : out.data_ptr());
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = p_attention(&kv, xt, qp, ldq, q_heads, yp, ldy, iM, scale, causal, window, cap, slopes,
                     prefix, max_len, ws, ws_bytes, stream);
    Py_END_ALLOW_THREADS
    return rc < 0 ? status_object(rc) : give(a[13], out_t, out);
}

}  // namespace

PyObject *binding_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(rope_checked, a, n);
}
PyObject *binding_kv_store(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(kv_store_checked, a, n);
}
PyObject *binding_kv_load(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(kv_load_checked, a, n);
}
PyObject *binding_attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(attend_checked, a, n);
}

bool bind_attention(PyObject *dict) {
    bool ok = true;
    auto get = [&](auto &fn, const char *name) { ok = get_entry(dict, fn, name) && ok; };
    get(p_rope, "mq_rope");
    get(p_store, "mq_kv_store_q4");
    get(p_load, "mq_kv_load_q4");
    get(p_attention, "mq_attention_q4");
    get(p_attention_ws, "mq_attention_q4_workspace_bytes");
    g_bound = ok;
    return ok;
}
