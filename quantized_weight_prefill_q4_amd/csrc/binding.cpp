// The torch side of the layer operators (layers.py): argument checks, output
// and workspace allocation and the call of libmq's C entry points, in one
// native call per operator.  A single-token layer is a few microseconds of GPU
// time; the same checks made from Python and passed through ctypes take 10.5 us
// (linear) and 11.8 us (norm) of host time per call, here 5.8 and 6.2, of which
// the launch itself is 3.9.
//
// The module holds no library of its own: layers.py hands it the addresses of
// the entry points of the loaded libmq (bind()).  Checks that fail raise
// ValueError; a library status is returned as an int for the caller to raise.

#include "binding.h"

namespace {

// ---- the bound entry points ----
decltype(&mq_linear_workspace_bytes) p_linear_ws;
decltype(&mq_glu_workspace_bytes) p_glu_ws;
decltype(&mq_linear_f16cache) p_linear_f16cache;
decltype(&mq_linear_fused) p_linear_fused;
decltype(&mq_glu_f16cache) p_glu_f16cache;
decltype(&mq_glu_fused) p_glu_fused;
decltype(&mq_add_rms_norm) p_norm;
decltype(&mq_add_rms_norm_q8_1) p_norm_q8_1;
decltype(&mq_row_bytes) p_row_bytes;

bool g_bound = false;

// layer(stream, x, weight, fmt, N, K, bias, act, residual, glu, y_type,
// split_k, out, ws): fmt 0 is the f16 cache, whose N is its row count (halved
// when glu); K None: x's width.
PyObject *layer_checked(PyObject *const *a, Py_ssize_t n) {
    need_bound(g_bound, n, 14, "layer");
    void *stream = PyLong_AsVoidPtr(a[0]);
    if (!stream && PyErr_Occurred()) throw Refused{};
    const at::Tensor &x = tensor(a[1], "x");
    matrix_form(x, "x");
    const int dev = device_of(x, "x");
    const int xt = element_type(x, "x");
    const int fmt = to_int(integer(a[3]));
    const at::Tensor &w = tensor(a[2], fmt ? "wq" : "w16");
    const bool glu = a[9] == Py_True;
    int64_t N = integer(a[4]);
    const int64_t M = x.size(0), K = a[5] == Py_None ? x.size(1) : integer(a[5]);
    if (fmt == 0) {
        matrix_form(w, "w16");
        if (glu && w.size(0) % 2)
            refuse("w16 must have an even number of rows, got %lld", (long long)w.size(0));
        N = glu ? w.size(0) / 2 : w.size(0);
    }
    const int64_t rows = glu ? 2 * N : N;
    const int ldx = matrix(x, dev, M, K, "x");
    int ldw = 0;
    if (fmt == 0) {
        if (w.scalar_type() != at::kHalf)
            refuse("w16 must be torch.float16, got %s", type_name(w));
        ldw = matrix(w, dev, rows, K, "w16");
    } else {
        if (w.scalar_type() != at::kByte)
            refuse("wq must be torch.uint8, got %s", type_name(w));
        if (!w.is_contiguous()) refuse("%s", "wq must be contiguous");
        const int64_t row = p_row_bytes(fmt, K);
        if (row < 0) return status_object((int)row);
        if (rows > 0 && w.numel() / row < rows)
            refuse("wq holds %lld bytes; %lld rows of K = %lld need %lld", (long long)w.numel(),
                   (long long)rows, (long long)K, (long long)(rows * row));
        same_device(w, dev, "wq");
    }
    const at::Tensor *bias_t = optional(a[6], "bias");
    const float *bias = bias_t ? vector(*bias_t, dev, rows, "bias") : nullptr;
    const int act = to_int(integer(a[7]));
    const at::Tensor *res = optional(a[8], "residual");
    int rt = MQ_F32, ldr = 0;
    if (res) {
        rt = element_type(*res, "residual");
        ldr = matrix(*res, dev, M, N, "residual");
    }
    const int split_k = to_int(integer(a[11]));
    const int iM = to_int(M), iN = to_int(N), iK = to_int(K);
    // the sizes are checked before anything is allocated for them
    const int64_t need = (glu ? p_glu_ws : p_linear_ws)(fmt, xt, iM, iN, iK, split_k);
    if (need < 0) return status_object((int)need);

    const at::Tensor *out_t = optional(a[12], "out");
    at::Tensor out;
    int yt = to_int(integer(a[10])), ldy = to_int(N);
    if (out_t) {
        out = *out_t;
        yt = element_type(out, "out");
        ldy = matrix(out, dev, M, N, "out");
    } else {
        out = make(x, {M, N}, scalar(yt));
    }
    at::Tensor own_ws;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    if (const at::Tensor *ws_t = optional(a[13], "ws")) {
        if (!ws_t->is_contiguous() || !ws_t->is_cuda() || ws_t->get_device() != dev)
            refuse("%s", "ws must be contiguous, on the same GPU as the activations");
        ws = ws_t->data_ptr();
        ws_bytes = ws_t->nbytes();
    } else if (need > 0) {
        own_ws = make(x, {need}, at::kByte);
        ws = own_ws.data_ptr();
        ws_bytes = (size_t)need;
    }
    const void *xp = x.const_data_ptr(), *wp = w.const_data_ptr();
    const void *rp = res ? res->const_data_ptr() : nullptr;
    void *yp = out.data_ptr();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    if (glu)
        rc = fmt ? p_glu_fused(xt, xp, ldx, fmt, wp, bias, act, yt, yp, ldy, iM, iN, iK, ws,
                               ws_bytes, split_k, stream)
                 : p_glu_f16cache(xt, xp, ldx, (const uint16_t *)wp, ldw, bias, act, yt, yp, ldy, iM,
                                  iN, iK, ws, ws_bytes, split_k, stream);
    else
        rc = fmt ? p_linear_fused(xt, xp, ldx, fmt, wp, bias, act, rt, rp, ldr, yt, yp, ldy, iM, iN,
                                  iK, ws, ws_bytes, split_k, stream)
                 : p_linear_f16cache(xt, xp, ldx, (const uint16_t *)wp, ldw, bias, act, rt, rp, ldr,
                                     yt, yp, ldy, iM, iN, iK, ws, ws_bytes, split_k, stream);
    Py_END_ALLOW_THREADS
    if (rc < 0) return status_object(rc);
    if (out_t) {
        Py_INCREF(a[12]);
        return a[12];
    }
    return THPVariable_Wrap(std::move(out));
}

// norm(stream, x, weight, residual, eps, y_type, out, ds, residual_out):
// (y, h) for y_type MQ_F32 / MQ_F16; (xq, ds, h) for y_type < 0.  h is None
// without a residual.
PyObject *norm_checked(PyObject *const *a, Py_ssize_t n) {
    need_bound(g_bound, n, 9, "norm");
    void *stream = PyLong_AsVoidPtr(a[0]);
    if (!stream && PyErr_Occurred()) throw Refused{};
    const at::Tensor &x = tensor(a[1], "x");
    matrix_form(x, "x");
    const int dev = device_of(x, "x");
    const int xt = element_type(x, "x");
    const int64_t M = x.size(0), K = x.size(1);
    const int ldx = matrix(x, dev, M, K, "x");
    const double eps = PyFloat_AsDouble(a[4]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused{};
    const int want = to_int(integer(a[5]));
    const bool q8 = want < 0;
    if (M == 0 || K == 0 || (q8 && K % 32)) return status_object(MQ_ERR_SHAPE);
    const float *w = vector(tensor(a[2], "weight"), dev, K, "weight");

    const at::Tensor *res = optional(a[3], "residual"), *h_t = optional(a[8], "residual_out");
    if (!res && h_t) refuse("%s", "residual_out needs a residual");
    int rt = MQ_F32, ldr = 0, ldh = to_int(K);
    at::Tensor h;
    if (res) {
        rt = element_type(*res, "residual");
        ldr = matrix(*res, dev, M, K, "residual");
        if (h_t) {
            if (h_t->scalar_type() != res->scalar_type())
                refuse("residual_out must be %s, got %s", type_name(*res), type_name(*h_t));
            h = *h_t;
            ldh = matrix(h, dev, M, K, "residual_out");
        } else {
            h = make(x, {M, K}, res->scalar_type());
        }
    }
    const at::Tensor *y_t = optional(a[6], q8 ? "xq" : "out"), *ds_t = optional(a[7], "ds");
    at::Tensor y, ds;
    int yt = want, ldy;
    if (q8) {
        if (y_t && y_t->scalar_type() != at::kChar)
            refuse("xq must be torch.int8, got %s", type_name(*y_t));
        y = y_t ? *y_t : make(x, {M, (K + 15) / 16 * 16}, at::kChar);
        ldy = matrix(y, dev, M, K, "xq");
        if (ds_t && (ds_t->scalar_type() != at::kFloat || !ds_t->is_contiguous() ||
                     !ds_t->is_cuda() || ds_t->get_device() != dev || ds_t->numel() < M * (K / 16)))
            refuse("%s", "ds must be contiguous float32 with M*K/16 elements, on x's GPU");
        ds = ds_t ? *ds_t : make(x, {M, K / 32, 2}, at::kFloat);
    } else if (y_t) {
        y = *y_t;
        yt = element_type(y, "out");
        ldy = matrix(y, dev, M, K, "out");
    } else {
        y = make(x, {M, K}, scalar(yt));
        ldy = to_int(K);
    }
    const void *xp = x.const_data_ptr(), *rp = res ? res->const_data_ptr() : nullptr;
    void *hp = res ? h.data_ptr() : nullptr, *yp = y.data_ptr();
    float *dp = q8 ? (float *)ds.data_ptr() : nullptr;
    const int iM = to_int(M), iK = to_int(K);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = q8 ? p_norm_q8_1(xt, xp, ldx, rt, rp, ldr, w, (float)eps, hp, ldh, (int8_t *)yp, ldy, dp, iM,
                          iK, stream)
            : p_norm(xt, xp, ldx, rt, rp, ldr, w, (float)eps, hp, ldh, yt, yp, ldy, iM, iK, stream);
    Py_END_ALLOW_THREADS
    if (rc < 0) return status_object(rc);
    auto give = [](PyObject *given, const at::Tensor *t, at::Tensor &made) {
        if (t || !made.defined()) {   // the caller's own tensor, or None
            Py_INCREF(given);
            return given;
        }
        return THPVariable_Wrap(std::move(made));
    };
    PyObject *items[3] = {give(a[6], y_t, y), nullptr, nullptr};
    int count = 1;
    if (q8) items[count++] = give(a[7], ds_t, ds);
    items[count++] = give(a[8], h_t, h);
    PyObject *result = PyTuple_New(count);
    for (int i = 0; i < count; ++i) {
        if (result && items[i])
            PyTuple_SET_ITEM(result, i, items[i]);
        else
            Py_XDECREF(items[i]);
    }
    if (result && PyErr_Occurred()) {   // an output that could not be wrapped
        Py_DECREF(result);
        return nullptr;
    }
    return result;
}

PyObject *layer(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(layer_checked, a, n);
}

PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) { return guarded(norm_checked, a, n); }

// bind({name: address}): the entry points of the loaded library.
PyObject *bind(PyObject *, PyObject *dict) {
    bool ok = true;
    auto get = [&](auto &fn, const char *name) { ok = get_entry(dict, fn, name) && ok; };
    get(p_linear_ws, "mq_linear_workspace_bytes");
    get(p_glu_ws, "mq_glu_workspace_bytes");
    get(p_linear_f16cache, "mq_linear_f16cache");
    get(p_linear_fused, "mq_linear_fused");
    get(p_glu_f16cache, "mq_glu_f16cache");
    get(p_glu_fused, "mq_glu_fused");
    get(p_norm, "mq_add_rms_norm");
    get(p_norm_q8_1, "mq_add_rms_norm_q8_1");
    get(p_row_bytes, "mq_row_bytes");
    ok = bind_attention(dict) && ok;
    if (!ok) {
        g_bound = false;
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: an entry point is missing");
        return nullptr;
    }
    g_bound = true;
    Py_RETURN_NONE;
}

#define FASTCALL(f) (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr

PyMethodDef methods[] = {
    {"layer", FASTCALL(layer)},
    {"norm", FASTCALL(norm)},
    {"rope", FASTCALL(binding_rope)},
    {"kv_store", FASTCALL(binding_kv_store)},
    {"kv_load", FASTCALL(binding_kv_load)},
    {"attend", FASTCALL(binding_attend)},
    {"bind", bind, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module_def); }
