// C ABI of libmq: argument validation, launch planning, error reporting.
// Every check happens before anything is enqueued, so a rejected call has no
// side effect (Fucina "Eager GPU Offload Without A Compute Graph", ordering
// section: submission failures are reported before return; faults after
// submission surface at the host boundary).

#include "mq.h"
#include "mq_internal.h"

#include <mutex>
#include <stdint.h>

// The K-split partial tiles of mq_gemm_fused_noalloc, for callers that cannot
// allocate.  Each GPU the library runs on holds its own copy for the life of
// the process.  In host code `scratch` names a host-side stand-in: kernels get
// the device address that hipGetSymbolAddress returns for the device
// (scratch_ptr below), never the array's name.
static __device__ __align__(256) float scratch[MQ_NOALLOC_SCRATCH_BYTES / 4];

namespace {

thread_local int g_last_hip_error = 0;

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

bool quant_fmt(int fmt) { return mq::block_elems(fmt) > 0; }

int check_dims(int M, int N, int K) {
    if (M <= 0 || N <= 0 || K <= 0 || M > MQ_MAX_DIM || N > MQ_MAX_DIM || K > MQ_MAX_K)
        return MQ_ERR_SHAPE;
    return MQ_OK;
}

bool ld_ok(int64_t ld, int64_t K) { return ld >= K && ld % 8 == 0 && ld <= MQ_MAX_K + 64; }

// int8 code rows: 16-byte aligned, at most MQ_MAX_K bytes apart.
bool ldq_ok(int64_t ld, int64_t K) { return ld >= K && ld % 16 == 0 && ld <= MQ_MAX_K; }

// f32 activation rows: 16-byte aligned (ld a multiple of 4), at most MQ_MAX_K
// elements apart (a 256-row tile then spans at most 2^31 bytes).
bool ld32_ok(int64_t ld, int64_t K) { return ld >= K && ld % 4 == 0 && ld <= MQ_MAX_K; }

int hip_status(hipError_t e) {
    if (e == hipSuccess) return MQ_OK;
    g_last_hip_error = (int)e;
    return MQ_ERR_HIP;
}

// Checks of one decode (mq_dequant_to_f16 and each job of a batch).
int check_dequant(int fmt, const void *wq, int N, int K, const uint16_t *w16, int ld) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    if (!wq || !w16) return MQ_ERR_NULL;
    if (check_dims(1, N, K) || K % mq::block_elems(fmt)) return MQ_ERR_SHAPE;
    if (!ld_ok(ld, K)) return MQ_ERR_LD;
    if (!aligned16(wq) || !aligned16(w16)) return MQ_ERR_ALIGN;
    if ((int64_t)N * ld / 8 >= ((int64_t)1 << 31)) return MQ_ERR_SHAPE;
    return MQ_OK;
}

// An element type of the norm and the linear layers, and a pointer aligned to it.
bool type_ok(int type) { return type == MQ_F32 || type == MQ_F16; }
bool elem_aligned(const void *p, int type) {
    return ((uintptr_t)p & (type == MQ_F32 ? 3 : 1)) == 0;
}

// The rows of a buffer that a call reads or writes.
struct Span {
    const char *p;
    int64_t stride, row, rows;   // bytes, bytes, count
};
Span span(const void *p, int64_t ld, int64_t K, int64_t elem, int64_t rows) {
    return Span{(const char *)p, ld * elem, K * elem, rows};
}
bool same_span(const Span &a, const Span &b) {
    return a.p == b.p && a.row == b.row && (a.stride == b.stride || a.rows == 1);
}
// Rows at one stride with disjoint columns (slices of one buffer) do not
// overlap; ranges that meet at different strides count as overlapping.
bool overlap(const Span &a, const Span &b) {
    if (a.p + (a.rows - 1) * a.stride + a.row <= b.p ||
        b.p + (b.rows - 1) * b.stride + b.row <= a.p)
        return false;
    if (a.stride != b.stride && a.rows > 1 && b.rows > 1) return true;
    const int64_t s = a.rows > 1 ? a.stride : b.stride;
    if (s <= 0 || (a.rows == 1 && b.rows == 1)) return true;
    const int64_t d = ((b.p - a.p) % s + s) % s;
    return d < a.row || d + b.row > s;
}

// The overlap rules of the norm: an output is elementwise the input itself or
// disjoint from it, and disjoint from the other output and the weights.
int check_norm_overlap(const mq::NormSpec &n, int64_t y_elem) {
    auto bytes = [](int type) { return (int64_t)(type == MQ_F32 ? 4 : 2); };
    const Span x = span(n.x, n.ldx, n.K, bytes(n.x_type), n.M);
    const Span y = span(n.y, n.ldy, n.K, y_elem, n.M);
    const Span w = span(n.w, n.K, n.K, 4, 1);
    const bool q8 = n.y_type == mq::kTypeI8;
    auto clash = [](const Span &out, const Span &in, bool may_be_same) {
        return overlap(out, in) && !(may_be_same && same_span(out, in));
    };
    if (clash(y, x, !q8) || clash(y, w, false)) return MQ_ERR_OVERLAP;
    const Span ds = span(n.ds, n.K / 16, n.K / 16, 4, n.M);
    if (q8 && (clash(ds, x, false) || clash(ds, w, false) || clash(ds, y, false)))
        return MQ_ERR_OVERLAP;
    if (n.r) {
        const Span r = span(n.r, n.ldr, n.K, bytes(n.r_type), n.M);
        const Span h = span(n.h, n.ldh, n.K, bytes(n.r_type), n.M);
        if (clash(y, r, !q8) || clash(y, h, false) || clash(h, x, true) || clash(h, r, true) ||
            clash(h, w, false))
            return MQ_ERR_OVERLAP;
        if (q8 && (clash(ds, r, false) || clash(ds, h, false))) return MQ_ERR_OVERLAP;
    }
    return MQ_OK;
}

// Checks of the norm's inputs and residual stream; fills their part of `n`.
int check_norm(int x_type, const void *X, int ldx, int r_type, const void *R, int ldr,
               const float *w, float eps, void *H, int ldh, int M, int K, mq::NormSpec *n) {
    if (!X || !w || (R && !H)) return MQ_ERR_NULL;
    if (!type_ok(x_type) || (R && !type_ok(r_type))) return MQ_ERR_TYPE;
    if (ldx < K || (R && (ldr < K || ldh < K))) return MQ_ERR_LD;
    if (!elem_aligned(X, x_type) || !elem_aligned(w, MQ_F32) ||
        (R && (!elem_aligned(R, r_type) || !elem_aligned(H, r_type))))
        return MQ_ERR_ALIGN;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return MQ_ERR_EPS;
    *n = mq::NormSpec{};
    n->x = X;
    n->ldx = ldx;
    n->x_type = x_type;
    n->w = w;
    n->eps = eps;
    n->M = M;
    n->K = K;
    if (R) {
        n->r = R;
        n->h = H;
        n->ldr = ldr;
        n->ldh = ldh;
        n->r_type = r_type;
    }
    return MQ_OK;
}

// How a GEMM with f32 activations runs.  Up to kInTileMaxM rows the kernel
// rounds X to f16 while staging its tiles; above, X is converted once into
// the front of the workspace and the f16-activation kernel (with its own
// plan, 256 × 256 tiles included) reads it: every column tile re-reads the
// X panel, so converting inside the tile costs N/BN conversions and twice
// the A-operand bytes per element, against one 6-byte pass.
constexpr int kInTileMaxM = 64;

struct XPlan {
    bool convert_first;
    int ld16;               // row stride of the converted X (convert_first)
    int64_t x16_bytes;      // its workspace bytes, a multiple of 256 (else 0)
    mq::GemmPlan gemm;      // split planes follow the converted X in the workspace
};

XPlan xf32_plan(int fmt, int M, int N, int K, int split_k) {
    XPlan xp;
    xp.convert_first = M > kInTileMaxM;
    if (xp.convert_first) {
        xp.ld16 = (int)mq_f16cache_ld(K);
        xp.x16_bytes = ((int64_t)M * xp.ld16 * 2 + 255) / 256 * 256;
        xp.gemm = mq::plan_gemm(fmt, M, N, K, split_k, false);
    } else {
        xp.ld16 = 0;
        xp.x16_bytes = 0;
        xp.gemm = mq::plan_gemm(fmt, M, N, K, split_k, true);
    }
    return xp;
}

// Device address of `scratch` on the device that owns `stream` (the current
// device for the null stream), looked up once per device with that device
// current and kept.
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices];

int scratch_ptr(hipStream_t stream, void **out) {
    int cur = 0, dev = 0;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return hip_status(e);
    dev = cur;
    if (stream) {
        e = hipStreamGetDevice(stream, &dev);
        if (e != hipSuccess) return hip_status(e);
    }
    if (dev < 0 || dev >= kMaxDevices) return hip_status(hipErrorInvalidDevice);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        if (dev != cur && (e = hipSetDevice(dev)) != hipSuccess) return hip_status(e);
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (dev != cur) {
            const hipError_t back = hipSetDevice(cur);
            if (e == hipSuccess) e = back;
        }
        if (e != hipSuccess) return hip_status(e);
        if (!p) return hip_status(hipErrorInvalidSymbol);
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return MQ_OK;
}

// Shared checks of both GEMM entry points; fills the plan on success.
int check_gemm(int fmt, const void *X, int ldx, const void *W, int64_t ldw_elems, const float *Y,
               int ldy, int M, int N, int K, const void *ws, size_t ws_bytes, int split_k,
               mq::GemmPlan *plan, bool x_f32 = false, XPlan *xplan = nullptr) {
    if (!X || !W || !Y) return MQ_ERR_NULL;
    if (fmt != mq::kFmtF16 && !quant_fmt(fmt)) return MQ_ERR_FORMAT;
    if (int rc = check_dims(M, N, K)) return rc;
    const int step = fmt == mq::kFmtF16 ? 8 : mq::block_elems(fmt);
    if (K % step) return MQ_ERR_SHAPE;
    if (!(x_f32 ? ld32_ok(ldx, K) : ld_ok(ldx, K)) || ldy < N) return MQ_ERR_LD;
    if (fmt == mq::kFmtF16 && !ld_ok(ldw_elems, K)) return MQ_ERR_LD;
    if (!aligned16(X) || !aligned16(W) || !aligned16(Y)) return MQ_ERR_ALIGN;
    if (split_k < 0 || split_k > MQ_MAX_SPLIT_K) return MQ_ERR_SPLIT;
    if (split_k > 1 && (int64_t)M * N >= ((int64_t)1 << 31)) return MQ_ERR_SPLIT;
    int64_t need;
    if (x_f32) {
        *xplan = xf32_plan(fmt, M, N, K, split_k);
        *plan = xplan->gemm;
        need = xplan->x16_bytes + plan->ws_bytes;
    } else {
        *plan = mq::plan_gemm(fmt, M, N, K, split_k);
        need = plan->ws_bytes;
    }
    if (need > 0 && (!ws || !aligned16(ws) || ws_bytes < (size_t)need)) return MQ_ERR_WORKSPACE;
    return MQ_OK;
}

// The f32-activation GEMM: in-tile conversion, or convert into the
// workspace and the f16-activation kernel.
int run_xf32(int fmt, const float *X, int ldx, const void *W, int64_t ldw, float *Y, int ldy,
             int M, int N, int K, void *ws, const XPlan &xp, hipStream_t stream) {
    if (!xp.convert_first)
        return hip_status(mq::launch_gemm_xf32(fmt, X, ldx, W, ldw, Y, ldy, M, N, K, xp.gemm,
                                               (float *)ws, stream));
    uint16_t *x16 = (uint16_t *)ws;
    if (int rc = hip_status(mq::launch_convert_f32_to_f16(X, ldx, x16, xp.ld16, M, K, stream)))
        return rc;
    return hip_status(mq::launch_gemm(fmt, x16, xp.ld16, W, ldw, Y, ldy, M, N, K, xp.gemm,
                                      (float *)((char *)ws + xp.x16_bytes), stream));
}

// How a linear layer runs.  Few rows with the split left to the library: one
// kernel that needs no workspace.  Else the tile GEMM: f32 activations are
// rounded to f16 into the front of the workspace, as xf32_plan does; the
// product's planes follow.
struct LinearPlan {
    bool rows;              // the few-row kernel
    int ld16;               // row stride of the converted X, 0 when X is f16
    int64_t x16_bytes;
    mq::GemmPlan gemm;
    int64_t ws_bytes;
};

LinearPlan linear_plan(int fmt, int x_type, int M, int rows, int K, int split_k) {
    LinearPlan p{};
    p.rows = split_k == 0 && mq::linear_rows_fit(fmt, M, rows, K);
    if (p.rows) return p;
    if (x_type == MQ_F32) {
        p.ld16 = (int)mq_f16cache_ld(K);
        p.x16_bytes = ((int64_t)M * p.ld16 * 2 + 255) / 256 * 256;
    }
    p.gemm = mq::plan_gemm(fmt, M, rows, K, split_k);
    // A short K over a quarter of a round of tiles or more is not worth the
    // planes and the second kernel of a split (f16 512 x 2048 x 512: 11.5 us
    // split two ways, 8.3 whole; Q4_K 200 x 8192 x 512 14.8 / 11.1, x 1024 17.6 /
    // 16.0; with 48 tiles the split is ahead from K = 1024 on, 10.2 / 11.1).
    if (split_k == 0 && p.gemm.split > 1 && p.gemm.dp_tiles == 0 && p.gemm.tail_tiles >= 64 &&
        K <= 1024)
        p.gemm = mq::plan_gemm(fmt, M, rows, K, 1);
    p.ws_bytes = p.x16_bytes + p.gemm.ws_bytes;
    return p;
}

// Sizes, format and split of a linear layer (`rows` rows of weights).
int check_linear_shape(int fmt, int x_type, int M, int rows, int K, int split_k) {
    if (fmt != mq::kFmtF16 && !quant_fmt(fmt)) return MQ_ERR_FORMAT;
    if (!type_ok(x_type)) return MQ_ERR_TYPE;
    if (int rc = check_dims(M, rows, K)) return rc;
    if (K % (fmt == mq::kFmtF16 ? 8 : mq::block_elems(fmt))) return MQ_ERR_SHAPE;
    if (split_k < 0 || split_k > MQ_MAX_SPLIT_K) return MQ_ERR_SPLIT;
    if (split_k > 1 && (int64_t)M * rows >= ((int64_t)1 << 31)) return MQ_ERR_SPLIT;
    return MQ_OK;
}

// Rows of weights of a layer with N output columns; -1 (a bad shape) for an N
// that has none.
int weight_rows(int N, bool glu) { return N <= 0 || N > MQ_MAX_DIM ? -1 : glu ? 2 * N : N; }

int64_t linear_workspace(int fmt, int x_type, int M, int N, int K, int split_k, bool glu) {
    const int rows = weight_rows(N, glu);
    if (int rc = check_linear_shape(fmt, x_type, M, rows, K, split_k)) return rc;
    return linear_plan(fmt, x_type, M, rows, K, split_k).ws_bytes;
}

// Checks and runs a linear layer; ldw in halves for the f16 cache, unused else.
int run_linear(int fmt, int x_type, const void *X, int ldx, const void *W, int64_t ldw, int y_type,
               void *Y, int ldy, int M, int N, int K, const mq::EpiSpec &epi, void *ws,
               size_t ws_bytes, int split_k, hipStream_t stream) {
    const int rows = weight_rows(N, epi.glu);
    if (int rc = check_linear_shape(fmt, x_type, M, rows, K, split_k)) return rc;
    if (!X || !W || !Y) return MQ_ERR_NULL;
    if (!type_ok(y_type) || (epi.res && !type_ok(epi.res_type))) return MQ_ERR_TYPE;
    if (epi.act < MQ_ACT_NONE || epi.act > MQ_ACT_GELU_TANH) return MQ_ERR_ACT;
    if (!(x_type == MQ_F32 ? ld32_ok(ldx, K) : ld_ok(ldx, K)) || ldy < N ||
        (epi.res && epi.ldr < N))
        return MQ_ERR_LD;
    if (fmt == mq::kFmtF16 ? !ld_ok(ldw, K) : false) return MQ_ERR_LD;
    if (!aligned16(X) || !aligned16(W) || !elem_aligned(Y, y_type) ||
        !elem_aligned(epi.bias, MQ_F32) || (epi.res && !elem_aligned(epi.res, epi.res_type)))
        return MQ_ERR_ALIGN;
    const LinearPlan p = linear_plan(fmt, x_type, M, rows, K, split_k);
    if (p.ws_bytes > 0 && (!ws || !aligned16(ws) || ws_bytes < (size_t)p.ws_bytes))
        return MQ_ERR_WORKSPACE;
    const int64_t wbytes =
        fmt == mq::kFmtF16 ? ldw * 2 : (int64_t)K / mq::block_elems(fmt) * mq::block_bytes(fmt);
    auto bytes = [](int type) { return (int64_t)(type == MQ_F32 ? 4 : 2); };
    const Span y = span(Y, ldy, N, bytes(y_type), M);
    // an absent buffer has no rows' bytes and overlaps nothing
    auto clash = [](const Span &p, const Span &q) {
        return p.row > 0 && q.row > 0 && overlap(p, q);
    };
    const Span x = span(X, ldx, K, bytes(x_type), M);
    const Span w{(const char *)W, wbytes, fmt == mq::kFmtF16 ? 2 * (int64_t)K : wbytes, rows};
    const Span b = span(epi.bias, rows, epi.bias ? rows : 0, 4, 1);
    const Span r = span(epi.res, epi.ldr, epi.res ? N : 0, bytes(epi.res_type), M);
    const Span work = span(ws, p.ws_bytes, p.ws_bytes, 1, 1);
    if (clash(y, x) || clash(y, w) || clash(y, b) || (clash(y, r) && !same_span(y, r)))
        return MQ_ERR_OVERLAP;
    if (clash(work, x) || clash(work, w) || clash(work, b) || clash(work, r) || clash(work, y))
        return MQ_ERR_OVERLAP;
    if (p.rows)
        return hip_status(mq::launch_linear_rows(fmt, x_type == MQ_F32, X, ldx, W,
                                                 fmt == mq::kFmtF16 ? ldw : wbytes, Y, ldy, M, N,
                                                 K, epi, stream));
    const uint16_t *x16 = (const uint16_t *)X;
    if (p.ld16) {
        uint16_t *to = (uint16_t *)ws;
        if (int rc = hip_status(
                mq::launch_convert_f32_to_f16((const float *)X, ldx, to, p.ld16, M, K, stream)))
            return rc;
        x16 = to;
        ldx = p.ld16;
    }
    float *planes = (float *)((char *)ws + p.x16_bytes);
    return hip_status((epi.glu ? mq::launch_gemm_glu : mq::launch_gemm_linear)(
        fmt, x16, ldx, W, fmt == mq::kFmtF16 ? ldw : wbytes, Y, ldy, M, N, K, p.gemm, planes, epi,
        stream));
}

// The units of kernels that number a batch's work come to fewer than 2^24 blocks
// of 256 threads (a launch holds fewer than 2^32 threads).
constexpr int64_t kMaxBlocks = (1 << 24) - 1;

// Checks of a cache and of the batch of M rows that goes with it; fills `kv`.
int check_kv(const mq_kv_q4 *c, int M, mq::KvSpec *kv) {
    if (!c || !c->cache || !c->table || !c->lens) return MQ_ERR_NULL;
    if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 256)
        return MQ_ERR_SHAPE;
    if (c->heads <= 0 || c->heads > MQ_MAX_HEADS || c->page <= 0 || c->page % 32 ||
        c->page > mq::kMaxLen || c->pages <= 0 || c->batch <= 0 || c->table_width <= 0)
        return MQ_ERR_SHAPE;
    if (M <= 0 || M > MQ_MAX_DIM || c->batch > MQ_MAX_DIM) return MQ_ERR_SHAPE;
    if (!c->cu_rows && M % c->batch) return MQ_ERR_SHAPE;
    if (M / 8 + 2 * (int64_t)c->batch > kMaxBlocks) return MQ_ERR_SHAPE;
    if (c->page_bytes < mq_kv_q4_page_bytes(c->heads, c->page, c->head_dim) || c->page_bytes % 16 ||
        (c->batch > 1 && c->table_ld < c->table_width))
        return MQ_ERR_LD;
    if (!aligned16(c->cache) || (uintptr_t)c->table % 4 || (uintptr_t)c->lens % 4 ||
        (uintptr_t)c->cu_rows % 4)
        return MQ_ERR_ALIGN;
    kv->cache = (char *)c->cache;
    kv->page_bytes = c->page_bytes;
    kv->table = c->table;
    kv->lens = c->lens;
    kv->cu = c->cu_rows;
    kv->table_ld = c->table_ld;
    kv->pages = c->pages;
    kv->heads = c->heads;
    kv->page = c->page;
    kv->D = c->head_dim;
    kv->width = c->table_width;
    kv->batch = c->batch;
    kv->rows = M / c->batch;
    kv->M = M;
    return MQ_OK;
}
Span cache_span(const mq::KvSpec &kv) {
    return span(kv.cache, kv.page_bytes, mq_kv_q4_page_bytes(kv.heads, kv.page, kv.D), 1, kv.pages);
}
int64_t type_bytes(int type) { return type == MQ_F32 ? 4 : 2; }

// Whether an output lies over n values of a vector that the call reads (null: none).
bool over(const Span &out, const void *p, int64_t n, int64_t elem) {
    return p && overlap(out, span(p, n, n, elem, 1));
}
// ... over what says where the batch's rows and tokens are.
bool over_batch(const Span &out, const mq::KvSpec &kv) {
    // (the table's rows, or all of it as one: it may lie between an output's rows as a whole)
    const int64_t all = (kv.batch - 1) * kv.table_ld + kv.width;
    return (overlap(out, span(kv.table, kv.table_ld, kv.width, 4, kv.batch)) &&
            over(out, kv.table, all, 4)) ||
           over(out, kv.lens, kv.batch, 4) || over(out, kv.cu, (int64_t)kv.batch + 1, 4);
}

// A rotation's frequencies: n_rot even and at most the head.
int check_rotation(const double *freqs, int n_rot, int layout, float mscale, int head_dim) {
    if (layout != MQ_ROPE_HALF && layout != MQ_ROPE_INTERLEAVED) return MQ_ERR_FORMAT;
    if (n_rot <= 0 || n_rot % 2 || n_rot > head_dim) return MQ_ERR_SHAPE;
    if (!(mscale > -3.0e38f && mscale < 3.0e38f)) return MQ_ERR_EPS;
    if ((uintptr_t)freqs % 8) return MQ_ERR_ALIGN;
    return MQ_OK;
}

bool heads_ok(int heads, int head_dim) {
    return heads > 0 && heads <= MQ_MAX_HEADS && (int64_t)heads * head_dim <= MQ_MAX_K;
}

// Checks of an attention call that its workspace depends on.
int check_attention(const mq::KvSpec &kv, int q_heads, int64_t max_len) {
    if (!heads_ok(q_heads, kv.D) || q_heads % kv.heads || max_len < 0) return MQ_ERR_SHAPE;
    // the kernels number a key/value head's rows, and work beyond them, as ints
    if ((int64_t)kv.M * (q_heads / kv.heads) > (1 << 30)) return MQ_ERR_SHAPE;
    return MQ_OK;
}
bool plan_ok(const mq::AttnPlan &p) { return p.items <= kMaxBlocks / 2; }

}  // namespace

extern "C" {

int mq_block_elems(int fmt) {
    const int v = mq::block_elems(fmt);
    return v < 0 ? MQ_ERR_FORMAT : v;
}

int mq_block_bytes(int fmt) {
    const int v = mq::block_bytes(fmt);
    return v < 0 ? MQ_ERR_FORMAT : v;
}

int64_t mq_row_bytes(int fmt, int64_t K) {
    const int be = mq::block_elems(fmt);
    if (be < 0) return MQ_ERR_FORMAT;
    if (K <= 0 || K > MQ_MAX_K || K % be) return MQ_ERR_SHAPE;
    return K / be * mq::block_bytes(fmt);
}

int64_t mq_f16cache_ld(int64_t K) {
    if (K <= 0 || K > MQ_MAX_K) return MQ_ERR_SHAPE;
    return (2 * K) % 2048 == 0 ? K + 64 : K;
}

int mq_dequant_to_f16(int fmt, const void *wq, int N, int K, uint16_t *w16, int ld,
                      void *stream) {
    if (int rc = check_dequant(fmt, wq, N, K, w16, ld)) return rc;
    return hip_status(mq::launch_dequant(fmt, wq, N, K, w16, ld, (hipStream_t)stream));
}

int mq_dequant_to_f16_batch(const mq_dequant_job *jobs, int n, void *stream) {
    if (n < 0) return MQ_ERR_SHAPE;
    if (n == 0) return MQ_OK;
    if (!jobs) return MQ_ERR_NULL;
    for (int i = 0; i < n; ++i) {
        const mq_dequant_job &j = jobs[i];
        if (int rc = check_dequant(j.fmt, j.wq, j.N, j.K, j.w16, j.ld)) return rc;
    }
    constexpr int kChunk = 64;
    mq::DequantSpec specs[kChunk];
    for (int first = 0; first < n; first += kChunk) {
        const int m = n - first < kChunk ? n - first : kChunk;
        for (int i = 0; i < m; ++i) {
            const mq_dequant_job &j = jobs[first + i];
            specs[i] = mq::DequantSpec{j.fmt, j.N, j.K, j.ld, j.wq, j.w16};
        }
        if (int rc = hip_status(mq::launch_dequant_batch(specs, m, (hipStream_t)stream))) return rc;
    }
    return MQ_OK;
}

static int64_t workspace_bytes(int fmt, int M, int N, int K, int split_k, bool x_f32) {
    if (fmt != mq::kFmtF16 && !quant_fmt(fmt)) return MQ_ERR_FORMAT;
    if (int rc = check_dims(M, N, K)) return rc;
    if (K % (fmt == mq::kFmtF16 ? 8 : mq::block_elems(fmt))) return MQ_ERR_SHAPE;
    if (split_k < 0 || split_k > MQ_MAX_SPLIT_K) return MQ_ERR_SPLIT;
    if (split_k > 1 && (int64_t)M * N >= ((int64_t)1 << 31)) return MQ_ERR_SPLIT;
    if (!x_f32) return mq::plan_gemm(fmt, M, N, K, split_k).ws_bytes;
    const XPlan xp = xf32_plan(fmt, M, N, K, split_k);
    return xp.x16_bytes + xp.gemm.ws_bytes;
}

int64_t mq_gemm_workspace_bytes(int fmt, int M, int N, int K, int split_k) {
    return workspace_bytes(fmt, M, N, K, split_k, false);
}

int64_t mq_gemm_xf32_workspace_bytes(int fmt, int M, int N, int K, int split_k) {
    return workspace_bytes(fmt, M, N, K, split_k, true);
}

int mq_gemm_f16cache(const uint16_t *X, int ldx, const uint16_t *W16, int ldw, float *Y,
                     int ldy, int M, int N, int K, void *ws, size_t ws_bytes, int split_k,
                     void *stream) {
    mq::GemmPlan plan;
    if (int rc = check_gemm(mq::kFmtF16, X, ldx, W16, ldw, Y, ldy, M, N, K, ws, ws_bytes,
                            split_k, &plan))
        return rc;
    return hip_status(mq::launch_gemm(mq::kFmtF16, X, ldx, W16, ldw, Y, ldy, M, N, K, plan,
                                      (float *)ws, (hipStream_t)stream));
}

int mq_gemm_fused(int fmt, const uint16_t *X, int ldx, const void *wq, float *Y, int ldy,
                  int M, int N, int K, void *ws, size_t ws_bytes, int split_k, void *stream) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    mq::GemmPlan plan;
    if (int rc = check_gemm(fmt, X, ldx, wq, 0, Y, ldy, M, N, K, ws, ws_bytes, split_k, &plan))
        return rc;
    const int64_t row_bytes = (int64_t)K / mq::block_elems(fmt) * mq::block_bytes(fmt);
    return hip_status(mq::launch_gemm(fmt, X, ldx, wq, row_bytes, Y, ldy, M, N, K, plan,
                                      (float *)ws, (hipStream_t)stream));
}

int mq_gemm_fused_noalloc(int fmt, const uint16_t *X, int ldx, const void *wq, float *Y,
                          int ldy, int M, int N, int K, int split_k, void *stream) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    // the plan's partial tiles must fit the static scratch
    const int64_t need = mq_gemm_workspace_bytes(fmt, M, N, K, split_k);
    if (need < 0) return (int)need;
    if (need > MQ_NOALLOC_SCRATCH_BYTES) return MQ_ERR_SCRATCH;
    void *ws = nullptr;
    if (need > 0) {
        if (int rc = scratch_ptr((hipStream_t)stream, &ws)) return rc;
    }
    mq::GemmPlan plan;
    if (int rc = check_gemm(fmt, X, ldx, wq, 0, Y, ldy, M, N, K, ws,
                            need > 0 ? (size_t)MQ_NOALLOC_SCRATCH_BYTES : 0, split_k, &plan))
        return rc;
    const int64_t row_bytes = (int64_t)K / mq::block_elems(fmt) * mq::block_bytes(fmt);
    return hip_status(mq::launch_gemm(fmt, X, ldx, wq, row_bytes, Y, ldy, M, N, K, plan,
                                      (float *)ws, (hipStream_t)stream));
}

int mq_gemm_f16cache_xf32(const float *X, int ldx, const uint16_t *W16, int ldw, float *Y,
                          int ldy, int M, int N, int K, void *ws, size_t ws_bytes, int split_k,
                          void *stream) {
    mq::GemmPlan plan;
    XPlan xp;
    if (int rc = check_gemm(mq::kFmtF16, X, ldx, W16, ldw, Y, ldy, M, N, K, ws, ws_bytes,
                            split_k, &plan, true, &xp))
        return rc;
    return run_xf32(mq::kFmtF16, X, ldx, W16, ldw, Y, ldy, M, N, K, ws, xp, (hipStream_t)stream);
}

int mq_gemm_fused_xf32(int fmt, const float *X, int ldx, const void *wq, float *Y, int ldy,
                       int M, int N, int K, void *ws, size_t ws_bytes, int split_k,
                       void *stream) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    mq::GemmPlan plan;
    XPlan xp;
    if (int rc = check_gemm(fmt, X, ldx, wq, 0, Y, ldy, M, N, K, ws, ws_bytes, split_k, &plan,
                            true, &xp))
        return rc;
    const int64_t row_bytes = (int64_t)K / mq::block_elems(fmt) * mq::block_bytes(fmt);
    return run_xf32(fmt, X, ldx, wq, row_bytes, Y, ldy, M, N, K, ws, xp, (hipStream_t)stream);
}

int mq_convert_f32_to_f16(const float *X, int ldx, uint16_t *X16, int ld16, int M, int K,
                          void *stream) {
    if (!X || !X16) return MQ_ERR_NULL;
    if (check_dims(M, 1, K) || K % 8) return MQ_ERR_SHAPE;
    if (!ld32_ok(ldx, K) || !ld_ok(ld16, K)) return MQ_ERR_LD;
    if (!aligned16(X) || !aligned16(X16)) return MQ_ERR_ALIGN;
    return hip_status(mq::launch_convert_f32_to_f16(X, ldx, X16, ld16, M, K, (hipStream_t)stream));
}

int mq_quantize_q8_1(const float *X, int ldx, int8_t *Xq, int ldq, float *ds, int M, int K,
                     void *stream) {
    if (!X || !Xq || !ds) return MQ_ERR_NULL;
    if (check_dims(M, 1, K) || K % 32) return MQ_ERR_SHAPE;
    if (!ld32_ok(ldx, K) || !ldq_ok(ldq, K)) return MQ_ERR_LD;
    if (!aligned16(X) || !aligned16(Xq) || !aligned16(ds)) return MQ_ERR_ALIGN;
    return hip_status(mq::launch_quantize_q8_1(X, ldx, Xq, ldq, ds, M, K, (hipStream_t)stream));
}

int64_t mq_gemm_mmq_workspace_bytes(int fmt, int M, int N, int K, int split_k) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    if (int rc = check_dims(M, N, K)) return rc;
    if (K % mq::block_elems(fmt) || K % 32) return MQ_ERR_SHAPE;
    if (split_k < 0 || split_k > MQ_MAX_SPLIT_K) return MQ_ERR_SPLIT;
    if (split_k > 1 && (int64_t)M * N >= ((int64_t)1 << 31)) return MQ_ERR_SPLIT;
    return mq::plan_mmq(M, N, K, split_k).ws_bytes;
}

int mq_gemm_mmq(int fmt, const int8_t *Xq, int ldq, const float *ds, const void *wq, float *Y,
                int ldy, int M, int N, int K, void *ws, size_t ws_bytes, int split_k,
                void *stream) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    if (!Xq || !ds || !wq || !Y) return MQ_ERR_NULL;
    if (int rc = check_dims(M, N, K)) return rc;
    if (K % mq::block_elems(fmt) || K % 32) return MQ_ERR_SHAPE;
    if (!ldq_ok(ldq, K) || ldy < N) return MQ_ERR_LD;
    if (!aligned16(Xq) || !aligned16(ds) || !aligned16(wq) || !aligned16(Y)) return MQ_ERR_ALIGN;
    if (split_k < 0 || split_k > MQ_MAX_SPLIT_K) return MQ_ERR_SPLIT;
    if (split_k > 1 && (int64_t)M * N >= ((int64_t)1 << 31)) return MQ_ERR_SPLIT;
    const mq::GemmPlan plan = mq::plan_mmq(M, N, K, split_k);
    if (plan.ws_bytes > 0 && (!ws || !aligned16(ws) || ws_bytes < (size_t)plan.ws_bytes))
        return MQ_ERR_WORKSPACE;
    const int64_t row_bytes = (int64_t)K / mq::block_elems(fmt) * mq::block_bytes(fmt);
    return hip_status(mq::launch_mmq(fmt, Xq, ldq, ds, wq, row_bytes, Y, ldy, M, N, K, plan,
                                     (float *)ws, (hipStream_t)stream));
}

int64_t mq_linear_workspace_bytes(int fmt, int x_type, int M, int N, int K, int split_k) {
    return linear_workspace(fmt, x_type, M, N, K, split_k, false);
}

int64_t mq_glu_workspace_bytes(int fmt, int x_type, int M, int N, int K, int split_k) {
    return linear_workspace(fmt, x_type, M, N, K, split_k, true);
}

int mq_linear_f16cache(int x_type, const void *X, int ldx, const uint16_t *W16, int ldw,
                       const float *bias, int act, int r_type, const void *R, int ldr, int y_type,
                       void *Y, int ldy, int M, int N, int K, void *ws, size_t ws_bytes,
                       int split_k, void *stream) {
    const mq::EpiSpec epi{bias, R, ldr, act, r_type, y_type, false};
    return run_linear(mq::kFmtF16, x_type, X, ldx, W16, ldw, y_type, Y, ldy, M, N, K, epi, ws,
                      ws_bytes, split_k, (hipStream_t)stream);
}

int mq_linear_fused(int x_type, const void *X, int ldx, int fmt, const void *wq,
                    const float *bias, int act, int r_type, const void *R, int ldr, int y_type,
                    void *Y, int ldy, int M, int N, int K, void *ws, size_t ws_bytes, int split_k,
                    void *stream) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    const mq::EpiSpec epi{bias, R, ldr, act, r_type, y_type, false};
    return run_linear(fmt, x_type, X, ldx, wq, 0, y_type, Y, ldy, M, N, K, epi, ws, ws_bytes,
                      split_k, (hipStream_t)stream);
}

int mq_glu_f16cache(int x_type, const void *X, int ldx, const uint16_t *W16, int ldw,
                    const float *bias, int act, int y_type, void *Y, int ldy, int M, int N, int K,
                    void *ws, size_t ws_bytes, int split_k, void *stream) {
    const mq::EpiSpec epi{bias, nullptr, 0, act, MQ_F32, y_type, true};
    return run_linear(mq::kFmtF16, x_type, X, ldx, W16, ldw, y_type, Y, ldy, M, N, K, epi, ws,
                      ws_bytes, split_k, (hipStream_t)stream);
}

int mq_glu_fused(int x_type, const void *X, int ldx, int fmt, const void *wq, const float *bias,
                 int act, int y_type, void *Y, int ldy, int M, int N, int K, void *ws,
                 size_t ws_bytes, int split_k, void *stream) {
    if (!quant_fmt(fmt)) return MQ_ERR_FORMAT;
    const mq::EpiSpec epi{bias, nullptr, 0, act, MQ_F32, y_type, true};
    return run_linear(fmt, x_type, X, ldx, wq, 0, y_type, Y, ldy, M, N, K, epi, ws, ws_bytes,
                      split_k, (hipStream_t)stream);
}

int mq_add_rms_norm(int x_type, const void *X, int ldx, int r_type, const void *R, int ldr,
                    const float *w, float eps, void *H, int ldh, int y_type, void *Y, int ldy,
                    int M, int K, void *stream) {
    mq::NormSpec n;
    if (int rc = check_dims(M, 1, K)) return rc;   // an empty tensor's pointers are NULL
    if (!Y) return MQ_ERR_NULL;
    if (!type_ok(y_type)) return MQ_ERR_TYPE;
    if (int rc = check_norm(x_type, X, ldx, r_type, R, ldr, w, eps, H, ldh, M, K, &n)) return rc;
    if (ldy < K) return MQ_ERR_LD;
    if (!elem_aligned(Y, y_type)) return MQ_ERR_ALIGN;
    n.y = Y;
    n.ldy = ldy;
    n.y_type = y_type;
    if (int rc = check_norm_overlap(n, y_type == MQ_F32 ? 4 : 2)) return rc;
    return hip_status(mq::launch_add_rms_norm(n, (hipStream_t)stream));
}

int mq_add_rms_norm_q8_1(int x_type, const void *X, int ldx, int r_type, const void *R, int ldr,
                         const float *w, float eps, void *H, int ldh, int8_t *Xq, int ldq,
                         float *ds, int M, int K, void *stream) {
    mq::NormSpec n;
    if (int rc = check_dims(M, 1, K)) return rc;
    if (!Xq || !ds) return MQ_ERR_NULL;
    if (int rc = check_norm(x_type, X, ldx, r_type, R, ldr, w, eps, H, ldh, M, K, &n)) return rc;
    if (K % 32) return MQ_ERR_SHAPE;
    if (!ldq_ok(ldq, K)) return MQ_ERR_LD;
    if (!aligned16(Xq) || !aligned16(ds)) return MQ_ERR_ALIGN;
    n.y = Xq;
    n.ldy = ldq;
    n.ds = ds;
    n.y_type = mq::kTypeI8;
    if (int rc = check_norm_overlap(n, 1)) return rc;
    return hip_status(mq::launch_add_rms_norm(n, (hipStream_t)stream));
}

int mq_rope(int x_type, const void *X, int ldx, const int32_t *positions, const double *freqs,
            int n_rot, int layout, float mscale, int heads, int head_dim, int y_type, void *Y,
            int ldy, int M, void *stream) {
    if (int rc = check_dims(M, 1, 1)) return rc;
    if (!X || !positions || !freqs || !Y) return MQ_ERR_NULL;
    if (!type_ok(x_type) || !type_ok(y_type)) return MQ_ERR_TYPE;
    if (head_dim <= 0 || head_dim > MQ_MAX_ROPE_DIM || !heads_ok(heads, head_dim))
        return MQ_ERR_SHAPE;
    if (int rc = check_rotation(freqs, n_rot, layout, mscale, head_dim)) return rc;
    const int width = heads * head_dim;
    if (ldx < width || ldy < width) return MQ_ERR_LD;
    if (!elem_aligned(X, x_type) || !elem_aligned(Y, y_type) || (uintptr_t)positions % 4)
        return MQ_ERR_ALIGN;
    const Span x = span(X, ldx, width, type_bytes(x_type), M);
    const Span y = span(Y, ldy, width, type_bytes(y_type), M);
    if ((overlap(y, x) && !same_span(y, x)) || overlap(y, span(positions, M, M, 4, 1)) ||
        overlap(y, span(freqs, n_rot / 2, n_rot / 2, 8, 1)))
        return MQ_ERR_OVERLAP;
    const mq::RopeSpec s{X,    Y,        positions, freqs, ldx,    ldy,    M,
                         heads, head_dim, n_rot,     x_type, y_type, layout == MQ_ROPE_INTERLEAVED,
                         mscale};
    return hip_status(mq::launch_rope(s, (hipStream_t)stream));
}

int64_t mq_kv_q4_page_bytes(int heads, int page, int head_dim) {
    if (heads <= 0 || heads > MQ_MAX_HEADS || page <= 0 || page % 32 || page > mq::kMaxLen ||
        (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 256))
        return MQ_ERR_SHAPE;
    return (int64_t)heads * (page / 32) * 36 * head_dim;
}

int mq_kv_store_q4(const mq_kv_q4 *cache, int x_type, const void *K, int ldk, const void *V, int ldv,
                   const double *freqs, int n_rot, int layout, float mscale,
                   const int32_t *positions, const void *Q, int ldq, int q_heads, int q_type,
                   void *QO, int ldqo, int M, void *stream) {
    mq::KvSpec kv;
    if (int rc = check_kv(cache, M, &kv)) return rc;
    if (!K || !V || (Q && !QO)) return MQ_ERR_NULL;
    if (!type_ok(x_type) || (Q && !type_ok(q_type))) return MQ_ERR_TYPE;
    if (freqs)
        if (int rc = check_rotation(freqs, n_rot, layout, mscale, kv.D)) return rc;
    const int width = kv.heads * kv.D;
    if (!heads_ok(kv.heads, kv.D) || (Q && !heads_ok(q_heads, kv.D))) return MQ_ERR_SHAPE;
    if (ldk < width || ldv < width) return MQ_ERR_LD;
    if (!elem_aligned(K, x_type) || !elem_aligned(V, x_type) || (uintptr_t)positions % 4)
        return MQ_ERR_ALIGN;
    const Span k = span(K, ldk, width, type_bytes(x_type), M);
    const Span v = span(V, ldv, width, type_bytes(x_type), M);
    const Span c = cache_span(kv);
    const int pairs = freqs ? n_rot / 2 : 0;
    auto over_tables = [&](const Span &out) {
        return over_batch(out, kv) || over(out, positions, M, 4) || over(out, freqs, pairs, 8);
    };
    if (overlap(c, k) || overlap(c, v) || over_tables(c)) return MQ_ERR_OVERLAP;
    if (Q) {
        const int qw = q_heads * kv.D;
        if (ldq < qw || ldqo < qw) return MQ_ERR_LD;
        if (!elem_aligned(Q, x_type) || !elem_aligned(QO, q_type)) return MQ_ERR_ALIGN;
        const Span q = span(Q, ldq, qw, type_bytes(x_type), M);
        const Span o = span(QO, ldqo, qw, type_bytes(q_type), M);
        if ((overlap(o, q) && !same_span(o, q)) || overlap(o, k) || overlap(o, v) ||
            overlap(o, c) || overlap(c, q) || over_tables(o))
            return MQ_ERR_OVERLAP;
    }
    const mq::StoreSpec s{K,   V,    Q,      QO,     positions, freqs,
                          ldk, ldv,  ldq,    ldqo,   x_type,    q_type,
                          freqs ? n_rot : 0, q_heads, layout == MQ_ROPE_INTERLEAVED, mscale};
    return hip_status(mq::launch_kv_store(kv, s, (hipStream_t)stream));
}

int mq_kv_load_q4(const mq_kv_q4 *cache, int y_type, void *K, int ldk, void *V, int ldv, int M,
                  void *stream) {
    mq::KvSpec kv;
    if (int rc = check_kv(cache, M, &kv)) return rc;
    if (!K || !V) return MQ_ERR_NULL;
    if (!type_ok(y_type)) return MQ_ERR_TYPE;
    const int width = kv.heads * kv.D;
    if (!heads_ok(kv.heads, kv.D)) return MQ_ERR_SHAPE;
    if (ldk < width || ldv < width) return MQ_ERR_LD;
    if (!elem_aligned(K, y_type) || !elem_aligned(V, y_type)) return MQ_ERR_ALIGN;
    const Span k = span(K, ldk, width, type_bytes(y_type), M);
    const Span v = span(V, ldv, width, type_bytes(y_type), M);
    const Span c = cache_span(kv);
    if (overlap(k, v) || overlap(c, k) || overlap(c, v) || over_batch(k, kv) || over_batch(v, kv))
        return MQ_ERR_OVERLAP;
    return hip_status(mq::launch_kv_load(kv, y_type, K, ldk, V, ldv, (hipStream_t)stream));
}

int64_t mq_attention_q4_workspace_bytes(const mq_kv_q4 *cache, int q_heads, int M,
                                        int64_t max_len) {
    mq::KvSpec kv;
    if (int rc = check_kv(cache, M, &kv)) return rc;
    if (int rc = check_attention(kv, q_heads, max_len)) return rc;
    mq::AttnSpec s{};
    s.q_heads = q_heads;
    s.max_len = max_len;
    const mq::AttnPlan p = mq::plan_attention(kv, s);
    return plan_ok(p) ? p.ws_bytes : MQ_ERR_SHAPE;
}

int mq_attention_q4(const mq_kv_q4 *cache, int x_type, const void *Q, int ldq, int q_heads,
                    uint16_t *Y, int ldy, int M, float scale, int causal, int window, float cap,
                    const float *slopes, const int32_t *prefix, int64_t max_len, void *ws,
                    size_t ws_bytes, void *stream) {
    mq::KvSpec kv;
    if (int rc = check_kv(cache, M, &kv)) return rc;
    if (!Q || !Y) return MQ_ERR_NULL;
    if (!type_ok(x_type)) return MQ_ERR_TYPE;
    if (int rc = check_attention(kv, q_heads, max_len)) return rc;
    if (!(scale > -3.0e38f && scale < 3.0e38f) || !(cap >= 0.0f && cap < 3.0e38f) || window < 0)
        return MQ_ERR_EPS;
    const int width = q_heads * kv.D;
    if (ldq < width || ldy < width) return MQ_ERR_LD;
    if (!elem_aligned(Q, x_type) || !elem_aligned(Y, MQ_F16) || (uintptr_t)slopes % 4 ||
        (uintptr_t)prefix % 4)
        return MQ_ERR_ALIGN;
    const mq::AttnSpec s{Q,   Y,   ldq,         ldy,    x_type, q_heads, scale,
                         cap, causal != 0, window, slopes, prefix,  max_len};
    const mq::AttnPlan p = mq::plan_attention(kv, s);
    if (!plan_ok(p)) return MQ_ERR_SHAPE;
    if (p.ws_bytes > 0 && (!ws || !aligned16(ws) || ws_bytes < (size_t)p.ws_bytes))
        return MQ_ERR_WORKSPACE;
    const Span q = span(Q, ldq, width, type_bytes(x_type), M);
    const Span y = span(Y, ldy, width, 2, M);
    const Span c = cache_span(kv);
    const Span w = span(ws, p.ws_bytes, p.ws_bytes, 1, 1);
    auto over_tables = [&](const Span &out) {
        return over_batch(out, kv) || over(out, slopes, q_heads, 4) || over(out, prefix, kv.batch, 4);
    };
    if (overlap(y, q) || overlap(y, c) || over_tables(y)) return MQ_ERR_OVERLAP;
    if (p.ws_bytes > 0 && (overlap(w, q) || overlap(w, y) || overlap(w, c) || over_tables(w)))
        return MQ_ERR_OVERLAP;
    return hip_status(mq::launch_attention(kv, s, p, (float *)ws, (hipStream_t)stream));
}

int mq_gemm_plan_query(int path, int fmt, int M, int N, int K, int split_k,
                       mq_gemm_plan_info *out) {
    if (!out) return MQ_ERR_NULL;
    if (path < 0 || path > 2) return MQ_ERR_FORMAT;
    const bool mmq = path == 2;
    if (mmq ? !quant_fmt(fmt) : (fmt != mq::kFmtF16 && !quant_fmt(fmt))) return MQ_ERR_FORMAT;
    if (int rc = check_dims(M, N, K)) return rc;
    if (K % (fmt == mq::kFmtF16 ? 8 : mq::block_elems(fmt)) || (mmq && K % 32))
        return MQ_ERR_SHAPE;
    if (split_k < 0 || split_k > MQ_MAX_SPLIT_K) return MQ_ERR_SPLIT;
    if (split_k > 1 && (int64_t)M * N >= ((int64_t)1 << 31)) return MQ_ERR_SPLIT;
    mq::GemmPlan p;
    int64_t x16_bytes = 0;
    bool has_kernel;
    if (mmq) {
        p = mq::plan_mmq(M, N, K, split_k);
        has_kernel = mq::mmq_plan_has_kernel(p);
    } else if (path == 1) {
        const XPlan xp = xf32_plan(fmt, M, N, K, split_k);
        p = xp.gemm;
        x16_bytes = xp.x16_bytes;
        has_kernel = (xp.convert_first
                          ? mq::launch_gemm(fmt, nullptr, 0, nullptr, 0, nullptr, 0, M, N, K, p,
                                            nullptr, nullptr, true)
                          : mq::launch_gemm_xf32(fmt, nullptr, 0, nullptr, 0, nullptr, 0, M, N,
                                                 K, p, nullptr, nullptr, true)) == hipSuccess;
    } else {
        p = mq::plan_gemm(fmt, M, N, K, split_k);
        has_kernel = mq::launch_gemm(fmt, nullptr, 0, nullptr, 0, nullptr, 0, M, N, K, p,
                                     nullptr, nullptr, true) == hipSuccess;
    }
    out->bm = p.bm;
    out->bn = p.bn;
    out->tiles_m = p.tiles_m;
    out->tiles_n = p.tiles_n;
    out->k_steps = p.k_steps;
    out->dp_tiles = p.dp_tiles;
    out->tail_tiles = p.tail_tiles;
    out->split = p.split;
    out->steps_per_split = p.steps_per_split;
    out->has_kernel = has_kernel ? 1 : 0;
    out->ws_bytes = x16_bytes + p.ws_bytes;
    return MQ_OK;
}

const char *mq_strerror(int code) {
    switch (code) {
    case MQ_OK: return "success";
    case MQ_ERR_NULL: return "a required pointer is NULL";
    case MQ_ERR_FORMAT: return "unknown weight format or rotary layout";
    case MQ_ERR_SHAPE: return "a size out of range (M, N, K, heads, pages, batch), or K not a multiple of the block size";
    case MQ_ERR_LD: return "a leading dimension is too small, too large or not a multiple of 8 (4 for f32 rows, 16 for int8 codes)";
    case MQ_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case MQ_ERR_WORKSPACE: return "workspace missing, misaligned or smaller than required";
    case MQ_ERR_SPLIT: return "split_k out of range for this problem";
    case MQ_ERR_HIP: return "the HIP runtime rejected a launch";
    case MQ_ERR_SCRATCH: return "the K-split partial tiles exceed the static scratch (MQ_NOALLOC_SCRATCH_BYTES)";
    case MQ_ERR_TYPE: return "an element type that is not f32 or f16";
    case MQ_ERR_EPS: return "eps, a scale, a cap or a window is negative or not finite";
    case MQ_ERR_OVERLAP: return "an output overlaps another buffer of the call";
    case MQ_ERR_ACT: return "unknown activation";
    default: return "unknown error code";
    }
}

int mq_last_hip_error(void) { return g_last_hip_error; }

}  // extern "C"
