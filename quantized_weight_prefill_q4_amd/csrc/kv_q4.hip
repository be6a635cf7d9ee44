// Store into and load from the 4-bit key/value cache (kv_q4.h has its layout).
//
// Store: a sequence's new keys, rotated by their positions, and values become
// blocks of 32 elements: with v the first of the elements of largest magnitude,
//   d = f16(v / −8),   q = clamp(floor(x/d + 8.5), 0, 15)   (8 where d is 0)
// so v itself is code 0 and the range is used whole.  All in f32 (the f16 d
// widened).  A block with an infinity or a NaN, or with |d| > 8188 (an element of 65520 or
// more), gets a NaN as its d: what attention multiplies are f16 numbers d·(q − 8), and f16
// ends at 65504 = 8 · 8188.  The queries of the same rows are rotated by the same launch: a
// single token's layer is launch-bound.
//
// A workgroup takes eight consecutive positions [8u, 8u + 8) of one sequence, the tokens
// that share the values' dwords, of one head or a few: it alone writes them, so neighbours'
// codes in a dword that a call fills in part are merged without atomics.
//
// Both directions move bytes: 1750 rows of f32 (32 query heads, 8 key/value heads of 128)
// in 15 us, 4.3 TB/s.  Few rows wait for three loads and the f64 angles one after the
// other, 5.8 us.
#include "kv_q4.h"
#include "rotary.h"

namespace mq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;   // of a head of 256

struct StoreArgs {
    KvSpec kv;
    const void *k, *v, *q;
    void *qo;
    const int32_t *pos;    // rotary positions of the rows, or null: their places
    const double *freqs;   // null: no rotation
    int64_t ldk, ldv, ldq, ldqo;
    int x_type, qo_type, n_rot, interleaved, q_heads, q_part, in_place;
    float mscale;
    unsigned per_seq;      // units of each sequence (equal rows)
    int kv_part;           // key/value heads of a workgroup
};

// The eight elements [8·oct, + 8) of row x of a head, rotated.
__device__ __forceinline__ void load_rotated(const StoreArgs &a, const void *x, int64_t at, int oct,
                                             const float2 *cs, float v[8]) {
    load_eight(x, a.x_type, at + 8 * oct, v);
    const int e0 = 8 * oct, np = a.n_rot / 2;
    if (!a.freqs || e0 >= 2 * np) return;
    if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            if (e0 + e < 2 * np) {
                const float2 r = cs[(e0 + e) / 2];
                const float p = v[e], q = v[e + 1];
                v[e] = p * r.x - q * r.y;
                v[e + 1] = q * r.x + p * r.y;
            }
        return;
    }
    float w[8];
    const bool whole = (np & 7) == 0;   // the partners are an octet too
    if (whole) load_eight(x, a.x_type, at + (e0 < np ? e0 + np : e0 - np), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = e0 + e;
        if (i >= 2 * np) continue;
        const bool low = i < np;
        const float2 r = cs[low ? i : i - np];
        const float o = whole ? w[e] : load_elem(x, a.x_type, at + (low ? i + np : i - np));
        v[e] = low ? v[e] * r.x - o * r.y : v[e] * r.x + o * r.y;
    }
}

// Codes of eight of a block's elements (its four threads are lanes 4i .. 4i + 3)
// and the block's d.
__device__ __forceinline__ uint16_t quantize_q4(const float v[8], int q[8]) {
    float a = -1.0f, top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float m = fabsf(v[e]);
        bad = bad || !(m < __builtin_inff());
        if (m > a) {
            a = m;
            top = v[e];
        }
    }
    int any = bad;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const float a2 = __shfl_xor(a, o), t2 = __shfl_xor(top, o);
        any |= __shfl_xor(any, o);
        // the lower lane holds the lower elements: it wins a tie
        const bool take = (threadIdx.x & o) ? a2 >= a : a2 > a;
        a = take ? a2 : a;
        top = take ? t2 : top;
    }
    uint16_t bits = (uint16_t)pack_f16x2(top / -8.0f, 0.0f);
    const float d = f16_bits_to_f32(bits);
    if (any || !(fabsf(d) <= kMostScale)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = 8;
        return 0x7E00;
    }
    // x/d from the correctly rounded 1/d, one residual exact by fma: correctly rounded too
    // (Markstein), in three instructions where a division is eleven.  (A quotient so small
    // that the residual underflows gives 8 either way.)
    const float inv = d == 0.0f ? 0.0f : 1.0f / d;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = v[e] * inv;
        const float t = floorf(__builtin_fmaf(__builtin_fmaf(-x, d, v[e]), inv, x) + 8.5f);
        q[e] = (int)fminf(fmaxf(t, 0.0f), 15.0f);
    }
    return d == 0.0f ? 0 : bits;
}

__global__ __launch_bounds__(kThreads) void kv_store_kernel(StoreArgs a) {
    __shared__ float2 cs[8][kMaxPairs];
    __shared__ uint8_t codes[8][256];
    const KvSpec &kv = a.kv;
    const int D = kv.D, NS = D / 32, octs = D / 8;
    Octet o;
    if (!find_octet(kv, blockIdx.x, a.per_seq, o)) return;
    const int p0 = o.p0, e_lo = o.e_lo, e_hi = o.e_hi;
    const int64_t row0 = o.row0;
    const int np = a.freqs ? a.n_rot / 2 : 0;
    for (int i = threadIdx.x; i < 8 * np; i += kThreads) {
        const int e = i / np, j = i - e * np;
        if (e >= e_lo && e < e_hi)
            cs[e][j] = rotation(a.pos ? a.pos[row0 + e] : p0 + e, a.freqs[j], a.mscale);
    }
    __syncthreads();
    const int kv_blocks = (kv.heads + a.kv_part - 1) / a.kv_part;
    if ((int)blockIdx.y >= kv_blocks) {   // queries
        const HeadItems h = head_items(D, a.freqs ? a.n_rot : 0, a.in_place);
        const int per_head = h.rot + h.copy;
        const int h0 = ((int)blockIdx.y - kv_blocks) * a.q_part;
        const int heads = a.q_heads - h0 < a.q_part ? a.q_heads - h0 : a.q_part;
        const int per_row = per_head * heads;
        for (int i = threadIdx.x; i < (e_hi - e_lo) * per_row; i += kThreads) {
            const int e = i / per_row, k = i - e * per_row;
            const int head = k / per_head, item = k - head * per_head;
            const int64_t row = row0 + e_lo + e, at = (int64_t)(h0 + head) * D;
            rotate_item(item, h, D, a.interleaved, cs[e_lo + e], a.q, a.x_type, row * a.ldq + at,
                        a.qo, a.qo_type, row * a.ldqo + at);
        }
        return;
    }
    const int hi = o.keys - p0 < e_hi ? o.keys - p0 : e_hi;   // beyond the table: no place
    char *tile = p0 < o.keys ? kv_tile(kv, o.b, 0, p0 / kTile) : nullptr;
    if (!tile) return;
    const int t0 = p0 & (kTile - 1);
    const int y0 = blockIdx.y * a.kv_part, y1 = y0 + a.kv_part < kv.heads ? y0 + a.kv_part : kv.heads;
    const int64_t head_bytes = (int64_t)(kv.page / kTile) * kv_tile_bytes(D);
    tile += y0 * head_bytes;
    for (int y = y0; y < y1; ++y, tile += head_bytes) {
        if (y > y0) __syncthreads();   // codes are read
        for (int i = threadIdx.x; i < 16 * octs; i += kThreads) {
            const bool value = i >= 8 * octs;
            const int k = value ? i - 8 * octs : i;
            const int e = k / octs, oct = k - e * octs;
            if (e < e_lo || e >= hi) continue;   // the block's four threads together
            const int64_t row = row0 + e;
            float x[8];
            if (value)
                load_eight(a.v, a.x_type, row * a.ldv + (int64_t)y * D + 8 * oct, x);
            else
                load_rotated(a, a.k, row * a.ldk + (int64_t)y * D, oct, cs[e], x);
            int q[8];
            const uint16_t d = quantize_q4(x, q);
            if (value) {
#pragma unroll
                for (int j = 0; j < 8; ++j) codes[e][8 * oct + j] = (uint8_t)q[j];
                if ((oct & 3) == 0)
                    ((uint16_t *)(tile + kv_vscale_at(D)))[((t0 >> 3) * NS + (oct >> 2)) * 8 + e] = d;
            } else {
                uint32_t w = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) w |= (uint32_t)q[j] << kv_shift(j);
                ((uint32_t *)tile)[kv_key_dword(t0 + e, oct, NS)] = w;
                if ((oct & 3) == 0)
                    ((uint16_t *)(tile + kv_kscale_at(D)))[kv_key_place(t0 + e) * NS + (oct >> 2)] = d;
            }
        }
        __syncthreads();
        uint32_t *vc = (uint32_t *)(tile + kv_vcode_at(D)) + (t0 >> 3) * D;
        for (int d = threadIdx.x; d < D; d += kThreads) {
            uint32_t w = e_lo == 0 && hi == 8 ? 0 : vc[d];
            for (int e = e_lo; e < hi; ++e)
                w = (w & ~(15u << kv_shift(e))) | ((uint32_t)codes[e][d] << kv_shift(e));
            vc[d] = w;
        }
    }
}

struct LoadArgs {
    KvSpec kv;
    void *k, *v;
    int64_t ldk, ldv;
    unsigned per_seq;
    int y_type;
};

__global__ __launch_bounds__(kThreads) void kv_load_kernel(LoadArgs a) {
    const KvSpec &kv = a.kv;
    const int D = kv.D, NS = D / 32, octs = D / 8;
    Octet o;
    if (!find_octet(kv, blockIdx.x, a.per_seq, o)) return;
    const int y = blockIdx.y;
    char *tile = o.p0 < o.keys ? kv_tile(kv, o.b, y, o.p0 / kTile) : nullptr;
    const int t0 = o.p0 & (kTile - 1);
    for (int i = threadIdx.x; i < 16 * octs; i += kThreads) {
        const bool value = i >= 8 * octs;
        const int k = value ? i - 8 * octs : i;
        const int e = k / octs, oct = k - e * octs;
        if (e < o.e_lo || e >= o.e_hi) continue;
        const int64_t row = o.row0 + e;
        float x[8];
        if (!tile || o.p0 + e >= o.keys) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
        } else if (value) {
            const float d = f16_bits_to_f32(
                ((const uint16_t *)(tile + kv_vscale_at(D)))[((t0 >> 3) * NS + (oct >> 2)) * 8 + e]);
            const u32x4 *w =
                (const u32x4 *)((const uint32_t *)(tile + kv_vcode_at(D)) + (t0 >> 3) * D + 8 * oct);
            const u32x4 w0 = w[0], w1 = w[1];
            const uint32_t ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = d * (float)((int)((ws[j] >> kv_shift(e)) & 15) - 8);
        } else {
            const float d = f16_bits_to_f32(
                ((const uint16_t *)(tile + kv_kscale_at(D)))[kv_key_place(t0 + e) * NS + (oct >> 2)]);
            const uint32_t w = ((const uint32_t *)tile)[kv_key_dword(t0 + e, oct, NS)];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = d * (float)((int)((w >> kv_shift(j)) & 15) - 8);
        }
        store_eight(value ? a.v : a.k, a.y_type,
                    row * (value ? a.ldv : a.ldk) + (int64_t)y * D + 8 * oct, x);
    }
}

}  // namespace

hipError_t launch_kv_store(const KvSpec &kv, const StoreSpec &s, hipStream_t stream) {
    StoreArgs a;
    a.kv = kv;
    a.k = s.k;
    a.v = s.v;
    a.q = s.q;
    a.qo = s.qo;
    a.pos = s.pos;
    a.freqs = s.freqs;
    a.ldk = s.ldk;
    a.ldv = s.ldv;
    a.ldq = s.ldq;
    a.ldqo = s.ldqo;
    a.x_type = s.x_type;
    a.qo_type = s.qo_type;
    a.n_rot = s.n_rot;
    a.interleaved = s.interleaved;
    a.mscale = s.mscale;
    a.q_heads = s.q ? s.q_heads : 0;
    a.in_place = s.q == s.qo;
    a.per_seq = units_per_seq(kv);
    // query heads of a workgroup: enough work for its threads
    a.q_part = 8;
    const int q_blocks = (a.q_heads + a.q_part - 1) / a.q_part;
    // key/value heads of a workgroup: the look-up and the angles are then made once for
    // them (1750 rows of 8 heads, keys, values and queries and the load behind: 23.6 us with
    // one, 21.0 with two, 22.7 with four; 131072 rows 352, 287, 258 without queries)
    const int64_t work = total_units(kv) * kv.heads;
    a.kv_part = work < 1500 ? 1 : work < 4096 ? 2 : 4;
    const int kv_blocks = (kv.heads + a.kv_part - 1) / a.kv_part;
    const dim3 grid((unsigned)total_units(kv), (unsigned)(kv_blocks + q_blocks));
    hipLaunchKernelGGL(kv_store_kernel, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_kv_load(const KvSpec &kv, int y_type, void *K, int64_t ldk, void *V, int64_t ldv,
                          hipStream_t stream) {
    LoadArgs a;
    a.kv = kv;
    a.k = K;
    a.v = V;
    a.ldk = ldk;
    a.ldv = ldv;
    a.per_seq = units_per_seq(kv);
    a.y_type = y_type;
    const dim3 grid((unsigned)total_units(kv), (unsigned)kv.heads);
    hipLaunchKernelGGL(kv_load_kernel, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mq
