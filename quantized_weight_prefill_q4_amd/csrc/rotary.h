// Rotary positions: the angle of a pair, its cosine and sine, and the rotation.
//
// Pair j of a head turns by a = fl64(position · f_j), f_j in f64.  A position of
// 10^6 times a frequency of 1 leaves an f32 angle 0.06 off, so the angle is
// formed and reduced in f64, which this chip does at the f32 rate: a − k·π/2 with
// π/2 in two parts (k·hi by one fma is exact to 2^-53 of the remainder), then the
// Taylor sums of sine and cosine on [−π/4, π/4], cut where the next term is
// below 1e-13.  cos and sin are multiplied by the magnitude in f64 and rounded
// once to f32; x0·c − x1·s and x1·c + x0·s are f32, each operation rounded.
#pragma once

#include "mq_device.h"
#include "mq_internal.h"

namespace mq {
namespace {

__device__ __forceinline__ float2 rotation(int position, double freq, float mscale) {
    const double a = (double)position * freq;
    const double k = rint(a * 0.63661977236758134308);
    double r = fma(-k, 1.5707963267948965580, a);
    r = fma(-k, 6.1232339957367660359e-17, r);
    const double t = r * r;
    double s = fma(t, 1.0 / 6227020800.0, -1.0 / 39916800.0);
    s = fma(t, s, 1.0 / 362880.0);
    s = fma(t, s, -1.0 / 5040.0);
    s = fma(t, s, 1.0 / 120.0);
    s = fma(t, s, -1.0 / 6.0);
    s = fma(t * r, s, r);
    double c = fma(t, -1.0 / 87178291200.0, 1.0 / 479001600.0);
    c = fma(t, c, -1.0 / 3628800.0);
    c = fma(t, c, 1.0 / 40320.0);
    c = fma(t, c, -1.0 / 720.0);
    c = fma(t, c, 1.0 / 24.0);
    c = fma(t, c, -0.5);
    c = fma(t, c, 1.0);
    const int q = (int)fma(-4.0, floor(k * 0.25), k);   // k mod 4
    const double cq = q & 1 ? s : c, sq = q & 1 ? c : s;
    float2 cs;
    cs.x = (float)(((q + 1) & 2 ? -cq : cq) * (double)mscale);
    cs.y = (float)((q & 2 ? -sq : sq) * (double)mscale);
    return cs;
}

__device__ __forceinline__ float load_elem(const void *p, int type, int64_t i) {
    return type == kTypeF32 ? ((const float *)p)[i] : f16_bits_to_f32(((const uint16_t *)p)[i]);
}
__device__ __forceinline__ void store_elem(void *p, int type, int64_t i, float v) {
    if (type == kTypeF32)
        ((float *)p)[i] = v;
    else
        ((uint16_t *)p)[i] = (uint16_t)pack_f16x2(v, 0.0f);
}

typedef uint32_t rot_u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float rot_f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void load_eight(const void *p, int type, int64_t i, float v[8]) {
    if (type == kTypeF32) {
        const rot_f32x4_a4 *q = reinterpret_cast<const rot_f32x4_a4 *>((const float *)p + i);
        const f32x4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const u32x4 a = *reinterpret_cast<const rot_u32x4_a2 *>((const uint16_t *)p + i);
        v[0] = f16_bits_to_f32(a.x); v[1] = f16_bits_to_f32(a.x >> 16);
        v[2] = f16_bits_to_f32(a.y); v[3] = f16_bits_to_f32(a.y >> 16);
        v[4] = f16_bits_to_f32(a.z); v[5] = f16_bits_to_f32(a.z >> 16);
        v[6] = f16_bits_to_f32(a.w); v[7] = f16_bits_to_f32(a.w >> 16);
    }
}
__device__ __forceinline__ void store_eight(void *p, int type, int64_t i, const float v[8]) {
    if (type == kTypeF32) {
        rot_f32x4_a4 *q = reinterpret_cast<rot_f32x4_a4 *>((float *)p + i);
        q[0] = f32x4{v[0], v[1], v[2], v[3]};
        q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *reinterpret_cast<rot_u32x4_a2 *>((uint16_t *)p + i) =
            u32x4{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                  pack_f16x2(v[6], v[7])};
    }
}

// The work of one head in items of 16 elements: its pairs eight at a time, then
// the elements behind them (copied; an in-place call has none of those).
struct HeadItems {
    int np;          // pairs
    int rot, copy;   // items of each kind
};
__device__ __host__ __forceinline__ HeadItems head_items(int head_dim, int n_rot, bool in_place) {
    const int np = n_rot / 2;
    return HeadItems{np, (np + 7) / 8, in_place ? 0 : (head_dim - n_rot + 15) / 16};
}

// One item of the head whose first element is x[xi] and y[yi] (which may be the
// same head); the pairs are (j, j + np), or (2j, 2j + 1) when interleaved, and
// cs their rotations.
__device__ __forceinline__ void rotate_item(int item, const HeadItems &h, int head_dim,
                                            bool interleaved, const float2 *cs, const void *x,
                                            int xt, int64_t xi, void *y, int yt, int64_t yi) {
    if (item < h.rot) {
        const int j0 = 8 * item;
        const int a = interleaved ? 2 * j0 : j0, b = interleaved ? 2 * j0 + 8 : h.np + j0;
        float u[8], v[8];
        if (j0 + 8 <= h.np) {
            load_eight(x, xt, xi + a, u);
            load_eight(x, xt, xi + b, v);
            if (interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float(&w)[8] = e < 4 ? u : v;
                    const int k = 2 * (e & 3);
                    const float2 r = cs[j0 + e];
                    const float p = w[k], q = w[k + 1];
                    w[k] = p * r.x - q * r.y;
                    w[k + 1] = q * r.x + p * r.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 r = cs[j0 + e];
                    const float p = u[e], q = v[e];
                    u[e] = p * r.x - q * r.y;
                    v[e] = q * r.x + p * r.y;
                }
            }
            store_eight(y, yt, yi + a, u);
            store_eight(y, yt, yi + b, v);
            return;
        }
        for (int j = j0; j < h.np; ++j) {
            const int p0 = interleaved ? 2 * j : j, p1 = interleaved ? 2 * j + 1 : h.np + j;
            const float p = load_elem(x, xt, xi + p0), q = load_elem(x, xt, xi + p1);
            const float2 r = cs[j];
            store_elem(y, yt, yi + p0, p * r.x - q * r.y);
            store_elem(y, yt, yi + p1, q * r.x + p * r.y);
        }
        return;
    }
    const int e0 = 2 * h.np + 16 * (item - h.rot);
    if (e0 + 16 <= head_dim) {
        float u[8];
        load_eight(x, xt, xi + e0, u);
        store_eight(y, yt, yi + e0, u);
        load_eight(x, xt, xi + e0 + 8, u);
        store_eight(y, yt, yi + e0 + 8, u);
        return;
    }
    for (int e = e0; e < head_dim; ++e) store_elem(y, yt, yi + e, load_elem(x, xt, xi + e));
}

}  // namespace
}  // namespace mq
