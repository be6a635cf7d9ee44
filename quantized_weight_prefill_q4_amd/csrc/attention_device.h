// Device helpers shared by the attention kernels.
#pragma once

#include "attention_view.h"
#include "mq_device.h"

namespace mq {
namespace {

constexpr float kLog2e = 1.44269502f;
constexpr float kShift = 15.0f;       // weights are held times 2^15

// 1 − 2 / (1 + e^2u), and below 1/4, where that cancels, u − u³/3 + 2u⁵/15 − 17u⁷/315
// (the next term is 3e-7 of the value at 1/4).
__device__ __forceinline__ float tanh_f32(float u) {
    const float e = __builtin_amdgcn_exp2f(u * (2.0f * kLog2e));
    const float t = u * u;
    float p = __builtin_fmaf(t, -17.0f / 315.0f, 2.0f / 15.0f);
    p = __builtin_fmaf(t, p, -1.0f / 3.0f);
    p = __builtin_fmaf(t * u, p, u);
    return fabsf(u) < 0.25f ? p : 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e);
}

typedef uint32_t q_u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float q_f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight query elements as f16.
__device__ __forceinline__ half8 load_q8(const void *q, int f32, int64_t at) {
    if (!f32)
        return __builtin_bit_cast(
            half8, (u32x4)*reinterpret_cast<const q_u32x4_a2 *>((const uint16_t *)q + at));
    const q_f32x4_a4 *p = reinterpret_cast<const q_f32x4_a4 *>((const float *)q + at);
    const f32x4 x = p[0], y = p[1];
    return __builtin_bit_cast(half8, u32x4{pack_f16x2(x.x, x.y), pack_f16x2(x.z, x.w),
                                           pack_f16x2(y.x, y.y), pack_f16x2(y.z, y.w)});
}

// The eight (q − 8) of a code dword, exact.  A nibble under the exponent of 1024
// is 1024 + q, one place of four bits higher 1024 + 16·q.
__device__ __forceinline__ void widen(uint32_t w, half2v h[4]) {
    const half2v c = {(_Float16)1032.0f, (_Float16)1032.0f};
    const half2v s = {(_Float16)0.0625f, (_Float16)0.0625f};
    const half2v o = {(_Float16)-72.0f, (_Float16)-72.0f};
    const uint32_t u = w >> 8;
    h[0] = __builtin_bit_cast(half2v, (w & 0x000F000Fu) | 0x64006400u) - c;
    h[1] = __builtin_elementwise_fma(
        __builtin_bit_cast(half2v, (w & 0x00F000F0u) | 0x64006400u), s, o);
    h[2] = __builtin_bit_cast(half2v, (u & 0x000F000Fu) | 0x64006400u) - c;
    h[3] = __builtin_elementwise_fma(
        __builtin_bit_cast(half2v, (u & 0x00F000F0u) | 0x64006400u), s, o);
}

__device__ __forceinline__ half8 join8(const half2v h[4]) {
    return half8{h[0].x, h[0].y, h[1].x, h[1].y, h[2].x, h[2].y, h[3].x, h[3].y};
}

__device__ __forceinline__ half2v as_half2(uint32_t w) { return __builtin_bit_cast(half2v, w); }

// N dwords at the alignment of the widest load that N allows.
template <int N>
__device__ __forceinline__ void load_dwords(const uint32_t *p, uint32_t (&w)[N]) {
    typedef uint32_t v2 __attribute__((ext_vector_type(2)));
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u32x4 x = *(const u32x4 *)(p + i);
            w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const v2 x = *(const v2 *)(p + i);
            w[i] = x.x; w[i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = p[i];
    }
}

// A value that is the same in all lanes, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ void make_uniform(View &v) {
    v.b = uniform(v.b);
    v.rt = uniform(v.rt);
    v.rows.first = uniform(v.rows.first);
    v.rows.n = uniform(v.rows.n);
    v.len = uniform(v.len);
    v.keys = uniform(v.keys);
    v.prefix = uniform(v.prefix);
    v.first_pos = uniform(v.first_pos);
    v.p_min = uniform(v.p_min);
    v.p_max = uniform(v.p_max);
    v.pre = uniform(v.pre);
    v.lo = uniform(v.lo);
    v.n = uniform(v.n);
}

// f16 words whose exponent is all ones (infinities, NaN), as 1.0 / 0.0 each.
__device__ __forceinline__ uint32_t bad_halves(uint32_t w) {
    return ((w & 0x7C00u) == 0x7C00u ? 0x3C00u : 0u) |
           ((w & 0x7C000000u) == 0x7C000000u ? 0x3C000000u : 0u);
}
__device__ __forceinline__ uint32_t keep_halves(uint32_t w, bool lo, bool hi) {
    return (lo ? w & 0xFFFFu : 0u) | (hi ? w & 0xFFFF0000u : 0u);
}

}  // namespace
}  // namespace mq
