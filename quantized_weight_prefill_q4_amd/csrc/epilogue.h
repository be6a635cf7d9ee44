// The epilogue of a linear layer's product, shared by the tile kernels, the
// K-split reduce and the few-row kernels: bias, activation, residual and the
// output's rounding, applied to the f32 sums.
//
//   linear:  y = act(v + bias) + residual
//   gated:   y = act(g + bias_g) · (u + bias_u), g and u the sums of the gate's
//            and the up matrix's rows
// All in f32, rounded once to the output type.  Bias and residual are read,
// and y written, at their elements' own alignment (odd N and odd strides): 16
// bytes at a time where 8 columns are whole, else element by element.

#pragma once

#include "mq_device.h"
#include "mq_internal.h"

namespace mq {
namespace {

// 16 bytes at the alignment of an f16 / an f32 element.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// e^x to about one unit in the last place: 2^(x·log2 e) with the product's
// rounding error carried into the fraction.  Clamped where the result is 0 or
// infinite anyway, so an infinite x gives e^x's limit; NaN is not kept (the
// activations below multiply by a NaN argument themselves).
__device__ __forceinline__ float exp_f32(float x) {
    constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596303e-8f;
    x = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);
    const float n = __builtin_rintf(x * kLog2e);
    const float f = __builtin_fmaf(x, kLog2eLo, __builtin_fmaf(x, kLog2e, -n));
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}

// v / (1 + e^−t).  silu: t = v; gelu_tanh: t = 2·sqrt(2/π)·(v + 0.044715·v³),
// which is 0.5·v·(1 + tanh(t/2)) without the cancellation at negative v.
__device__ __forceinline__ float gate_f32(float v, float t) {
    return v * __builtin_amdgcn_rcpf(1.0f + exp_f32(-t));
}

// v[0 .. N) = act(v); one uniform branch per call.
template <int N>
__device__ __forceinline__ void apply_act(int act, float (&v)[N]) {
    if (act == kActSilu) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = gate_f32(v[j], v[j]);
    } else if (act == kActGeluTanh) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float p = v[j] * __builtin_fmaf(v[j] * v[j], 0.0713548163f, 1.59576912f);
            v[j] = gate_f32(v[j], p);
        }
    } else if (act == kActGelu) {
        // 0.5·v·erfc(−v/√2), exact to f32 also where 1 + erf cancels
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = 0.5f * v[j] * erfcf(-0.707106781f * v[j]);
    } else if (act == kActRelu) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];   // keeps NaN
    }
}

// v[0 .. n) of n <= 8 consecutive elements of `type` (the rest 0).
__device__ __forceinline__ void load_upto8(const void *row, int type, int64_t col, int n,
                                           float (&v)[8]) {
    if (n >= 8) {
        if (type == kTypeF32) {
            const f32x4_a4 *p = reinterpret_cast<const f32x4_a4 *>((const float *)row + col);
            const f32x4 a = p[0], b = p[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4_a2 *>((const uint16_t *)row + col);
            v[0] = f16_bits_to_f32(a.x); v[1] = f16_bits_to_f32(a.x >> 16);
            v[2] = f16_bits_to_f32(a.y); v[3] = f16_bits_to_f32(a.y >> 16);
            v[4] = f16_bits_to_f32(a.z); v[5] = f16_bits_to_f32(a.z >> 16);
            v[6] = f16_bits_to_f32(a.w); v[7] = f16_bits_to_f32(a.w >> 16);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (j < n)
            v[j] = type == kTypeF32 ? ((const float *)row)[col + j]
                                    : f16_bits_to_f32(((const uint16_t *)row)[col + j]);
    }
}

// The first n <= 8 of v to consecutive elements of `type`, each rounded once.
// The output is not read again by the kernel: whole groups are streamed out
// with non-temporal stores.
__device__ __forceinline__ void store_upto8(void *row, int type, int64_t col, int n,
                                            const float (&v)[8]) {
    if (n >= 8) {
        if (type == kTypeF32) {
            f32x4_a4 *p = reinterpret_cast<f32x4_a4 *>((float *)row + col);
            const f32x4_a4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
            __builtin_nontemporal_store(a, p);
            __builtin_nontemporal_store(b, p + 1);
        } else {
            const u32x4_a2 a = {pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]),
                                pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7])};
            __builtin_nontemporal_store(a, reinterpret_cast<u32x4_a2 *>((uint16_t *)row + col));
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) {
            if (type == kTypeF32)
                ((float *)row)[col + j] = v[j];
            else
                ((uint16_t *)row)[col + j] = (uint16_t)pack_f16x2(v[j], 0.0f);
        }
}

// load_upto8 / store_upto8 for groups of four.
__device__ __forceinline__ void load_upto4(const void *row, int type, int64_t col, int n,
                                           float (&v)[4]) {
    if (n >= 4) {
        if (type == kTypeF32) {
            const f32x4 a = *reinterpret_cast<const f32x4_a4 *>((const float *)row + col);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        } else {
            const u32x2 a = *reinterpret_cast<const u32x2_a2 *>((const uint16_t *)row + col);
            v[0] = f16_bits_to_f32(a.x); v[1] = f16_bits_to_f32(a.x >> 16);
            v[2] = f16_bits_to_f32(a.y); v[3] = f16_bits_to_f32(a.y >> 16);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = 0.0f;
        if (j < n)
            v[j] = type == kTypeF32 ? ((const float *)row)[col + j]
                                    : f16_bits_to_f32(((const uint16_t *)row)[col + j]);
    }
}

__device__ __forceinline__ void store_upto4(void *row, int type, int64_t col, int n,
                                            const float (&v)[4]) {
    if (n >= 4) {
        if (type == kTypeF32)
            *reinterpret_cast<f32x4_a4 *>((float *)row + col) = f32x4{v[0], v[1], v[2], v[3]};
        else
            *reinterpret_cast<u32x2_a2 *>((uint16_t *)row + col) =
                u32x2{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) {
            if (type == kTypeF32)
                ((float *)row)[col + j] = v[j];
            else
                ((uint16_t *)row)[col + j] = (uint16_t)pack_f16x2(v[j], 0.0f);
        }
}

}  // namespace
}  // namespace mq
