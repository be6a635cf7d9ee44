// The epilogue of a linear layer's product, shared by the tile kernels, the
// K-split reduce and the few-row kernels: bias, activation, residual and the
// output's rounding, applied to the f32 sums.
//
//   linear:  y = act(v + bias) + residual
//   gated:   y = act(g + bias_g) · (u + bias_u), g and u the sums of the gate's
//            and the up matrix's rows
// All in f32, rounded once to the output type.  Bias and residual are read,
// and y written, at their elements' own alignment (odd N and odd strides): 16
// bytes at a time where 4 or 8 columns are whole, else element by element.

#pragma once

#include "mq_device.h"
#include "mq_internal.h"

namespace mq {
namespace {

// 16 bytes at the alignment of an f16 / an f32 element.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// v / (1 + e^−t).  silu: t = v; gelu_tanh: t = 2·sqrt(2/π)·(v + 0.044715·v³),
// which is 0.5·v·(1 + tanh(t/2)) without the cancellation at negative v.  e^−t
// is 2^(−t·log2 e): the product's rounding costs |t|·2^-24 of it, which only
// shows where the result is itself e^−|t| small.  An infinite e^−t gives 0 (or
// NaN for an infinite v), as the formula does.
__device__ __forceinline__ float gate_f32(float v, float t) {
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269502f * t));
}

// 0.5·v·(1 + erf(v/√2)) without the cancellation at negative v: with
// z = |v|/√2, 0.5·erfc(z) = e^(−v²/2) · h(z) and h = 0.5·e^(z²)·erfc(z), a
// smooth function that falls from 0.5 to about 0.06 at z = 4.7.  h is a
// polynomial of degree 10 in t = (z − 3)/(z + 3), fitted to the function by
// iteratively reweighted least squares for the smallest relative error (1.2e-8
// with its coefficients rounded to f32; evaluated in f32 with an exact division
// 3.5·2^-24).  A third of the instructions of erfcf.
__device__ __forceinline__ float gelu_f32(float v) {
    const float z = fminf(0.707106781f * fabsf(v), 16.0f);   // beyond, e^(−v²/2) is 0
    const float t = (z - 3.0f) * __builtin_amdgcn_rcpf(z + 3.0f);
    float h = 2.7769003e-05f;
    h = __builtin_fmaf(h, t, 1.39897702e-05f);
    h = __builtin_fmaf(h, t, -2.97506282e-04f);
    h = __builtin_fmaf(h, t, 3.58054851e-04f);
    h = __builtin_fmaf(h, t, 2.13459646e-03f);
    h = __builtin_fmaf(h, t, -1.21971341e-02f);
    h = __builtin_fmaf(h, t, 3.58329043e-02f);
    h = __builtin_fmaf(h, t, -7.50578940e-02f);
    h = __builtin_fmaf(h, t, 1.22801900e-01f);
    h = __builtin_fmaf(h, t, -1.63116783e-01f);
    h = __builtin_fmaf(h, t, 8.95005763e-02f);
    const float e = h * __builtin_amdgcn_exp2f(-0.721347520f * (v * v));
    return v * (v < 0.0f ? e : 1.0f - e);
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
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = gelu_f32(v[j]);
    } else if (act == kActRelu) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = v[j] < 0.0f ? 0.0f : v[j];   // keeps NaN
    }
}

// Eight f16 outputs as one 16-byte store, each rounded once.  Outputs are not
// read again by the kernel: whole groups are streamed out with non-temporal
// stores.
__device__ __forceinline__ void store8_f16(void *row, int64_t col, const float (&v)[8]) {
    const u32x4_a2 a = {pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                        pack_f16x2(v[6], v[7])};
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4_a2 *>((uint16_t *)row + col));
}

// v[0 .. n) of n <= 4 consecutive elements of `type` (the rest 0), and the
// first n <= 4 of v to consecutive elements, each rounded once (n <= 0: none).
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
        if (type == kTypeF32) {
            const f32x4_a4 a = {v[0], v[1], v[2], v[3]};
            __builtin_nontemporal_store(a, reinterpret_cast<f32x4_a4 *>((float *)row + col));
        } else {
            const u32x2_a2 a = {pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
            __builtin_nontemporal_store(a, reinterpret_cast<u32x2_a2 *>((uint16_t *)row + col));
        }
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
