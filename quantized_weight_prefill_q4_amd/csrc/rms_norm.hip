// Residual addition and root-mean-square norm of activation rows, with the
// output in the type the next product reads: f16 (the f16-cache and fused
// GEMMs), f32, or the Q8_1-style int8 blocks of the int8 product.
//
// Per row of K elements, everything in f32:
//   h = x + r                     (an f32 sum, rounded to r's type and written; without
//                                  r, h = x)
//   y = (h · 1/sqrt(Σh²/K + eps)) · w
//   f16 / f32 output: y rounded once; Q8_1 output: per 32-element block the
//   codes and (d, s) that mq_quantize_q8_1 gives for the f32 y, bit for bit
//   (same arithmetic, quantize8 in mq_device.h).
//
// The operator moves bytes: at K = 3584 with f32 x, residual and sum and f16
// y it is 14 bytes against about 6 operations per element.  So each row is
// read once and stays in registers between the sum of squares and the output:
// T threads own a row, each C chunks of 8 consecutive elements (two 16-byte
// f32 loads, or one f16 one).  Rows longer than 32768 elements do not fit the
// registers of a workgroup and are read again for the output, from the sum
// that the same thread wrote (or x).  Rows need no alignment: 16-byte
// accesses at the element's own alignment; only a last chunk of fewer than 8
// elements goes element by element.
// Measured: 2048 x 3584 (f32 in, f16 or Q8_1 out) 20.7 us = 4.96 TB/s, 2048 x
// 8192 41.7 us = 5.6 TB/s (a plain device copy: 4.9), 4099 x 1001 f16 at an odd
// stride 9.9 us = 3.3 TB/s (one short row per two waves: latency), one row of
// 3584 2.8 us (2.5 in a kernel trace), the least a kernel of one round trip takes.

#include "mq_device.h"
#include "mq_internal.h"

namespace mq {
namespace {

// 16 bytes at the alignment of an f16 / an f32 element.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

struct NormArgs {
    const void *x, *r;
    const float *w;
    void *h, *y;
    float *ds;
    int64_t ldx, ldr, ldh, ldy;
    int M, K;
    int x_type, r_type, y_type;   // kTypeF32 / kTypeF16; y also kTypeI8 (Q8_1 blocks)
    float eps;
};

__device__ __forceinline__ float half_lo(uint32_t w) { return f16_bits_to_f32(w); }
__device__ __forceinline__ float half_hi(uint32_t w) { return f16_bits_to_f32(w >> 16); }

// Elements [8c, 8c + 8) of a row of `type`, elements at or past K as zeros.
__device__ __forceinline__ void load8(const void *row, int type, int c, int K, float v[8]) {
    const int e = 8 * c;
    if (e + 8 <= K) {
        if (type == kTypeF32) {
            const f32x4_a4 *p = reinterpret_cast<const f32x4_a4 *>((const float *)row + e);
            const f32x4 a = p[0], b = p[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4_a2 *>((const uint16_t *)row + e);
            v[0] = half_lo(a.x); v[1] = half_hi(a.x); v[2] = half_lo(a.y); v[3] = half_hi(a.y);
            v[4] = half_lo(a.z); v[5] = half_hi(a.z); v[6] = half_lo(a.w); v[7] = half_hi(a.w);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (e + j < K)
            v[j] = type == kTypeF32 ? ((const float *)row)[e + j]
                                    : f16_bits_to_f32(((const uint16_t *)row)[e + j]);
    }
}

__device__ __forceinline__ void store8(void *row, int type, int c, int K, const float v[8]) {
    const int e = 8 * c;
    if (e + 8 <= K) {
        if (type == kTypeF32) {
            f32x4_a4 *p = reinterpret_cast<f32x4_a4 *>((float *)row + e);
            p[0] = f32x4{v[0], v[1], v[2], v[3]};
            p[1] = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            *reinterpret_cast<u32x4_a2 *>((uint16_t *)row + e) =
                u32x4{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                      pack_f16x2(v[6], v[7])};
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (e + j < K) {
            if (type == kTypeF32)
                ((float *)row)[e + j] = v[j];
            else
                ((uint16_t *)row)[e + j] = (uint16_t)pack_f16x2(v[j], 0.0f);
        }
}

__device__ __forceinline__ int64_t elem_bytes(int type) { return type == kTypeF32 ? 4 : 2; }

// Sum over the T threads of a row group (T a power of two: part of a wave, or
// whole waves).
template <int T>
__device__ __forceinline__ float group_sum(float s, float *lds) {
#pragma unroll
    for (int o = T < 64 ? T / 2 : 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if constexpr (T > 64) {
        const int wave = threadIdx.x >> 6, first = wave & ~(T / 64 - 1);
        if ((threadIdx.x & 63) == 0) lds[wave] = s;
        __syncthreads();
        s = lds[first];
#pragma unroll
        for (int i = 1; i < T / 64; ++i) s += lds[first + i];
    }
    return s;
}

// x and r of one chunk summed into h (rounded to r's type, which is what is
// written and normed).
__device__ __forceinline__ void add_round(const NormArgs &a, const float r[8], float h[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        h[j] += r[j];
        if (a.r_type == kTypeF16) h[j] = (float)(_Float16)as_f32(h[j]);
    }
}

// y of one chunk from its h, written in the output type.  For Q8_1 the four
// lanes of a block call this together (K is a multiple of 32).
__device__ __forceinline__ void finish8(const NormArgs &a, int64_t row, int c, float inv,
                                        const float h[8]) {
    float w[8], y[8];
    load8(a.w, kTypeF32, c, a.K, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = (h[j] * inv) * w[j];
    if (a.y_type != kTypeI8) {
        store8((char *)a.y + row * a.ldy * elem_bytes(a.y_type), a.y_type, c, a.K, y);
        return;
    }
    uint2 codes;
    float2 ds;
    quantize8(y, codes, ds);
    *reinterpret_cast<uint2 *>((int8_t *)a.y + row * a.ldy + 8 * c) = codes;
    if ((c & 3) == 0) *reinterpret_cast<float2 *>(a.ds + 2 * (row * (a.K / 32) + (c >> 2))) = ds;
}

// T threads per row, C chunks of 8 elements each (chunk t + T·i); TB threads
// per workgroup.  Every chunk's loads are issued before the first use.
template <int T, int C, int TB>
__global__ __launch_bounds__(TB) void add_rms_norm_kernel(NormArgs a) {
    __shared__ float lds[TB / 64];
    const int t = threadIdx.x & (T - 1);
    const int64_t row = (int64_t)blockIdx.x * (TB / T) + threadIdx.x / T;
    const int chunks = row < a.M ? (a.K + 7) >> 3 : 0;   // a row past M owns nothing
    const char *xr = (const char *)a.x + row * a.ldx * elem_bytes(a.x_type);
    float h[C][8];
    auto all = [&](auto &&f) {
#pragma unroll
        for (int i = 0; i < C; ++i) f(i, t + T * i);
    };
    if (a.x_type == kTypeF32)
        all([&](int i, int c) { load8(xr, kTypeF32, c, c < chunks ? a.K : 0, h[i]); });
    else
        all([&](int i, int c) { load8(xr, kTypeF16, c, c < chunks ? a.K : 0, h[i]); });
    if (a.r) {
        const char *rr = (const char *)a.r + row * a.ldr * elem_bytes(a.r_type);
        char *hr = (char *)a.h + row * a.ldh * elem_bytes(a.r_type);
        float r[C][8];
        if (a.r_type == kTypeF32)
            all([&](int i, int c) { load8(rr, kTypeF32, c, c < chunks ? a.K : 0, r[i]); });
        else
            all([&](int i, int c) { load8(rr, kTypeF16, c, c < chunks ? a.K : 0, r[i]); });
        all([&](int i, int c) {
            add_round(a, r[i], h[i]);
            if (c < chunks) store8(hr, a.r_type, c, a.K, h[i]);
        });
    }
    float s = 0.0f;
    all([&](int i, int) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(h[i][j], h[i][j], s);
    });
    s = group_sum<T>(s, lds);
    const float inv = 1.0f / sqrtf(s / (float)a.K + a.eps);
    all([&](int i, int c) {
        if (c < chunks) finish8(a, row, c, inv, h[i]);
    });
}

// Rows too long for the registers: one workgroup of T threads per row, the
// row read twice.
template <int T>
__global__ __launch_bounds__(T) void add_rms_norm_long_kernel(NormArgs a) {
    __shared__ float lds[T / 64];
    const int64_t row = blockIdx.x;
    const int chunks = (a.K + 7) >> 3;
    const char *xr = (const char *)a.x + row * a.ldx * elem_bytes(a.x_type);
    const char *rr = (const char *)a.r + row * a.ldr * elem_bytes(a.r_type);
    char *hr = (char *)a.h + row * a.ldh * elem_bytes(a.r_type);
    float s = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += T) {
        float h[8];
        load8(xr, a.x_type, c, a.K, h);
        if (a.r) {
            float r[8];
            load8(rr, a.r_type, c, a.K, r);
            add_round(a, r, h);
            store8(hr, a.r_type, c, a.K, h);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(h[j], h[j], s);
    }
    s = group_sum<T>(s, lds);
    const float inv = 1.0f / sqrtf(s / (float)a.K + a.eps);
    for (int c = threadIdx.x; c < chunks; c += T) {
        float h[8];   // this thread's own chunk: of the sum it wrote above, or of x
        if (a.r)
            load8(hr, a.r_type, c, a.K, h);
        else
            load8(xr, a.x_type, c, a.K, h);
        finish8(a, row, c, inv, h);
    }
}

template <int T, int C, int TB>
hipError_t launch_rows(const NormArgs &a, hipStream_t stream) {
    const int rows = TB / T;
    hipLaunchKernelGGL((add_rms_norm_kernel<T, C, TB>), dim3((a.M + rows - 1) / rows), dim3(TB), 0,
                       stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rms_norm(const NormSpec &n, hipStream_t stream) {
    NormArgs a;
    a.x = n.x;
    a.r = n.r;
    a.w = n.w;
    a.h = n.h;
    a.y = n.y;
    a.ds = n.ds;
    a.ldx = n.ldx;
    a.ldr = n.ldr;
    a.ldh = n.ldh;
    a.ldy = n.ldy;
    a.M = n.M;
    a.K = n.K;
    a.x_type = n.x_type;
    a.r_type = n.r_type;
    a.y_type = n.y_type;
    a.eps = n.eps;
    // One chunk per thread, T the power of two that covers the row: for one row,
    // fewer threads leave too few loads in flight (1 x 3584, f32 in, f16 out: 512
    // threads 2.8 us, 256 of 2 chunks 3.5, 64 of 8 chunks 6.6); for many, more
    // stand idle (16384 x 128 f32: 16 threads 7.7 us, 64 11.0; 4099 x 1001 f16:
    // 128 threads 9.9, 256 11.5).  With enough rows to fill the chip, two chunks
    // per thread save half the cross-wave sums: taken from 257 chunks on (2048 x
    // 3584: 20.7 us against 21.5 with 512 threads of one), where they gain 4 %;
    // below, the gain is 2 to 3 % (4099 x 1001, 64 threads of two against 128 of
    // one: f16 9.6 / 9.9, f32 13.9 / 14.2) and one chunk serves both.
    const int chunks = (n.K + 7) / 8;
    if (chunks <= 16) return launch_rows<16, 1, 256>(a, stream);
    if (chunks <= 32) return launch_rows<32, 1, 256>(a, stream);
    if (chunks <= 64) return launch_rows<64, 1, 256>(a, stream);
    if (chunks <= 128) return launch_rows<128, 1, 256>(a, stream);
    if (chunks <= 256) return launch_rows<256, 1, 256>(a, stream);
    if (chunks <= 512 && n.M >= 1024) return launch_rows<256, 2, 256>(a, stream);
    if (chunks <= 512) return launch_rows<512, 1, 512>(a, stream);
    if (chunks <= 1024) return launch_rows<1024, 1, 1024>(a, stream);
    if (chunks <= 2048) return launch_rows<1024, 2, 1024>(a, stream);
    if (chunks <= 4096) return launch_rows<1024, 4, 1024>(a, stream);
    hipLaunchKernelGGL((add_rms_norm_long_kernel<1024>), dim3(n.M), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mq
