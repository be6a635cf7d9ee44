// Device helpers shared by the attention kernels.
#pragma once

#include "attention_view.h"
#include "mq_device.h"

#define MQ_INLINE __attribute__((always_inline))   // on a lambda that is used more than once

namespace mq {
namespace {

constexpr float kLog2e = 1.44269502f;

// A row's weights are e^(s − m) with m a maximum that follows the scores only when
// they exceed it by kSlack (in powers of two): the sums are rescaled rarely.  The f16
// parts of a weight are held times 2^kShift, at most 2^15; the largest of a row is 2^7 at
// least, so those down to 2^-21 of it keep the first part's 11 bits, and 2^-31 of it is the
// step of either part.
constexpr float kShift = 7.0f, kSlack = 8.0f;

// tanh u = 1 − 2 / (1 + e^2u), and below 1/4, where that cancels,
// u − u³/3 + 2u⁵/15 − 17u⁷/315 (the next term is 3e-7 of the value at 1/4).
__device__ __forceinline__ float tanh_f32(float u) {
    const float e = __builtin_amdgcn_exp2f(u * (2.0f * kLog2e));
    const float t = u * u;
    float p = __builtin_fmaf(t, -17.0f / 315.0f, 2.0f / 15.0f);
    p = __builtin_fmaf(t, p, -1.0f / 3.0f);
    p = __builtin_fmaf(t * u, p, u);
    return fabsf(u) < 0.25f ? p : 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e);
}

__device__ __forceinline__ float finite(float v) { return fminf(fmaxf(v, -3.0e38f), 3.0e38f); }

// Products to scores: scale (a.scale, over what the row's queries were multiplied by) and
// cap, and the bias of N tokens, of which number i is `to − at(i)` positions before the
// row's.
// The cancellation of tanh's quotient is of no account where the cap is small: the
// score is off by 2^-21 of the cap at most, 2^-14 for kQuickCap, which changes a weight by
// an eighth of the half step that the output is rounded to.  (Five instructions per score
// instead of twelve: 512 rows over 16512 tokens with a cap 321 us to 291.)
constexpr float kQuickCap = 128.0f;
template <int N, class At>
__device__ __forceinline__ void bias_scores(const AttnArgs &a, float (&s)[N], float scale,
                                            float slope, int to, At at) {
    if (a.cap > kQuickCap) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = a.cap * tanh_f32(s[i] * scale * a.inv_cap);
    } else if (a.cap > 0.0f) {
        // (finite: a score of 0 stays one)
        const float c2 = -2.0f * a.cap, k = finite(scale * a.inv_cap * (2.0f * kLog2e));
#pragma unroll
        for (int i = 0; i < N; ++i)
            s[i] = __builtin_fmaf(
                c2, __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s[i] * k)), a.cap);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] *= scale;
    }
    if (a.slopes) {
        const float d = (float)to;   // (rounded beyond 2^24, like the distance itself)
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = __builtin_fmaf(-slope, fabsf(d - (float)at(i)), s[i]);
    }
}

typedef uint32_t q_u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float q_f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight query elements.
__device__ __forceinline__ half8 load_q8(const uint16_t *q, int64_t at) {
    return __builtin_bit_cast(half8, (u32x4)*reinterpret_cast<const q_u32x4_a2 *>(q + at));
}
__device__ __forceinline__ void load_q8(const float *q, int64_t at, float (&v)[8]) {
    const q_f32x4_a4 *p = reinterpret_cast<const q_f32x4_a4 *>(q + at);
    const f32x4 x = p[0], y = p[1];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < 4 ? x[e & 3] : y[e & 3];
}
__device__ __forceinline__ float largest_of(const float (&v)[8], float m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
    return m;
}
// f32 queries enter as two f16 numbers, of 22 bits together, down to f16's last step.  So
// that f16's range is no limit, a row goes in times a power of two that puts its largest
// element between 2^14 and 2^15 (the last step is then 2^-39 of it or less), and its
// scores' scale takes it out again, both exactly.  (The scale is then each lane's own: with
// f32 queries up to 4% of the time, for heads of 256, elsewhere 0 to 3%.)
__device__ __forceinline__ int query_shift(float largest) {
    return 15 - __builtin_amdgcn_frexp_expf(largest);   // (of 0, infinity and NaN: 15)
}
__device__ __forceinline__ float shifted_scale(float scale, int shift) {
    return finite(__builtin_amdgcn_ldexpf(scale, -shift));
}
__device__ __forceinline__ void split_q8(const float (&v)[8], int shift, half8 &high, half8 &low) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = __builtin_amdgcn_ldexpf(v[e], shift);
        high[e] = (_Float16)x;
        low[e] = (_Float16)(x - (float)high[e]);
    }
}

// The eight (q − 8) of a code dword, exact.  A nibble under the exponent of 1024
// is 1024 + q, one place of four bits higher 1024 + 16·q.
// (magic() sits in a vector register: an and-or takes one scalar operand, the mask.)
__device__ __forceinline__ uint32_t magic() { return opaque(0x64006400u); }
__device__ __forceinline__ void widen(uint32_t w, uint32_t magic, half2v h[4]) {
    const half2v c = {(_Float16)1032.0f, (_Float16)1032.0f};
    const half2v s = {(_Float16)0.0625f, (_Float16)0.0625f};
    const half2v o = {(_Float16)-72.0f, (_Float16)-72.0f};
    const uint32_t u = w >> 8;
    h[0] = __builtin_bit_cast(half2v, (w & 0x000F000Fu) | magic) - c;
    h[1] = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (w & 0x00F000F0u) | magic), s, o);
    h[2] = __builtin_bit_cast(half2v, (u & 0x000F000Fu) | magic) - c;
    h[3] = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (u & 0x00F000F0u) | magic), s, o);
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
    v.full_pre = uniform(v.full_pre);
    v.full_lo = uniform(v.full_lo);
    v.full_hi = uniform(v.full_hi);
}

// An even share of the batch's tiles for a.target workgroups (all lanes together).
__device__ __forceinline__ int even_share(const AttnArgs &a, int rows_per_tile) {
    if (a.splits == 1) return 0;
    float s = 0.0f;
    if (a.kv.batch == 1) {
        s = tiles_of_seq(a, 0, rows_per_tile);
    } else {
        for (int b = threadIdx.x & 63; b < a.kv.batch; b += 64) s += tiles_of_seq(a, b, rows_per_tile);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    }
    const float share = s * (float)a.kv.heads / (float)a.target;
    return uniform(share < 1e9f ? (int)ceilf(share) : 1000000000);
}

// The work of a workgroup of the kernel for few rows, or (BY_JOB) of the one that joins
// the parts of a job: number `index`.  All lanes of a wave together, a sequence each.
struct Work {
    View view;          // of the row tile, with pre, lo and n of the sequence's rows
    int head, split;
    Parts parts;
    int first;          // number of the job's first part
};
template <int R, bool BY_JOB>
__device__ __forceinline__ bool find_work(const AttnArgs &a, int index, Work &w) {
    const int lane = threadIdx.x & 63, batch = a.kv.batch;
    SeqWork mine = seq_work<R>(a, lane < batch ? lane : batch - 1);
    int share = 0;
    if (a.splits > 1) {
        float cost = lane < batch ? mine.cost : 0.0f;
        for (int b = lane + 64; b < batch; b += 64) cost += seq_work<R>(a, b).cost;
#pragma unroll
        for (int o = 1; o < 64; o *= 2)
            if (o < batch) cost += __shfl_xor(cost, o);
        share = uniform(share_of(a, cost));
    }
    int jobs0 = 0, items0 = 0;
    for (int b0 = 0; b0 < batch; b0 += 64) {
        if (b0 > 0) mine = seq_work<R>(a, b0 + lane < batch ? b0 + lane : batch - 1);
        const Parts parts = parts_of(a, mine.span.n, share);
        const bool here = b0 + lane < batch;
        const int jobs = here ? mine.jobs : 0, items = here ? items_of(mine, parts) : 0;
        int job_sum = jobs, item_sum = items;   // of the lanes up to this one
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
            if (o < batch) {
                const int x = __shfl_up(job_sum, o), y = __shfl_up(item_sum, o);
                if (lane >= o) {
                    job_sum += x;
                    item_sum += y;
                }
            }
        }
        const uint64_t past = __ballot(BY_JOB ? jobs0 + job_sum > index : items0 + item_sum > index);
        if (past) {
            const int l = uniform(__builtin_ctzll(past));
            const int job_base = jobs0 + __builtin_amdgcn_readlane(job_sum - jobs, l);
            const int item_base = items0 + __builtin_amdgcn_readlane(item_sum - items, l);
            w.parts.per = __builtin_amdgcn_readlane(parts.per, l);
            w.parts.count = __builtin_amdgcn_readlane(parts.count, l);
            const int within = BY_JOB ? (index - job_base) * w.parts.count : index - item_base;
            const int job = (int)((unsigned)within / (unsigned)w.parts.count);
            w.split = within - job * w.parts.count;
            w.first = item_base + job * w.parts.count;
            const int rt = (int)((unsigned)job / (unsigned)a.kv.heads);
            w.head = job - rt * a.kv.heads;
            w.view.b = b0 + l;
            const bool found = tile_view<R>(a, rt, w.view);
            w.view.pre = __builtin_amdgcn_readlane(mine.span.pre, l);
            w.view.lo = __builtin_amdgcn_readlane(mine.span.lo, l);
            w.view.n = __builtin_amdgcn_readlane(mine.span.n, l);
            return found;
        }
        jobs0 = clampi(jobs0 + __builtin_amdgcn_readlane(job_sum, 63), 0, 1 << 30);
        items0 = clampi(items0 + __builtin_amdgcn_readlane(item_sum, 63), 0, 1 << 30);
    }
    return false;
}

// The maximum over the lanes that hold the same column: l and l ^ 32, and with 16
// columns l ^ 16 too.
__device__ __forceinline__ float max_across32(float v) {
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto p = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
}
__device__ __forceinline__ float max_across16(float v) {
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
}

// The score where its bit is set, else −∞ (two instructions: no condition registers).
__device__ __forceinline__ float masked(float s, uint32_t bits, int bit) {
    const uint32_t keep = (uint32_t)((int32_t)(bits << (31 - bit)) >> 31);
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, s) & keep) | (0xFF800000u & ~keep));
}

// Values' scales in tiles that are masked in part.  A weight of 0 times an infinity or
// a NaN is not 0, so scales of tokens past the sequence (never written, perhaps) and
// scales that are not finite are taken out, and the rows that see one of the latter
// get a NaN in the elements of its block at the end.  Likewise finite ones from 8192 on
// (the three upper bits of the exponent): their products are infinite in f16.  The store
// writes none (kMostScale), but a token that no row sees may never have been stored.
__device__ __forceinline__ uint32_t bad_halves(uint32_t w) {   // bit 0: the low, 1: the high one
    return ((w & 0x7000u) == 0x7000u ? 1u : 0u) | ((w & 0x70000000u) == 0x70000000u ? 2u : 0u);
}
__device__ __forceinline__ uint32_t keep_halves(uint32_t w, bool lo, bool hi) {
    return (lo ? w & 0xFFFFu : 0u) | (hi ? w & 0xFFFF0000u : 0u);
}

// Pair e of an octet's scales as it enters, `tokens` of the octet existing; collects
// in bad the bits of those taken out that exist.
__device__ __forceinline__ uint32_t clean_scales(uint32_t s, int tokens, int e, uint32_t &bad) {
    s = keep_halves(s, tokens > 2 * e, tokens > 2 * e + 1);
    const uint32_t x = bad_halves(s);
    bad |= x << (2 * e);
    return keep_halves(s, !(x & 1), !(x & 2));
}
// The blocks (bit per 32 elements) that a row must give NaN in, for the tokens of one
// octet of a tile that it sees.  Rare: reads the scales again.
template <int NS>
__device__ __forceinline__ uint32_t bad_blocks(const char *tile, int octet, int tokens, uint32_t seen) {
    uint32_t blocks = 0;
#pragma unroll 1
    for (int b = 0; b < NS; ++b) {
        const u32x4 s = ((const u32x4 *)(tile + kv_vscale_at(32 * NS)))[octet * NS + b];
        uint32_t bad = 0;
        clean_scales(s.x, tokens, 0, bad);
        clean_scales(s.y, tokens, 1, bad);
        clean_scales(s.z, tokens, 2, bad);
        clean_scales(s.w, tokens, 3, bad);
        if (bad & seen & 0xFFu) blocks |= 1u << b;
    }
    return blocks;
}

// A key's scale as two f16 whose products with a code are exact: seven bits of it (times
// four of the code), and the four bits that are left.
__device__ __forceinline__ void split_scales(uint32_t d, half2v &high, half2v &low) {
    high = as_half2(d & 0xFFF0FFF0u);
    low = as_half2(d) - high;
}

// Two weights as f16, and what that rounding left of them as f16 (exact differences).
__device__ __forceinline__ void pack_weights(float a, float b, uint32_t &high, uint32_t &low) {
    const half2v v = {(_Float16)a, (_Float16)b};
    // (opaque: the pair is converted once, not each half again for its difference)
    high = opaque(__builtin_bit_cast(uint32_t, v));
    const half2v h = as_half2(high);
    const half2v l = {(_Float16)__builtin_fmaf((float)h.x, -1.0f, a),
                      (_Float16)__builtin_fmaf((float)h.y, -1.0f, b)};
    low = __builtin_bit_cast(uint32_t, l);
}

}  // namespace
}  // namespace mq
