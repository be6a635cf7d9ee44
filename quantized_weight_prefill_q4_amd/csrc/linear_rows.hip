// Linear and gated layers for a few activation rows (one generated token, or a
// handful of sequences decoded together): Y = epilogue(X·Wᵀ) with M <= 32.
//
// Mathematics and bound.  Every weight is used M times and read once, so the
// product is bound by the weight's bytes (0.56 to 2 per weight) and, for the
// block formats, by the instructions that expand them (3 to 5 per weight; the
// f16 values that feed the matrix cores are the cache's, bit for bit).  Tiles
// of 64 × 128 outputs would need a K split with partial planes and a second
// kernel to fill the chip, and would compute mostly rows that do not exist.
//
// Layout.  The matrix instruction is v_mfma_f32_16x16x32_f16 with the weight
// rows as its 16 rows and the activation rows as its 16 columns: lane l holds
// weight row l % 16 and, with g = l / 16, a quarter of the k range.  Since a sum
// does not care in which order its k are taken, a lane's quarter is what is
// contiguous in the block format (64 elements: two 32-element blocks, or a
// quarter of a super-block with one pair of scales), and the activations are
// read for the same k.  Bytes are loaded in whole 16-byte chunks of consecutive
// lanes and reach the lanes that use them through a strip of LDS that belongs
// to the wave alone, so there is no barrier in the loop.  A wave takes RT tiles
// of 16 weight rows (for a gated layer a gate tile and its up tile) on the same
// activations; the waves of a workgroup take the units of 256 k in turn, and
// their sums are joined in LDS in a fixed order, so one launch does the whole
// layer and results are deterministic.  A wave has one unit's raw bytes in
// registers: as soon as they are in the strip, the next unit's loads go into
// the same registers and are in flight while the fragments are expanded and
// multiplied.
//
// Measured (one token, weights cold in L2, graph replays): f16 28672 x 4096 42.9
// us = 5.6 TB/s, 14336 x 4096 22.9, 3584 x 3584 7.4; gated 2 x 14336 x 4096: f16
// 45 us (5.3 TB/s), Q8_0 30 (4.2), Q6_K 29, Q5_0 26, Q5_K 25, Q5_1 23.5, Q4_0 and
// Q4_K 20.5 (3.3).  16 rows of Q4_K 14336 x 4096: 16.8 us; 32: 21.3.  The f16 cache
// is bound by memory, the block formats by the expansion (3.2 vector
// instructions per weight for Q8_0, 3.3 for Q4_K, 5.2 for Q6_K, all told) of the
// last units, which no load covers, and a small layer by the memory's first
// answer (about 3 us from a cold start).

#include "epilogue.h"
#include "mq_device.h"
#include "mq_internal.h"

#include <type_traits>

namespace mq {
namespace {

constexpr int kCUs = 256;   // MI355X compute units

struct RowsArgs {
    const void *X;
    const uint8_t *W;
    void *Y;
    const float *bias;
    const void *res;
    int64_t ldw;       // bytes per weight row
    int64_t ldr;
    int ldx, ldy;
    int M, N, K;       // N: output columns (a gated layer's weight has 2·N rows)
    int act, res_type, y_type;
};

// Eight expanded weights (one MFMA operand), fl32(A·q + C) rounded to f16, from
// four dwords of two codes each: e0, e1 hold elements 0 and 2, 1 and 3 in their
// 16-bit halves, e2, e3 elements 4 and 6, 5 and 7.  A code q in the low bits of
// a half is the f16 subnormal q·2^-24, which v_fma_mix_f32 widens while it
// multiplies: with A scaled by 2^24 (exact) the fma's one rounding is the
// decode's, and no separate integer conversion is spent (2.1 instructions per
// Q4_K weight instead of 2.9).  Codes 4 bits up are scaled by 2^20 instead.
constexpr float kCode = 16777216.0f;        // 2^24
constexpr float kCodeHigh = 1048576.0f;     // 2^20
__device__ __forceinline__ half8 frag_codes(uint32_t e0, uint32_t e1, uint32_t e2, uint32_t e3,
                                            float A, float C) {
    auto lo = [&](uint32_t e) { return __builtin_fmaf(A, f16_bits_to_f32(e), C); };
    auto hi = [&](uint32_t e) { return __builtin_fmaf(A, f16_bits_to_f32(e >> 16), C); };
    const u32x4 v = {pack_f16x2(lo(e0), lo(e1)), pack_f16x2(hi(e0), hi(e1)),
                     pack_f16x2(lo(e2), lo(e3)), pack_f16x2(hi(e2), hi(e3))};
    return __builtin_bit_cast(half8, v);
}

// Where the value is one product of the f16 scale and a small integer, d·(u -
// OFF), its f32 product is exact and the f16 product rounds alike: from two
// dwords of byte codes u, as the f16 numbers 1024 + u (0x6400 | u), two
// weights to an instruction (1.5 per weight; Q8_0 2.5 and Q4_0 2.2 by the fma
// above.  v_fma_mixlo_f16 / mixhi, one per weight in place of fma and
// conversion, measured 4 to 7 % slower than those).
template <int OFF>
__device__ __forceinline__ half8 frag_products(uint32_t w0, uint32_t w1, uint32_t d2) {
    typedef _Float16 half2v __attribute__((ext_vector_type(2)));
    const half2v d = __builtin_bit_cast(half2v, d2);
    constexpr _Float16 o = (_Float16)(1024.0f + OFF);
    auto two = [&](uint32_t w, uint32_t bytes) {
        const uint32_t u = __builtin_amdgcn_perm(0x64646464u, w, bytes);
        return __builtin_bit_cast(uint32_t, (__builtin_bit_cast(half2v, u) - half2v{o, o}) * d);
    };
    constexpr uint32_t lo = 0x04010400u, hi = 0x04030402u;
    const u32x4 v = {two(w0, lo), two(w0, hi), two(w1, lo), two(w1, hi)};
    return __builtin_bit_cast(half8, v);
}

// frag_codes of two dwords of byte codes (at most 8 bits each).
__device__ __forceinline__ half8 frag_bytes(uint32_t w0, uint32_t w1, float A, float C) {
    constexpr uint32_t B = 0x00FF00FFu;
    return frag_codes(w0 & B, (w0 >> 8) & B, w1 & B, (w1 >> 8) & B, A, C);
}

// frag_codes of the low (HIGH = 0) or high nibbles of two dwords; A scaled by
// kCode or kCodeHigh accordingly.
template <int HIGH>
__device__ __forceinline__ half8 frag_nibbles(uint32_t w0, uint32_t w1, float A, float C) {
    constexpr uint32_t L = HIGH ? 0x00F000F0u : 0x000F000Fu;
    return frag_codes(w0 & L, (w0 >> 8) & L, w1 & L, (w1 >> 8) & L, A, C);
}

// The same with a byte h of fifth bits, element i's at bit i.  One pair of shifts lays the bits of
// elements 0 and 2 beside their nibbles, and one more shift each those of 1 and
// 3, 4 and 6, 5 and 7 (spreading a nibble's bits over a dword by a
// multiplication costs 4 cycles' worth of instructions for each).
template <int HIGH>
__device__ __forceinline__ half8 frag_fifths(uint32_t w0, uint32_t w1, uint32_t h, float A,
                                             float C) {
    constexpr uint32_t L = HIGH ? 0x00F000F0u : 0x000F000Fu, B = HIGH ? 0x01000100u : 0x00100010u;
    const uint32_t z = (h << (HIGH ? 8 : 4)) | (h << (HIGH ? 22 : 18));
    return frag_codes((w0 & L) | (z & B), ((w0 >> 8) & L) | ((z >> 1) & B),
                      (w1 & L) | ((z >> 4) & B), ((w1 >> 8) & L) | ((z >> 5) & B), A, C);
}

// ---------------------------------------------------------------------------
// One unit of k of a tile of 16 weight rows, as a wave holds it.  load(): the
// raw bytes into registers, zeros when the unit is not live; unpack(): the
// form that lane (row r, quarter g) makes its fragments from; frag<S>(): the
// eight weights of fragment S, whose k is kofs(g, S) within the unit.  The
// fragments of half h of a unit, S = 4h .. 4h + 3, cover 16 of its 32 chunks of
// 8 elements: half_chunk(h, i), i = 0 .. 15; half_slot(g, S) is the i of theirs.
// ---------------------------------------------------------------------------
template <int FMT>
struct RowUnit;

// f16: 256 contiguous bytes of each row (four rows per load) through the wave's
// strip of LDS; chunk c of row r lies at c ^ r, so that the 16 rows of a
// fragment lie in distinct banks.
template <>
struct RowUnit<kFmtF16> {
    static constexpr int NF = 4, UK = 128, STRIP = 256;
    u32x4 v[NF];
    struct Place {
        uint32_t o;
        int64_t ld4;
        __device__ __forceinline__ void init(int lane, int64_t ldw) {
            o = (uint32_t)((lane >> 4) * ldw) + 16u * (lane & 15);
            ld4 = 4 * ldw;
        }
    };
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t, const Place &at, int u,
                                         int lane, int K, bool live) {
        const int k = u * UK + 8 * (lane & 15);
        const uint32_t o = live && k < K ? at.o + (uint32_t)u * (2 * UK) : kOOB;
#pragma unroll
        for (int j = 0; j < NF; ++j) v[j] = buf_load16(rs, o + (uint32_t)(j * at.ld4));
    }
    struct Unpacked {
        u32x4 v[NF];
        template <int S>
        __device__ __forceinline__ half8 frag() const {
            return __builtin_bit_cast(half8, v[S]);
        }
    };
    __device__ __forceinline__ Unpacked unpack(u32x4 *strip, uint32_t, int64_t, int, int lane,
                                               int) const {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const int r = 4 * j + (lane >> 4);
            strip[16 * r + ((lane & 15) ^ r)] = v[j];
        }
        asm volatile("" ::: "memory");
        Unpacked p;
        const int r = lane & 15, g = lane >> 4;
#pragma unroll
        for (int s = 0; s < NF; ++s) p.v[s] = strip[16 * r + ((4 * s + g) ^ r)];
        return p;
    }
    static __device__ __forceinline__ int kofs(int g, int s) { return 32 * s + 8 * g; }
    static __device__ __forceinline__ int half_chunk(int, int i) { return i; }
    static __device__ __forceinline__ int half_slot(int, int) { return 0; }
};

// The block formats' bytes: UB bytes per row and unit, loaded as the WB / 16
// chunks of 16 bytes that cover them from the 16-byte boundary at or below
// their start (the 18, 22, 34 and 210-byte blocks are only 2-byte aligned),
// chunk by chunk of row after row over the 64 lanes, and handed to the lanes
// that expand them through a strip of LDS of the wave's own.  Loading each
// lane's bytes directly touches every cache line several times and is bound by
// the first-level cache (gated 14336 x 4096 at M = 1: Q8_0 36 us, Q6_K 36 us);
// chunks at dword alignment cost the address unit twice the cycles.
template <int UB_, int WB_>
struct Staged {
    static constexpr int UB = UB_, WB = WB_, CPR = WB / 16, NCH = 16 * CPR, NJ = (NCH + 63) / 64;
    static constexpr int STRIP = NJ * 64;   // chunks of LDS
    static_assert(WB % 16 == 0 && WB >= UB, "whole chunks");
    // The chunks' alignment: where UB bytes at any even start fit, the 16-byte
    // boundary below it; Q4_K's and Q5_K's rows start on one anyway, and Q5_1's
    // on 8 bytes (a 13th chunk for their other half costs a fourth load:
    // gated 14336 x 4096 at M = 1 25.4 -> 28.3 us).
    static constexpr uint32_t kAlign = WB >= UB + 14 ? 16 : 4;
    u32x4 v[NJ];
    struct Place {
        uint32_t o[NJ];
        __device__ __forceinline__ void init(int lane, int64_t ldw) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int id = 64 * j + lane, r = id / CPR;
                o[j] = id < NCH ? (uint32_t)(r * ldw) + 16u * (id - r * CPR) : kOOB;
            }
        }
    };
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t lead, const Place &at,
                                         int u, int, int, bool live) {
        const uint32_t base = lead + (uint32_t)u * UB;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            v[j] = buf_load16(rs, live && at.o[j] < kOOB ? (at.o[j] + base) & ~(kAlign - 1) : kOOB);
    }
    // to the strip; returns row lane % 16 of it
    __device__ __forceinline__ const uint32_t *stage(u32x4 *strip, int lane) const {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int j = 0; j < NJ; ++j) strip[64 * j + lane] = v[j];
        asm volatile("" ::: "memory");
        return reinterpret_cast<const uint32_t *>(strip + (lane & 15) * CPR);
    }
    // where in the strip's row the bytes of row lane % 16 start (even)
    static __device__ __forceinline__ uint32_t shift(uint32_t lead, int64_t ldw, int u, int lane) {
        return (lead + (uint32_t)((lane & 15) * ldw) + (uint32_t)u * UB) & 15;
    }
    static __device__ __forceinline__ u32x4 chunk(const uint32_t *w, int i) {
        return reinterpret_cast<const u32x4 *>(w)[i];
    }
};

// Q4_K, Q5_K: quarter g of the super-block, sub-blocks 2g (low nibbles) and
// 2g + 1 (high nibbles).
template <int FMT>
struct KUnit : Staged<FMT == kFmtQ5_K ? 176 : 144, FMT == kFmtQ5_K ? 176 : 144> {
    static constexpr int NF = 8, UK = 256;
    static constexpr bool Q5 = FMT == kFmtQ5_K;
    struct Unpacked {
        float A[2], C[2];
        u32x4 q[2], h[Q5 ? 2 : 1];
        template <int S>
        __device__ __forceinline__ half8 frag() const {
            constexpr int c = S & 3;             // 8 of the 32 quant bytes
            constexpr int high = S >= 4;
            const u32x4 w = q[c >> 1];
            uint32_t w0 = (c & 1) ? w.z : w.x, w1 = (c & 1) ? w.w : w.y;
            if constexpr (Q5) {
                w0 = (high ? w0 >> 4 : w0) & 0x0F0F0F0Fu;
                w1 = (high ? w1 >> 4 : w1) & 0x0F0F0F0Fu;
                const u32x4 b = h[c >> 1];
                const uint32_t b0 = (c & 1) ? b.z : b.x, b1 = (c & 1) ? b.w : b.y;
                w0 |= ((high ? b0 >> 1 : b0) & 0x01010101u) << 4;
                w1 |= ((high ? b1 >> 1 : b1) & 0x01010101u) << 4;
                return frag_bytes(w0, w1, A[high], C[high]);
            } else {
                return frag_nibbles<high>(w0, w1, A[high], C[high]);
            }
        }
    };
    __device__ __forceinline__ Unpacked unpack(u32x4 *strip, uint32_t, int64_t, int, int lane,
                                               int) const {
        const int g = lane >> 4;
        const uint32_t *w = this->stage(strip, lane);
        const u32x4 hdr = this->chunk(w, 0);
        Unpacked p;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            p.q[i] = this->chunk(w, (Q5 ? 3 : 1) + 2 * g + i);
            if constexpr (Q5) p.h[i] = this->chunk(w, 1 + i) >> (2 * g);   // bit 2g to bit 0
        }
        // Sub-blocks 2g, 2g + 1: bytes 2(g & 1) and the next of the scale dwords.
        // Of the first four the 6 bits lie together; of the last four the low 4
        // are nibbles of the third dword and the top 2 the first four's top bits.
        const uint32_t sh = 16 * (g & 1);
        const uint32_t lo = hdr.y >> sh, mid = hdr.z >> sh, hi = hdr.w >> sh;
        const uint32_t low = g < 2 ? 0x3F3Fu : 0x0F0Fu, top = g < 2 ? 0u : 0x3030u;
        const uint32_t sc = ((g < 2 ? lo : hi) & low) | ((lo >> 2) & top);
        const uint32_t mn = ((g < 2 ? mid : hi >> 4) & low) | ((mid >> 2) & top);
        const float d = kCode * f16_bits_to_f32(hdr.x), dmin = f16_bits_to_f32(hdr.x >> 16);
        p.A[0] = d * ubyte_f32<0>(sc);
        p.C[0] = -(dmin * ubyte_f32<0>(mn));
        p.A[1] = (Q5 ? d : d * (kCodeHigh / kCode)) * ubyte_f32<1>(sc);
        p.C[1] = -(dmin * ubyte_f32<1>(mn));
        return p;
    }
    static __device__ __forceinline__ int kofs(int g, int s) { return 64 * g + 8 * s; }
    static __device__ __forceinline__ int half_chunk(int h, int i) { return 8 * (i >> 2) + 4 * h + (i & 3); }
    static __device__ __forceinline__ int half_slot(int g, int s) { return 4 * g + (s & 3); }
};
template <> struct RowUnit<kFmtQ4_K> : KUnit<kFmtQ4_K> {};
template <> struct RowUnit<kFmtQ5_K> : KUnit<kFmtQ5_K> {};

// Q6_K: half h = g / 2 of the super-block, elements 16p .. 16p + 15 (p = g % 2)
// of its four 32-element groups.
template <>
struct RowUnit<kFmtQ6_K> : Staged<210, 224> {
    static constexpr int NF = 8, UK = 256;
    struct Unpacked {
        u32x4 a, b, h;
        float A[4], C[4];
        template <int S>
        __device__ __forceinline__ half8 frag() const {
            constexpr int grp = S >> 1, c = S & 1;
            const u32x4 l = (grp & 1) ? b : a;
            uint32_t w0 = c ? l.z : l.x, w1 = c ? l.w : l.y;
            const uint32_t h0 = c ? h.z : h.x, h1 = c ? h.w : h.y;
            w0 = (grp >= 2 ? w0 >> 4 : w0) & 0x0F0F0F0Fu;
            w1 = (grp >= 2 ? w1 >> 4 : w1) & 0x0F0F0F0Fu;
            w0 |= ((h0 >> (2 * grp)) & 0x03030303u) << 4;
            w1 |= ((h1 >> (2 * grp)) & 0x03030303u) << 4;
            // (d·s)·(q − 32): ds·q and 32·ds are exact, so one fma is
            return frag_bytes(w0, w1, A[grp], C[grp]);
        }
    };
    // the 16 bytes at w[4i] + s bytes (s = 0 or 2)
    static __device__ __forceinline__ u32x4 realign(const uint32_t *w, int i, uint32_t s) {
        const uint32_t *q = w + 4 * i;
        const uint32_t t[5] = {q[0], q[1], q[2], q[3], q[4]};
        return u32x4{__builtin_amdgcn_alignbyte(t[1], t[0], s), __builtin_amdgcn_alignbyte(t[2], t[1], s),
                     __builtin_amdgcn_alignbyte(t[3], t[2], s), __builtin_amdgcn_alignbyte(t[4], t[3], s)};
    }
    __device__ __forceinline__ Unpacked unpack(u32x4 *strip, uint32_t lead, int64_t ldw, int u,
                                               int lane, int) const {
        const int g = lane >> 4, h = g >> 1, pp = g & 1;
        const uint32_t off = shift(lead, ldw, u, lane), sh = off & 2;
        const uint32_t *w = stage(strip, lane) + (off >> 2);
        Unpacked p;
        p.a = realign(w, 4 * h + pp, sh);
        p.b = realign(w, 4 * h + 2 + pp, sh);
        p.h = realign(w, 8 + 2 * h + pp, sh);
        // the half's eight scales; this lane's are bytes pp, pp + 2, pp + 4, pp + 6
        const uint32_t *sc = w + 48 + 2 * h;
        uint32_t s0 = __builtin_amdgcn_alignbyte(sc[1], sc[0], sh);
        uint32_t s1 = __builtin_amdgcn_alignbyte(sc[2], sc[1], sh);
        s0 >>= 8 * pp;
        s1 >>= 8 * pp;
        const float d = f16_bits_to_f32(w[52] >> (8 * sh));
        const float ds[4] = {d * sbyte_f32<0>(s0), d * sbyte_f32<2>(s0), d * sbyte_f32<0>(s1),
                             d * sbyte_f32<2>(s1)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p.A[i] = kCode * ds[i];
            p.C[i] = -32.0f * ds[i];
        }
        return p;
    }
    static __device__ __forceinline__ int kofs(int g, int s) {
        return 128 * (g >> 1) + 32 * (s >> 1) + 16 * (g & 1) + 8 * (s & 1);
    }
    static __device__ __forceinline__ int half_chunk(int h, int i) { return 16 * (i >> 3) + 8 * h + (i & 7); }
    static __device__ __forceinline__ int half_slot(int g, int s) {
        return 8 * (g >> 1) + (s & 2) * 2 + 2 * (g & 1) + (s & 1);
    }
};

// The 32-element formats: blocks 2g and 2g + 1 of the unit's eight.  A block
// past the row's last has its factors cleared (its bytes are the next row's).
constexpr int b32_bytes(int fmt) {
    return fmt == kFmtQ4_0 ? 18 : fmt == kFmtQ5_0 ? 22 : fmt == kFmtQ5_1 ? 24 : 34;
}
template <int FMT>
struct BUnit : Staged<8 * b32_bytes(FMT),
                      FMT == kFmtQ5_1 ? 192 : (8 * b32_bytes(FMT) + 14 + 15) / 16 * 16> {
    static constexpr int NF = 8, UK = 256, BB = b32_bytes(FMT);
    struct Unpacked {
        static constexpr int NC = 2 * BB / 4;
        uint32_t c[NC];                  // the two blocks from byte 0
        float A[2], C[2];                // Q5_0, Q5_1: factor and offset
        uint32_t d2[2];                  // Q4_0, Q8_0: the f16 scale, twice
        // the dword at even byte offset T of the two blocks
        template <int TO>
        __device__ __forceinline__ uint32_t dw() const {
            if constexpr (TO % 4 == 0)
                return c[TO / 4];
            else
                return __builtin_amdgcn_alignbyte(c[TO / 4 + 1], c[TO / 4], 2);
        }
        template <int S>
        __device__ __forceinline__ half8 frag() const {
            constexpr int b = S >> 2, ch = S & 3, base = b * BB;   // block, 8-element chunk
            if constexpr (FMT == kFmtQ8_0) {
                // q + 128 as an unsigned byte
                constexpr uint32_t S8 = 0x80808080u;
                return frag_products<128>(dw<base + 2 + 8 * ch>() ^ S8, dw<base + 6 + 8 * ch>() ^ S8,
                                          d2[b]);
            } else {
                constexpr int QS = FMT == kFmtQ4_0 ? 2 : FMT == kFmtQ5_0 ? 6 : 8;
                const uint32_t w0 = dw<base + QS + 8 * (ch & 1)>();
                const uint32_t w1 = dw<base + QS + 4 + 8 * (ch & 1)>();
                if constexpr (FMT == kFmtQ4_0) {
                    constexpr uint32_t L = 0x0F0F0F0Fu;
                    return frag_products<8>((ch >= 2 ? w0 >> 4 : w0) & L,
                                            (ch >= 2 ? w1 >> 4 : w1) & L, d2[b]);
                } else {
                    constexpr int QH = FMT == kFmtQ5_0 ? 2 : 4;
                    return frag_fifths<(ch >> 1)>(w0, w1, (dw<base + QH>() >> (8 * ch)) & 255,
                                                  ch >= 2 ? A[b] * (kCodeHigh / kCode) : A[b],
                                                  C[b]);
                }
            }
        }
    };
    __device__ __forceinline__ Unpacked unpack(u32x4 *strip, uint32_t lead, int64_t ldw, int u,
                                               int lane, int K) const {
        const int g = lane >> 4, exist = (K >> 5) - (8 * u + 2 * g);
        const uint32_t *w = this->stage(strip, lane);
        Unpacked p;
        if constexpr (FMT == kFmtQ5_1) {
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const u32x4 v = this->chunk(w, 3 * g + i);
                p.c[4 * i] = v.x; p.c[4 * i + 1] = v.y; p.c[4 * i + 2] = v.z; p.c[4 * i + 3] = v.w;
            }
        } else {
            // the lane's two blocks start 2·BB·g bytes into the row's, a whole
            // number of dwords
            const uint32_t off = this->shift(lead, ldw, u, lane), sh = off & 2;
            const uint32_t *b = w + (off >> 2) + (2 * BB / 4) * g;
            uint32_t t[Unpacked::NC + 1];
#pragma unroll
            for (int i = 0; i <= Unpacked::NC; ++i) t[i] = b[i];
#pragma unroll
            for (int i = 0; i < Unpacked::NC; ++i)
                p.c[i] = __builtin_amdgcn_alignbyte(t[i + 1], t[i], sh);
        }
        const uint32_t h0 = p.c[0], h1 = BB % 4 ? p.c[BB / 4] >> 16 : p.c[BB / 4];
        if constexpr (FMT == kFmtQ4_0 || FMT == kFmtQ8_0) {
            p.d2[0] = exist > 0 ? __builtin_amdgcn_perm(h0, h0, 0x01000100u) : 0u;
            p.d2[1] = exist > 1 ? __builtin_amdgcn_perm(h1, h1, 0x01000100u) : 0u;
        } else {
            p.A[0] = exist > 0 ? kCode * f16_bits_to_f32(h0) : 0.0f;
            p.A[1] = exist > 1 ? kCode * f16_bits_to_f32(h1) : 0.0f;
            if constexpr (FMT == kFmtQ5_1) {
                p.C[0] = exist > 0 ? f16_bits_to_f32(h0 >> 16) : 0.0f;
                p.C[1] = exist > 1 ? f16_bits_to_f32(h1 >> 16) : 0.0f;
            } else {
                // the codes' offset; d times it is exact
                p.C[0] = (-16.0f / kCode) * p.A[0];
                p.C[1] = (-16.0f / kCode) * p.A[1];
            }
        }
        return p;
    }
    static __device__ __forceinline__ int kofs(int g, int s) { return 64 * g + 8 * s; }
    static __device__ __forceinline__ int half_chunk(int h, int i) { return 8 * (i >> 2) + 4 * h + (i & 3); }
    static __device__ __forceinline__ int half_slot(int g, int s) { return 4 * g + (s & 3); }
};
template <> struct RowUnit<kFmtQ4_0> : BUnit<kFmtQ4_0> {};
template <> struct RowUnit<kFmtQ5_0> : BUnit<kFmtQ5_0> {};
template <> struct RowUnit<kFmtQ5_1> : BUnit<kFmtQ5_1> {};
template <> struct RowUnit<kFmtQ8_0> : BUnit<kFmtQ8_0> {};

// A unit's activations: MR rows of UK elements (with PH = 2 half a unit at a
// time, so that 32 rows fit), loaded in row segments of at least 64 bytes one
// step ahead, rounded to f16 when they are f32, and handed through a strip of
// LDS that belongs to the wave alone, so without a barrier.  Fragment loads
// straight from global memory touch a cache line per lane instead (M = 16,
// gated 14336 x 4096 Q4_K: 46 us).  Slot c of row r is stored at c ^ (r mod
// 16): the 16 rows that a ds_read_b128 serves together then lie in distinct
// banks.
template <class U, int MR, bool XF32, int PH>
struct XUnit {
    static constexpr int CH = U::UK / 8 / PH;     // chunks per row and step: 32 or 16
    static constexpr int RPI = 64 / CH;           // rows per load
    static constexpr int NX = MR / RPI;
    static_assert(NX >= 1 && NX * RPI == MR, "whole loads");
    static_assert(PH == 1 || CH == 16, "halves of 16 chunks");
    u32x4 v[NX][XF32 ? 2 : 1];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, uint32_t ldb, int u, int ph,
                                         int lane, int M, int K, bool live) {
        const int c = lane & (CH - 1), r0 = lane / CH;
        const int k = u * U::UK + 8 * (PH == 1 ? c : U::half_chunk(ph, c));
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int r = r0 + RPI * i;
            const uint32_t o = live && k < K && r < M ? (uint32_t)r * ldb + (XF32 ? 4 : 2) * k : kOOB;
            v[i][0] = buf_load16(rs, o);
            if constexpr (XF32) v[i][1] = buf_load16(rs, o + 16);
        }
    }
    __device__ __forceinline__ void store(u32x4 *lds, int lane) const {
        const int c = lane & (CH - 1), r0 = lane / CH;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int r = r0 + RPI * i;
            u32x4 h = v[i][0];
            if constexpr (XF32) {
                auto f = [](uint32_t w) { return __builtin_bit_cast(float, w); };
                const u32x4 p = v[i][0], q = v[i][1];
                h = u32x4{pack_f16x2(f(p.x), f(p.y)), pack_f16x2(f(p.z), f(p.w)),
                          pack_f16x2(f(q.x), f(q.y)), pack_f16x2(f(q.z), f(q.w))};
            }
            lds[r * CH + (c ^ (r & 15))] = h;
        }
    }
    // Fragment s of lane (row, g), activation rows 16·f + row.  Columns of the
    // product past M are never written out, so rows past MR may read any row's
    // chunk.
    static __device__ __forceinline__ half8 frag(const u32x4 *lds, int f, int row, int g, int s) {
        const int r = (16 * f + row) & (MR - 1);
        const int c = PH == 1 ? U::kofs(g, s) >> 3 : U::half_slot(g, s);
        return __builtin_bit_cast(half8, lds[r * CH + (c ^ (r & 15))]);
    }
};

template <int I, int N, class F>
__device__ __forceinline__ void for_const(F &&f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        for_const<I + 1, N>(f);
    }
}

// Steps per unit: the 32-chunk units' activations in halves where a whole unit
// of 32 rows, or of 16 in f32, would not fit the registers (16 f16 rows in
// halves: gated 14336 x 4096 Q4_K 26 -> 31 us).
template <class Unit, int MR, bool XF32>
constexpr int kPhases = Unit::UK == 256 && (MR > 16 || (MR == 16 && XF32)) ? 2 : 1;

// The LDS strip of a wave: its activations and a tile's raw bytes, then its
// sums.
template <class Unit, int RT, int MR, bool XF32>
constexpr int strip_chunks() {
    const int need = MR * Unit::UK / 8 / kPhases<Unit, MR, XF32> + Unit::STRIP;
    const int sums = RT * (MR > 16 ? MR / 16 : 1) * 64;
    return need > sums ? need : sums;
}

// Waves that share a compute unit, which caps their registers: 4 per SIMD (with
// half of them the loads in flight do not cover the memory's latency), 3 or 2
// where more rows' activations and sums, or two tiles of a gated layer, would
// spill (gated 9472 x 3584, 7 rows, 4 -> 3 waves: Q8_0 32 -> 22 us, f32 rows 56
// -> 24.5, Q6_K 27 -> 24, Q4_K 17.7 -> 16.4; 14336 x 4096: Q8_0 38 -> 33, Q4_K
// 21.7 -> 23.1; ungated Q8_0 6144 x 4096, 7 f32 rows, 12.5 -> 11.9).
constexpr int max_waves(int fmt, int MR, bool GLU, bool XF32) {
    if (MR > 16) return 8;
    if (GLU && fmt == kFmtQ8_0) return MR > 8 && XF32 ? 8 : 12;
    return MR > (GLU || (XF32 && fmt == kFmtQ8_0) ? 4 : 8) ? 12 : 16;
}

// RT tiles of 16 weight rows per workgroup of blockDim.x / 64 waves, at least
// the RT·MF whose sums they finish (gated: a gate tile and its up tile, RT =
// 2); MR: activation rows held (4, 8, 16 or 32).
template <int FMT, int RT, bool GLU, bool XF32, int MR>
__global__ __launch_bounds__(64 * max_waves(FMT, MR, GLU, XF32),
                             max_waves(FMT, MR, GLU, XF32) / 4) void
linear_rows_kernel(RowsArgs a) {
    static_assert(!GLU || RT == 2, "a gate tile and an up tile");
    using Unit = RowUnit<FMT>;
    constexpr int PH = kPhases<Unit, MR, XF32>, MF = MR > 16 ? MR / 16 : 1;
    using XU = XUnit<Unit, MR, XF32, PH>;
    constexpr int NF = Unit::NF, SC = strip_chunks<Unit, RT, MR, XF32>();
    extern __shared__ u32x4 strips[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int NW = (int)blockDim.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * (GLU ? 16 : 16 * RT);   // first output column

    // what the epilogue needs, requested first: wave (tile t, row block f)
    // finishes rows 16f + lane % 16 of y, columns n0 + 16t + 4g .. + 3
    constexpr int OT = GLU ? 1 : RT;
    const int ot = wave / MF, of = wave % MF, row = 16 * of + r16;
    const int col = n0 + 16 * ot + 4 * g;
    const int n = ot < OT && row < a.M ? min(4, a.N - col) : 0;
    float b0[4] = {}, b1[4] = {}, res[4] = {};
    if (n > 0) {
        if (a.bias) {
            load_upto4(a.bias, kTypeF32, col, n, b0);
            if constexpr (GLU) load_upto4(a.bias, kTypeF32, (int64_t)a.N + col, n, b1);
        }
        if (!GLU && a.res)
            load_upto4((const char *)a.res + row * a.ldr * (a.res_type == kTypeF32 ? 4 : 2),
                       a.res_type, col, n, res);
    }

    __amdgpu_buffer_rsrc_t rsw[RT];
    uint32_t lead[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int first = n0 + (GLU ? 0 : 16 * t);
        const int valid = min(16, a.N - first);
        const int64_t start = ((int64_t)first + (GLU && t ? a.N : 0)) * a.ldw;
        lead[t] = FMT == kFmtF16 ? 0 : (uint32_t)(((uintptr_t)a.W + start) & 15);
        const int64_t last = FMT == kFmtF16 ? 2 * (int64_t)a.K : a.ldw;
        // a tile past N reads nothing
        const int64_t bytes =
            valid > 0 ? (lead[t] + (valid - 1) * a.ldw + last + 3) & ~(int64_t)3 : 0;
        rsw[t] = make_rsrc(valid > 0 ? a.W + start - lead[t] : a.W, (uint32_t)bytes);
    }
    typename Unit::Place place;
    place.init(lane, a.ldw);
    constexpr int XE = XF32 ? 4 : 2;
    const __amdgpu_buffer_rsrc_t rsx =
        make_rsrc(a.X, (uint32_t)(((int64_t)(a.M - 1) * a.ldx + a.K) * XE));
    const uint32_t ldb = (uint32_t)a.ldx * XE;

    const int units = (a.K + Unit::UK - 1) / Unit::UK;
    f32x4 acc[RT][MF];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int f = 0; f < MF; ++f) acc[t][f] = f32x4{};
    Unit w[RT];
    XU x;
    u32x4 *const xl = strips + wave * SC, *const wl = xl + MR * XU::CH;
    // Look-aheads past the last unit load zeros: a branch around the loads
    // would make the compiler wait for all of them at its join.
    auto load_w = [&](int t, int u) { w[t].load(rsw[t], lead[t], place, u, lane, a.K, u < units); };
    // The activations' strip: the previous step's reads come before in the
    // wave's LDS order; only the compiler must keep both.
    auto next_x = [&](int u, int ph) {
        asm volatile("" ::: "memory");
        x.store(xl, lane);
        asm volatile("" ::: "memory");
        x.load(rsx, ldb, u, ph, lane, a.M, a.K, u < units);
    };
    auto unpack = [&](int t, int u) {
        const auto p = w[t].unpack(wl, lead[t], a.ldw, u, lane, a.K);
        load_w(t, u + NW);
        return p;
    };
    auto multiply = [&](int t, auto &&p, auto f, const half8 (&xf)[MF]) {
        const half8 wf = p.template frag<decltype(f)::value>();
#pragma unroll
        for (int i = 0; i < MF; ++i)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wf, xf[i], acc[t][i], 0, 0, 0);
    };
    auto x_frags = [&](int s, half8 (&xf)[MF]) {
#pragma unroll
        for (int i = 0; i < MF; ++i) xf[i] = XU::frag(xl, i, r16, g, s);
    };
    int u = wave;
    x.load(rsx, ldb, u, 0, lane, a.M, a.K, u < units);
#pragma unroll
    for (int t = 0; t < RT; ++t) load_w(t, u);
    for (; u < units; u += NW) {
        if constexpr (PH == 1) {
            next_x(u + NW, 0);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const auto p = unpack(t, u);
                for_const<0, NF>([&](auto f) {
                    half8 xf[MF];
                    x_frags(decltype(f)::value, xf);
                    multiply(t, p, f, xf);
                });
            }
        } else {
            next_x(u, 1);
            typename Unit::Unpacked p[RT];
#pragma unroll
            for (int t = 0; t < RT; ++t) p[t] = unpack(t, u);
            for_const<0, NF>([&](auto f) {
                constexpr int S = decltype(f)::value;
                if constexpr (S == NF / 2) next_x(u + NW, 0);
                half8 xf[MF];
                x_frags(S, xf);
#pragma unroll
                for (int t = 0; t < RT; ++t) multiply(t, p[t], f, xf);
            });
        }
    }

    asm volatile("" ::: "memory");
    f32x4 *const sums = reinterpret_cast<f32x4 *>(strips);
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int f = 0; f < MF; ++f) sums[wave * SC + (t * MF + f) * 64 + lane] = acc[t][f];
    __syncthreads();
    if (n <= 0) return;
    const int at = (GLU ? of : wave) * 64 + lane;
    f32x4 s = sums[at];
    for (int i = 1; i < NW; ++i) s += sums[i * SC + at];
    float y[4] = {s.x + b0[0], s.y + b0[1], s.z + b0[2], s.w + b0[3]};
    apply_act(a.act, y);
    if constexpr (GLU) {
        const int up = (MF + of) * 64 + lane;
        f32x4 v = sums[up];
        for (int i = 1; i < NW; ++i) v += sums[i * SC + up];
        y[0] *= v.x + b1[0];
        y[1] *= v.y + b1[1];
        y[2] *= v.z + b1[2];
        y[3] *= v.w + b1[3];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] += res[j];
    }
    store_upto4((char *)a.Y + (int64_t)row * a.ldy * (a.y_type == kTypeF32 ? 4 : 2), a.y_type, col,
                n, y);
}

template <int FMT, int RT, bool GLU, bool XF32, int MR>
hipError_t launch_rows(const RowsArgs &a, hipStream_t stream) {
    using Unit = RowUnit<FMT>;
    const int cols = GLU ? 16 : 16 * RT;
    const int tiles = (a.N + cols - 1) / cols;
    const int units = (a.K + Unit::UK - 1) / Unit::UK;
    // As many waves per workgroup as let all workgroups be resident at once
    // (a second round of a few left over costs as much as the first: 288 tiles
    // on 256 compute units, f16 4608 x 3584 at M = 24, 15.5 us with 8 waves
    // each, 13.8 with 4), but 4 where that is 5 to 7, which do not spread evenly
    // over four SIMDs, and where it is 1 or 2; no more than there are units, and
    // at least the RT·MF that finish the sums.  Both sides, us:
    //   6 -> 4: gated Q8_0 6144 x 4096, 1 row, 22.4 -> 17.8, 16 rows 24.5 -> 19.6;
    //     gated Q6_K 4608 x 3584, 8 rows, 22.7 -> 18.1; 16 rows: Q8_0 6144 x 4096
    //     14.9 -> 12.3, f16 15.2 -> 14.1, Q4_K 10.4 -> 9.8; Q4_K 4608 x 3584, 13
    //     f32 rows, and gated 6144 x 4096, 8 rows, level;
    //   5 -> 4: 1 row, 11008 x 4096: Q8_0 18.5 -> 13.0, Q6_K 15.7 -> 12.8, f16 and
    //     Q4_K level; gated Q4_K 20.3 -> 15.9, Q6_K 30.7 -> 23.8, f16 37.5 -> 34;
    //   3 stay 3, all of them resident; with 4: gated Q8_0 14336 x 4096, 1 row,
    //     29.4 -> 33.7, 13824 x 5120, 4 rows, 38 -> 45; gated Q6_K 14336 x 4096, 8
    //     rows, 31.4 -> 34.3; 16 rows: Q8_0 21.6 -> 23.5, Q4_K 16.7 -> 17.5, Q6_K
    //     19.8 -> 20.2; gated 18944 x 3584, 1 row: Q6_K 33.5 -> 35.3, Q4_K 22.9 ->
    //     23.5; ungated f16 and Q4_K level; gated Q4_K 14336 x 4096, 8 rows, 21.8 ->
    //     21.4.
    const int per_cu = (tiles + kCUs - 1) / kCUs;
    int nw = max_waves(FMT, MR, GLU, XF32) / per_cu;
    if (nw < 3 || (nw > 4 && nw < 8)) nw = 4;
    if (nw > units) nw = units;
    const int finish = (GLU ? 1 : RT) * (MR > 16 ? MR / 16 : 1);
    if (nw < finish) nw = finish;
    static_assert(max_waves(FMT, MR, GLU, XF32) * strip_chunks<Unit, RT, MR, XF32>() * 16 <=
                      160 * 1024,
                  "the strips of the most waves fit a compute unit's LDS");
    const size_t lds = nw * (size_t)(strip_chunks<Unit, RT, MR, XF32>()) * 16;
    hipLaunchKernelGGL((linear_rows_kernel<FMT, RT, GLU, XF32, MR>), dim3(tiles), dim3(64 * nw),
                       lds, stream, a);
    return hipGetLastError();
}

template <int FMT, bool XF32, int MR>
hipError_t launch_rows_fmt(const RowsArgs &a, bool glu, hipStream_t stream) {
    if (glu) return launch_rows<FMT, 2, true, XF32, MR>(a, stream);
    // Two weight tiles per wave on the same activations where loading those
    // costs more than the tile's own registers do: with 32 rows, and with 16 for
    // the f16 cache, once one tile per workgroup would be more than two rounds of
    // the chip (M = 32, 14336 x 4096: Q4_K 31 -> 21 us, Q8_0 38 -> 28; M = 16 f16
    // 27 -> 25, but Q8_0 24 -> 26).
    if constexpr (MR > 16 || (MR == 16 && FMT == kFmtF16)) {
        if (a.N > 16 * 2 * kCUs) return launch_rows<FMT, 2, false, XF32, MR>(a, stream);
    }
    return launch_rows<FMT, 1, false, XF32, MR>(a, stream);
}

template <bool XF32, int MR>
hipError_t launch_rows_any(int fmt, const RowsArgs &a, bool glu, hipStream_t stream) {
    switch (fmt) {
    case kFmtF16: return launch_rows_fmt<kFmtF16, XF32, MR>(a, glu, stream);
    case kFmtQ4_0: return launch_rows_fmt<kFmtQ4_0, XF32, MR>(a, glu, stream);
    case kFmtQ5_0: return launch_rows_fmt<kFmtQ5_0, XF32, MR>(a, glu, stream);
    case kFmtQ5_1: return launch_rows_fmt<kFmtQ5_1, XF32, MR>(a, glu, stream);
    case kFmtQ8_0: return launch_rows_fmt<kFmtQ8_0, XF32, MR>(a, glu, stream);
    case kFmtQ4_K: return launch_rows_fmt<kFmtQ4_K, XF32, MR>(a, glu, stream);
    case kFmtQ5_K: return launch_rows_fmt<kFmtQ5_K, XF32, MR>(a, glu, stream);
    case kFmtQ6_K: return launch_rows_fmt<kFmtQ6_K, XF32, MR>(a, glu, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_linear_rows(int fmt, bool x_f32, const void *X, int ldx, const void *W,
                              int64_t ldw, void *Y, int ldy, int M, int N, int K,
                              const EpiSpec &epi, hipStream_t stream) {
    RowsArgs a;
    a.X = X;
    a.W = (const uint8_t *)W;
    a.Y = Y;
    a.bias = epi.bias;
    a.res = epi.res;
    a.ldw = fmt == kFmtF16 ? 2 * ldw : ldw;
    a.ldr = epi.ldr;
    a.ldx = ldx;
    a.ldy = ldy;
    a.M = M;
    a.N = N;
    a.K = K;
    a.act = epi.act;
    a.res_type = epi.res_type;
    a.y_type = epi.y_type;
    if (M <= 4)
        return x_f32 ? launch_rows_any<true, 4>(fmt, a, epi.glu, stream)
                     : launch_rows_any<false, 4>(fmt, a, epi.glu, stream);
    if (M <= 8)
        return x_f32 ? launch_rows_any<true, 8>(fmt, a, epi.glu, stream)
                     : launch_rows_any<false, 8>(fmt, a, epi.glu, stream);
    if (M <= 16)
        return x_f32 ? launch_rows_any<true, 16>(fmt, a, epi.glu, stream)
                     : launch_rows_any<false, 16>(fmt, a, epi.glu, stream);
    return x_f32 ? launch_rows_any<true, 32>(fmt, a, epi.glu, stream)
                 : launch_rows_any<false, 32>(fmt, a, epi.glu, stream);
}

}  // namespace mq
