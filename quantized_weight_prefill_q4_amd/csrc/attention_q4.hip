// Attention over the 4-bit key/value cache (kv_q4.h has its layout).
//
// Row i of a sequence with n new rows and len tokens stands at p = len − n + i.
// For each of its heads, with q the row's query and k_j, v_j the cache's:
//   s_j = scale · q·k_j;  s_j = cap · tanh(s_j / cap);  s_j −= slope · |p − j|
//   o   = Σ_j e^(s_j − m) v_j / Σ_j e^(s_j − m),  over the visible j, m their maximum
// and zeros where none is visible.
//
// Few rows of a key/value head (this file; more in attention_prompt.hip): the
// time is that of reading the cache.  A workgroup takes R rows (16 or 32; row = token ·
// group + head of the group, so that the query heads of a key/value head share its
// tiles) of one key/value head and a part of the keys; its four waves take the part's
// tiles of 32 tokens in turn, each loading one tile ahead, and their results are joined
// at the end.  Per tile, in one pass with the running maximum and sum:
//   Sᵀ[t, n] = Σ_b d_b[t] · (q − 8)[t, b] · Q[n, b]   over the blocks b of 32 elements:
//                                   matrix instructions 16 x 16 x 32, a block's codes as A,
//                                   times its scale in f32; f32 queries' low part a second
//   Oᵀ[d, n] += Vᵀ[d, t] · Pᵀ[t, n]  values as A, twice: both parts of the weights
// A lane holds of Sᵀ exactly the eight tokens whose weights it has to give as the
// second product's B operand, because row r of the first product's tile m is
// token 8·(r/4) + 4·m + r%4: nothing moves between lanes but the maximum of a
// column.  Codes become f16 in the registers that loaded them.
//
// Numerics: the keys' codes are exact in f16 and their scales multiply f32 sums; f32
// queries enter as two f16 numbers (their row scaled into f16's range: split_q8), the
// weights e^(s − m) as two (2^-22 of the weight).  Products are summed in f32, statistics are f32.  The values d·(q − 8) enter as one f16,
// rounded once: errors of either sign that the sum over the tokens averages, 0.75 of the
// output's own rounding in effect.  Keys rounded to one f16 would add 1.6 of it, weights
// 0.8.
//
// What bounds it, at one token of 32 heads (8 key/value heads, D = 128) over 131072
// tokens, 151 MB: 33.5 us when the cache lies in the chip's last-level cache, of which the
// vector instructions that expand the codes (380 a tile and wave) are 20, and 35 from
// memory (4.3 TB/s; a large copy 4.8); the join 5.6.  (Keys as two f16 parts, eight more
// matrix and 50 more vector instructions a tile: 36.)  Short contexts: the chain of loads
// (lengths, page numbers, tiles) and two launches, 10 us over 4096 tokens.
#include "attention_device.h"

namespace mq {
namespace {

constexpr int kWaves = 4;
constexpr int kMaxSplits = 256;
// Workgroups that the keys are dealt to: the three that fit on each unit.  (One token over
// 131072: 40.6 us with 512, 40.3 with 768, 42.4 with 1024; 64 sequences of up to 8000 54.0,
// 49.5, 46.6.)
constexpr int kFewRowsTarget = 768;

// A tile as loaded: code dwords of the lane's operands and the scales they need.
// Lane l is row r = l % 16 of the A operands and their inner octet g = l / 16.
// Values' operand i holds element d(r, i) of tokens [8g, + 8): d = (D/16)·r + i,
// where one scale per token serves all of a lane's operands, or for D = 96, whose
// 16ths straddle blocks, d = 16·i + r.
template <int NS>
struct Tile {
    static constexpr bool kRuns = (NS & (NS - 1)) == 0;
    static constexpr int kScaleSets = kRuns ? 1 : NS;
    static constexpr int KS2 = (NS + 1) / 2;
    // (vectors: arrays that live on from one trip of a loop to the next went to memory)
    typedef uint32_t Codes __attribute__((ext_vector_type(2 * NS)));
    typedef uint32_t KeyScales __attribute__((ext_vector_type(2 * KS2)));
    typedef uint32_t ValueScales __attribute__((ext_vector_type(4 * kScaleSets)));
    Codes k, v;           // [m][block], [operand]
    KeyScales ks;         // [m][pair of blocks]
    ValueScales vs;       // [set][pair of tokens]
};

template <int NS>
__device__ __forceinline__ void load_tile(const char *tile, int r, int g, Tile<NS> &t) {
    constexpr int D = 32 * NS, KS2 = Tile<NS>::KS2;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        uint32_t k[NS], ks[KS2];
        load_dwords((const uint32_t *)tile + ((4 * m + g) * 16 + r) * NS, k);
        const uint16_t *s = (const uint16_t *)(tile + kv_kscale_at(D)) + (16 * m + r) * NS;
        if constexpr (NS % 2 == 0) {
            load_dwords((const uint32_t *)s, ks);
        } else {
#pragma unroll
            for (int i = 0; i < KS2; ++i)
                ks[i] = s[2 * i] | (2 * i + 1 < NS ? (uint32_t)s[2 * i + 1] << 16 : 0u);
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) t.k[m * NS + i] = k[i];
#pragma unroll
        for (int i = 0; i < KS2; ++i) t.ks[m * KS2 + i] = ks[i];
    }
    const uint32_t *vc = (const uint32_t *)(tile + kv_vcode_at(D)) + g * D;
    const u32x4 *vs = (const u32x4 *)(tile + kv_vscale_at(D)) + g * NS;
    uint32_t v[2 * NS];
    if constexpr (Tile<NS>::kRuns) {
        load_dwords(vc + 2 * NS * r, v);
        vs += (2 * NS * r) / 32;
    } else {
#pragma unroll
        for (int i = 0; i < 2 * NS; ++i) v[i] = vc[16 * i + r];
    }
#pragma unroll
    for (int i = 0; i < 2 * NS; ++i) t.v[i] = v[i];
#pragma unroll
    for (int i = 0; i < Tile<NS>::kScaleSets; ++i) {
        const u32x4 x = vs[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) t.vs[4 * i + e] = x[e];
    }
}

// The values' operand i.
template <int NS>
__device__ __forceinline__ half8 value_operand(const Tile<NS> &t, int i, uint32_t mg) {
    const int set = Tile<NS>::kRuns ? 0 : i / 2;
    half2v h[4];
    widen(t.v[i], mg, h);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] *= as_half2(t.vs[4 * set + e]);
    return join8(h);
}

// Waves per SIMD that the registers have to leave room for.
template <int NS, int NT, bool WIDE>
constexpr int kWavesPerSimd = NS * NT <= 4 ? 3 : NS * NT == 8 && NT == 1 && WIDE ? 1 : 2;

template <int NS, int NT, bool BIAS, bool WIDE>
__global__ __launch_bounds__(256, (kWavesPerSimd<NS, NT, WIDE>)) void attention_kernel(AttnArgs a) {
    constexpr int D = 32 * NS, R = 16 * NT, MT = 2 * NS;   // MT: output tiles of 16 elements
    constexpr int CH = MT < 8 ? MT : 8;                    // of them joined at a time
    __shared__ float join[kWaves][CH * 4][64];
    __shared__ float2 wave_stats[kWaves][R];
    __shared__ uint32_t wave_nan[kWaves][R];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    Work work;
    if (!find_work<R, false>(a, blockIdx.x, work)) return;
    View &view = work.view;
    make_uniform(view);
    const int head = work.head, t_begin = work.split * work.parts.per;
    const int t_end = t_begin + work.parts.per < view.n ? t_begin + work.parts.per : view.n;

    // this lane's column in each of the NT column tiles: row 16·c + r
    half8 q[NT][NS], q_low[NT][WIDE ? NS : 1];
    int pos[NT];
    Range range[NT];
    float slope[NT], scale[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int row = view.rt * R + 16 * c + r;
        const int i = (int)((unsigned)row / (unsigned)a.group), h = head * a.group + row - i * a.group;
        const bool live = i < view.rows.n;
        pos[c] = view.first_pos + i;
        range[c] = row_range(a, view, pos[c]);
        slope[c] = BIAS && a.slopes && live ? a.slopes[h] : 0.0f;
        const int64_t at = (int64_t)(view.rows.first + (live ? i : 0)) * a.ldq +
                           (int64_t)(live ? h : head * a.group) * D + 8 * g;
        scale[c] = a.scale;
        if constexpr (WIDE) {
            float x[NS][8], top = 0.0f;
#pragma unroll
            for (int s = 0; s < NS; ++s) load_q8((const float *)a.q, at + 32 * s, x[s]);
#pragma unroll
            for (int s = 0; s < NS; ++s) top = largest_of(x[s], top);
            const int shift = query_shift(max_across32(max_across16(top)));
            scale[c] = shifted_scale(a.scale, shift);
#pragma unroll
            for (int s = 0; s < NS; ++s) split_q8(x[s], shift, q[c][s], q_low[c][s]);
        } else {
#pragma unroll
            for (int s = 0; s < NS; ++s) q[c][s] = load_q8((const uint16_t *)a.q, at + 32 * s);
        }
    }
    f32x4 o[NT][MT];
    float m[NT], l[NT];
    uint32_t nan_blocks[NT];   // blocks of the column's row that must become NaN
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        m[c] = -__builtin_inff();
        l[c] = 0.0f;
        nan_blocks[c] = 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[c][i] = f32x4{0, 0, 0, 0};
    }
    const float to_log2 = BIAS ? kLog2e : a.scale * kLog2e;
    const uint32_t mg = magic();

    auto tile_of = [&](int t) { return t < view.pre ? t : t - view.pre + view.lo; };
    const int per_page = a.kv.page / kTile;
    // The work on one tile; hole: there is no such page, its tokens are not visible.
    auto use_tile = [&](Tile<NS> &now, const char *p, int t, bool hole) MQ_INLINE {
        const int tile = tile_of(t), j0 = tile * kTile;
        f32x4 s[NT][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            // scales of the lane's four tokens: row 4g + b of the operand is lane 4g + b's
            uint32_t d[Tile<NS>::KS2][4];
#pragma unroll
            for (int i = 0; i < Tile<NS>::KS2; ++i)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    d[i][b] = __builtin_amdgcn_ds_bpermute(
                        16 * g + 4 * b, now.ks[mt * Tile<NS>::KS2 + i]);
#pragma unroll
            for (int c = 0; c < NT; ++c) s[c][mt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                half2v h[4];
                widen(now.k[mt * NS + k], mg, h);
                const half8 op = join8(h);
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    f32x4 x = __builtin_amdgcn_mfma_f32_16x16x32_f16(op, q[c][k], f32x4{0, 0, 0, 0}, 0,
                                                                     0, 0);
                    if constexpr (WIDE)
                        x = __builtin_amdgcn_mfma_f32_16x16x32_f16(op, q_low[c][k], x, 0, 0, 0);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const half2v pair = as_half2(d[k / 2][b]);
                        s[c][mt][b] =
                            __builtin_fmaf((float)(k & 1 ? pair.y : pair.x), x[b], s[c][mt][b]);
                    }
                    asm volatile("" : "+v"(s[c][mt]));   // here, not where they are used
                }
            }
        }
        // element b of s[c][mt]: token j0 + 8g + 4·mt + b
        const bool edge = hole || !all_visible(view, tile);
        if constexpr (BIAS) {
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = s[c][e / 4][e % 4];
                bias_scores(a, x, scale[c], slope[c], pos[c] - j0 - 8 * g, [](int e) { return e; });
#pragma unroll
                for (int e = 0; e < 8; ++e) s[c][e / 4][e % 4] = x[e];
            }
        }
        uint32_t seen[NT];   // bit 4·mt + b of column c: visible
        if (edge) {
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                seen[c] = hole ? 0u : visible_bits(range[c], view.prefix, j0) >> (8 * g);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int b = 0; b < 4; ++b) s[c][mt][b] = masked(s[c][mt][b], seen[c], 4 * mt + b);
            }
        }
        half8 w[NT], w_low[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            float top = -__builtin_inff();
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int b = 0; b < 4; ++b) top = fmaxf(top, s[c][mt][b]);
            top = max_across32(max_across16(top)) * to_log2;
            if (__any(top > m[c] + kSlack)) {
                const float mc = fmaxf(m[c], top);
                const float f = mc == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m[c] - mc);
                l[c] *= f;
#pragma unroll
                for (int i = 0; i < MT; ++i) o[c][i] *= f;
                m[c] = mc;
            }
            const float base = m[c] == -__builtin_inff() ? 0.0f : m[c] - kShift;
            float e[8];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    e[4 * mt + b] =
                        __builtin_amdgcn_exp2f(__builtin_fmaf(s[c][mt][b], to_log2, -base));
            l[c] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            uint32_t high[4], low[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pack_weights(e[2 * i], e[2 * i + 1], high[i], low[i]);
            w[c] = __builtin_bit_cast(half8, u32x4{high[0], high[1], high[2], high[3]});
            w_low[c] = __builtin_bit_cast(half8, u32x4{low[0], low[1], low[2], low[3]});
        }
        if (edge) {
            uint32_t bad = 0;
            const int tokens = hole ? 0 : view.keys - j0 - 8 * g;   // of this octet
#pragma unroll
            for (int i = 0; i < Tile<NS>::kScaleSets; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    now.vs[4 * i + e] = clean_scales(now.vs[4 * i + e], tokens, e, bad);
            if (__any(bad != 0)) {
#pragma unroll
                for (int c = 0; c < NT; ++c) nan_blocks[c] |= bad_blocks<NS>(p, g, tokens, seen[c]);
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const half8 op = value_operand(now, i, mg);
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                o[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(op, w[c], o[c][i], 0, 0, 0);
                o[c][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(op, w_low[c], o[c][i], 0, 0, 0);
            }
        }
    };
    // The wave's tiles: where they lie is looked up 64 at a time, one a lane, and each is
    // loaded while the one before is worked on.
    for (int t0 = t_begin + wave; t0 < t_end; t0 += 64 * kWaves) {
        int64_t at = -1;
        if (t0 + kWaves * lane < t_end) {
            const int tile = tile_of(t0 + kWaves * lane);
            const int page = (int)((unsigned)tile / (unsigned)per_page);
            const int id = a.kv.table[view.b * a.kv.table_ld + page];
            if ((unsigned)id < (unsigned)a.kv.pages)
                at = kv_tile_at(a.kv, head, id, tile - page * per_page);
        }
        auto place = [&](int k, bool &hole) {   // (of the cache's first tile without)
            const int64_t x = (int64_t)__builtin_amdgcn_readlane((int)(at >> 32), k) << 32 |
                              (uint32_t)__builtin_amdgcn_readlane((int)at, k);
            hole = x < 0;
            return (const char *)a.kv.cache + (hole ? 0 : x);
        };
        const int left = (t_end - t0 + kWaves - 1) / kWaves, n = left < 64 ? left : 64;
        bool hole;
        const char *p = place(0, hole);
        Tile<NS> now;
        load_tile(p, r, g, now);
        for (int k = 0; k + 1 < n; ++k) {
            bool next_hole;
            const char *next_p = place(k + 1, next_hole);
            Tile<NS> next;
            load_tile(next_p, r, g, next);
            use_tile(now, p, t0 + kWaves * k, hole);
            now = next;
            p = next_p;
            hole = next_hole;
        }
        use_tile(now, p, t0 + kWaves * (n - 1), hole);
    }

    // Join the waves: every wave's results at the common maximum.
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        l[c] += __shfl_xor(l[c], 16);
        l[c] += __shfl_xor(l[c], 32);
        nan_blocks[c] |= __shfl_xor(nan_blocks[c], 16);
        nan_blocks[c] |= __shfl_xor(nan_blocks[c], 32);
        if (g == 0) {
            wave_stats[wave][16 * c + r] = float2{m[c], l[c]};
            wave_nan[wave][16 * c + r] = nan_blocks[c];
        }
    }
    __syncthreads();
    const int64_t part = blockIdx.x;
    const bool partial = work.parts.count > 1;   // else the rows are done
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        float mc = -__builtin_inff(), lc = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) mc = fmaxf(mc, wave_stats[i][16 * c + r].x);
        const float base = mc == -__builtin_inff() ? 0.0f : mc;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            const float2 x = wave_stats[i][16 * c + r];
            lc += x.y * __builtin_amdgcn_exp2f(x.x - base);
        }
        uint32_t nan = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) nan |= wave_nan[i][16 * c + r];
        const float f = __builtin_amdgcn_exp2f(m[c] - base);
        const float inv = lc == 0.0f ? 0.0f : 1.0f / lc;
        const int row = view.rt * R + 16 * c + r;
        const int i = (int)((unsigned)row / (unsigned)a.group), h = head * a.group + row - i * a.group;
        const bool live = i < view.rows.n;
        if (partial && wave == 0 && g == 0 && live) {
            float *st = a.stats + (part * R + 16 * c + r) * 2;
            st[0] = mc;
            st[1] = lc;
        }
#pragma unroll
        for (int i0 = 0; i0 < MT; i0 += CH) {
            if (c > 0 || i0 > 0) __syncthreads();
#pragma unroll
            for (int k = 0; k < CH && i0 + k < MT; ++k)
#pragma unroll
                for (int b = 0; b < 4; ++b) join[wave][4 * k + b][lane] = o[c][i0 + k][b] * f;
            __syncthreads();
            // wave b' = `wave` finishes element row 4g + b' of each tile
            float x[CH];
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                x[k] = 0.0f;
                if (i0 + k < MT)
#pragma unroll
                    for (int v = 0; v < kWaves; ++v) x[k] += join[v][4 * k + wave][lane];
            }
            const int dr = 4 * g + wave;   // row of the output tiles
            if (nan) {
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const int d = Tile<NS>::kRuns ? MT * dr + i0 + k : 16 * (i0 + k) + dr;
                    if (nan >> (d / 32) & 1) x[k] = __builtin_nanf("");
                }
            }
            if (live && partial) {
                float *y = a.partial + (part * R + 16 * c + r) * D;
#pragma unroll
                for (int k = 0; k < CH; ++k)
                    if (i0 + k < MT) y[Tile<NS>::kRuns ? MT * dr + i0 + k : 16 * (i0 + k) + dr] = x[k];
            } else if (live) {
                uint16_t *y = a.y + (int64_t)(view.rows.first + i) * a.ldy + (int64_t)h * D;
#pragma unroll
                for (int k = 0; k < CH; ++k)
                    if (i0 + k < MT)
                        y[Tile<NS>::kRuns ? MT * dr + i0 + k : 16 * (i0 + k) + dr] =
                            (uint16_t)pack_f16x2(x[k] * inv, 0.0f);
            }
        }
    }
}

// Joins the parts of the rows that have more than one.
//   out = Σ_s f_s · o_s / Σ_s f_s · l_s,  f_s = e^(m_s − max m)

template <int NS>
__device__ __forceinline__ void store_row(const AttnArgs &a, const View &v, int head, int R, int n,
                                          const float (&x)[(32 * NS + 63) / 64], float sum) {
    constexpr int D = 32 * NS;
    const int lane = threadIdx.x & 63;
    const int row = v.rt * R + n;
    const int i = (int)((unsigned)row / (unsigned)a.group), h = head * a.group + row - i * a.group;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *out = a.y + (int64_t)(v.rows.first + i) * a.ldy + (int64_t)h * D;
#pragma unroll
    for (int e = 0; e < (D + 63) / 64; ++e)
        if (lane + 64 * e < D) out[lane + 64 * e] = (uint16_t)pack_f16x2(x[e] * inv, 0.0f);
}

// Few rows and many parts: a workgroup per row of R per job, part s to wave s % 8.
template <int NS, int R>
__global__ __launch_bounds__(512) void attention_join_parts(AttnArgs a) {
    constexpr int D = 32 * NS, E = (D + 63) / 64, W = 8;
    __shared__ float factor[kMaxSplits];
    __shared__ float sums[W][E * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = blockIdx.x % R;
    Work work;
    if (!find_work<R, true>(a, blockIdx.x / R, work)) return;
    const View &view = work.view;
    const Parts &parts = work.parts;
    const int head = work.head;
    if (view.rt * R + n >= view.rows.n * a.group) return;
    if (parts.count == 1 || work.first + parts.count > a.items) return;
    const int64_t base = work.first;
    const float2 *st = (const float2 *)a.stats + base * R + n;
    float m = -__builtin_inff(), sum = 0.0f;
    float2 t[kMaxSplits / 64];
#pragma unroll
    for (int k = 0; k < kMaxSplits / 64; ++k) {
        const int s = lane + 64 * k;
        t[k] = s < parts.count ? st[(int64_t)s * R] : float2{-__builtin_inff(), 0.0f};
        m = fmaxf(m, t[k].x);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    if (m == -__builtin_inff()) m = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxSplits / 64; ++k) {
        const float f = __builtin_amdgcn_exp2f(t[k].x - m);
        sum = __builtin_fmaf(t[k].y, f, sum);
        if (wave == 0 && lane + 64 * k < parts.count) factor[lane + 64 * k] = f;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    __syncthreads();
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.0f;
    const float *y = a.partial + (base * R + n) * D;
#pragma unroll 4
    for (int s = wave; s < parts.count; s += W) {
        const float f = factor[s];
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 64 * e < D)
                x[e] = __builtin_fmaf(y[(int64_t)s * R * D + lane + 64 * e], f, x[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[wave][64 * e + lane] = x[e];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w)
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] += sums[w][64 * e + lane];
    store_row<NS>(a, view, head, R, n, x, sum);
}

// Many rows and few parts: a workgroup per a.join_rows rows of a job, four elements per
// thread, four parts at a time with a running maximum.
template <int NS, int R>
__global__ __launch_bounds__(256) void attention_join_rows(AttnArgs a) {
    constexpr int D = 32 * NS, Q = D / 4, PASS = 256 / Q;   // threads per row, rows per pass
    constexpr int P = 4;
    const int groups = R / a.join_rows, job = (int)((unsigned)blockIdx.x / (unsigned)groups);
    Work work;
    if constexpr (R > 32) {   // the kernel for many rows: a.splits places for each job
        work.head = job % a.kv.heads;
        work.first = job * a.splits;
        if (!find_view<R>(a, job / a.kv.heads, work.view)) return;
        work.parts = parts_of(a, work.view.n, even_share(a, R));
    } else {
        if (!find_work<R, true>(a, job, work)) return;
        if (work.first + work.parts.count > a.items) return;
    }
    const View &view = work.view;
    const Parts &parts = work.parts;
    const int head = work.head;
    if (parts.count == 1) return;
    const int n0 = ((int)blockIdx.x - job * groups) * a.join_rows, e = threadIdx.x % Q * 4;
    const int rows = view.rows.n * a.group - view.rt * R;   // of this tile on
    const int end = n0 + a.join_rows < rows ? n0 + a.join_rows : rows;
    const int64_t base = (int64_t)work.first * R;
    for (int n = n0 + threadIdx.x / Q; n < end && threadIdx.x < Q * PASS; n += PASS) {
        float m = -__builtin_inff(), sum = 0.0f;
        f32x4 x = {0, 0, 0, 0};
        for (int s0 = 0; s0 < parts.count; s0 += P) {
            float2 st[P];
            f32x4 y[P];
#pragma unroll
            for (int k = 0; k < P; ++k) {   // parts beyond the last: that, with no weight
                const int s = s0 + k < parts.count ? s0 + k : parts.count - 1;
                const int64_t at = base + (int64_t)s * R + n;
                st[k] = ((const float2 *)a.stats)[at];
                y[k] = *(const f32x4 *)(a.partial + at * D + e);
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < P; ++k) top = fmaxf(top, st[k].x);
            const float shift = top == -__builtin_inff() ? 0.0f : top;
            const float f = __builtin_amdgcn_exp2f(m - shift);
            m = top;
            sum *= f;
            x *= f;
#pragma unroll
            for (int k = 0; k < P; ++k) {
                if (s0 + k >= parts.count) break;
                const float w = __builtin_amdgcn_exp2f(st[k].x - shift);
                sum = __builtin_fmaf(st[k].y, w, sum);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __builtin_fmaf(y[k][i], w, x[i]);
            }
        }
        const int row = view.rt * R + n;
        const int i = (int)((unsigned)row / (unsigned)a.group), h = head * a.group + row - i * a.group;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
        *(u2 *)(a.y + (int64_t)(view.rows.first + i) * a.ldy + (int64_t)h * D + e) =
            u2{pack_f16x2(x[0] * inv, x[1] * inv), pack_f16x2(x[2] * inv, x[3] * inv)};
    }
}

template <int NS, int R>
void launch_join(AttnArgs a, hipStream_t stream) {
    const unsigned jobs = (unsigned)a.units * a.kv.heads;
    if constexpr (R <= 32) {
        if (a.splits > 8 && jobs * R <= 512) {
            hipLaunchKernelGGL((attention_join_parts<NS, R>), dim3(jobs * R), dim3(512), 0, stream, a);
            return;
        }
    }
    a.join_rows = R <= 32 ? R : jobs <= 32 ? 8 : 32;
    hipLaunchKernelGGL((attention_join_rows<NS, R>), dim3(jobs * (R / a.join_rows)), dim3(256), 0,
                       stream, a);
}

template <int NS, int NT>
void launch_rows(const AttnArgs &a, bool bias, hipStream_t stream) {
    const dim3 grid(a.items), block(256);
    if (a.q_f32)   // (with the scores' general form: one kernel less)
        hipLaunchKernelGGL((attention_kernel<NS, NT, true, true>), grid, block, 0, stream, a);
    else if (bias)
        hipLaunchKernelGGL((attention_kernel<NS, NT, true, false>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((attention_kernel<NS, NT, false, false>), grid, block, 0, stream, a);
}

template <int NS>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, hipStream_t stream) {
    // without a cap or bias the scale goes into the exponent's factor, after the
    // mask's −∞: it has to be positive and in range there
    const bool bias = a.cap > 0.0f || a.slopes || !(a.scale > 1e-30f && a.scale < 1e30f);
    hipError_t e = hipSuccess;
    if (p.rows > 32) {
        e = launch_attention_prompt(a, bias, stream);
    } else {
        if (p.rows == 16)
            launch_rows<NS, 1>(a, bias, stream);
        else if constexpr (NS <= 4)
            launch_rows<NS, 2>(a, bias, stream);
        e = hipGetLastError();
    }
    if (e != hipSuccess || a.splits == 1) return e;
    if (p.rows == 16)
        launch_join<NS, 16>(a, stream);
    else if (p.rows > 32)
        launch_join<NS, NS <= 4 ? 256 : 128>(a, stream);
    else if constexpr (NS <= 4)
        launch_join<NS, 32>(a, stream);
    return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(const KvSpec &kv, const AttnSpec &s) {
    AttnPlan p;
    const int group = s.q_heads / kv.heads;
    // (row counts are on the device: one plan for all, by their mean.  A prompt of 2048 rows
    // beside 60 single tokens of up to 8000: 467 us so, 129 in two calls.)
    const int64_t mean = kv.cu ? ((int64_t)kv.M + kv.batch - 1) / kv.batch : kv.rows;
    const int64_t rows = mean * group;   // of a key/value head and sequence
    // Rows of a workgroup.  Up to 16 rows one column tile, up to 64 two (up to 128 where
    // contexts may be long), for heads of 256 one up to 96 (their second does not fit the
    // registers), and beyond that the kernel for many rows.  One sequence over 30000 tokens /
    // 32 sequences over 3000 / over 200, 8 key/value heads (4 of 256), us:
    //   D = 128  24 rows  16: 25.7 / 54.3 / 12.2   32: 30.2 / 49.1 / 12.4   256: 72.3 / 168 / 18.5
    //            40 rows  16: 32.7 / 72.1 / 14.8   32: 35.8 / 74.6 / 17.1   256: 67.7 / 168 / 19.1
    //            64 rows  16: 39.8 / 90.5 / 22.5   32: 37.1 / 77.7 / 22.7   256: 68.3 / 172 / 19.4
    //           128 rows  16: 63.4 / 159 / 35.7    32: 86.0 / 134 / 36.6    256: 71.2 / 176 / 20.5
    //   D = 64   96 rows  16: 35.5 / 76.5 / 15.4   32: 46.3 / 62.3 / 12.4   256: 53.6 / 115 / 14.4
    //   D = 256  32 rows  16: 35.6 / 58.1 / 14.1                            128: 83.1 / 132 / 26.0
    //            96 rows  16: 55.1 / 126 / 30.0                             128: 89.3 / 143 / 27.0
    //           128 rows  16: 70.2 / 157 / 34.1                             128: 90.7 / 141 / 27.3
    const bool wide = kv.D == 256;
    const int64_t most = wide ? 96 : s.max_len < 1024 ? 64 : 128;
    p.rows = rows <= 16 ? 16 : rows > most ? attention_prompt_rows(kv.D) : wide ? 16 : 32;
    p.row_tiles = kv.cu ? (int64_t)kv.M * group / p.rows + kv.batch
                        : (rows + p.rows - 1) / p.rows * kv.batch;
    // Parts of the keys.  (The workspace's size is asked for without the mask: none of this
    // may depend on it.)
    const int64_t jobs = p.row_tiles * kv.heads;
    const int64_t max_len = s.max_len < kMaxLen ? s.max_len : kMaxLen;
    const int64_t tiles = (max_len + kTile - 1) / kTile;
    int64_t splits;
    if (p.rows <= 32) {   // dealt out over the batch (find_work)
        p.target = kFewRowsTarget;
        splits = kMaxSplits;
    } else {
        // one workgroup per unit (512 rows over 16512 tokens 254 us; 270 with 200, 343 with
        // 300, 269 with 512)
        p.target = 256;
        splits = (1024 + jobs - 1) / jobs;
        if (kv.batch == 1) {   // the longest of the jobs against their mean, if causal
            const double mean = max_len > kv.M ? max_len - kv.M / 2 : max_len / 2 + 1;
            splits = (int64_t)(p.target / (double)jobs * (max_len / mean) + 0.5);
        }
        // few jobs: the parts' time falls with their number and the join's grows, equal at
        // some 2·√tiles (256 rows of one head of 64 over 19500 tokens 90 us with 8 parts, 39 with
        // 50; over 131000 tokens 514 with 8, 82 with 128)
        int64_t most = 8;
        while (most * jobs < 512 && most * most < 4 * tiles) ++most;
        if (splits > most) splits = most;
    }
    // Parts of four tiles, one a wave, where the few jobs leave most of the chip idle (one
    // token over 4096, four heads: 10.3 us against 11.5 with eight); with more jobs they
    // cost more to join than they give (8 sequences of 5 rows, heads of 256: 19.8 against
    // 18.4).
    p.min_tiles = p.rows <= 32 && jobs <= 64 ? 4 : 8;
    if (splits > tiles / p.min_tiles) splits = tiles / p.min_tiles;
    if (splits > kMaxSplits) splits = kMaxSplits;
    if (splits < 1) splits = 1;
    p.splits = (int)splits;
    p.items = jobs * splits;
    if (p.rows <= 32 && p.items > jobs + p.target + 8) p.items = jobs + p.target + 8;
    p.ws_bytes = splits == 1 ? 0 : p.items * p.rows * (kv.D + 2) * 4;
    return p;
}

hipError_t launch_attention(const KvSpec &kv, const AttnSpec &s, const AttnPlan &p, float *ws,
                            hipStream_t stream) {
    AttnArgs a;
    a.kv = kv;
    a.q = s.q;
    a.y = s.y;
    a.ldq = s.ldq;
    a.ldy = s.ldy;
    a.scale = s.scale;
    a.cap = s.cap;
    // (a cap below 1e-30 is as good as 0: finite all the same)
    a.inv_cap = s.cap > 1e-30f ? 1.0f / s.cap : s.cap > 0.0f ? 1e30f : 0.0f;
    a.q_f32 = s.x_type == kTypeF32;
    a.group = s.q_heads / kv.heads;
    a.causal = s.causal;
    a.window = s.window < kMaxLen ? s.window : kMaxLen;   // no sequence is longer
    a.splits = p.splits;
    a.target = p.target;
    a.min_tiles = p.min_tiles;
    a.slopes = s.slopes;
    a.prefix = s.prefix;
    a.stats = ws;
    a.items = (int)p.items;
    a.partial = ws + p.items * p.rows * 2;
    a.units = (int)p.row_tiles;
    a.per_seq = kv.cu ? 0 : (unsigned)(((int64_t)kv.rows * a.group + p.rows - 1) / p.rows);
    switch (kv.D) {
    case 64: return launch_dim<2>(a, p, stream);
    case 96: return launch_dim<3>(a, p, stream);
    case 128: return launch_dim<4>(a, p, stream);
    default: return launch_dim<8>(a, p, stream);
    }
}

}  // namespace mq
