// Attention over the 4-bit cache for many query rows (attention_q4.hip has the
// definition and the numerics; here the keys d·(q − 8) enter as two f16 numbers whose sum
// they are, which keeps blocks in one sum, and f32 queries lose 2^-18 of a product, that of
// both low parts).
//
// With many rows the work is the matrix products and the exponentials: 4·D
// operations and one exponential per visible pair, and the expansion of the codes
// is paid once per workgroup.  A workgroup takes 32 rows of one key/value head for
// each of its waves (eight; four for heads of 256, which need the registers of two)
// and goes through the keys 32 tokens at a time: each wave expands its share of the
// tile's operands into LDS and reads all of them.
//   Sᵀ[t, n] = K[t, :] · Q[n, :]    matrix instructions 32 x 32 x 16, keys as A, twice:
//                                   both parts of the keys; f32 queries' low part a third
//   Oᵀ[d, n] += Vᵀ[d, t] · Pᵀ[t, n]  values as A, twice: both parts of the weights
// Operands lie in LDS as the lanes hold them, 16 bytes per lane in lane order: no
// bank conflicts on either side.  Row ρ = 8a + 4h + b of a key operand is token
// 16·(a/2) + 8h + 4·(a%2) + b, which puts the eight tokens that a lane has to give
// to the second product's step u into its own registers 8u .. 8u + 7.
//
// In one step the scores of the next tile are multiplied while this tile's weights are
// computed, and this tile's values while later operands are expanded (keys two tiles
// ahead, values one).  The codes go to LDS as they lie, 16 bytes a lane (each wave
// loading its own operands' codes is five loads of 2 to 16 bytes a lane instead of
// one), three tiles ahead of their use and loaded two steps before.  One barrier per
// step.
//
// What bounds it: the matrix instructions.  A step of 256 rows by 32 tokens (D = 128) takes
// 3270 cycles, at the 2.0 to 2.1 GHz that the power limit leaves with all compute units at
// work, and they fill 2048; over long contexts (512 rows over 16512 tokens, 254 us without a
// cap, 9 of them the join's) they run at 1.1 PFLOP/s, where a large matrix product alone
// reaches 1.17.  Starting a workgroup takes 9000 cycles (three loads one after the other:
// lengths, page numbers, tiles), ending it 3900.
// What the parts cost there, in one measurement: keys and weights as one f16 each 188 us,
// keys as two 225, both 266; the error against 64 bits, in units of the output's own
// rounding, is 2.4, 1.5 and 1.25.
// Tried without gain: the values' products a step later, beside the maximum (within 3%
// either way); with one f16 each (then 2480 cycles a step): two tiles per barrier (the
// same), waves of a SIMD half a step apart by a second barrier (2900), 128 rows per
// workgroup and two workgroups per unit (261 us against 192), 64 rows per wave (operands in
// accumulation registers have to be copied).
#include "attention_device.h"

namespace mq {
namespace {

__device__ __forceinline__ half8 load_operand(const u32x4 *p) {
    return __builtin_bit_cast(half8, *p);
}

// What the wave's lanes wrote to LDS is there for all of them.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int V>
struct Int {
    static constexpr int value = V;
};

// One wave's share of a tile's keys or values, as loaded: PW operands (number PW·wave
// + k: k-steps of the keys; values by token half and tile of elements) and the scales of
// their pairs (a key's is one, in x).  Waves past the last operand have none.
template <int NS, int PW>
struct Codes {
    static constexpr bool kRuns = (NS & (NS - 1)) == 0;   // one set of scales serves all values
    static constexpr int SETS = kRuns ? (PW + 1) / 2 : PW;
    static constexpr int key_set(int k) { return kRuns ? k / 2 : k; }
    static constexpr int value_set(int k) { return kRuns ? 0 : k; }
    uint32_t c[PW];
    u32x4 s[SETS];
};

template <int NS, int WAVES, bool BIAS, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void attention_prompt_kernel(AttnArgs a) {
    constexpr int D = 32 * NS, KS = 2 * NS;   // KS: k-steps of the first product
    constexpr int ROWS = 32 * WAVES;
    constexpr int PW = (KS + WAVES - 1) / WAVES;   // operands that a wave expands
    constexpr int CHUNKS = kv_tile_bytes(D) / 16, PIECES = (CHUNKS + 64 * WAVES - 1) / (64 * WAVES);
    constexpr int kRowChunks = D / 8 + 1;   // 16 bytes each; odd: no bank conflicts
    typedef Codes<NS, PW> Share;
    constexpr bool kRuns = Share::kRuns, kWhole = PW * WAVES == KS;
    static_assert(KS % PW == 0 && (!kRuns || NS % PW == 0), "a wave's operands share their scales");
    // operands: [buffer][keys, what their rounding left, values][operand][lane], and in the
    // same place a wave's rows of queries on their way in and of results on their way out
    constexpr int OPS = 2 * 3 * KS * 64, ROWS_LDS = WAVES * 32 * kRowChunks;
    __shared__ u32x4 lds[OPS > ROWS_LDS ? OPS : ROWS_LDS];
    u32x4(*const ops)[3][KS][64] = (u32x4(*)[3][KS][64])lds;
    __shared__ u32x4 raw[3][CHUNKS];   // tiles as they lie in the cache
    // of a tile masked in part: tokens whose scale is not finite, a byte by h and token half
    __shared__ uint32_t bad_tokens[2][NS];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    int split, job, head;
    find_job(a, blockIdx.x, split, job, head);
    // the last row tiles see the most keys: first
    const int unit = a.units - 1 - job / a.kv.heads;
    job = unit * a.kv.heads + head;
    View view;
    if (!find_view<ROWS>(a, unit, view)) return;
    make_uniform(view);
    Parts parts = parts_of(a, view.n, even_share(a, ROWS));
    parts.per = uniform(parts.per);
    parts.count = uniform(parts.count);
    if (split >= parts.count) return;
    const int t_begin = split * parts.per;
    const int t_end = t_begin + parts.per < view.n ? t_begin + parts.per : view.n;

    // this lane's row
    const int slot = 32 * wave + r;
    const int row = view.rt * ROWS + slot;
    const int qi = (int)((unsigned)row / (unsigned)a.group), qh = head * a.group + row - qi * a.group;
    const bool live = qi < view.rows.n;
    const int pos = view.first_pos + qi;
    const Range range = row_range(a, view, pos);
    const float slope = BIAS && a.slopes && live ? a.slopes[qh] : 0.0f;
    f32x16 o[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;
    uint32_t nan_blocks = 0;   // blocks of the lane's row that must become NaN
    const float to_log2 = BIAS ? kLog2e : a.scale * kLog2e;
    const uint32_t mg = magic();

    // The tiles in turn: [0, pre), then from lo on.  Where they lie is looked up 64 at a
    // time, one a lane (a page walked in scalar instructions, one waiting for the other, was
    // 500 cycles of a step): byte offsets (the cache's
    // first tile where there is none), and a bit each for those masked in part or wholly
    // and for holes among them (no such page, or behind the part).
    const int per_page = a.kv.page / kTile;
    const int32_t *const table = a.kv.table + view.b * a.kv.table_ld;
    auto tile_of = [&](int t) { return t < view.pre ? t : t - view.pre + view.lo; };
    int64_t place_at;
    uint64_t hole_bits, edge_bits;
    auto look_up = [&](int t0) {
        const int t = t0 + lane, tile = tile_of(t);
        const int page = (int)((unsigned)tile / (unsigned)per_page);
        const int id = t < t_end ? table[page] : -1;
        const bool hole = (unsigned)id >= (unsigned)a.kv.pages;
        place_at = hole ? 0 : kv_tile_at(a.kv, head, id, tile - page * per_page);
        hole_bits = __ballot(hole);
        edge_bits = __ballot(hole || !all_visible(view, tile));
    };
    auto place = [&](int k) {
        return a.kv.cache + ((int64_t)__builtin_amdgcn_readlane((int)(place_at >> 32), k) << 32 |
                             (uint32_t)__builtin_amdgcn_readlane((int)place_at, k));
    };
    // Bits of the tiles in the pipeline, this one's first.
    uint32_t holes, edges;

    // Lane's token of a key operand: row r = 8·ra + 4·rh + rb.  K-step s takes octet 2s + h
    // of the token's elements, which lies in block s / 2.  Byte offsets within a tile:
    const int mine = kWhole || PW * wave < KS ? wave : 0;
    const int token_place = 16 * ((r >> 3) & 1) + 4 * (2 * (r >> 4) + ((r >> 2) & 1)) + (r & 3);
    const int s0 = PW * mine, o8 = 2 * (s0 / NS) + h;   // o8: octet of the value operands
    const uint32_t kcode_at =
        4 * (((4 * (token_place >> 4) + h) * 16 + (token_place & 15)) * NS + 32 * NS * (s0 & 1) + s0 / 2);
    const uint32_t kscale_at = kv_kscale_at(D) + 2 * (token_place * NS + s0 / 2);
    const uint32_t vcode_at = kv_vcode_at(D) + 4 * (o8 * D + NS * r + s0 % NS);
    const uint32_t vscale_at = kv_vscale_at(D) + 16 * (o8 * NS + NS * r / 32);
    auto load_piece = [&](const char *p, u32x4 (&x)[PIECES]) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int chunk = 64 * (WAVES * i + wave) + lane;
            if (chunk < CHUNKS) x[i] = ((const u32x4 *)p)[chunk];
        }
    };
    auto store_piece = [&](const u32x4 (&x)[PIECES], u32x4 *to) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int chunk = 64 * (WAVES * i + wave) + lane;
            if (chunk < CHUNKS) to[chunk] = x[i];
        }
    };
    auto read_key_codes = [&](const u32x4 *tile, Share &c) {
        const char *const p = (const char *)tile;
#pragma unroll
        for (int k = 0; k < PW; ++k)
            c.c[k] = *(const uint32_t *)(p + kcode_at + 128 * NS * (k & 1) + 4 * (k / 2));
#pragma unroll
        for (int k = 0; k < PW; ++k)
            if (k == 0 || Share::key_set(k) > Share::key_set(k - 1))
                c.s[Share::key_set(k)].x = *(const uint16_t *)(p + kscale_at + 2 * (k / 2));
    };
    auto read_value_codes = [&](const u32x4 *tile, Share &c) {
        const char *const p = (const char *)tile;
        if constexpr (kRuns) {
            load_dwords((const uint32_t *)(p + vcode_at), c.c);
            c.s[0] = *(const u32x4 *)(p + vscale_at);
        } else {
#pragma unroll
            for (int k = 0; k < PW; ++k) {
                const int x = 2 * ((s0 + k) / NS) + h, i = (s0 + k) % NS;
                c.c[k] = *(const uint32_t *)(p + kv_vcode_at(D) + 4 * (x * D + 32 * i + r));
                c.s[k] = *(const u32x4 *)(p + kv_vscale_at(D) + 16 * (x * NS + i));
            }
        }
    };
    // Takes scales out of a tile that is masked in part (clean_scales).
    auto clean_values = [&](Share &c, int t, bool hole, int buf) {
#pragma unroll
        for (int k = 0; k <= Share::value_set(PW - 1); ++k) {
            const int u = (s0 + k) / NS;
            const int tokens = hole ? 0 : view.keys - tile_of(t) * kTile - 8 * (2 * u + h);
            uint32_t bad = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) c.s[k][e] = clean_scales(c.s[k][e], tokens, e, bad);
            ((uint8_t *)&bad_tokens[buf][kRuns ? NS * r / 32 : (s0 + k) % NS])[2 * h + u] =
                (uint8_t)bad;
        }
    };
    // Operand k of a share, into LDS.
    auto expand_key = [&](const Share &c, int k, int buf) {
        half2v w[4], low[4], dh, dl;
        widen(c.c[k], mg, w);
        split_scales(c.s[Share::key_set(k)].x, dh, dl);
        const half2v hh = {dh.x, dh.x}, ll = {dl.x, dl.x};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            low[e] = w[e] * ll;
            w[e] *= hh;
        }
        if (kWhole || PW * wave < KS) {
            ops[buf][0][PW * wave + k][lane] = __builtin_bit_cast(u32x4, join8(w));
            ops[buf][1][PW * wave + k][lane] = __builtin_bit_cast(u32x4, join8(low));
        }
    };
    auto expand_value = [&](const Share &c, int k, int buf) {
        half2v w[4];
        widen(c.c[k], mg, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] *= as_half2(c.s[Share::value_set(k)][e]);
        if (kWhole || PW * wave < KS)   // [half][element tile]
            ops[buf][2][PW * wave + k][lane] = __builtin_bit_cast(u32x4, join8(w));
    };
    // K-step k of the first product, its operands one after the other.
    auto key_operand = [&](int buf, int i) { return load_operand(&ops[buf][i & 1][i / 2][lane]); };

    // Fill the pipeline.
    look_up(t_begin);
    // Global memory is read and written along the rows, 16 bytes a lane: lanes of 32
    // different rows would cost a cycle each (a 256-row workgroup: 4 us of 2.5 + 8).
    u32x4 *const stage = lds + wave * 32 * kRowChunks;
    half8 q[KS];
    const int64_t q_row = (int64_t)(view.rows.first + (live ? qi : 0)) * a.ldq +
                          (int64_t)(live ? qh : head * a.group) * D;
    int64_t q_at[KS];
    half8 q_in[KS], q_low_in[WIDE ? KS : 1];
    float scale = a.scale;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
        const int chunk = 64 * k + lane, n = chunk / (D / 8);
        q_at[k] = __shfl(q_row, n) + 8 * (chunk - n * (D / 8));
    }
    if constexpr (WIDE) {
        float x[KS][8];
#pragma unroll
        for (int k = 0; k < KS; ++k) load_q8((const float *)a.q, q_at[k], x[k]);
        // the largest of each chunk, and by them that of the lane's row
        float *const tops = (float *)stage;
#pragma unroll
        for (int k = 0; k < KS; ++k) tops[64 * k + lane] = largest_of(x[k], 0.0f);
        wave_sync();
        f32x4 top = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const f32x4 t = ((const f32x4 *)tops)[r * (D / 32) + i];
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], t[e]);
        }
        const int shift = query_shift(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
        scale = shifted_scale(a.scale, shift);
#pragma unroll
        for (int k = 0; k < KS; ++k)
            split_q8(x[k], __shfl(shift, (64 * k + lane) / (D / 8)), q_in[k], q_low_in[k]);
        wave_sync();   // the place is used again
    } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) q_in[k] = load_q8((const uint16_t *)a.q, q_at[k]);
    }
    u32x4 pa[PIECES], pb[PIECES];   // the wave's share of two tiles on their way to LDS
    {
        u32x4 first[3][PIECES];
#pragma unroll
        for (int k = 0; k < 3; ++k) load_piece(place(k), first[k]);
        load_piece(place(3), pa);
        load_piece(place(4), pb);
        holes = (uint32_t)hole_bits & 31;
        edges = (uint32_t)edge_bits & 31;
#pragma unroll
        for (int k = 0; k < 3; ++k) store_piece(first[k], raw[k]);
    }
    half8 q_low[WIDE ? KS : 1];
    auto turn = [&](const half8 (&in)[KS], half8 (&out)[KS]) MQ_INLINE {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int chunk = 64 * k + lane, n = chunk / (D / 8);
            stage[chunk + n] = __builtin_bit_cast(u32x4, in[k]);
        }
        wave_sync();
#pragma unroll
        for (int s = 0; s < KS; ++s) out[s] = load_operand(&stage[r * kRowChunks + 2 * s + h]);
    };
    turn(q_in, q);
    if constexpr (WIDE) {
        wave_sync();
        turn(q_low_in, q_low);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        Share c;
        read_key_codes(raw[i], c);
#pragma unroll
        for (int k = 0; k < PW; ++k) expand_key(c, k, i);
    }
    {
        Share c;
        read_value_codes(raw[0], c);
        if (edges & 1) clean_values(c, t_begin, holes & 1, 0);
#pragma unroll
        for (int k = 0; k < PW; ++k) expand_value(c, k, 0);
    }
    int raw1 = 1, raw2 = 2, raw3 = 0;   // raw buffers of the next three tiles
    __syncthreads();
    f32x16 s;
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
        const half8 op = key_operand(0, i);
        s = __builtin_amdgcn_mfma_f32_32x32x16_f16(op, q[i / 2], s, 0, 0, 0);
        if constexpr (WIDE)
            if (i % 2 == 0) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(op, q_low[i / 2], s, 0, 0, 0);
    }
    __syncthreads();
    constexpr int kAhead = 4;   // operands are read as far ahead of their use
    uint32_t w[8], w_low[8];   // a tile's weights by pairs
    // The elements of s that the lane's row sees, a bit each, in a tile masked in part.
    auto seen_bits = [&](int t) {
        const uint32_t seen =
            holes & 1 ? 0u : visible_bits(range, view.prefix, tile_of(t) * kTile) >> (8 * h);
        return (seen & 0xFFu) | (seen >> 8 & 0xFF00u);
    };
    // Marks blocks of the row that saw a value with a scale that is not finite.
    auto mark_bad = [&](int buf, int t) {
        uint32_t bad[NS], any = 0;
#pragma unroll
        for (int b = 0; b < NS; ++b) any |= bad[b] = bad_tokens[buf][b];
        if (uniform(any)) {
            const uint32_t seen = seen_bits(t);
#pragma unroll
            for (int b = 0; b < NS; ++b)
                nan_blocks |= (bad[b] >> (16 * h) & seen ? 1u : 0u) << b;
        }
    };
    // The weights of tile t from its scores, beside the scores of the next.
    auto weigh = [&](auto parity, int t) MQ_INLINE {
        constexpr int BUF = decltype(parity)::value;
        if constexpr (BIAS) {
            float x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = s[e];
            bias_scores(a, x, scale, slope, pos - tile_of(t) * kTile - 8 * h,
                        [](int e) { return 16 * (e >> 3) + (e & 7); });
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = x[e];
        }
        if (edges & 1) {
            const uint32_t seen = seen_bits(t);
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = masked(s[e], seen, e);
        }
        half8 kop[2 * KS];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) kop[i] = key_operand(BUF ^ 1, i);
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, s[e]);
        top = max_across32(top) * to_log2;
        if (__any(top > m + kSlack)) {
            const float mc = fmaxf(m, top);
            const float f = mc == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - mc);
            l *= f;
#pragma unroll
            for (int i = 0; i < NS; ++i) o[i] *= f;
            m = mc;
        }
        const float base = m == -__builtin_inff() ? 0.0f : m - kShift;
        // The order below is the order of issue (the scheduler would put each LDS read
        // right before its use): between two matrix instructions, what they leave time for.
        // The next tile's scores beside this one's weights and the reading of its values.
        f32x16 ahead;
#pragma unroll
        for (int e = 0; e < 16; ++e) ahead[e] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int i = 2 * k; i < 2 * k + 2; ++i) {
                ahead = __builtin_amdgcn_mfma_f32_32x32x16_f16(kop[i], q[k], ahead, 0, 0, 0);
                if constexpr (WIDE)
                    if (i == 2 * k)
                        ahead =
                            __builtin_amdgcn_mfma_f32_32x32x16_f16(kop[i], q_low[k], ahead, 0, 0, 0);
                if (i + kAhead < 2 * KS) kop[i + kAhead] = key_operand(BUF ^ 1, i + kAhead);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (x * KS / 8 == k) {
                    const float e0 =
                        __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * x], to_log2, -base));
                    const float e1 =
                        __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * x + 1], to_log2, -base));
                    l += e0 + e1;
                    pack_weights(e0, e1, w[x], w_low[x]);
                    asm volatile("" : "+v"(w[x]), "+v"(w_low[x]));   // here, not where they are used
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        s = ahead;
    };
    // Their products with its values, beside the expansion of keys kc (two tiles ahead) and
    // values vc (one).
    auto multiply = [&](auto parity, const Share &kc, const Share &vc) MQ_INLINE {
        constexpr int BUF = decltype(parity)::value;
        half8 vop[KS];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) vop[k] = load_operand(&ops[BUF][2][k][lane]);
#pragma unroll
        for (int k = 0; k < KS; ++k) {   // operand [half][element tile]
            const int u = k / NS, i = k % NS;
            const u32x4 x = {w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]};
            const u32x4 y = {w_low[4 * u], w_low[4 * u + 1], w_low[4 * u + 2], w_low[4 * u + 3]};
            o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vop[k], __builtin_bit_cast(half8, x), o[i],
                                                          0, 0, 0);
            if (k + kAhead < KS) vop[k + kAhead] = load_operand(&ops[BUF][2][k + kAhead][lane]);
            o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vop[k], __builtin_bit_cast(half8, y), o[i],
                                                          0, 0, 0);
#pragma unroll
            for (int z = 0; z < 2 * PW; ++z)
                if (z * KS / (2 * PW) == k) {
                    if (z < PW)
                        expand_key(kc, z, BUF);
                    else
                        expand_value(vc, z - PW, BUF ^ 1);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // One step.  p: of tile t + 3, to LDS now; that of tile t + 5 is loaded.
    auto step = [&](auto parity, int t, u32x4 (&p)[PIECES]) MQ_INLINE {
        constexpr int BUF = decltype(parity)::value;
        Share kc, vc;
        read_key_codes(raw[raw2], kc);
        read_value_codes(raw[raw1], vc);
        // the wave with more vector instructions before the other of its SIMD (a 2048-token
        // prompt 98 us without, 90 with)
        __builtin_amdgcn_s_setprio(1);
        weigh(parity, t);
        __builtin_amdgcn_s_setprio(0);
        if (edges & 1) mark_bad(BUF, t);
        if (edges & 2) clean_values(vc, t + 1, holes & 2, BUF ^ 1);
        multiply(parity, kc, vc);
        store_piece(p, raw[raw3]);
        const int k = (t + 5 - t_begin) & 63;
        if (k == 0) look_up(t + 5);
        load_piece(place(k), p);
        holes = holes >> 1 | (uint32_t)(hole_bits >> k & 1) << 4;
        edges = edges >> 1 | (uint32_t)(edge_bits >> k & 1) << 4;
        const int next = raw1;
        raw1 = raw2;
        raw2 = raw3;
        raw3 = next;
        __syncthreads();
    };
    for (int t = t_begin; t < t_end; ++t) {
        step(Int<0>{}, t, pa);
        if (++t >= t_end) break;
        step(Int<1>{}, t, pb);
    }

    // The row's place is computed again: the loop has no registers to keep it in.
    const int lane_again = (int)opaque((uint32_t)lane);
    {
        const int lane = lane_again, r = lane & 31, h = lane >> 5, slot = 32 * wave + r;
        const int row = view.rt * ROWS + slot, qi = (int)((unsigned)row / (unsigned)a.group);
        const int qh = head * a.group + row - qi * a.group;
        l += __shfl_xor(l, 32);
        nan_blocks |= __shfl_xor(nan_blocks, 32);
        // register 4a + b of o[i]: row ρ = 8a + 4h + b, element NS·ρ + i (or 32·i + ρ)
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t part = ((int64_t)job * a.splits + split) * ROWS + slot;
        const bool partial = parts.count > 1;   // else the row is done
        const int total = view.rows.n * a.group;
        if (partial && h == 0 && row < total) {
            a.stats[2 * part] = m;
            a.stats[2 * part + 1] = l;
        }
        if (__any(nan_blocks != 0)) {
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int rho = 8 * (e / 4) + 4 * h + e % 4, d = kRuns ? NS * rho + i : 32 * i + rho;
                    if (nan_blocks >> (d / 32) & 1) o[i][e] = __builtin_nanf("");
                }
        }
        // quads of a row's elements: number j of o's registers 4·ra .. 4·ra + 3 is
        // kRuns: elements NS·(8·ra + 4·h) + 4·j and on, else 32·j + 8·ra + 4·h and on
        auto quad = [&](int ra, int j) {
            f32x4 x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = kRuns ? o[(4 * j + e) % NS][4 * ra + (4 * j + e) / NS] : o[j][4 * ra + e];
            return x;
        };
        if (partial) {   // half the elements at a time: f32 rows are twice as long
            f32x4 *const py = (f32x4 *)(a.partial + (part - slot + 32 * wave) * D);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wave_sync();
#pragma unroll
                for (int rb = 0; rb < 2; ++rb)
#pragma unroll
                    for (int j = 0; j < NS; ++j)
                        stage[r * kRowChunks + (kRuns ? NS * (2 * rb + h) + j : 4 * j + 2 * rb + h)] =
                            __builtin_bit_cast(u32x4, quad(2 * half + rb, j));
                wave_sync();
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int chunk = 64 * k + lane, n = chunk / (D / 8), c = chunk - n * (D / 8);
                    if (row - r + n < total)
                        py[n * (D / 4) + (kRuns ? half * (D / 8) + c : 8 * (c / 4) + 4 * half + c % 4)] =
                            __builtin_bit_cast(f32x4, stage[chunk + n]);
                }
            }
        } else {
            const int64_t mine = (int64_t)(view.rows.first + qi) * a.ldy + (int64_t)qh * D;
            typedef uint32_t u2 __attribute__((ext_vector_type(2)));
            wave_sync();
#pragma unroll
            for (int ra = 0; ra < 4; ++ra)
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    const f32x4 x = quad(ra, j);
                    const int at = kRuns ? NS * (2 * ra + h) + j : 8 * j + 2 * ra + h;
                    ((u2 *)&stage[r * kRowChunks])[at] =
                        u2{pack_f16x2(x[0] * inv, x[1] * inv), pack_f16x2(x[2] * inv, x[3] * inv)};
                }
            wave_sync();
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int chunk = 64 * k + lane, n = chunk / (D / 8), c = chunk - n * (D / 8);
                const int64_t at = __shfl(mine, n) + 8 * c;
                if (row - r + n < total) *(q_u32x4_a2 *)(a.y + at) = stage[chunk + n];
            }
        }
    }
}

template <int NS, int WAVES>
hipError_t launch(const AttnArgs &a, bool bias, hipStream_t stream) {
    const dim3 grid((unsigned)(a.units * a.kv.heads * a.splits)), block(64 * WAVES);
    if (a.q_f32)   // (with the scores' general form: one kernel less)
        hipLaunchKernelGGL((attention_prompt_kernel<NS, WAVES, true, true>), grid, block, 0, stream, a);
    else if (bias)
        hipLaunchKernelGGL((attention_prompt_kernel<NS, WAVES, true, false>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((attention_prompt_kernel<NS, WAVES, false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

int attention_prompt_rows(int D) { return D <= 128 ? 256 : 128; }

hipError_t launch_attention_prompt(const AttnArgs &a, bool bias, hipStream_t stream) {
    switch (a.kv.D) {
    case 64: return launch<2, 8>(a, bias, stream);
    case 96: return launch<3, 8>(a, bias, stream);
    case 128: return launch<4, 8>(a, bias, stream);
    default: return launch<8, 4>(a, bias, stream);
    }
}

}  // namespace mq
