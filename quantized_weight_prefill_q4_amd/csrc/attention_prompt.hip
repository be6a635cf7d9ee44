// Attention over the 4-bit cache for many query rows (attention_q4.hip has the
// definition and the numerics, which are the same here).
//
// With many rows the work is the matrix products and the exponentials: 4·D
// operations and one exponential per visible pair, and the expansion of the codes
// is paid once per workgroup.  A workgroup takes 128 rows of one key/value head,
// 32 for each of its four waves, and goes through the keys ST·32 tokens at a time:
// the waves expand a quarter of the tokens' operands each, into LDS, and every wave
// reads all of them.
//   Sᵀ[t, n] = K[t, :] · Q[n, :]    matrix instructions 32 x 32 x 16, keys as A
//   Oᵀ[d, n] += Vᵀ[d, t] · Pᵀ[t, n]  values as A
// Operands lie in LDS as the lanes hold them, 16 bytes per lane in lane order: no
// bank conflicts on either side.  Row ρ = 8a + 4h + b of a key operand is token
// 16·(a/2) + 8h + 4·(a%2) + b, which puts the eight tokens that a lane has to give
// to the second product's step u into its own registers 8u .. 8u + 7.
// Two LDS buffers: the next tokens' operands are expanded (from codes loaded one
// step earlier) while these are used; one barrier per step.
#include "attention_device.h"

namespace mq {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;

// One wave's share of a 32-token tile's expansion: the key operands of one parity
// of k-steps, or the value operands of one half of the tokens; NS of either.
template <int NS>
struct Codes {
    uint32_t c[NS];
    uint32_t s[4];   // keys: NS scales; values: eight of them (NS = 3: see below)
};

__device__ __forceinline__ half8 load_operand(const u32x4 *p) {
    return __builtin_bit_cast(half8, *p);
}

template <int NS, int ST, bool BIAS>
__global__ __launch_bounds__(kThreads, NS <= 4 ? 2 : 1) void attention_prompt_kernel(AttnArgs a) {
    constexpr int D = 32 * NS, KS = 2 * NS;   // KS: k-steps of the first product
    constexpr bool kRuns = (NS & (NS - 1)) == 0;
    // operands: [buffer][tile][keys KS, values 2·NS][lane]
    __shared__ u32x4 ops[2][ST][2 * KS][64];
    __shared__ int flags[2][4];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int split = blockIdx.x % a.splits;
    int job = blockIdx.x / a.splits;
    const int head = job % a.kv.heads;
    // the last row tiles see the most keys: first
    const int unit = a.units - 1 - job / a.kv.heads;
    job = unit * a.kv.heads + head;
    View view;
    if (!find_view<kRows>(a, unit, view)) return;
    make_uniform(view);
    const int chunk = part_tiles(view.n, a.splits);
    const int t_begin = split * chunk;
    const int t_end = t_begin + chunk < view.n ? t_begin + chunk : view.n;
    if (t_begin >= t_end && split > 0) return;
    const int steps = t_end > t_begin ? (t_end - t_begin + ST - 1) / ST : 0;

    // this lane's row
    const int64_t row = (int64_t)view.rt * kRows + 32 * wave + r;
    const int qi = (int)(row / a.group), qh = head * a.group + (int)(row - (int64_t)qi * a.group);
    const bool live = qi < view.rows.n;
    const int pos = view.first_pos + qi;
    const Range range = row_range(a, view, pos);
    const float slope = BIAS && a.slopes && live ? a.slopes[qh] : 0.0f;
    half8 q[KS];
    {
        const int64_t at = (int64_t)(view.rows.first + (live ? qi : 0)) * a.ldq +
                           (int64_t)(live ? qh : head * a.group) * D + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; ++s) q[s] = load_q8(a.q, a.q_f32, at + 16 * s);
    }
    f32x16 o[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
    float m = -__builtin_inff(), l = 0.0f;
    const float to_log2 = BIAS ? kLog2e : a.scale * kLog2e;

    // What a wave expands.  ST = 2: keys and values of tile wave % 2, of parity and
    // token half wave / 2.  ST = 1: waves 0 and 1 keys, 2 and 3 values, of wave % 2.
    constexpr int UNITS = ST;
    const int my_tile = ST == 2 ? wave & 1 : 0, sub = ST == 2 ? wave >> 1 : wave & 1;
    auto is_keys = [&](int n) { return ST == 2 ? n == 0 : wave < 2; };
    auto tile_of = [&](int t) { return t < view.pre ? t : t - view.pre + view.lo; };
    const int per_page = a.kv.page / kTile;
    // the page of this wave's tile of a step: read a step before its codes are
    auto page_of = [&](int step) {
        const int t = t_begin + step * ST + my_tile;
        return t < t_end ? a.kv.table[view.b * a.kv.table_ld + tile_of(t) / per_page] : -1;
    };
    Codes<NS> codes[UNITS];
    const char *tile = nullptr;   // of the codes; null: no such page, or behind the part
    auto fetch = [&](int step, int id) {
        id = uniform(id);
        const int index = tile_of(t_begin + step * ST + my_tile);
        tile = (unsigned)id < (unsigned)a.kv.pages
                   ? a.kv.cache + id * a.kv.page_bytes +
                         ((int64_t)head * per_page + index % per_page) * kv_tile_bytes(D)
                   : nullptr;
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            Codes<NS> &c = codes[n];
            if (!tile) {   // zeros: its tokens are masked
#pragma unroll
                for (int i = 0; i < NS; ++i) c.c[i] = 0x88888888u;
                c.s[0] = c.s[1] = c.s[2] = c.s[3] = 0;
                continue;
            }
            if (is_keys(n)) {
                // lane's token: row r = 8·ra + 4·rh + rb
                const int ra = r >> 3, rh = (r >> 2) & 1, rb = r & 3;
                const int place = 16 * (ra & 1) + 4 * (2 * (ra >> 1) + rh) + rb;
                const int g = 2 * sub + h;   // octets g, g + 4, ...: k-steps sub, sub + 2, ...
                load_dwords((const uint32_t *)tile + ((4 * (place >> 4) + g) * 16 + (place & 15)) * NS,
                            c.c);
                const char *sp = tile + kv_kscale_at(D) + 2 * place * NS;
                if constexpr (NS == 2) {
                    c.s[0] = *(const uint32_t *)sp;
                } else if constexpr (NS == 4) {
                    const u32x2 x = *(const u32x2 *)sp;
                    c.s[0] = x.x; c.s[1] = x.y;
                } else if constexpr (NS == 8) {
                    load_dwords((const uint32_t *)sp, c.s);
                } else {
#pragma unroll
                    for (int i = 0; i < (NS + 1) / 2; ++i)
                        c.s[i] = ((const uint16_t *)sp)[2 * i] |
                                 (2 * i + 1 < NS ? (uint32_t)((const uint16_t *)sp)[2 * i + 1] << 16 : 0u);
                }
            } else {
                const int o8 = 2 * sub + h;
                const uint32_t *p = (const uint32_t *)(tile + kv_vcode_at(D)) + o8 * D;
                if constexpr (kRuns) {
                    load_dwords(p + NS * r, c.c);
                    load_dwords((const uint32_t *)(tile + kv_vscale_at(D)) +
                                    4 * (o8 * NS + NS * r / 32), c.s);
                } else {
#pragma unroll
                    for (int i = 0; i < NS; ++i) c.c[i] = p[32 * i + r];
                }
            }
        }
    };
    // A value scale pair as it enters: those of tokens past the sequence, and in tiles
    // that are masked in part any that is not finite, are taken out.
    auto clean = [&](uint32_t s, int tokens, int e, bool &bad) {
        s = keep_halves(s, tokens > 2 * e, tokens > 2 * e + 1);
        const uint32_t x = bad_halves(s);
        bad = bad || x;
        return keep_halves(s, !(x & 0xFFFFu), !(x >> 16));
    };
    auto expand = [&](int step) {
        const int buf = step & 1;
        bool bad = false;
#pragma unroll
        for (int n = 0; n < UNITS; ++n) {
            const Codes<NS> &c = codes[n];
            if (is_keys(n)) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    half2v w[4];
                    widen(c.c[i], w);
                    const half2v pair = as_half2(c.s[i / 2]);
                    const _Float16 d = i & 1 ? pair.y : pair.x;
                    const half2v dd = {d, d};
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] *= dd;
                    ops[buf][my_tile][2 * i + sub][lane] = __builtin_bit_cast(u32x4, join8(w));
                }
            } else {
                const int o8 = 2 * sub + h;
                const int j0 = tile_of(t_begin + step * ST + my_tile) * kTile;
                const bool edge = !all_visible(a, view, j0);
                uint32_t s[4] = {c.s[0], c.s[1], c.s[2], c.s[3]};
                if (kRuns && edge)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[e] = clean(s[e], view.keys - j0 - 8 * o8, e, bad);
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    if constexpr (!kRuns) {   // a lane's operands are of different blocks
                        u32x4 x = {0, 0, 0, 0};
                        if (tile) x = ((const u32x4 *)(tile + kv_vscale_at(D)))[o8 * NS + i];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[e] = edge ? clean(x[e], view.keys - j0 - 8 * o8, e, bad) : x[e];
                    }
                    half2v w[4];
                    widen(c.c[i], w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] *= as_half2(s[e]);
                    ops[buf][my_tile][KS + 2 * i + sub][lane] = __builtin_bit_cast(u32x4, join8(w));
                }
            }
        }
        const bool any = __any(bad);
        if (lane == 0) flags[buf][wave] = (any ? 1 : 0) | (tile ? 0 : 2);
    };

    int next = page_of(0);
    if (steps > 0) {
        fetch(0, next);
        next = page_of(1);
        expand(0);
        fetch(1, next);
        next = page_of(2);
    }
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
        const int buf = step & 1;
        f32x16 s[ST];
#pragma unroll
        for (int t = 0; t < ST; ++t) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(load_operand(&ops[buf][t][k][lane]), q[k],
                                                              s[t], 0, 0, 0);
        }
        if (step + 1 < steps) {
            expand(step + 1);
            fetch(step + 2, next);
            next = page_of(step + 3);
        }
        // bits of the four waves: 1 a scale that is not finite, 2 no such tile
        int flag[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) flag[i] = uniform(flags[buf][i]);
        // element 8u + 4v + b of s[t]: token j0 + 16u + 8h + 4v + b
        bool edge = false;
        uint32_t seen[ST];
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            const int tt = t_begin + step * ST + t;
            const bool none = tt >= t_end;
            const int j0 = none ? 0 : tile_of(tt) * kTile;
            if constexpr (BIAS) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x = s[t][e] * a.scale;
                    if (a.cap > 0.0f) x = a.cap * tanh_f32(x * a.inv_cap);
                    const int j = j0 + 16 * (e >> 3) + 8 * h + (e & 7);
                    s[t][e] = x - slope * (float)(pos > j ? pos - j : j - pos);
                }
            }
            seen[t] = 0xFFFFu;
            const bool hole = none || (flag[t] & 2);   // wave t expands tile t
            if (hole || !all_visible(a, view, j0)) {
                edge = true;
                seen[t] = 0;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool see = !hole &
                        in_range(range, view.prefix, j0 + 16 * (e >> 3) + 8 * h + (e & 7));
                    seen[t] |= (uint32_t)see << e;
                    s[t][e] = see ? s[t][e] : -__builtin_inff();
                }
            }
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[t][e]);
        top = fmaxf(top, __shfl_xor(top, 32));
        top *= to_log2;
        const float mc = fmaxf(m, top);
        if (__any(mc > m)) {
            const float f = mc == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(m - mc);
            l *= f;
#pragma unroll
            for (int i = 0; i < NS; ++i) o[i] *= f;
            m = mc;
        }
        const float base = mc == -__builtin_inff() ? 0.0f : mc - kShift;
        half8 w[ST][2];
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    e[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][8 * u + k], to_log2, -base));
                    l += e[k];
                }
                w[t][u] = __builtin_bit_cast(half8, u32x4{pack_f16x2(e[0], e[1]), pack_f16x2(e[2], e[3]),
                                                          pack_f16x2(e[4], e[5]), pack_f16x2(e[6], e[7])});
            }
        if (edge && ((flag[0] | flag[1] | flag[2] | flag[3]) & 1)) {
            // scales that are not finite, taken out above: NaN for the rows that see them
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                const int tt = t_begin + step * ST + t;
                const char *tile = tt < t_end ? kv_tile(a.kv, view.b, head, tile_of(tt)) : nullptr;
                if (!tile) continue;
                const int j0 = tile_of(tt) * kTile;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int o8 = 2 * u + h, tokens = view.keys - j0 - 8 * o8;
                    u32x4 see;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        see[e] = (seen[t] >> (8 * u + 2 * e) & 1 ? 0x3C00u : 0u) |
                                 (seen[t] >> (8 * u + 2 * e + 1) & 1 ? 0x3C000000u : 0u);
#pragma unroll
                    for (int i = 0; i < NS; ++i) {
                        const int group = kRuns ? NS * r / 32 : i;
                        const u32x4 sc = ((const u32x4 *)(tile + kv_vscale_at(D)))[o8 * NS + group];
                        u32x4 ind;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            ind[e] = bad_halves(keep_halves(sc[e], tokens > 2 * e, tokens > 2 * e + 1));
                        f32x16 hit;
#pragma unroll
                        for (int e = 0; e < 16; ++e) hit[e] = 0.0f;
                        hit = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                            __builtin_bit_cast(half8, ind), __builtin_bit_cast(half8, see), hit, 0, 0, 0);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[i][e] = hit[e] > 0.0f ? __builtin_nanf("") : o[i][e];
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        load_operand(&ops[buf][t][KS + 2 * i + u][lane]), w[t][u], o[i], 0, 0, 0);
        __syncthreads();
    }

    l += __shfl_xor(l, 32);
    if (!live) return;
    // register 4a + b of o[i]: row ρ = 8a + 4h + b, element NS·ρ + i (or 32·i + ρ)
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t part = ((int64_t)job * a.splits + split) * kRows + 32 * wave + r;
    if (a.splits > 1 && h == 0) {
        a.stats[2 * part] = m;
        a.stats[2 * part + 1] = l;
    }
    uint16_t *y = a.y + (int64_t)(view.rows.first + qi) * a.ldy + (int64_t)qh * D;
    float *py = a.partial + part * D;
#pragma unroll
    for (int ra = 0; ra < 4; ++ra) {
        float x[4 * NS];   // kRuns: elements NS·(8a + 4h) + [0, 4·NS)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < NS; ++i) x[kRuns ? NS * b + i : 4 * i + b] = o[i][4 * ra + b];
        const int rho = 8 * ra + 4 * h;
#pragma unroll
        for (int e = 0; e < 4 * NS; e += 4) {
            const int d = kRuns ? NS * rho + e : 32 * (e / 4) + rho;
            if (a.splits > 1) {
                *(f32x4 *)(py + d) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
            } else {
                typedef uint32_t u2 __attribute__((ext_vector_type(2), aligned(2)));
                *(u2 *)(y + d) = u2{pack_f16x2(x[e] * inv, x[e + 1] * inv),
                                    pack_f16x2(x[e + 2] * inv, x[e + 3] * inv)};
            }
        }
    }
}

template <int NS, int ST>
hipError_t launch(const AttnArgs &a, bool bias, hipStream_t stream) {
    const dim3 grid((unsigned)(a.units * a.kv.heads * a.splits));
    if (bias)
        hipLaunchKernelGGL((attention_prompt_kernel<NS, ST, true>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((attention_prompt_kernel<NS, ST, false>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_prompt(const AttnArgs &a, bool bias, hipStream_t stream) {
    switch (a.kv.D) {
    case 64: return launch<2, 2>(a, bias, stream);
    case 96: return launch<3, 2>(a, bias, stream);
    case 128: return launch<4, 2>(a, bias, stream);
    default: return launch<8, 1>(a, bias, stream);
    }
}

}  // namespace mq
