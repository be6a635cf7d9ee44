// What a workgroup of the attention kernels sees: its rows of the batch, and the
// tiles of keys that any of them reads.
#pragma once

#include "kv_q4.h"

namespace mq {

struct AttnArgs {
    KvSpec kv;
    const void *q;
    uint16_t *y;
    int64_t ldq, ldy;
    float scale, cap, inv_cap;        // cap 0: none
    int q_f32, q_heads, group, causal, window, splits;
    const float *slopes;
    const int32_t *prefix;
    float *stats, *partial;           // workspace: [row tile][head][split][R][2] and [..][R][D]
    int64_t per_seq;                  // row tiles of a sequence (equal rows)
    int units;                        // row tiles of the batch
};

// The kernel for many rows (attention_prompt.hip); launches it alone.
hipError_t launch_attention_prompt(const AttnArgs &a, bool bias, hipStream_t stream);

namespace {

constexpr int kMinTiles = 8;   // tiles of a part: fewer do not pay for the join

// What a workgroup's rows see: tiles [0, pre) and [lo, lo + n − pre).
struct View {
    int b, rt;                // sequence, row tile within it
    SeqRows rows;
    int len, keys, prefix;
    int first_pos;            // of the sequence's first new row (may be negative)
    int p_min, p_max;         // of the row tile's rows
    int pre, lo, n;
};

template <int R>
MQ_INDEX bool find_view(const AttnArgs &a, int64_t unit, View &v) {
    int64_t within;
    v.b = find_seq(a.kv, unit, a.group, R, 1, a.per_seq, &within);
    v.rows = seq_rows(a.kv, v.b);
    const int64_t total = (int64_t)v.rows.n * a.group;
    if (within < 0 || within * R >= total) return false;
    v.rt = (int)within;
    v.len = seq_len(a.kv, v.b);
    v.keys = seq_keys(a.kv, v.len);
    v.first_pos = v.len - v.rows.n;
    const int64_t last = (within + 1) * R < total ? (within + 1) * R : total;
    v.p_min = v.first_pos + (int)(within * R / a.group);
    v.p_max = v.first_pos + (int)((last - 1) / a.group);
    v.prefix = a.prefix ? clampi(a.prefix[v.b], 0, v.keys) : 0;
    int64_t lo = 0, hi = v.keys;
    if (a.window) {
        lo = (int64_t)v.p_min - a.window + 1;
        if (lo < 0) lo = 0;
        if ((int64_t)v.p_max + a.window < hi) hi = (int64_t)v.p_max + a.window;
    }
    if (a.causal && (int64_t)v.p_max + 1 < hi) hi = (int64_t)v.p_max + 1;
    if (hi < v.prefix) hi = v.prefix;
    if (hi < 0) hi = 0;
    v.pre = (v.prefix + kTile - 1) / kTile;
    v.lo = (int)(lo / kTile);
    const int end = (int)((hi + kTile - 1) / kTile);
    if (v.pre >= v.lo) v.pre = v.lo = 0;
    v.n = v.pre + (end > v.lo ? end - v.lo : 0);
    return true;
}

// Tiles of a part: a multiple of four, so that the waves share it evenly.
MQ_INDEX int part_tiles(int n, int splits) {
    const int c = ((n + splits - 1) / splits + 3) & ~3;
    return c < kMinTiles ? kMinTiles : c;
}

// The tokens that the row at position p sees: [lo, hi), and those before the prefix.
struct Range {
    int lo, hi;
};
MQ_INDEX Range row_range(const AttnArgs &a, const View &v, int p) {
    Range r{0, v.keys};
    if (a.window) {
        const int64_t lo = (int64_t)p - a.window + 1, hi = (int64_t)p + a.window;
        if (lo > 0) r.lo = (int)lo;
        if (hi < r.hi) r.hi = (int)hi;
    }
    if (a.causal && p + 1 < r.hi) r.hi = p + 1;
    return r;
}
// (without branches: eight of these per lane and column of a tile)
MQ_INDEX bool in_range(const Range &r, int prefix, int j) {
    return ((j >= r.lo) & (j < r.hi)) | (j < prefix);
}

// Whether every row of the workgroup sees all of tokens [j, j + 32).
MQ_INDEX bool all_visible(const AttnArgs &a, const View &v, int j) {
    const int last = j + kTile - 1;
    if (last >= v.keys) return false;
    if (last < v.prefix) return true;
    if (a.causal && last > v.p_min) return false;
    return !a.window || (j > v.p_max - a.window && last < (int64_t)v.p_min + a.window);
}

}  // namespace
}  // namespace mq
