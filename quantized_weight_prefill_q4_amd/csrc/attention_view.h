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
    int q_f32, group, causal, window;
    int splits, target;               // parts of the keys: at most, workgroups to fill
    int min_tiles;                    // of a part: fewer do not pay for the join
    int items;                        // workgroups of the kernel for few rows
    int join_rows;                    // rows of a workgroup of the join
    const float *slopes;
    const int32_t *prefix;
    float *stats, *partial;           // workspace: [part][R][2] and [part][R][D], those of a
                                      // row tile and head side by side
    unsigned per_seq;                 // row tiles of a sequence (equal rows)
    int units;                        // row tiles of the batch
};

// The kernel for many rows (attention_prompt.hip), and how many a workgroup takes.
int attention_prompt_rows(int D);
hipError_t launch_attention_prompt(const AttnArgs &a, bool bias, hipStream_t stream);

namespace {

// What a workgroup's rows see: tiles [0, pre) and [lo, lo + n − pre).
struct View {
    int b, rt;                // sequence, row tile within it
    SeqRows rows;
    int len, keys, prefix;
    int first_pos;            // of the sequence's first new row (may be negative)
    int p_min, p_max;         // of the row tile's rows
    int pre, lo, n;
    int full_pre, full_lo, full_hi;   // tiles [0, full_pre) and [full_lo, full_hi): all rows
                                      // see all of them
};

// What rows [first, last] of sequence v.b see (rows of a key/value head: token · group +
// query head); v.rows is known.
MQ_INDEX void set_view(const AttnArgs &a, View &v, int first, int last) {
    v.len = seq_len(a.kv, v.b);
    v.keys = seq_keys(a.kv, v.len);
    v.first_pos = v.len - v.rows.n;
    v.p_min = v.first_pos + (int)((unsigned)first / (unsigned)a.group);
    v.p_max = v.first_pos + (int)((unsigned)last / (unsigned)a.group);
    v.prefix = a.prefix ? clampi(a.prefix[v.b], 0, v.keys) : 0;
    // positions lie within 2^30 of 0, the window is cut to 2^30: no sum passes an int
    int lo = 0, hi = v.keys, from = 0, to = v.keys;
    if (a.window) {
        lo = v.p_min - a.window + 1;
        from = v.p_max - a.window + 1;
        if (v.p_max + a.window < hi) hi = v.p_max + a.window;
        if (v.p_min + a.window < to) to = v.p_min + a.window;
        if (lo < 0) lo = 0;
        if (from < 0) from = 0;
    }
    if (a.causal) {
        if (v.p_max + 1 < hi) hi = v.p_max + 1;
        if (v.p_min + 1 < to) to = v.p_min + 1;
    }
    if (hi < v.prefix) hi = v.prefix;
    if (hi < 0) hi = 0;
    if (to < 0) to = 0;
    v.pre = (v.prefix + kTile - 1) / kTile;
    v.lo = lo / kTile;
    const int end = (hi + kTile - 1) / kTile;
    if (v.pre >= v.lo) v.pre = v.lo = 0;
    v.n = v.pre + (end > v.lo ? end - v.lo : 0);
    v.full_pre = v.prefix / kTile;
    v.full_lo = (from + kTile - 1) / kTile;
    v.full_hi = to / kTile;
}

// The view of row tile `rt` of sequence v.b, false without such rows.
template <int R>
MQ_INDEX bool tile_view(const AttnArgs &a, int rt, View &v) {
    v.rows = seq_rows(a.kv, v.b);
    const int total = v.rows.n * a.group;
    if (rt < 0 || (int64_t)rt * R >= total) return false;
    v.rt = rt;
    set_view(a, v, rt * R, total - rt * R < R ? total - 1 : rt * R + R - 1);
    return true;
}
template <int R>
MQ_INDEX bool find_view(const AttnArgs &a, int unit, View &v) {
    int within;
    v.b = find_seq(a.kv, unit, a.group, R, 1, a.per_seq, &within);
    return tile_view<R>(a, within, v);
}

// The keys of a row tile in parts, each a workgroup's, of `per` tiles (a multiple of
// four: the waves share a part evenly): about as many tiles as a part holds if all
// tiles of the batch are dealt to a.target workgroups (even_share), at least a.min_tiles,
// and at most a.splits parts.  One part needs no joining.
struct Parts {
    int per, count;
};
MQ_INDEX Parts parts_of(const AttnArgs &a, int n, int share) {
    const int c = share < a.min_tiles ? a.min_tiles : share;
    int want = (n + c / 2) / c;
    if (want > a.splits) want = a.splits;
    if (want < 1) want = 1;
    int per = ((n + want - 1) / want + 3) & ~3;
    if (per < a.min_tiles) per = a.min_tiles;
    const int count = (n + per - 1) / per;
    return Parts{per, count < 1 ? 1 : count};
}
// A workgroup's part and job (row tile · heads + head).  Workgroups go to the eight
// XCDs in turn, and many have no part: with the parts outermost those that have are
// neighbours and fill all XCDs (with the parts innermost, four of which two are
// empty, half the chip stands idle: a 2048-row prompt 166 us against 88).  The last
// parts first: only the longest jobs have them.
MQ_INDEX void find_job(const AttnArgs &a, unsigned block, int &split, int &job, int &head) {
    const unsigned jobs = (unsigned)a.units * a.kv.heads;
    split = a.splits - 1 - (int)(block / jobs);
    job = (int)(block % jobs);
    head = job % a.kv.heads;
}

// Tiles that the row tiles of sequence b read, about, per head.
MQ_INDEX float tiles_of_seq(const AttnArgs &a, int b, int rows_per_tile) {
    const SeqRows r = seq_rows(a.kv, b);
    int keys = seq_keys(a.kv, seq_len(a.kv, b));
    if (a.causal) keys -= r.n / 2;
    if (a.window && keys > a.window + r.n) keys = a.window + r.n;
    if (keys < 0) keys = 0;
    return (float)((r.n * a.group + rows_per_tile - 1) / rows_per_tile) * (float)(keys / kTile + 1);
}

// The kernel for few rows deals a sequence's keys out as a whole: all its row tiles
// (one, mostly) have the same parts, of the tiles that any of its rows sees.  Parts are
// numbered with those of the sequences before, job by job (row tile · heads + head):
// every number below `items` of the last sequence is a workgroup's work, and there are
// at most jobs + a.target of them, plus the sum's rounding (plan_attention).
struct SeqWork {
    View span;    // pre, lo and n of all rows
    int jobs;
    float cost;   // tiles to read
};
template <int R>
MQ_INDEX SeqWork seq_work(const AttnArgs &a, int b) {
    SeqWork w;
    w.span.b = b;
    w.span.rows = seq_rows(a.kv, b);
    const int total = w.span.rows.n * a.group;
    if (total == 0) {
        w.span.pre = w.span.lo = w.span.n = w.span.keys = w.jobs = 0;
        w.cost = 0.0f;
        return w;
    }
    set_view(a, w.span, 0, total - 1);
    w.jobs = (total + R - 1) / R * a.kv.heads;
    w.cost = (float)w.jobs * (float)w.span.n;
    return w;
}
MQ_INDEX int share_of(const AttnArgs &a, float cost) {
    const float share = ceilf(cost / (float)a.target);
    return share < 1e9f ? (int)share : 1000000000;
}
constexpr int kMostItems = 1 << 24;   // of a sequence or a call (the host's limit too)
MQ_INDEX int items_of(const SeqWork &w, const Parts &p) {
    const int64_t n = (int64_t)w.jobs * p.count;
    return n < kMostItems ? (int)n : kMostItems;
}

// The tokens that the row at position p sees: [lo, hi), and those before the prefix.
struct Range {
    int lo, hi;
};
MQ_INDEX Range row_range(const AttnArgs &a, const View &v, int p) {
    Range r{0, v.keys};
    if (a.window) {
        if (p - a.window + 1 > 0) r.lo = p - a.window + 1;
        if (p + a.window < r.hi) r.hi = p + a.window;
    }
    if (a.causal && p + 1 < r.hi) r.hi = p + 1;
    return r;
}
// The 32 tokens from j0 on that a row with this range sees, a bit each.
MQ_INDEX uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
MQ_INDEX uint32_t visible_bits(const Range &r, int prefix, int j0) {
    return (bits_below(r.hi - j0) & ~bits_below(r.lo - j0)) | bits_below(prefix - j0);
}

// Whether every row of the workgroup sees all of a tile.
MQ_INDEX bool all_visible(const View &v, int tile) {
    return tile < v.full_pre || (tile >= v.full_lo && tile < v.full_hi);
}

}  // namespace
}  // namespace mq
