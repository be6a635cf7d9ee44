// The 4-bit key/value cache: its layout, and how a batch's rows find their
// tokens in it.
//
// A cache is pages of page tokens (a multiple of 32).  Within a page the tokens
// of one head are tiles of 32, a tile holding its keys and then its values, each
// as 16·D bytes of codes and 2·D bytes of f16 scales: 36·D bytes per tile.  An
// element is d·(q − 8), one d for 32 consecutive elements of a token's head.
//
// The order inside a tile is the one matrix instructions take their operands
// in, so that attention loads whole operands with 16-byte loads and exchanges
// nothing between lanes:
//   keys    dword ((4·m + g)·16 + r)·NS + s, NS = D/32, holds elements
//           [32·s + 8·g, + 8) of token 8·(r/4) + 4·m + r%4; scale (16·m + r)·NS + s
//   values  dword o·D + d holds element d of tokens [8·o, + 8);
//           scale (o·NS + d/32)·8 + e is that of token 8·o + e
// In a dword, of eight consecutive elements (keys) or tokens (values) number 2j
// is nibble j and number 2j + 1 nibble j + 4: (w >> 4j) & 0x000F000F is a pair of
// neighbours in the two halves of a register.
#pragma once

#include "mq_internal.h"

// Index arithmetic, also run on the host by the tests that walk a batch's bounds.
#define MQ_INDEX __host__ __device__ inline

namespace mq {
namespace {

constexpr int kTile = 32;
constexpr float kMostScale = 8188.0f;   // of a block: 8 of it are f16's largest number

MQ_INDEX constexpr int kv_tile_bytes(int D) { return 36 * D; }

// Keys' codes at 0; then
MQ_INDEX int kv_kscale_at(int D) { return 16 * D; }
MQ_INDEX int kv_vcode_at(int D) { return 18 * D; }
MQ_INDEX int kv_vscale_at(int D) { return 34 * D; }

// Place of token t (0..31) among the keys' scales, and of its elements
// [8·oct, + 8) among the keys' code dwords.
MQ_INDEX int kv_key_place(int t) {
    return 16 * ((t >> 2) & 1) + 4 * (t >> 3) + (t & 3);
}
MQ_INDEX int kv_key_dword(int t, int oct, int NS) {
    const int p = kv_key_place(t);
    return ((4 * (p >> 4) + (oct & 3)) * 16 + (p & 15)) * NS + (oct >> 2);
}
// Bit position of element or token e (0..7) in its dword.
MQ_INDEX int kv_shift(int e) { return 4 * (e >> 1) + 16 * (e & 1); }

MQ_INDEX int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Rows [first, first + n) of the batch are sequence b's.  Row counts outside the
// batch are cut to it: no index below leaves [0, M).
struct SeqRows {
    int first, n;
};
MQ_INDEX SeqRows seq_rows(const KvSpec &kv, int b) {
    if (!kv.cu) return SeqRows{b * kv.rows, kv.rows};
    const int c0 = clampi(kv.cu[b], 0, kv.M);
    return SeqRows{c0, clampi(kv.cu[b + 1], c0, kv.M) - c0};
}

// Tokens of sequence b, its new rows included (0 for a negative entry).
MQ_INDEX int seq_len(const KvSpec &kv, int b) { return clampi(kv.lens[b], 0, kMaxLen); }
// Those of them that the table has pages for.
MQ_INDEX int seq_keys(const KvSpec &kv, int len) {
    const int64_t room = (int64_t)kv.width * kv.page;
    return len < room ? len : (int)room;
}

// A sequence's work in units of `per` (rows times scale, or positions) is
// numbered with those of the others: sequence b's units begin at
// cu[b]·scale / per + extra·b, which leaves it at least as many as it needs.
// Finds the sequence of a unit, and the unit's number within it (negative before
// the first row, beyond what the sequence needs behind its last).  The host refuses
// batches whose rows times scale, or units, pass an int: 64-bit divisions are a
// hundred instructions each, fetched cold by every workgroup.
MQ_INDEX int unit_base(const KvSpec &kv, int b, int scale, unsigned per, int extra) {
    return (int)((unsigned)(clampi(kv.cu[b], 0, kv.M) * scale) / per) + extra * b;
}
MQ_INDEX int find_seq(const KvSpec &kv, int unit, int scale, unsigned per, int extra,
                      unsigned per_seq, int *within) {
    if (!kv.cu) {
        const int b = kv.batch == 1 ? 0 : (int)((unsigned)unit / per_seq);
        *within = unit - b * (int)per_seq;
        return b;
    }
    int lo = 0;   // the last b whose base is at most unit
#ifdef __HIP_DEVICE_COMPILE__
    // 64 of them at a time, one a lane: a search by halves waits for a load in each step
    for (int n = kv.batch; n > 1;) {
        const int step = (n + 63) / 64, at = (int)(threadIdx.x & 63) * step;
        const uint64_t below =
            __ballot(at < n && unit_base(kv, at < n ? lo + at : lo, scale, per, extra) <= unit);
        const int found = 63 - __builtin_clzll(below | 1);
        lo += found * step;
        n = n - found * step < step ? n - found * step : step;
    }
#else
    for (int hi = kv.batch - 1; lo < hi;) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit_base(kv, mid, scale, per, extra) <= unit)
            lo = mid;
        else
            hi = mid - 1;
    }
#endif
    *within = unit - unit_base(kv, lo, scale, per, extra);
    return lo;
}

// Eight positions [p0, p0 + 8) of sequence b, of which [e_lo, e_hi), one at least, are rows
// of the batch (position p0 + e is row row0 + e); positions at or past keys have no place.
// Units of eight positions are numbered as above; n rows from any position on
// touch at most n/8 + 2.  Rows at negative positions are in no unit.
struct Octet {
    int b, p0, e_lo, e_hi, keys;
    int64_t row0;
};
MQ_INDEX bool find_octet(const KvSpec &kv, int unit, unsigned per_seq, Octet &o) {
    int within;
    o.b = find_seq(kv, unit, 1, 8, 2, per_seq, &within);
    const SeqRows rows = seq_rows(kv, o.b);
    const int len = seq_len(kv, o.b), start = len - rows.n;
    // (within is below 2^24 + 2, start below 2^30)
    o.p0 = 8 * ((start > 0 ? start / 8 : 0) + within);
    if (within < 0 || o.p0 >= len) return false;
    o.e_lo = start > o.p0 ? start - o.p0 : 0;
    o.e_hi = len - o.p0 < 8 ? len - o.p0 : 8;
    // a sequence without rows has its end in an octet, and no work there: the store would
    // put the dwords of other tokens back as it read them, over another workgroup's
    if (o.e_lo >= o.e_hi) return false;
    o.keys = seq_keys(kv, len);
    o.row0 = (int64_t)rows.first + o.p0 - start;
    return true;
}
inline unsigned units_per_seq(const KvSpec &kv) { return kv.rows / 8 + 2; }
inline int64_t total_units(const KvSpec &kv) {
    return kv.cu ? (int64_t)kv.M / 8 + 2 * (int64_t)kv.batch : (int64_t)units_per_seq(kv) * kv.batch;
}

// Bytes from the cache's start to a tile: number `off` of a page's.
MQ_INDEX int64_t kv_tile_at(const KvSpec &kv, int head, int page, int off) {
    return page * kv.page_bytes +
           ((int64_t)head * (kv.page / kTile) + off) * kv_tile_bytes(kv.D);
}
// The tile of tokens [32·tile, + 32) of sequence b's head, or null where the
// table names no page of the cache.
MQ_INDEX char *kv_tile(const KvSpec &kv, int b, int head, int tile) {
    const int per = kv.page / kTile, p = tile / per;
    const int id = kv.table[b * kv.table_ld + p];
    if ((unsigned)id >= (unsigned)kv.pages) return nullptr;
    return kv.cache + kv_tile_at(kv, head, id, tile - p * per);
}

}  // namespace
}  // namespace mq
