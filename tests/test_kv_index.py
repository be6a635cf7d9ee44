"""The index arithmetic of the 4-bit cache's kernels, walked on the host: every unit of
work that a launch starts stays inside the batch, the table and the cache, whatever
lens, cu_rows and table hold, and for a sound batch every row is worked on exactly once.
Compiled with the host compiler; no GPU."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_weight_prefill_q4_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <random>
#include <vector>
#include "attention_view.h"
using namespace mq;

#define CHECK(c) do { if (!(c)) { printf("line %d: %s (seed %d)\n", __LINE__, #c, seed); return 1; } } while (0)

template <int R>
static int views(const KvSpec &kv, const AttnArgs &a, int64_t units, bool sound, int seed) {
    std::vector<int> seen(kv.M * a.group);
    for (int64_t u = 0; u < units; ++u) {
        View v;
        if (!find_view<R>(a, u, v)) continue;
        CHECK(v.b >= 0 && v.b < kv.batch && v.rt >= 0);
        CHECK(v.rows.first >= 0 && v.rows.n >= 0 && v.rows.first + v.rows.n <= kv.M);
        CHECK(v.keys >= 0 && v.keys <= (int64_t)kv.width * kv.page);
        CHECK(v.n >= 0 && v.pre >= 0 && v.pre <= v.n);
        for (int n = 0; n < R; ++n) {
            const int64_t row = (int64_t)v.rt * R + n, i = row / a.group;
            if (i < v.rows.n) ++seen[(v.rows.first + i) * a.group + row % a.group];
        }
        // every tile it may touch has an entry in the table; every pair that a row
        // sees lies in one of them, and a tile taken whole is seen whole by all rows
        std::vector<char> in(v.keys / kTile + 2, 0);
        for (int t = 0; t < v.n; ++t) {
            const int tile = t < v.pre ? t : t - v.pre + v.lo;
            CHECK(tile >= 0 && (int64_t)tile * kTile < (int64_t)kv.width * kv.page);
            CHECK(tile * kTile < v.keys);
            CHECK(!in[tile]);
            in[tile] = 1;
            char *p = kv_tile(kv, v.b, kv.heads - 1, tile);
            if (p) {
                CHECK(p >= kv.cache);
                CHECK(p + kv_tile_bytes(kv.D) <= kv.cache + kv.pages * kv.page_bytes);
            }
        }
        for (int n = 0; n < R; ++n) {
            const int64_t i = ((int64_t)v.rt * R + n) / a.group;
            if (i >= v.rows.n) break;
            const int p = v.first_pos + (int)i;
            CHECK(p >= v.p_min && p <= v.p_max);
            for (int j = 0; j < v.keys; ++j) {
                const bool see =
                    visible_bits(row_range(a, v, p), v.prefix, j / kTile * kTile) >> (j % kTile) & 1;
                const int64_t far = p > j ? (int64_t)p - j : (int64_t)j - p;
                CHECK(see == (((!a.causal || j <= p) && (!a.window || far < a.window)) || j < v.prefix));
                if (see) CHECK(in[j / kTile]);
                if (!see && in[j / kTile]) CHECK(!all_visible(v, j / kTile));
            }
        }
        for (int tile = 0; tile * kTile < v.keys; ++tile)
            if ((tile + 1) * kTile > v.keys) CHECK(!all_visible(v, tile));
        // the parts are the tiles, once each, in no more than were planned for
        for (int splits = 1; splits < 20; ++splits)
            for (int share : {0, 1, 3, 9, 40, 1000000000}) {
                AttnArgs s = a;
                s.splits = splits;
                s.min_tiles = splits % 2 ? 4 : 8;
                const Parts p = parts_of(s, v.n, share);
                CHECK(p.count >= 1 && p.count <= splits && p.per % 4 == 0 && p.per >= s.min_tiles);
                CHECK((int64_t)p.count * p.per >= v.n && (v.n == 0 || (int64_t)(p.count - 1) * p.per < v.n));
            }
    }
    if (sound)
        for (int x : seen) CHECK(x == 1);
    return 0;
}

// The kernel for few rows: no more parts than it has workgroups and room for, and every
// tile that a row tile reads is in its sequence's span.
template <int R>
static int works(const KvSpec &kv, AttnArgs a, bool sound, int seed) {
    const int64_t most_jobs = ((int64_t)kv.M * a.group / R + kv.batch) * kv.heads;
    for (int target : {1, 5, 40, 768})
        for (int splits : {1, 2, 256}) {
            a.target = target;
            a.splits = splits;
            a.min_tiles = target % 2 ? 4 : 8;
            float cost = 0.0f;
            for (int b = 0; b < kv.batch; ++b) cost += seq_work<R>(a, b).cost;
            const int share = share_of(a, cost);
            int64_t jobs = 0, items = 0;
            for (int b = 0; b < kv.batch; ++b) {
                const SeqWork w = seq_work<R>(a, b);
                const Parts p = parts_of(a, w.span.n, share);
                CHECK(w.jobs >= 0 && w.jobs % kv.heads == 0);
                jobs += w.jobs;
                items += items_of(w, p);
                std::vector<char> in(w.span.keys / kTile + 2, 0);
                for (int t = 0; t < w.span.n; ++t)
                    in[t < w.span.pre ? t : t - w.span.pre + w.span.lo] = 1;
                for (int rt = 0; rt * kv.heads < w.jobs; ++rt) {
                    View v;
                    v.b = b;
                    CHECK(tile_view<R>(a, rt, v));
                    for (int t = 0; t < v.n; ++t) CHECK(in[t < v.pre ? t : t - v.pre + v.lo]);
                }
                View v;
                v.b = b;
                CHECK(!tile_view<R>(a, w.jobs / kv.heads, v) && !tile_view<R>(a, -1, v));
            }
            if (!sound) continue;
            CHECK(jobs <= most_jobs);
            CHECK(splits > 1 ? items <= most_jobs + target + 8 : items == jobs);
        }
    return 0;
}

int main() {
    for (int seed = 0; seed < 600; ++seed) {
        std::mt19937 rng(seed);
        auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
        const bool sound = seed % 2 == 0, ragged = seed % 3 != 0;
        KvSpec kv{};
        AttnArgs a{};
        kv.batch = pick(1, 6);
        kv.page = 32 * pick(1, 4);
        kv.width = pick(1, 5);
        kv.pages = pick(1, 9);
        kv.heads = pick(1, 3);
        kv.D = 64;
        kv.page_bytes = (int64_t)kv.heads * (kv.page / 32) * 36 * kv.D + 16 * pick(0, 2);
        kv.cache = (char *)0x100000;
        kv.table_ld = kv.width + pick(0, 2);
        kv.rows = pick(1, 70);
        std::vector<int> n(kv.batch), cu(kv.batch + 1), lens(kv.batch);
        cu[0] = ragged && seed % 5 == 0 ? pick(0, 9) : 0;
        for (int b = 0; b < kv.batch; ++b) {
            n[b] = ragged ? pick(0, 3) * pick(0, 40) : kv.rows;
            cu[b + 1] = cu[b] + n[b];
        }
        kv.M = cu[kv.batch] + (ragged ? pick(0, 5) : 0);
        if (kv.M == 0) continue;
        if (!ragged) kv.M = kv.rows * kv.batch;
        const int room = kv.width * kv.page;
        for (int b = 0; b < kv.batch; ++b) lens[b] = n[b] + pick(0, room);
        std::vector<int> table(kv.batch * kv.table_ld);
        for (int &t : table) t = pick(0, kv.pages - 1);
        if (!sound) {
            const int odd[] = {-1, INT32_MIN, INT32_MAX, 1 << 30, -7, 3, 1000000};
            for (int &t : table) if (pick(0, 2) == 0) t = odd[pick(0, 6)];
            for (int &t : lens) if (pick(0, 2) == 0) t = odd[pick(0, 6)];
            for (int &t : cu) if (pick(0, 2) == 0) t = odd[pick(0, 6)];
        }
        kv.table = table.data();
        kv.lens = lens.data();
        kv.cu = ragged ? cu.data() : nullptr;
        std::vector<int> rows(kv.M);
        const unsigned per = units_per_seq(kv);
        const int64_t units = total_units(kv);
        for (int64_t u = 0; u < units; ++u) {
            Octet o;
            if (!find_octet(kv, u, per, o)) continue;
            CHECK(o.b >= 0 && o.b < kv.batch && o.p0 >= 0 && o.p0 % 8 == 0);
            CHECK(o.e_lo >= 0 && o.e_hi <= 8);
            for (int e = o.e_lo; e < o.e_hi; ++e) {
                CHECK(o.row0 + e >= 0 && o.row0 + e < kv.M);
                ++rows[o.row0 + e];
                if (o.p0 + e >= o.keys) continue;
                char *p = kv_tile(kv, o.b, kv.heads - 1, o.p0 / kTile);
                if (p) {
                    CHECK(p >= kv.cache);
                    CHECK(p + kv_tile_bytes(kv.D) <= kv.cache + kv.pages * kv.page_bytes);
                }
            }
        }
        if (sound) {
            for (int i = 0; i < kv.M; ++i)
                CHECK(rows[i] == (ragged ? i >= cu[0] && i < cu[kv.batch] : 1));
        }
        std::vector<int> prefix(kv.batch);
        for (int &p : prefix) p = pick(-5, room + 5);
        a.kv = kv;
        a.group = pick(1, 9);
        a.causal = pick(0, 1);
        a.window = pick(0, 1) ? pick(1, 200) : 0;
        if (seed % 7 == 0) a.window = kMaxLen;
        a.prefix = pick(0, 1) ? prefix.data() : nullptr;
        for (int b = 0; b < kv.batch; ++b)
            for (int R : {16, 256}) CHECK(tiles_of_seq(a, b, R) >= 0.0f);
        const bool whole = sound && (!ragged || (cu[0] == 0 && cu[kv.batch] == kv.M));
        for (int R : {16, 32, 128, 256}) {
            a.per_seq = kv.cu ? 0 : ((int64_t)kv.rows * a.group + R - 1) / R;
            const int64_t total = kv.cu ? (int64_t)kv.M * a.group / R + kv.batch : (int64_t)a.per_seq * kv.batch;
            const int rc = R == 16 ? views<16>(kv, a, total, whole, seed)
                         : R == 32 ? views<32>(kv, a, total, whole, seed)
                         : R == 128 ? views<128>(kv, a, total, whole, seed)
                                    : views<256>(kv, a, total, whole, seed);
            if (rc) return rc;
            if (R <= 32)
                if (const int rc = R == 16 ? works<16>(kv, a, whole, seed) : works<32>(kv, a, whole, seed))
                    return rc;
        }
    }
    {   // a page of more than 2^31 bytes
        const int seed = 0;
        KvSpec kv{};
        kv.page = 1 << 29;
        kv.heads = 2;
        kv.D = 256;
        kv.page_bytes = (int64_t)2 * (kv.page / 32) * 36 * 256;
        CHECK(kv_tile_at(kv, 1, 3, (1 << 24) - 1) == 4 * kv.page_bytes - 36 * 256);
    }
    // the byte layout: every nibble and scale of a tile has one place
    for (int D : {64, 96, 128, 256}) {
        const int seed = D, NS = D / 32;
        std::vector<int> k(4 * D), ks(D), vs(D);
        for (int t = 0; t < 32; ++t) {
            for (int o = 0; o < D / 8; ++o) ++k[kv_key_dword(t, o, NS)];
            for (int s = 0; s < NS; ++s) ++ks[kv_key_place(t) * NS + s];
        }
        for (int x : k) CHECK(x == 1);
        for (int x : ks) CHECK(x == 1);
        unsigned bits = 0;
        for (int e = 0; e < 8; ++e) bits |= 15u << kv_shift(e);
        CHECK(bits == 0xFFFFFFFFu);
        CHECK(kv_kscale_at(D) == 4 * 4 * D && kv_vcode_at(D) == kv_kscale_at(D) + 2 * D);
        CHECK(kv_vscale_at(D) == kv_vcode_at(D) + 16 * D && kv_tile_bytes(D) == kv_vscale_at(D) + 2 * D);
    }
    printf("ok\n");
    return 0;
}
"""


def test_indexes_stay_in_bounds(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("no host compiler or HIP headers")
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-g", "-w", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
                        "-I", "/opt/rocm/include", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout, r.stderr[-2000:])


EMPTY = r"""
#include <stdio.h>
#include <random>
#include <vector>
#include "kv_q4.h"
using namespace mq;

int main() {
    // a sequence without rows, of every length: none of its units has work
    for (int len = 0; len < 70; ++len)
        for (int at = 0; at < 3; ++at) {
            int table[12], lens[3] = {20, 20, 20}, cu[4] = {0, 20, 40, 60};
            for (int &t : table) t = 0;
            lens[at] = len;
            for (int b = at + 1; b < 4; ++b) cu[b] -= 20;
            KvSpec kv{};
            kv.batch = 3;
            kv.page = 32;
            kv.width = kv.table_ld = 4;
            kv.pages = 1;
            kv.heads = 1;
            kv.D = 64;
            kv.table = table;
            kv.lens = lens;
            kv.cu = cu;
            kv.M = 40;
            int rows = 0;
            for (int64_t u = 0; u < total_units(kv); ++u) {
                Octet o;
                if (!find_octet(kv, u, units_per_seq(kv), o)) continue;
                if (o.b == at || o.e_lo >= o.e_hi) {
                    printf("length %d at %d: unit %d, positions %d + [%d, %d)\n", len, at, (int)u, o.p0,
                           o.e_lo, o.e_hi);
                    return 1;
                }
                rows += o.e_hi - o.e_lo;
            }
            if (rows != 40) {
                printf("length %d at %d: %d rows\n", len, at, rows);
                return 1;
            }
        }
    // whatever lens and cu_rows hold, every unit with work has a row
    for (int seed = 0; seed < 20000; ++seed) {
        std::mt19937 rng(seed);
        auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
        const int odd[] = {-1, INT32_MIN, INT32_MAX, 1 << 30, -7, 3, 1000000};
        KvSpec kv{};
        kv.batch = pick(1, 5);
        kv.page = 32;
        kv.width = pick(1, 4);
        kv.M = pick(1, 60);
        std::vector<int> lens(kv.batch), cu(kv.batch + 1);
        for (int &x : lens) x = pick(0, 3) ? pick(0, 200) : odd[pick(0, 6)];
        for (int &x : cu) x = pick(0, 3) ? pick(0, kv.M) : odd[pick(0, 6)];
        kv.lens = lens.data();
        kv.cu = cu.data();
        for (int64_t u = 0; u < total_units(kv); ++u) {
            Octet o;
            if (find_octet(kv, u, 0, o) && o.e_lo >= o.e_hi) {
                printf("seed %d: a unit without rows\n", seed);
                return 1;
            }
        }
    }
    printf("ok\n");
    return 0;
}
"""


def test_sequences_without_rows_have_no_octets(tmp_path):
    """The store reads and rewrites whole dwords of an octet: one without rows must be
    nobody's work, or it puts old values back over those that another sequence stores."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("no host compiler or HIP headers")
    src, exe = tmp_path / "empty.cpp", tmp_path / "empty"
    src.write_text(EMPTY)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-g", "-w", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__",
                        "-I", "/opt/rocm/include", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout, r.stderr[-2000:])
