// kvb_pages.h -- what the operators on 16-bit and fp8 pages share (kv_attend_shared,
// kv_bound, kv_select, kv_attend_selected): parameter blocks, and how attention's work
// is cut into equal shares.  The functions here also compile as host C++ for the CPU
// tests.  Not part of the public ABI.
#pragma once

#include "kvb_vec.h"

namespace kvb {

// ------------------------------------------------------ attention: units of work
//
// A segment is a run of cached tokens with the queries that see it: the prefix of a group
// of requests, or the own tokens of one request.  A unit is one KV head and one tile of
// query rows of a segment; its cached tokens are counted in tiles of 2^kv_shift.  All tiles
// of a call, in the order segment, row tile, head, cached tokens, are cut into equal runs,
// one a worker, so that ragged lengths leave nobody idle; what a worker holds of a unit is a
// piece, and a kernel behind joins the pieces of each query row.  Unit u's piece at worker
// w has slot u + w of the workspace: from one piece to the next u, w or both go up, so
// slots are distinct.  More units than valid query ranges can have (ranges that overlap) are
// refused on the GPU: nothing of the call is done.

struct PageEngine {
    uint32_t on;              // launched for this call
    uint32_t prefix, own;     // which segments it takes: groups' prefixes first, then requests
    uint32_t whole;           // a worker takes one unit, and nothing is joined
    uint32_t unit_cost;       // what a unit takes to begin and end, in tiles
    uint32_t row_tile, kv_shift;   // query rows of a unit, log2 of the cached tokens of a tile
    uint32_t workers;
    uint32_t slot_rows;       // query rows of a slot
    uint32_t team;            // warps of a worker (kernel for few rows)
    uint64_t units;           // that the workspace has room for
    uint32_t small;           // the segments fit a block's table, units 24 bits and tiles 31
    float *part_o;            // [slot][slot_rows][D] sums
    float *part_ml;           // [slot][slot_rows][2] maxima (base 2), sums of weights
    uint64_t *seg_tiles;      // [segments + 1] tiles before each segment (written on the GPU)
    uint64_t *seg_units;      // [segments + 1]
    int32_t *seg_table;       // [segments][kSegWords], not where they are few
};

struct PageAttendArgs {
    Vecs q, out;
    float *lse;
    const int32_t *q_start, *lens, *pages;
    int64_t pages_stride;
    const int32_t *group_start, *prefix_lens, *prefix_pages;
    int64_t prefix_stride;
    const int32_t *picks;     // [tokens][H][budget], or null: all pages
    uint32_t budget;
    uint32_t *status;
    PoolLayer pool;
    uint32_t requests, tokens, max_q, max_len, groups, max_group, max_prefix;
    uint32_t q_heads, group;  // group: query heads of a KV head
    float scale_log2;         // scale * log2(e), the keys' scale included
    float v_scale;
    uint32_t join_heads;      // query heads that a warp of the join takes in turn
    uint32_t joined;          // a request's units take its group's prefix in front of its own tokens
    PageEngine rows, tc;      // kernel for few rows, kernel on tcgen05
};

struct PageSeg {
    int q0, n, len;           // first query token, query tokens, cached tokens
    bool prefix, bad;
    uint32_t index;           // of the group or request
    int in;                   // a request: the group whose prefix its queries see, or -1
    int before;               // tokens of that prefix where they are in front of its own (joined)
};

// A group's prefix with all query tokens of its requests (none where the group is out of order
// or holds more than max_group), or a request's own tokens with its queries (none where they are
// out of range); lengths brought into range.
KVB_HD PageSeg seg_of(const PageAttendArgs &a, bool prefix, uint32_t index) {
    PageSeg g;
    g.prefix = prefix;
    g.index = index;
    const int32_t *lens = g.prefix ? a.prefix_lens : a.lens;
    const int len = lens[g.index];
    int r0 = (int)g.index, r1 = r0 + 1;
    if (g.prefix) {
        r0 = a.group_start[g.index];
        r1 = a.group_start[g.index + 1];
    }
    bool out = r0 < 0 || r1 < r0 || r1 > (int)a.requests;
    const int q0 = out ? 0 : a.q_start[r0], q1 = out ? 0 : a.q_start[r1];
    const int most = (int)(g.prefix ? a.max_group : a.max_q), longest = (int)(g.prefix ? a.max_prefix : a.max_len);
    out = out || q0 < 0 || q1 < q0 || q1 > (int)a.tokens || q1 - q0 > most;
    g.bad = out || len < 0 || len > longest;
    g.q0 = out ? 0 : q0;
    g.n = out ? 0 : q1 - q0;
    g.len = len < 0 ? 0 : len > longest ? longest : len;
    g.in = -1;
    g.before = 0;
    return g;
}

KVB_HD PageSeg prefix_seg(const PageAttendArgs &a, uint32_t g) { return seg_of(a, true, g); }

// The group whose prefix request r's queries q0 .. q0 + n - 1 see, or -1.  Groups are in
// order; where they are not, whichever the search meets.
KVB_HD int group_of(const PageAttendArgs &a, uint32_t r, int q0, int n) {
    if (a.groups == 0) return -1;
    uint32_t lo = 0, hi = a.groups;              // last group that starts at r or before
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (a.group_start[mid] <= (int)r) lo = mid;
        else hi = mid;
    }
    // empty groups in front of the one that holds r start at the same request
    const PageSeg s = prefix_seg(a, lo);
    if (s.n == 0 || s.len == 0 || a.group_start[lo] > (int)r || a.group_start[lo + 1] <= (int)r) return -1;
    if (q0 < s.q0 || q0 + n > s.q0 + s.n) return -1;
    return (int)lo;
}

KVB_HD PageSeg own_seg(const PageAttendArgs &a, uint32_t r) {
    PageSeg s = seg_of(a, false, r);
    if (a.groups == 0 || s.n == 0) return s;
    s.in = group_of(a, r, s.q0, s.n);
    if (a.joined && s.in >= 0) s.before = prefix_seg(a, (uint32_t)s.in).len;
    return s;
}

KVB_HD uint32_t seg_count(const PageAttendArgs &a, const PageEngine &e) {
    return (e.prefix ? a.groups : 0) + (e.own ? a.requests : 0);
}

// Segment s of an engine's.
KVB_HD PageSeg seg_at(const PageAttendArgs &a, const PageEngine &e, uint32_t s) {
    const uint32_t before = e.prefix ? a.groups : 0;
    return s < before ? prefix_seg(a, s) : own_seg(a, s - before);
}

// Row tiles of a segment.  Rows are (query token, head of the group); where every token
// has pages of its own, a tile holds rows of one token.
KVB_HD int row_tiles(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s) {
    const int rt = (int)e.row_tile, g = (int)a.group;
    return a.picks != nullptr ? s.n * ((g + rt - 1) / rt) : (s.n * g + rt - 1) / rt;    // at most 2^30 rows
}

// Cached tokens of the segment's own that some row of a tile sees: [0, that).
KVB_HD int seen_tokens(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, int rt) {
    if (s.prefix) return s.len;
    if (a.picks != nullptr) {
        // whole pages of the list, as many as the request's last token may have
        const uint32_t all = div_T(a.pool, (uint32_t)s.len + a.pool.T - 1);
        return (int)((all < a.budget ? all : a.budget) * a.pool.T);
    }
    int last = (int)((((uint32_t)rt + 1) * e.row_tile - 1) / a.group);
    if (last > s.n - 1) last = s.n - 1;
    const int hi = s.len - s.n + last + 1;
    return hi < 0 ? 0 : hi;                      // at most len
}

KVB_HD uint32_t tiles_of(const PageEngine &e, int tokens) { return ((uint32_t)tokens + (1u << e.kv_shift) - 1) >> e.kv_shift; }
KVB_HD uint32_t unit_tiles(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, int rt) {
    return tiles_of(e, s.before) + tiles_of(e, seen_tokens(a, e, s, rt));
}

// What a unit counts when work is shared out: its tiles, and in front of them unit_cost.
KVB_HD uint32_t unit_span(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, int rt) {
    const uint32_t n = unit_tiles(a, e, s, rt);
    return n == 0 ? 0 : n + e.unit_cost;
}

// The spans of the row tiles before rt, for one head.
KVB_HD uint64_t tiles_before(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, int rt) {
    if (rt == 0) return 0;
    if (s.prefix || a.picks != nullptr) return (uint64_t)rt * unit_span(a, e, s, 0);
    uint64_t sum = 0;
    for (int i = 0; i < rt; ++i) sum += unit_span(a, e, s, i);
    return sum;
}

KVB_HD uint64_t seg_tiles(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s) {
    return s.n == 0 ? 0 : tiles_before(a, e, s, row_tiles(a, e, s)) * a.pool.H;
}

// Division, in 32 bits where that does.
KVB_HD uint64_t quotient(uint64_t a, uint64_t b) { return ((a | b) >> 32) == 0 ? (uint32_t)a / (uint32_t)b : a / b; }

// Tiles of a worker.
KVB_HD uint64_t share_of(uint64_t tiles, uint32_t workers) { return tiles == 0 ? 1 : quotient(tiles + workers - 1, workers); }

// Units of a segment.  Those without a token to see are left to the join, where there is one.
KVB_HD uint64_t seg_units(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, uint64_t tiles) {
    return tiles != 0 || e.whole ? (uint64_t)row_tiles(a, e, s) * a.pool.H : 0;
}

// Where a block sums up the segments itself (PageEngine::small): a segment's tiles, and its units in the high word.  Valid
// ranges make fewer than kSmallUnits units and 2^31 tiles in all; of ranges that overlap, each counts for one more
// than there is room for at most, so that kPlanSegs of them do not wrap the high word.
constexpr uint64_t kSmallUnits = 1u << 24;
KVB_HD uint64_t pack_work(const PageEngine &e, uint64_t tiles, uint64_t units) {
    return (uint32_t)tiles | (units > e.units ? e.units + 1 : units) << 32;
}

// A worker's tiles [k0, k1) of the n_tiles of a unit (none where its run ends in front of them), and how much of
// the run that is.
struct PagePiece {
    PageSeg s;
    int rt, head, k0, k1, n_tiles;
    uint32_t span;
    uint64_t slot;
};

// The segments of a call: what comes before each, and its members.  A block holds up to kPlanSegs of
// them in shared memory; a kernel of its own writes more to the workspace.
constexpr uint32_t kPlanSegs = 128;
struct PageTable {
    const uint64_t *tiles, *units;        // [segments + 1]
    const int32_t *seg;                   // [segments][kSegWords]: q0, n, len, in, before
};
constexpr uint32_t kSegWords = 5;
struct PageTableSpace {
    uint64_t tiles[kPlanSegs + 1], units[kPlanSegs + 1];
    int32_t seg[kPlanSegs * kSegWords];
};

KVB_HD void put_seg(int32_t *to, const PageSeg &s) {
    to[0] = s.q0;
    to[1] = s.n;
    to[2] = s.len;
    to[3] = s.in;
    to[4] = s.before;
}

// The segment that holds tile x.
KVB_HD uint32_t find_segment(const uint64_t *tiles, uint32_t n, uint64_t x) {
    uint32_t lo = 0, hi = n;              // tiles[lo] <= x < tiles[hi]
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (tiles[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The piece of `worker` that begins at x of its run (x < x1, the run's end); *seg: a segment at x or before.
// A segment counts fewer than 2^31.  Where workers take whole units, x counts those.
KVB_HD PagePiece piece_of(const PageAttendArgs &a, const PageEngine &e, const PageTable &t, uint32_t *seg, uint64_t x, uint64_t x1,
                          uint32_t worker) {
    uint32_t i = *seg;
    const uint64_t *counts = e.whole ? t.units : t.tiles;
    while (x >= counts[i + 1]) ++i;
    *seg = i;
    const uint32_t before = e.prefix ? a.groups : 0, H = a.pool.H;
    const int32_t *w = t.seg + (uint64_t)i * kSegWords;
    PagePiece p;
    p.s.q0 = w[0];
    p.s.n = w[1];
    p.s.len = w[2];
    p.s.in = w[3];
    p.s.before = w[4];
    p.s.bad = false;
    p.s.prefix = i < before;
    p.s.index = i < before ? i : i - before;
    uint32_t rel = (uint32_t)(x - counts[i]);
    if (e.whole) {
        p.rt = (int)(rel / H);
        p.head = (int)(rel - (uint32_t)p.rt * H);
        p.n_tiles = (int)unit_tiles(a, e, p.s, p.rt);
        p.k0 = 0;
        p.k1 = p.n_tiles;
        p.span = 1;
        p.slot = 0;
        return p;
    }
    uint32_t n = unit_span(a, e, p.s, 0);
    p.rt = 0;
    if (p.s.prefix || a.picks != nullptr) {
        p.rt = (int)(rel / (n * H));
        rel -= (uint32_t)p.rt * n * H;
    } else {
        while (rel >= n * H) {
            rel -= n * H;
            n = unit_span(a, e, p.s, ++p.rt);
        }
    }
    const uint32_t c = e.unit_cost;
    p.n_tiles = (int)(n - c);
    p.head = (int)(rel / n);
    const uint32_t v0 = rel - (uint32_t)p.head * n, v1 = x1 - x < n - v0 ? v0 + (uint32_t)(x1 - x) : n;
    p.k0 = v0 > c ? (int)(v0 - c) : 0;
    p.k1 = v1 > c ? (int)(v1 - c) : 0;
    p.span = v1 - v0;
    p.slot = t.units[i] + (uint64_t)p.rt * H + p.head + worker;
    return p;
}

// Where the pieces of a query row are: workers w0 .. w1, slots unit + w, row `row` of each.
struct RowPieces {
    uint64_t unit, w0, w1;
    int row;
    bool any;
};

// The row tile of query token i and head j of the KV head's group, and which row of it that is.
KVB_HD int row_tile_of(const PageAttendArgs &a, const PageEngine &e, int i, int j, int *row) {
    const int rt_n = (int)e.row_tile, g = (int)a.group, at = a.picks != nullptr ? j : i * g + j;
    *row = at % rt_n;
    return a.picks != nullptr ? i * ((g + rt_n - 1) / rt_n) + at / rt_n : at / rt_n;
}

// Pieces of row `row` of row tile rt, whose units (one a KV head, each of `span`) begin `at` into the engine's run of
// shares; units_at units come before the segment's.
KVB_HD RowPieces row_pieces(const PageAttendArgs &a, const PageEngine &e, uint64_t share, uint64_t at, uint64_t units_at, uint32_t span,
                            int rt, int row, int head) {
    RowPieces p;
    p.any = span != 0;
    p.row = row;
    const uint64_t t0 = at + (uint64_t)head * span;
    p.w0 = quotient(t0 + (span != 0 ? e.unit_cost : 0), share);      // the first that holds tiles
    p.w1 = quotient(t0 + (span != 0 ? span : 1) - 1, share);
    p.unit = units_at + (uint64_t)rt * a.pool.H + head;
    return p;
}

// ------------------------------------------------------------ bounds of pages

constexpr uint32_t kTinyBits = 0x0d800000u;      // 2^-100: a group below it is zeros
constexpr float kMostScore = 3.402823466e38f;

KVB_HD uint32_t record_bytes(uint32_t D) { return (2 * D + D / 8 + 15) / 16 * 16; }

// The step of a group whose largest magnitude has these bits: the least power of two s
// with m <= 127 s; *inv = 1 / s.  0 and 0 below 2^-100, infinity and 0 for what is not finite.
KVB_HD float bound_step(uint32_t m, float *inv) {
    *inv = 0.0f;
    if (m < kTinyBits) return 0.0f;
    if (m >= 0x7f800000u) return f_bits(0x7f800000u);
    const uint32_t e = (m + 0x1ffffu) >> 23;     // 127 / 64 = 1.984375 is mantissa 0x7e0000
    *inv = f_bits((260u - e) << 23);
    return f_bits((e - 6u) << 23);
}

struct BoundArgs {
    uint8_t *bounds;          // [P][H] records
    const int32_t *lens, *first, *pages;
    int64_t pages_stride;
    uint32_t *status;
    PoolLayer pool;
    uint32_t requests, max_len, max_new;
    uint32_t most_pages;      // that one request's new tokens may touch
};

struct SelectArgs {
    const uint8_t *bounds;
    Vecs q;
    const int32_t *q_start, *lens, *pages;
    int64_t pages_stride;
    int32_t *picks;           // [tokens][H][budget]
    float *scores;            // [tokens][H][max_pages]
    uint32_t *status;
    uint32_t T, P, H;
    uint32_t requests, tokens, max_q, max_len, max_pages, q_heads, group;
    uint32_t budget, keep_first, keep_last;
    uint32_t block_pages;     // pages a block scores
};

// Pages of a request that query i of n sees: 0 .. that - 1.
KVB_HD int pages_seen(int len, int n, int i, uint32_t T) {
    const int pos = len - n + i;
    return pos < 0 ? 0 : (int)((uint32_t)pos / T) + 1;
}

}  // namespace kvb
