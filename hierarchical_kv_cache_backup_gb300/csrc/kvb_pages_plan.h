// kvb_pages_plan.h -- how attention over 16-bit and fp8 pages is cut: which kernel takes which
// segments, with how many workers, and the workspace.  Host code, of numbers alone, so that
// the CPU tests run it.  Not part of the public ABI.
#pragma once

#include "kvb_pages.h"

#include <algorithm>
#include <cmath>

namespace kvb {

// The kernel for few rows: warps of a block, query rows of a unit.
constexpr int kWarps = 4, kRowsP = 16;
// The kernel on tcgen05: a tile of query rows, log2 of the cached tokens of a tile; two tiles of rows a unit
// where tensor memory holds the sums of both.
constexpr int kTcTileQ = 128, kTcShift = 6;
KVB_HD constexpr int tc_q_tiles(int D) { return D > 128 ? 1 : 2; }
inline uint32_t pages_tc_rows(uint32_t D, uint64_t rows) { return tc_q_tiles((int)D) == 1 || rows <= (uint64_t)kTcTileQ ? kTcTileQ : 2 * kTcTileQ; }
// Heads of a group up to which a warp of the join takes several rows.
constexpr uint32_t kManyGroup = 128;

// How a call is cut, and its workspace.
struct PagePlan {
    PageEngine rows, tc;      // pointers are offsets from the workspace's start
    uint64_t bytes;
    bool wide_join;           // a row may have many pieces
    uint32_t join_heads;      // rows that a warp of the join takes in turn
    bool joined;              // units of own tokens take the prefix too
};

// Space in the workspace, 256 bytes aligned.
inline uint64_t take(uint64_t *at, uint64_t bytes) {
    const uint64_t p = *at;
    *at += (bytes + 255) / 256 * 256;
    return p;
}

// The most cached tokens that a list of pages stands for (whole pages of it, as many as the request has).
inline uint64_t list_tokens(uint32_t budget, uint32_t T, uint32_t max_len) {
    return std::min((uint64_t)budget * T, (uint64_t)max_len + T);
}

// The most units that an engine may meet.
inline uint64_t most_units(const PageEngine &e, uint32_t requests, uint32_t tokens, uint32_t max_q, uint32_t groups, uint32_t max_group,
                           uint32_t group, bool picked, uint32_t H) {
    uint64_t u = 0;
    auto tiles = [&](uint64_t segs, uint64_t most_tokens) {
        const uint64_t rt = e.row_tile;
        if (picked) return (uint64_t)tokens * ((group + rt - 1) / rt);
        // each segment alone, or all tokens cut once and one ragged tile a segment
        return std::min(segs * ((most_tokens * group + rt - 1) / rt), (uint64_t)tokens * group / rt + segs);
    };
    if (e.prefix) u += tiles(groups, max_group);
    if (e.own) u += tiles(requests, max_q);
    return u * H;
}

// `span`: the most cached tokens of a unit.
inline void place(PageEngine *e, uint64_t *at, uint64_t units, uint64_t segs, uint64_t span, uint32_t D) {
    e->units = units;
    const uint64_t tiles = units * ((span >> e->kv_shift) + 2 + e->unit_cost);      // at most
    e->small = segs <= kPlanSegs && units < kSmallUnits && tiles < (1ull << 31);
    if (!e->small) e->seg_table = (int32_t *)take(at, segs * kSegWords * 4);
    if (!e->small || !e->whole) {
        e->seg_tiles = (uint64_t *)take(at, (segs + 1) * 8);
        e->seg_units = (uint64_t *)take(at, (segs + 1) * 8);
    }
    if (e->whole) return;                 // nothing is joined
    const uint64_t rows = (units + e->workers) * e->slot_rows;
    e->part_ml = (float *)take(at, rows * 8);
    e->part_o = (float *)take(at, rows * D * 4);
}

// per_sm: blocks of the kernel for few rows that an SM holds.
inline PagePlan plan_pages(uint32_t requests, uint32_t tokens, uint32_t max_q, uint32_t max_len, uint32_t groups,
                           uint32_t max_group, uint32_t max_prefix, uint32_t budget, uint32_t T, uint32_t q_heads,
                           uint32_t kv_heads, uint32_t D, bool fp8, int sms, uint32_t per_sm) {
    PagePlan p{};
    const uint32_t group = q_heads / kv_heads;
    const bool picked = budget != 0;
    const uint32_t prefix_rows = (uint32_t)std::min<uint64_t>((uint64_t)max_group * group, 1u << 30);
    const uint32_t own_rows = picked ? group : max_q * group;
    // More rows than one tile of mma.sync: tcgen05.
    const bool tc_own = !picked && own_rows > kRowsP;
    // Where requests fill units on their own, reading the prefix with them saves the joining: where the call has at
    // most a third more units so than all its rows fill.  Units that a few single tokens take for themselves would
    // each read the prefix again.  Behind 8,192 tokens (us, prefix in front / apart): four chunks of 500 237 / 286, with
    // 8 single tokens beside them 288 / 301, 16 343 / 315, 32 451 / 343; a chunk of 512 beside 63 732 / 434; 8-bit
    // pages and heads of 256, chunks of 500 with 4, 8 and 16 beside them 231 / 232, 245 / 239 and 277 / 251.
    // Groups without any prefix are the same: nothing is in front, and no kernel is kept for them.
    PageEngine alone{};
    alone.own = 1;
    alone.row_tile = pages_tc_rows(D, own_rows);
    const uint64_t filled = ((uint64_t)tokens * group + alone.row_tile - 1) / alone.row_tile;
    const uint64_t most = most_units(alone, requests, tokens, max_q, 0, 0, group, false, 1);
    p.joined = groups != 0 && (max_prefix == 0 || (tc_own && own_rows >= 256 && 3 * most <= 4 * filled));
    const bool tc_prefix = groups != 0 && prefix_rows > kRowsP && !p.joined;
    const uint64_t span = picked ? list_tokens(budget, T, max_len) : p.joined ? (uint64_t)max_prefix + max_len : std::max(max_len, groups != 0 ? max_prefix : 0);
    uint64_t at = 0;
    const uint64_t segs = (p.joined ? 0 : (uint64_t)groups) + requests;
    PageEngine &t = p.tc, &e = p.rows;
    if (own_rows <= (uint32_t)kRowsP) {
        // A block a request (or query with a list) and head, the prefix in front of its own tokens, and nothing to join:
        // where that ends sooner.  In rounds of a block's four warps (64 tokens, 1.3 us at heads of 128): a unit begins
        // and ends in 4; cut in equal shares the join takes 4 more, and tcgen05 begins in 8.  Two requests of 30 behind
        // 150 tokens: 13.1 us cut.
        PageEngine w{};
        w.own = 1;
        w.row_tile = kRowsP;
        w.kv_shift = 6;
        const uint64_t units = most_units(w, requests, tokens, max_q, groups, max_group, group, picked, kv_heads);
        const uint64_t all = picked ? list_tokens(budget, T, max_len) : (uint64_t)max_len + (groups != 0 ? max_prefix : 0);
        const double rounds = (double)(all / 64 + 1), places = (double)sms * per_sm;
        const double by_units = std::ceil((double)units / places) * (rounds + 4.0);
        const double own_rounds = picked ? rounds : (double)(max_len / 64 + 1);
        const double cut = ((double)units * (own_rounds + 4.0) + (groups != 0 && max_prefix != 0 && !tc_prefix ? (double)groups * kv_heads * (max_prefix / 64.0 + 4.0) : 0.0)) / places;
        if (units < (1ull << 31) && by_units <= std::max(cut, 5.0) + 4.0 + (tc_prefix ? 8.0 : 0.0)) {
            e = w;
            e.on = 1;
            e.whole = 1;
            e.team = kWarps;
            e.slot_rows = 1;
            e.workers = (uint32_t)units;
            p.joined = groups != 0;
            place(&e, &at, units, segs, all, D);
            p.bytes = at;
            return p;
        }
    }
    uint64_t t_units = 0, e_units = 0;
    if (tc_prefix || tc_own) {
        const uint32_t most = std::max(tc_prefix ? prefix_rows : 0, tc_own ? own_rows : 0);
        t.on = 1;
        t.prefix = tc_prefix;
        t.own = tc_own;
        t.row_tile = pages_tc_rows(D, most);
        t.kv_shift = kTcShift;
        t.slot_rows = std::min(t.row_tile, most);
        t.team = 1;
        t.unit_cost = 10;                        // 14,000 cycles, 27,000 of a block's first piece
        t.workers = (uint32_t)sms;
        t_units = most_units(t, requests, tokens, max_q, groups, max_group, group, picked, kv_heads);
    }
    if (!(tc_prefix || p.joined || groups == 0) || !tc_own) {
        e.on = 1;
        e.prefix = groups != 0 && !tc_prefix && !p.joined;
        e.own = !tc_own;
        e.row_tile = kRowsP;
        e.slot_rows = std::min<uint32_t>(kRowsP, std::max(e.own ? own_rows : 0, e.prefix ? prefix_rows : 0));
        e_units = most_units(e, requests, tokens, max_q, groups, max_group, group, picked, kv_heads);
        uint32_t e_sms = (uint32_t)sms;
        if (t.on) {
            // The two kernels run side by side, each on SMs of its own, so that neither waits for the other's
            // beginning and end: as many for tcgen05 as its share of the cycles, 26 D a tile of 64
            // cached tokens against 25 D a warp's tile of 16, waits included.  64 requests of up to 1,000
            // tokens behind 8,192: 96 us one after the other on all SMs, side by side 72 / 66 / 68 with
            // 20 / 26 / 32 D.
            const double tc_cost = (double)t_units * ((t.prefix ? max_prefix : max_len) / 64 + 1) * (fp8 ? 24.0 : 26.0) * D;
            const double rows_cost = (double)e_units * ((e.prefix ? max_prefix : max_len) / 16 + 1) * 25.0 * D / (kWarps * per_sm);
            const double part = (double)sms * tc_cost / (tc_cost + rows_cost);
            t.workers = (uint32_t)std::min<double>(sms - 1, std::max(1.0, std::floor(part + 0.5)));
            e_sms = (uint32_t)sms - t.workers;
        }
        // A few places are left free: a block that found none at the start (the kernel in front still in it) would
        // begin when the others end (selected decode of 48 requests: 48 us, 80 where that happened).
        const uint32_t places = e_sms * per_sm, blocks = places - places / 32;
        // A warp works by itself (what a unit takes to begin and end is paid once); where that would make
        // more than 16 pieces of a unit, a block's four warps share one, so that fewer pieces have to be joined.
        e.team = 4 * e_units >= blocks ? 1 : kWarps;
        e.kv_shift = e.team == 1 ? 4 : 6;
        e.unit_cost = e.team == 1 ? 5 : 4;       // 10,000 cycles
        e.workers = blocks * (kWarps / e.team);
        place(&e, &at, e_units, segs, span, D);
        p.wide_join = e.workers > 6 * e_units;
    }
    if (t.on) place(&t, &at, t_units, segs, span, D);
    if (p.tc.on && p.tc.workers > 6 * p.tc.units) p.wide_join = true;
    // Rows of a token that a warp of the join takes: as many as make about two rounds of 32 warps an SM, four at
    // least where it is more than one.
    const uint64_t rounds = (uint64_t)tokens * q_heads / ((uint64_t)sms * 64);
    p.join_heads = rounds < 2 || group > kManyGroup ? 1 : (uint32_t)std::min<uint64_t>((rounds + 3) / 4 * 4, (q_heads + 3) / 4);
    p.bytes = at;
    return p;
}

// The kernels count the tiles of one segment, all its units with what each takes to begin and end, in 31 bits.
inline bool plan_counts_fit(const PagePlan &p, uint32_t max_q, uint32_t max_len, uint32_t max_group, uint32_t max_prefix,
                            uint32_t budget, uint32_t T, uint32_t q_heads, uint32_t kv_heads) {
    const double group = q_heads / kv_heads;
    // a list is taken for at most what the request has, and both stay far from 64 bits
    if (budget != 0 && (double)max_q * kv_heads * max_len >= 281474976710656.0) return false;
    for (const PageEngine *e : {&p.rows, &p.tc}) {
        if (!e->on) continue;
        const double rows = std::max(max_q * group, e->prefix ? max_group * group : 0.0);
        const double units = kv_heads * (budget != 0 ? max_q * std::ceil(group / e->row_tile) : rows / e->row_tile + 1);
        const double tokens = budget != 0 ? (double)list_tokens(budget, T, max_len) : (double)max_len + max_prefix;
        if (units * (tokens / (1u << e->kv_shift) + 2 + e->unit_cost) >= 2147483648.0) return false;
    }
    return true;
}

}  // namespace kvb
