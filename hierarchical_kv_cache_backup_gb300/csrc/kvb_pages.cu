// kvb_pages.cu -- attention over pages held in 16 bits or in fp8 (kv_attend_shared,
// kv_attend_selected): the kernel for few query rows, and the kernel that joins pieces.
//
// Mathematics.  A piece is some cached tokens t of a unit (KV head, 16 query rows).  With a
// running maximum m of x_t = scale log2(e) q . k_t, it keeps l = sum 2^(x_t - m) and
// o = sum 2^(x_t - m) v_t in float32; pieces join as o = sum o_i 2^(m_i - m), l likewise,
// and out = o / l.  Attention of a shared prefix is that: the prefix is a unit of its own,
// read once for all requests of the group, whose pieces join with those of each request's own
// tokens.
#include "kvb_pages.h"
#include "kvb_pages_device.h"
#include "kvb_pages_internal.h"
#include "kvb_pages_plan.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

namespace kvb {

namespace {

constexpr int kTile = 16;        // cached tokens a warp takes at a time (2^4)
constexpr float kNoMax = -3.0e38f;

// The 16-byte pieces of a token's values; in shared memory a token takes one more, so that
// the 8 rows of a fragment start in different banks (an odd multiple of 16 bytes apart).
__host__ __device__ constexpr int row_bytes(int D, bool f8) { return f8 ? D : 2 * D; }
__host__ __device__ constexpr int smem_stride(int D, bool f8) { return row_bytes(D, f8) + 16; }
__host__ __device__ constexpr int stage_bytes(int D, bool f8) { return 2 * kTile * smem_stride(D, f8); }
// Stages: few, for as many warps as registers allow (D = 128 of 16 bits: two stages and 12 warps of 168
// registers an SM; D = 64, 300 queries with 1,024 selected tokens each: 62 us with three stages and 12
// warps, 54 with two and 16).
__host__ __device__ constexpr int stages_of(int D, bool f8) { return row_bytes(D, f8) >= 128 ? 2 : 3; }
__host__ __device__ constexpr int ring_bytes(int D, bool f8) {
    const int ring = stages_of(D, f8) * stage_bytes(D, f8), join = kRowsP * (D + 4) * 4;
    return ring > join ? ring : join;
}
// Blocks of an SM that the registers are kept for.
__host__ __device__ constexpr int blocks_wanted(int D) { return D <= 64 ? 4 : D <= 128 ? 3 : 1; }

__device__ __forceinline__ void copy16(uint32_t smem, uint64_t gmem, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t smem, uint64_t gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void ldm(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kBf>
__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    if (kBf)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Threads of a team (worker) wait for one another.
__device__ __forceinline__ void team_sync(uint32_t team, uint32_t id) {
    if (team == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(team * 32) : "memory");
}

// ------------------------------------------------------------------- the plan
//
// Tiles and units before each segment, where a block's table cannot hold them: one block an engine
// (0: few rows, 1: tcgen05), 1,024 segments at a time.  Bound: a launch and two dependent reads; smaller calls go
// without (every block sums up to 128 segments itself).
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) kv_pages_plan_kernel(const __grid_constant__ PageAttendArgs a) {
    __shared__ unsigned long long sums[2][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const PageEngine &e = blockIdx.x == 0 ? a.rows : a.tc;
    if (!e.on || e.small) return;
    report_groups(a);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t n = seg_count(a, e);
    unsigned long long run_t = 0, run_u = 0;
    for (uint32_t s0 = 0; s0 < n; s0 += kPlanThreads) {
        const uint32_t s = s0 + tid;
        unsigned long long t = 0, u = 0;
        if (s < n) {
            const PageSeg g = seg_at(a, e, s);
            t = seg_tiles(a, e, g);
            u = seg_units(a, e, g, t);
            if (g.bad && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
        }
        const unsigned long long it = scan_add(t, lane), iu = scan_add(u, lane);
        __syncthreads();
        if (lane == 31) {
            sums[0][warp] = it;
            sums[1][warp] = iu;
        }
        __syncthreads();
        unsigned long long bt = run_t + it - t, bu = run_u + iu - u;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) {
                bt += sums[0][w];
                bu += sums[1][w];
            }
            run_t += sums[0][w];
            run_u += sums[1][w];
        }
        if (s < n) {
            e.seg_tiles[s] = bt;
            e.seg_units[s] = bu;
            put_seg(e.seg_table + (uint64_t)s * kSegWords, seg_at(a, e, s));
        }
    }
    if (tid == 0) {
        e.seg_tiles[n] = run_t;
        e.seg_units[n] = run_u;
        if (run_u > e.units && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
    }
}

// ------------------------------------------------------------- few query rows
//
// A worker is a team of 1 or 4 warps.  Warps take 16 cached tokens in turn, each with a
// private ring of cp.async stages (no barrier in the loop); query rows are the 16 rows of
// mma.sync m16n8k16, cached tokens the 8 columns of the first product and the 16 k of the
// second, so that weights go from one to the other in registers.  tcgen05 would leave 112 or more of
// its 128 rows empty here.  Bound: the latency of one warp's chain (of a tile of 16 tokens of 128 values
// 3,450 cycles with stamps of the clock in it: wait 150, scores 730, maximum 200, weights and sums 940, asking for the
// next tile 1,400) with the 12 warps that 168 registers leave an SM; 64 requests of up to 1,000 tokens of their own behind 8,192 common ones, with
// the kernel on tcgen05 beside it: 67 us, floor 34.6 by bytes.
template <int D, bool kF8, bool kHalf>
__global__ void __launch_bounds__(kWarps * 32, blocks_wanted(D))
    kv_pages_rows_kernel(const __grid_constant__ PageAttendArgs a) {
    constexpr bool kBf = !kF8 && !kHalf;          // type of the products' operands
    // Weights in two parts: bf16 (8 bits) alone errs as much as the output's rounding again, and
    // so does fp16 for fp16 outputs; fp16 is enough for bf16 outputs.
    constexpr bool kTwo = !kF8 || kHalf;
    // fp16 weights stand 2^7 higher, so that those down to 2^-21 of the largest keep their bits
    constexpr float kBits = kBf ? 0.0f : 7.0f;
    constexpr int RB = row_bytes(D, kF8), SV = smem_stride(D, kF8), PV = RB / 16, kStages = stages_of(D, kF8);
    constexpr int KS = D / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float join_m[kWarps][kRowsP], join_l[kWarps][kRowsP];
    __shared__ PageTableSpace space;
    __shared__ uint32_t masks[kWarps][kStages];
    // Behind the kernel on tcgen05, which lets this one start once what came before it is done, the two
    // have nothing to wait for in each other; this one ends after it, so that the join finds both done.
    if (!a.tc.on) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const PageEngine &e = a.rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const uint32_t team = e.team, team_id = warp / team, w_in = warp % team, teams = kWarps / team;
    const uint32_t worker = blockIdx.x * teams + team_id;
    unsigned long long x, x1;
    const PageTable table_of = table_and_share(a, e, blockIdx.x == 0, worker, space, &x, &x1);
    if (x >= x1) {                                // no barrier of the whole block follows
        if (a.tc.on) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    uint32_t seg = find_segment(e.whole ? table_of.units : table_of.tiles, seg_count(a, e), x);

    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * ring_bytes(D, kF8);
    float *mine = reinterpret_cast<float *>(smem + warp * ring_bytes(D, kF8));
    const int group = (int)a.group, H = (int)a.pool.H;
    const bool picked = a.picks != nullptr;
    // Tiles are copied 16 bytes a lane, a token's PV pieces by neighbouring lanes.  Lane i
    // (and i + 16) knows the place of token i and hands it round.
    constexpr int kAtOnce = 32 / PV;
    const int lane_tok = lane / PV, piece16 = lane - lane_tok * PV;
    const uint32_t to = ring + lane_tok * SV + piece16 * 16;

    while (x < x1) {
        const PagePiece piece = piece_of(a, e, table_of, &seg, x, x1, worker);
        const PageSeg &s = piece.s;
        const int rt = piece.rt, head = piece.head, k0 = piece.k0, k1 = piece.k1;
        x += piece.span;
        if (k0 >= k1 && !e.whole) continue;

        const int end = seen_tokens(a, e, s, rt);
        // rows of the tile: new token and head of the group
        const int per = (group + kRowsP - 1) / kRowsP;
        const int tok0 = picked ? rt / per : 0, row0 = picked ? rt % per * kRowsP : rt * kRowsP;
        const int rows = min(kRowsP, (picked ? group : s.n * group) - row0);
        const bool single = picked || (s.n == 1 && !s.prefix);       // rows of one token: no division
        auto new_token = [&](int row) { return single ? tok0 : (row0 + row) / group; };
        auto head_of = [&](int row) { return single ? row0 + row : (row0 + row) % group; };
        // tiles of the prefix come first where it stands in front of a request's own tokens
        const int pre = s.before, pre_tiles = (int)tiles_of(e, pre);
        const int32_t *table = s.prefix ? a.prefix_pages + (int64_t)s.index * a.prefix_stride
                                        : a.pages + (int64_t)s.index * a.pages_stride;
        const int32_t *pre_table = a.prefix_pages + (int64_t)max(s.in, 0) * a.prefix_stride;
        const int32_t *list = picked ? a.picks + ((int64_t)(s.q0 + tok0) * H + head) * a.budget : nullptr;
        const int pos0 = s.len - s.n + tok0;      // picked: the query's position
        const int pages0 = pages_seen(s.len, s.n, tok0, a.pool.T);
        const bool whole = !s.prefix && (s.in < 0 || a.joined) && k0 == 0 && k1 == piece.n_tiles;

        // Token of this lane in tile k (-1: none that is seen), and its page.  Where there is a list of pages,
        // its entry is read a tile before it is looked at.
        bool wrong_pick = false;
        auto first_of = [&](int k) { return ((k < pre_tiles ? k : k - pre_tiles) * (int)team + (int)w_in) * kTile; };
        auto place_in = [&](int k) { return first_of(k) + (lane & 15); };
        auto entry_of = [&](int k) {
            const int t = place_in(k);
            return picked && k < k1 && t < end ? list[div_T(a.pool, (uint32_t)t)] : -1;
        };
        auto token_of = [&](int k, int p) {
            const int t = place_in(k);
            if (k >= k1 || t >= (k < pre_tiles ? pre : end)) return -1;
            if (!picked) return t;
            if ((uint32_t)p >= (uint32_t)pages0) {
                wrong_pick |= p != -1;
                return -1;
            }
            const int real = p * (int)a.pool.T + (t - (int)(div_T(a.pool, (uint32_t)t) * a.pool.T));
            return real <= pos0 ? real : -1;
        };
        auto page_of = [&](int k, int t) { return t >= 0 ? (k < pre_tiles ? pre_table : table)[div_T(a.pool, (uint32_t)t)] : 0; };
        int tk[kStages + 1], entry[kStages + 2];
        int32_t pg[kStages + 1];
#pragma unroll
        for (int i = 0; i < kStages + 2; ++i) entry[i] = entry_of(k0 + i);
#pragma unroll
        for (int i = 0; i < kStages + 1; ++i) {
            tk[i] = token_of(k0 + i, entry[i]);
            pg[i] = page_of(k0 + i, tk[i]);
        }
        // Query rows first, so that they are there when the first tiles are.
        constexpr int SQ = 2 * D + 16;
        static_assert(kRowsP * SQ <= stage_bytes(D, kF8), "queries fit a stage");
        const uint32_t place = ring + (kStages - 1) * stage_bytes(D, kF8);
        int pos;
        {
            // through the last stage's place, neighbouring lanes a row's 16-byte pieces
            constexpr int PQ = D / 8, AQ = PQ <= 8 ? 4 : PQ <= 16 ? 2 : 1;
            const int sub = lane / PQ, ch = lane - sub * PQ;
            const bool on = (lane & 15) < rows;
            const int i = on ? new_token(lane & 15) : 0, j = on ? head_of(lane & 15) : 0;
            const long long mine_at = (long long)(s.q0 + i) * a.q.s_tok + (long long)(head * group + j) * a.q.s_head;
            pos = s.prefix || picked || !on ? end - 1 : s.len - s.n + i;
#pragma unroll
            for (int r0 = 0; r0 < kRowsP; r0 += AQ) {
                const int r = r0 + sub;
                const long long from = __shfl_sync(0xffffffffu, mine_at, r & 15);
                if (sub < AQ) copy16(place + r * SQ + ch * 16, a.q.data + from + ch * 16, r < rows);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        const uint64_t from_k = a.pool.base[0] + (uint64_t)head * a.pool.s_head + piece16 * 16;
        const uint64_t from_v = a.pool.base[1] + (uint64_t)head * a.pool.s_head + piece16 * 16;
        auto load = [&](int stage, int k, int t, int32_t page) {
            if (k < k1) {
                const bool bad = t >= 0 && (uint32_t)page >= a.pool.P, ok = t >= 0 && !bad;
                const uint32_t where = ok ? vector_index(a.pool, (uint32_t)page, (uint32_t)t) : 0;
                const uint32_t good = __ballot_sync(0xffffffffu, ok), bads = __ballot_sync(0xffffffffu, bad);
                if (lane == 0) masks[warp][stage] = (good & 0xffffu) | bads << 16;
                const uint32_t dst = to + stage * stage_bytes(D, kF8);
                if ((good & 0xffffu) == 0xffffu) {
#pragma unroll
                    for (int i = 0; i < (kTile + kAtOnce - 1) / kAtOnce; ++i) {
                        const int tok = i * kAtOnce + lane_tok;
                        const uint32_t w = __shfl_sync(0xffffffffu, where, tok & 15);
                        if (lane_tok < kAtOnce && (kTile % kAtOnce == 0 || tok < kTile)) {
                            copy16(dst + i * kAtOnce * SV, from_k + (uint64_t)w * (uint32_t)RB);
                            copy16(dst + (i * kAtOnce + kTile) * SV, from_v + (uint64_t)w * (uint32_t)RB);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < (kTile + kAtOnce - 1) / kAtOnce; ++i) {
                        const int tok = i * kAtOnce + lane_tok;
                        const uint32_t w = __shfl_sync(0xffffffffu, where, tok & 15);
                        if (lane_tok < kAtOnce && (kTile % kAtOnce == 0 || tok < kTile)) {
                            copy16(dst + i * kAtOnce * SV, from_k + (uint64_t)w * (uint32_t)RB, good >> (tok & 15) & 1);
                            copy16(dst + (i * kAtOnce + kTile) * SV, from_v + (uint64_t)w * (uint32_t)RB, good >> (tok & 15) & 1);
                        }
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // Query rows as A fragments.  fp8 keys meet fp16 queries: a bf16 row is scaled by
        // the power of two that brings its largest value to 2^14..2^15 (values under 2^-22
        // of it lose bits), which its scores undo.
        uint32_t qf[KS][4];
        float sc[2];
        int lim[2];
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) load(i, k0 + i, tk[i], pg[i]);
        {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 2; ++r) lim[r] = __shfl_sync(0xffffffffu, pos, g + 8 * r);
            if (kF8) {
                // fragments of fp8 come 4 values a lane: 4 c and 4 c + 2 of a run of 16 are the lane's pairs
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        uint32_t w[2];
                        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(place + (g + 8 * r) * SQ + 32 * ks + 8 * c) : "memory");
                        qf[ks][r] = w[0];
                        qf[ks][r + 2] = w[1];
                    }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) ldm(place + (lane & 15) * SQ + ks * 32 + (lane >> 4) * 16, qf[ks]);
            }
            __syncwarp();
        }
        load(kStages - 1, k0 + kStages - 1, tk[kStages - 1], pg[kStages - 1]);
        int entry_next = entry[kStages + 1];
        int t_next = tk[kStages];
        int32_t page_next = pg[kStages];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sc[r] = a.scale_log2;
            if (kF8 && !kHalf) {
                float top = 0.0f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 f = unpack2<true>(qf[ks][r + 2 * h]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t ex = max(__float_as_uint(top) >> 23, 15u);
                const float up = ex < 255 ? __uint_as_float((268u - ex) << 23) : 1.0f;
                sc[r] *= ex < 255 ? __uint_as_float((ex - 14u) << 23) : 1.0f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 f = unpack2<true>(qf[ks][r + 2 * h]);
                        qf[ks][r + 2 * h] = pack2<false>(f.x * up, f.y * up);
                    }
            }
        }
        const int all_see = s.prefix || picked ? end : s.len - s.n + new_token(0) + 1;   // tokens that every row sees

        float o[2 * KS][4], m[2] = {kNoMax, kNoMax}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.0f;

        // lane constants of the fragments' addresses
        const uint32_t k_at = kF8 ? ((lane >> 3 & 1) * 8 + (lane & 7)) * SV + (lane >> 4) * 16
                                  : ((lane >> 4) * 8 + (lane & 7)) * SV + (lane >> 3 & 1) * 16;
        const uint32_t v_at = ((lane >> 3 & 1) * 8 + (lane & 7)) * SV + (lane >> 4) * 16 + kTile * SV;
        int stage = 0;
        for (int k = k0; k < k1; ++k) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint32_t tile = ring + stage * stage_bytes(D, kF8);
            const uint32_t mask = masks[warp][stage];
            const int t0 = first_of(k);
            const bool edge = !picked && k >= pre_tiles && min(t0 + kTile, end) > all_see;      // rows see different tokens
            if (mask != 0) {                      // a token that some row sees
                float y[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[n][i] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < KS; ks += kF8 ? 2 : 1) {
                    uint32_t b[4];
                    ldm(tile + k_at + ks * (kF8 ? 16 : 32), b);
                    if (kF8) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int n = 0; n < 2; ++n)
                                mma<false>(y[n], qf[ks + h], e4m3x2(b[2 * h + n]), e4m3x2(b[2 * h + n] >> 16));
                    } else {
                        mma<kBf>(y[0], qf[ks], b[0], b[1]);
                        mma<kBf>(y[1], qf[ks], b[2], b[3]);
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[n][i] = y[n][i] * sc[i >> 1] - (m[i >> 1] == kNoMax ? 0.0f : m[i >> 1]);
                if (mask != 0xffffu || edge) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int in = 8 * n + 2 * c + (i & 1);
                            if (mask >> 16 >> in & 1) y[n][i] = __uint_as_float(kNanWord);
                            if (!((mask | mask >> 16) >> in & 1) || (edge && t0 + in > lim[i >> 1])) y[n][i] = -INFINITY;
                        }
                    if (mask >> 16 != 0 && a.status != nullptr && lane == 0) atomicOr(a.status, KV_STATUS_BAD_PAGE);
                    if (edge) {
                        // A value that is not finite must not reach rows that do not see it (0 x NaN): it
                        // makes its dim NaN in those that do, and leaves the tile.
                        uint32_t found = 0;
                        for (int i = lane; i < kTile * PV; i += 32) {
                            const uint32_t p = tile + (kTile + i / PV) * SV + i % PV * 16;
                            uint32_t w[4];
                            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p) : "memory");
                            found |= not_finite<kF8, kBf>(w[0]) | not_finite<kF8, kBf>(w[1]) | not_finite<kF8, kBf>(w[2]) | not_finite<kF8, kBf>(w[3]);
                        }
                        if (__any_sync(0xffffffffu, found != 0)) {
                            for (int t = 0; t < kTile; ++t)
#pragma unroll
                                for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const int d = kF8 ? 16 * (n >> 1) + 4 * c + 2 * (i & 1) + (n & 1) : 8 * n + 2 * c + (i & 1);
                                        const unsigned char *v = smem + (tile - (uint32_t)__cvta_generic_to_shared(smem)) + (kTile + t) * SV;
                                        const uint32_t w = kF8 ? v[d] * 0x01010101u : reinterpret_cast<const unsigned short *>(v)[d];
                                        if ((not_finite<kF8, kBf>(w) & (kF8 ? 0xffu : 0xffffu)) != 0 && t0 + t <= lim[i >> 1]) o[n][i] = __uint_as_float(kNanWord);
                                    }
                            __syncwarp();
                            for (int i = lane; i < kTile * RB / 4; i += 32) {
                                uint32_t *p = reinterpret_cast<uint32_t *>(smem + (tile - (uint32_t)__cvta_generic_to_shared(smem)) + (kTile + i / (RB / 4)) * SV) + i % (RB / 4);
                                *p &= ~not_finite<kF8, kBf>(*p);
                            }
                            __syncwarp();
                        }
                    }
                }
                // The maximum moves only when a score passes it by more than 2^8.
                const float over[2] = {fmaxf(fmaxf(y[0][0], y[0][1]), fmaxf(y[1][0], y[1][1])),
                                       fmaxf(fmaxf(y[0][2], y[0][3]), fmaxf(y[1][2], y[1][3]))};
                bool move = false;
#pragma unroll
                for (int r = 0; r < 2; ++r) move |= over[r] > kBits + 8.0f || m[r] == kNoMax;
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float t = over[r];
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                        if (t == -INFINITY) continue;
                        float up = 0.0f;
                        if (m[r] == kNoMax) {
                            up = t - kBits;
                            m[r] = up;
                        } else if (t > kBits + 8.0f) {
                            up = t - kBits;
                            m[r] += up;
                            const float f = exp2_fast(-up);
                            l[r] *= f;
#pragma unroll
                            for (int n = 0; n < 2 * KS; ++n) {
                                o[n][2 * r] *= f;
                                o[n][2 * r + 1] *= f;
                            }
                        }
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            y[n][2 * r] -= up;
                            y[n][2 * r + 1] -= up;
                        }
                    }
                }
                uint32_t p[4], rest[4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float u = exp2_fast(y[n][2 * r]), v = exp2_fast(y[n][2 * r + 1]);
                        l[r] += u + v;
                        p[2 * n + r] = pack2<kBf>(u, v);
                        if (kTwo) {
                            const float2 f = unpack2<kBf>(p[2 * n + r]);
                            rest[2 * n + r] = pack2<kBf>(u - f.x, v - f.y);
                        }
                    }
#pragma unroll
                for (int j = 0; j < 2 * KS; j += kF8 ? 4 : 2) {
                    uint32_t b[4];
                    ldm_t(tile + v_at + j * (kF8 ? 8 : 16), b);
                    if (kF8) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // even and odd dims of 16
                            const uint32_t e0 = e4m3x2(__byte_perm(b[2 * h], 0, 0x4420)), e1 = e4m3x2(__byte_perm(b[2 * h + 1], 0, 0x4420));
                            const uint32_t o0 = e4m3x2(__byte_perm(b[2 * h], 0, 0x4431)), o1 = e4m3x2(__byte_perm(b[2 * h + 1], 0, 0x4431));
                            mma<false>(o[j + 2 * h], p, e0, e1);
                            mma<false>(o[j + 2 * h + 1], p, o0, o1);
                            if (kTwo) {
                                mma<false>(o[j + 2 * h], rest, e0, e1);
                                mma<false>(o[j + 2 * h + 1], rest, o0, o1);
                            }
                        }
                    } else {
                        mma<kBf>(o[j], p, b[0], b[1]);
                        mma<kBf>(o[j + 1], p, b[2], b[3]);
                        if (kTwo) {
                            mma<kBf>(o[j], rest, b[0], b[1]);
                            mma<kBf>(o[j + 1], rest, b[2], b[3]);
                        }
                    }
                }
            }
            __syncwarp();
            load(stage, k + kStages, t_next, page_next);
            t_next = token_of(k + kStages + 1, entry_next);
            page_next = page_of(k + kStages + 1, t_next);
            entry_next = entry_of(k + kStages + 2);
            if (++stage == kStages) stage = 0;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
        if (wrong_pick && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_PAGE);

        const uint64_t to_row = piece.slot * e.slot_rows;
        if (team == 1) {
            // a warp's rows go out of its registers, pairs of neighbouring dims a lane (fp8: four)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float t = l[r];
                t += __shfl_xor_sync(0xffffffffu, t, 1);
                t += __shfl_xor_sync(0xffffffffu, t, 2);
                const int row = g + 8 * r;
                if (row >= rows) continue;
                const int64_t tok = s.q0 + new_token(row);
                const int qh = head * group + head_of(row);
                if (whole) {
                    const float inv = t != 0.0f ? a.v_scale / t : 0.0f;
                    const uint64_t dst = a.out.data + tok * a.out.s_tok + (int64_t)qh * a.out.s_head;
#pragma unroll
                    for (int n = 0; n < 2 * KS; ++n) {
                        if (!kF8)
                            *reinterpret_cast<uint32_t *>(dst + 16 * n + 4 * c) = pack2<!kHalf>(o[n][2 * r] * inv, o[n][2 * r + 1] * inv);
                        else if ((n & 1) == 0)
                            *reinterpret_cast<uint2 *>(dst + 16 * n + 8 * c) =
                                make_uint2(pack2<!kHalf>(o[n][2 * r] * inv, o[n + 1][2 * r] * inv), pack2<!kHalf>(o[n][2 * r + 1] * inv, o[n + 1][2 * r + 1] * inv));
                    }
                    if (c == 0 && a.lse != nullptr)
                        a.lse[tok * a.q_heads + qh] = t != 0.0f ? (m[r] + log2f(t)) * 0.693147180559945f : -INFINITY;
                } else {
                    float *dst = e.part_o + (to_row + row) * D;
#pragma unroll
                    for (int n = 0; n < 2 * KS; ++n) {
                        if (!kF8)
                            *reinterpret_cast<float2 *>(dst + 8 * n + 2 * c) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
                        else if ((n & 1) == 0)
                            *reinterpret_cast<float4 *>(dst + 8 * n + 4 * c) =
                                make_float4(o[n][2 * r], o[n + 1][2 * r], o[n][2 * r + 1], o[n + 1][2 * r + 1]);
                    }
                    if (c == 0) *reinterpret_cast<float2 *>(e.part_ml + (to_row + row) * 2) = make_float2(m[r], t);
                }
            }
            __syncwarp();                         // the ring is free again
            continue;
        }
        // Join the team's warps: accumulators go to the warp's own ring as [row][D + 4].
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float t = l[r];
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            const int row = g + 8 * r;
            if (c == 0) {
                join_m[warp][row] = m[r];
                join_l[warp][row] = t;
            }
            float *dst = mine + row * (D + 4);
#pragma unroll
            for (int n = 0; n < 2 * KS; ++n) {
                if (kF8) {
                    if ((n & 1) == 0)
                        *reinterpret_cast<float4 *>(dst + 16 * (n >> 1) + 4 * c) =
                            make_float4(o[n][2 * r], o[n + 1][2 * r], o[n][2 * r + 1], o[n + 1][2 * r + 1]);
                } else {
                    *reinterpret_cast<float2 *>(dst + 8 * n + 2 * c) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
                }
            }
        }
        team_sync(team, team_id);
        constexpr int D4 = D / 4;
        const int first = (int)(team_id * team);
        for (int it = (int)w_in * 32 + lane; it < rows * D4; it += (int)team * 32) {
            const int row = it / D4, d4 = it - row * D4;
            float top = kNoMax, sum = 0.0f;
            for (int w = first; w < first + (int)team; ++w)
                if (join_l[w][row] != 0.0f) top = fmaxf(top, join_m[w][row]);
            float4 acc = make_float4(0, 0, 0, 0);
            for (int w = first; w < first + (int)team; ++w) {
                const float lw = join_l[w][row];
                if (lw == 0.0f) continue;         // this warp saw nothing of the row
                const float f = exp2_fast(join_m[w][row] - top);
                const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(smem + w * ring_bytes(D, kF8)) +
                                                                   row * (D + 4) + d4 * 4);
                sum += lw * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
            if (whole) {
                const int64_t tok = s.q0 + new_token(row);
                const int qh = head * group + head_of(row);
                const float inv = sum != 0.0f ? a.v_scale / sum : 0.0f;
                *reinterpret_cast<uint2 *>(a.out.data + tok * a.out.s_tok + (int64_t)qh * a.out.s_head + d4 * 8) =
                    make_uint2(pack2<!kHalf>(acc.x * inv, acc.y * inv), pack2<!kHalf>(acc.z * inv, acc.w * inv));
                if (d4 == 0 && a.lse != nullptr)
                    a.lse[tok * a.q_heads + qh] = sum != 0.0f ? (top + log2f(sum)) * 0.693147180559945f : -INFINITY;
            } else {
                *reinterpret_cast<float4 *>(e.part_o + (to_row + row) * D + d4 * 4) = acc;
                if (d4 == 0) *reinterpret_cast<float2 *>(e.part_ml + (to_row + row) * 2) = make_float2(top, sum);
            }
        }
        team_sync(team, team_id);                 // rings are free again
    }
    if (a.tc.on) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------- the join
//
// A row (query token and head) takes the pieces of its prefix and of its own tokens, kW
// warps a row, each every kW-th piece, a lane D / 32 values.  Rows that one worker held alone
// were written by it.  Bound: a chain of three dependent reads (plan, maxima, sums), 3 to 7 us; several heads
// a warp were no faster.

// Pieces of head j of a KV head's group and query token i of a segment: `tiles` and `units` of the engine's come before it.
__device__ __forceinline__ RowPieces find_pieces(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, uint64_t tiles, uint64_t units,
                                                 uint64_t total, int i, int head, int j) {
    int row;
    const int rt = row_tile_of(a, e, i, j, &row);
    return row_pieces(a, e, share_of(total, e.workers), tiles + tiles_before(a, e, s, rt) * a.pool.H, units, unit_span(a, e, s, rt), rt, row, head);
}

template <int D, bool kHalf, int kW>
__global__ void __launch_bounds__(128) kv_pages_join_kernel(const __grid_constant__ PageAttendArgs a) {
    constexpr int NV = D / 32;
    __shared__ float acc_s[kW][D], m_s[kW], l_s[kW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int qh = kW == 1 ? blockIdx.x * 4 + warp : blockIdx.x, part = kW == 1 ? 0 : warp;
    const int i = blockIdx.y, r = blockIdx.z, group = (int)a.group;
    // the call's inputs were there before the kernels in front of this one began
    const PageSeg own = own_seg(a, r);
    const int in = a.joined ? -1 : own.in;
    const int64_t tok = own.q0 + i;
    const int head = qh / group, j = qh - head * group;
    const PageSeg pre = in >= 0 ? prefix_seg(a, (uint32_t)in) : own;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (qh >= (int)a.q_heads || i >= own.n) return;
    // all that says where the row's pieces are, in one go
    const PageEngine &e0 = a.tc.prefix ? a.tc : a.rows, &e1 = a.tc.own ? a.tc : a.rows;
    const uint32_t at1 = (e1.prefix ? a.groups : 0) + (uint32_t)r, n0 = seg_count(a, e0), n1 = seg_count(a, e1);
    unsigned long long tiles0 = 0, units0 = 0, total0 = 0, all0 = 0;
    if (in >= 0) {
        tiles0 = e0.seg_tiles[in];
        units0 = e0.seg_units[in];
        total0 = e0.seg_tiles[n0];
        all0 = e0.seg_units[n0];
    }
    const unsigned long long tiles1 = e1.seg_tiles[at1], units1 = e1.seg_units[at1], total1 = e1.seg_tiles[n1], all1 = e1.seg_units[n1];
    if ((in >= 0 && all0 > e0.units) || all1 > e1.units) return;
    const RowPieces p1 = find_pieces(a, e1, own, tiles1, units1, total1, i, head, j);
    if (in < 0 && p1.any && p1.w0 == p1.w1) return;
    int c0 = 0, c1 = p1.any ? (int)(p1.w1 - p1.w0) + 1 : 0;       // pieces of the prefix and of its own tokens
    unsigned long long from0 = 0;
    if (in >= 0) {
        const RowPieces p0 = find_pieces(a, e0, pre, tiles0, units0, total0, (int)(tok - pre.q0), head, j);
        c0 = p0.any ? (int)(p0.w1 - p0.w0) + 1 : 0;
        from0 = (p0.unit + p0.w0) * e0.slot_rows + p0.row;
    }
    const unsigned long long from1 = (p1.unit + p1.w0) * e1.slot_rows + p1.row;
    float top = kNoMax, sum = 0.0f, acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] = 0.0f;
    // A lane looks after a piece's maximum and sum, 32 pieces at a time; then all take the sums of each.
    for (int p = part; p < c0 + c1; p += 32 * kW) {
        const int mine = p + lane * kW, count = min(32, (c0 + c1 - p + kW - 1) / kW);
        float2 ml = make_float2(kNoMax, 0.0f);
        unsigned long long o_at = 0;
        if (mine < c0 + c1) {
            const bool one = mine < c0;
            const unsigned long long at = one ? from0 + (unsigned long long)mine * e0.slot_rows : from1 + (unsigned long long)(mine - c0) * e1.slot_rows;
            ml = *reinterpret_cast<const float2 *>((one ? e0.part_ml : e1.part_ml) + at * 2);
            o_at = reinterpret_cast<unsigned long long>((one ? e0.part_o : e1.part_o) + at * D);
        }
        float most = ml.y != 0.0f ? ml.x : kNoMax;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        most = fmaxf(most, top);
        // -1: nothing seen.  A weight that underflows still multiplies: 0 x NaN is what such a value gives.
        const float u = exp2_fast(top - most), f = ml.y != 0.0f ? exp2_fast(ml.x - most) : -1.0f;
        float add = ml.y != 0.0f ? ml.y * f : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
        top = most;
        sum = sum * u + add;
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] *= u;
#pragma unroll 4
        for (int k = 0; k < count; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const float *o = reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, o_at, k)) + lane;
            float x[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) x[v] = o[v * 32];
            if (fk < 0.0f) continue;
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] += x[v] * fk;
        }
    }
    if (kW > 1) {
        if (lane == 0) {
            m_s[warp] = top;
            l_s[warp] = sum;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) acc_s[warp][v * 32 + lane] = acc[v];
        __syncthreads();
        if (warp != 0) return;
        float most = kNoMax;
#pragma unroll
        for (int w = 0; w < kW; ++w)
            if (l_s[w] != 0.0f) most = fmaxf(most, m_s[w]);
        sum = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] = 0.0f;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (l_s[w] == 0.0f) continue;
            const float f = exp2_fast(m_s[w] - most);
            sum += l_s[w] * f;
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] += acc_s[w][v * 32 + lane] * f;
        }
        top = most;
    }
    const float inv = sum != 0.0f ? a.v_scale / sum : 0.0f;
    const uint64_t dst = a.out.data + tok * a.out.s_tok + (int64_t)qh * a.out.s_head;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const uint64_t to = dst + 2 * (v * 32 + lane);
        if (kHalf) *reinterpret_cast<__half *>(to) = __float2half_rn(acc[v] * inv);
        else *reinterpret_cast<__nv_bfloat16 *>(to) = __float2bfloat16_rn(acc[v] * inv);
    }
    if (lane == 0 && a.lse != nullptr)
        a.lse[tok * a.q_heads + qh] = sum != 0.0f ? (top + log2f(sum)) * 0.693147180559945f : -INFINITY;
}

// The same for calls with many rows, 8 lanes a row: a warp takes join_heads rows of a token, four at once, and
// works out once where their pieces are; sums are asked for together with the maxima that weigh them.  A
// token's rows lie in at most two row tiles of a segment (kManyGroup heads of a group), or have a list of pages.
// Bound: latency of the reads.  Four chunks of 500 tokens of 32 heads of 128 behind 8,192: the call took 233 us, 259 with the
// kernel above, 252 where that takes its rows in turn.

// What comes before row tile rt of a segment, by a warp.
__device__ __forceinline__ uint64_t warp_tiles_before(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, int rt, int lane) {
    if (s.prefix || a.picks != nullptr) return rt == 0 ? 0 : (uint64_t)rt * unit_span(a, e, s, 0);
    unsigned long long sum = 0;
    for (int k = lane; k < rt; k += 32) sum += unit_span(a, e, s, k);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

// A segment with the row tiles of one of its tokens.
struct JoinSide {
    unsigned long long tiles, units, share, at[2];
    uint32_t span[2];
    int i, rt;
    __device__ __forceinline__ void begin(const PageAttendArgs &a, const PageEngine &e, const PageSeg &s, unsigned long long total, int token,
                                          int lane) {
        int row;
        i = token;
        share = share_of(total, e.workers);
        rt = row_tile_of(a, e, i, 0, &row);
        const int rt1 = row_tile_of(a, e, i, (int)a.group - 1, &row);
        at[0] = tiles + warp_tiles_before(a, e, s, rt, lane) * a.pool.H;
        span[0] = unit_span(a, e, s, rt);
        at[1] = at[0] + (uint64_t)span[0] * a.pool.H;
        span[1] = rt1 != rt ? unit_span(a, e, s, rt1) : 0;
    }
    __device__ __forceinline__ RowPieces find(const PageAttendArgs &a, const PageEngine &e, int head, int j) const {
        int row;
        const int t = row_tile_of(a, e, i, j, &row);
        // with lists all units of a token are of one span
        if (a.picks != nullptr)
            return row_pieces(a, e, share, at[0] + (uint64_t)(t - rt) * span[0] * a.pool.H, units, span[0], t, row, head);
        return row_pieces(a, e, share, t != rt ? at[1] : at[0], units, t != rt ? span[1] : span[0], t, row, head);
    }
};

template <int D, bool kHalf>
__global__ void __launch_bounds__(128) kv_pages_join_many_kernel(const __grid_constant__ PageAttendArgs a) {
    constexpr int NV = D / 32, kAtOnce = D <= 128 ? 2 : 1;
    const int lane = threadIdx.x & 31, in8 = lane & 7;
    const int i = blockIdx.y, r = blockIdx.z, group = (int)a.group;
    const int first = (blockIdx.x * 4 + (threadIdx.x >> 5)) * (int)a.join_heads, last = min((int)a.q_heads, first + (int)a.join_heads);
    // the call's inputs were there before the kernels in front of this one began
    const PageSeg own = own_seg(a, r);
    const int in = a.joined ? -1 : own.in;
    const int64_t tok = own.q0 + i;
    const PageSeg pre = in >= 0 ? prefix_seg(a, (uint32_t)in) : own;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (first >= last || i >= own.n) return;
    const PageEngine &e0 = a.tc.prefix ? a.tc : a.rows, &e1 = a.tc.own ? a.tc : a.rows;
    const uint32_t at1 = (e1.prefix ? a.groups : 0) + (uint32_t)r, n0 = seg_count(a, e0), n1 = seg_count(a, e1);
    JoinSide d0{}, d1{};
    unsigned long long total0 = 0, all0 = 0;
    if (in >= 0) {
        d0.tiles = e0.seg_tiles[in];
        d0.units = e0.seg_units[in];
        total0 = e0.seg_tiles[n0];
        all0 = e0.seg_units[n0];
    }
    d1.tiles = e1.seg_tiles[at1];
    d1.units = e1.seg_units[at1];
    const unsigned long long total1 = e1.seg_tiles[n1], all1 = e1.seg_units[n1];
    if ((in >= 0 && all0 > e0.units) || all1 > e1.units) return;
    d1.begin(a, e1, own, total1, i, lane);
    if (in >= 0) d0.begin(a, e0, pre, total0, (int)(tok - pre.q0), lane);
    for (int q = first; q < last; q += 4) {
        const int qh = q + (lane >> 3);
        if (qh >= last) continue;                 // no shuffle follows
        const int head = qh / group, j = qh - head * group;
        const RowPieces p1 = d1.find(a, e1, head, j);
        if (in < 0 && p1.any && p1.w0 == p1.w1) continue;
        const int c1 = p1.any ? (int)(p1.w1 - p1.w0) + 1 : 0;
        int c0 = 0;
        unsigned long long from0 = 0;
        if (in >= 0) {
            const RowPieces p0 = d0.find(a, e0, head, j);
            c0 = p0.any ? (int)(p0.w1 - p0.w0) + 1 : 0;
            from0 = (p0.unit + p0.w0) * e0.slot_rows + p0.row;
        }
        const unsigned long long from1 = (p1.unit + p1.w0) * e1.slot_rows + p1.row;
        float top = kNoMax, sum = 0.0f;
        float4 acc[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p = 0; p < c0 + c1; p += kAtOnce) {
            float2 ml[kAtOnce];
            float4 x[kAtOnce][NV];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                ml[k] = make_float2(kNoMax, 0.0f);
                if (p + k >= c0 + c1) continue;
                const bool one = p + k < c0;
                const unsigned long long at = one ? from0 + (unsigned long long)(p + k) * e0.slot_rows : from1 + (unsigned long long)(p + k - c0) * e1.slot_rows;
                ml[k] = *reinterpret_cast<const float2 *>((one ? e0.part_ml : e1.part_ml) + at * 2);
                const float4 *o = reinterpret_cast<const float4 *>((one ? e0.part_o : e1.part_o) + at * D) + in8;
#pragma unroll
                for (int v = 0; v < NV; ++v) x[k][v] = o[8 * v];
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (ml[k].y == 0.0f) continue;    // nothing seen
                const float most = fmaxf(top, ml[k].x), u = exp2_fast(top - most), f = exp2_fast(ml[k].x - most);
                top = most;
                sum = sum * u + ml[k].y * f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    acc[v].x = acc[v].x * u + x[k][v].x * f;
                    acc[v].y = acc[v].y * u + x[k][v].y * f;
                    acc[v].z = acc[v].z * u + x[k][v].z * f;
                    acc[v].w = acc[v].w * u + x[k][v].w * f;
                }
            }
        }
        const float inv = sum != 0.0f ? a.v_scale / sum : 0.0f;
        const uint64_t dst = a.out.data + tok * a.out.s_tok + (int64_t)qh * a.out.s_head;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            *reinterpret_cast<uint2 *>(dst + 2 * (v * 32 + in8 * 4)) =
                make_uint2(pack2<!kHalf>(acc[v].x * inv, acc[v].y * inv), pack2<!kHalf>(acc[v].z * inv, acc[v].w * inv));
        if (in8 == 0 && a.lse != nullptr)
            a.lse[tok * a.q_heads + qh] = sum != 0.0f ? (top + log2f(sum)) * 0.693147180559945f : -INFINITY;
    }
}

typedef void(PagesFn)(PageAttendArgs);
struct Variant {
    uint32_t D;
    bool fp8, fp16;
    PagesFn *rows_fn, *join_fn, *join4_fn, *join_many_fn;
    int smem, blocks;      // blocks of an SM: set when the kernels are loaded
};
template <int D, bool kF8, bool kHalf>
constexpr Variant variant() {
    return Variant{(uint32_t)D, kF8, kHalf, kv_pages_rows_kernel<D, kF8, kHalf>, kv_pages_join_kernel<D, kHalf, 1>,
                   kv_pages_join_kernel<D, kHalf, 4>, kv_pages_join_many_kernel<D, kHalf>, kWarps * ring_bytes(D, kF8), 1};
}
#define KVB_PAGES(D) variant<D, false, false>(), variant<D, false, true>(), variant<D, true, false>(), variant<D, true, true>()
Variant g_variants[] = {KVB_PAGES(64), KVB_PAGES(96), KVB_PAGES(128), KVB_PAGES(192), KVB_PAGES(256)};

const Variant *find_variant(uint32_t D, bool fp8, bool fp16) {
    for (const Variant &v : g_variants)
        if (v.D == D && v.fp8 == fp8 && v.fp16 == fp16) return &v;
    return nullptr;
}

cudaError_t launch(PagesFn *fn, dim3 grid, int threads, int smem, cudaStream_t stream, bool pdl, const PageAttendArgs &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace

uint32_t pages_blocks(uint32_t D, bool fp8) { return (uint32_t)find_variant(D, fp8, false)->blocks; }

cudaError_t launch_pages(const PageAttendArgs &a, const PagePlan &p, uint32_t D, bool fp8, bool fp16, bool pdl,
                         cudaStream_t stream, int *launches) {
    (void)cudaGetLastError();
    const Variant *v = find_variant(D, fp8, fp16);
    if (v == nullptr) return cudaErrorInvalidValue;
    cudaError_t e;
    if ((a.rows.on && !a.rows.small) || (a.tc.on && !a.tc.small)) {
        e = launch(kv_pages_plan_kernel, dim3(2), kPlanThreads, 0, stream, pdl, a);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    if (a.tc.on) {
        e = launch_pages_tc(a, D, fp8, fp16, pdl, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    if (a.rows.on) {
        const uint32_t teams = kWarps / a.rows.team;
        e = launch(v->rows_fn, dim3((a.rows.workers + teams - 1) / teams), kWarps * 32, v->smem, stream, pdl, a);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    if (a.rows.whole) return cudaSuccess;
    if (p.wide_join) e = launch(v->join4_fn, dim3(a.q_heads, a.max_q, a.requests), 128, 0, stream, pdl, a);
    else e = launch(a.join_heads > 1 ? v->join_many_fn : v->join_fn,
                    dim3((a.q_heads + 4 * a.join_heads - 1) / (4 * a.join_heads), a.max_q, a.requests), 128, 0, stream, pdl, a);
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t preload_pages_kernels() {
    cudaFuncAttributes at;
    const cudaError_t e0 = cudaFuncGetAttributes(&at, (const void *)kv_pages_plan_kernel);
    if (e0 != cudaSuccess) return e0;
    for (Variant &v : g_variants) {
        cudaError_t e = cudaFuncGetAttributes(&at, (const void *)v.rows_fn);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute((const void *)v.rows_fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v.blocks, (const void *)v.rows_fn, kWarps * 32, (size_t)v.smem);
        if (e == cudaSuccess && v.blocks < 1) e = cudaErrorInvalidConfiguration;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, (const void *)v.join_fn);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, (const void *)v.join4_fn);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, (const void *)v.join_many_fn);
        // The same split of an SM's memory for all: an SM has to be empty to change it, and blocks of the next
        // kernel, launched early, would find no place beside the join's.
        for (PagesFn *fn : {v.rows_fn, v.join_fn, v.join4_fn, v.join_many_fn})
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
    }
    return preload_pages_tc_kernels();
}

}  // namespace kvb
