// kvb_pages_tc.cu -- attention of many query rows over pages held in 16 bits or in fp8
// (kv_attend_shared: the queries of a group over its prefix, a prompt chunk over its own
// tokens), on the fifth-generation tensor cores.
//
// A block is a worker (kvb_pages.h).  A unit's 256 query rows (128 for heads over 128
// values) are two tiles of 128, and a block walks the cached tokens of its piece 64 at a time.
// Warps have roles:
//   2 warps  16-bit pages: bring keys and values into swizzled tiles in shared memory by
//            cp.async.  TMA gathers of four tokens were measured: a warp issues one in 70 cycles, so
//            that the 64 of a tile took 4,300 cycles from one warp, 2,500 from three
//   4 warps  (8 for heads over 128) fp8 pages: the same through registers, as fp16, exact
//   1 warp   issues tcgen05.mma: scores S = Q K^T and sums O += P V
//   4 + 4    softmax of the two tiles (4 of one), one row a thread: scores come from tensor
//            memory, weights go back there, the A operand of P V
// Tensor memory holds two buffers of 64 scores a row for each tile (P overwrites S) and
// O0, O1 (D columns each; one of up to 256).
//
// Bound: a product of 64 keys reads 6 KB of shared memory for 32 cycles of arithmetic, 1,280 cycles a tile for
// both row tiles; measured are 1,640, and 14,000 for the beginning and end of a piece (27,000 of a block's first
// piece, cold).  Four chunks of 500 tokens behind 8,192: 238 us with the join, floor 147.4 by operations (1.17 PFLOP/s).
//
// What is rounded: a weight, to the operands' type (bf16: 2^-9 of itself at most, 2^-8 in
// steps of the type; fp16: 2^-11), once; a bf16 query against fp8 pages below 2^-22 of
// the row's largest.  16-bit queries and keys multiply exactly.
#include "kvb_pages.h"
#include "kvb_pages_device.h"
#include "kvb_pages_internal.h"
#include "kvb_tc.h"

#include <algorithm>

namespace kvb {

using namespace tc;

namespace {

constexpr int kTileQ = kTcTileQ, kTileK = 1 << kTcShift;
constexpr float kNoMax = -3.0e38f;
// 64 values (128 bytes, swizzled) of every row of a tile
constexpr uint32_t kBlockQ = kTileQ * 128, kBlockK = kTileK * 128;

__host__ __device__ constexpr int blocks_of(int D) { return (D + 63) / 64; }
// Softmax warps, and those that bring keys and values: 13 warps of fp8 (128 registers a thread), 11 or 7 of
// 16 bits.
__host__ __device__ constexpr int soft_warps(int D) { return 4 * tc_q_tiles(D); }
__host__ __device__ constexpr int load_warps(int D, bool f8) { return f8 ? 12 - soft_warps(D) : 2; }
__host__ __device__ constexpr int threads_of(int D, bool f8) { return 32 * (soft_warps(D) + load_warps(D, f8) + 1); }
// Stages of keys, and as many of values.
__host__ __device__ constexpr int stages_of(int D) { return D > 192 ? 2 : D > 64 ? 3 : 4; }
__host__ __device__ constexpr int smem_of(int D) {
    return blocks_of(D) * (int)(tc_q_tiles(D) * kBlockQ + 2 * stages_of(D) * kBlockK) + 1024;
}
static_assert(smem_of(128) <= 226 * 1024 && smem_of(192) <= 226 * 1024 && smem_of(256) <= 226 * 1024, "fits an SM");

// Place of 16 bytes (8 values from dim 8 chunk) of `row` in a swizzled tile.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, uint32_t block, uint32_t row, uint32_t chunk) {
    return tile + (chunk >> 3) * block + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(addr) : "memory");
    return w;
}

struct Shared {
    unsigned long long bars[32];
    uint2 place[4][kTileK];     // fp8: of a tile's tokens: vector count, and 0 past the end, 1 in the pool, 2 outside
    unsigned long long bad[8];  // 16-bit: tokens of a tile in pages outside the pool
    // the piece in hand, kept here so that no role carries what it does not use in registers
    PageTableSpace space;
    PageTable table;
    uint32_t seg;
    PagePiece piece;
    uint64_t x, x1;
    int seen, whole, none;
    uint32_t tmem;
    int gave_up, value_nan;
};

__device__ __forceinline__ void copy16(uint32_t smem, uint64_t gmem, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(on ? 16 : 0) : "memory");
}

template <int D, bool kF8, bool kHalf>
__global__ void __launch_bounds__(threads_of(D, kF8), 1) kv_pages_tc_kernel(const __grid_constant__ PageAttendArgs a) {
    constexpr int kSoftWarps = soft_warps(D), kLoadWarps = load_warps(D, kF8), kLoadThreads = 32 * kLoadWarps;
    constexpr bool kBf = !kF8 && !kHalf;              // type of the operands
    constexpr float kBits = kBf ? 0.0f : 7.0f;        // fp16 weights stand 2^7 higher
    constexpr int NB = blocks_of(D), NQ = tc_q_tiles(D), kStages = stages_of(D);
    constexpr uint32_t kBytesQ = NB * kBlockQ, kBytesK = NB * kBlockK;
    constexpr int RB = kF8 ? D : 2 * D;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");     // what comes next may count on all before this kernel
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t k_tile = base + NQ * kBytesQ, v_tile = k_tile + kStages * kBytesK;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t bars = smem_u32(sh.bars);
    const uint32_t k_full = bars, v_full = bars + 32, k_free = bars + 64, v_free = bars + 96,
                   s_full = bars + 128, p_full = bars + 160,      // [tile of rows][buffer]
                   o_last = bars + 192, q_full = bars + 208, o_full = bars + 216;
    const PageEngine &e = a.tc;
    if (tid == 0) sh.gave_up = 0;
    {
        unsigned long long x, x1;
        const PageTable t = table_and_share(a, e, blockIdx.x == 0, blockIdx.x, sh.space, &x, &x1);
        if (tid == 0) {
            sh.table = t;
            sh.x = x;
            sh.x1 = x1;
            sh.seg = x < x1 ? find_segment(t.tiles, seg_count(a, e), x) : 0;
        }
        if (warp == kSoftWarps + kLoadWarps) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    const int group = (int)a.group;

    for (bool first = true;; first = false) {
        bool found = false;
        while (tid == 0 && !found && sh.x < sh.x1) {
            sh.piece = piece_of(a, e, sh.table, &sh.seg, sh.x, sh.x1, blockIdx.x);
            sh.x += sh.piece.span;
            found = sh.piece.k0 < sh.piece.k1;
        }
        if (found) {
            const PageSeg &g = sh.piece.s;
            sh.seen = seen_tokens(a, e, g, sh.piece.rt);
            sh.whole = !g.prefix && sh.piece.k0 == 0 && sh.piece.k1 == sh.piece.n_tiles && (g.in < 0 || a.joined);
            if (!first)
                for (int i = 0; i < 28; ++i) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bars + 8 * i) : "memory");
            for (int i = 0; i < 4; ++i) {
                bar_init(k_full + 8 * i, kF8 ? kLoadThreads : 32);
                bar_init(v_full + 8 * i, kF8 ? kLoadThreads : 32);
                bar_init(k_free + 8 * i, 1);
                bar_init(v_free + 8 * i, 1);
                bar_init(s_full + 8 * i, 1);
                bar_init(p_full + 8 * i, kTileQ);
            }
            bar_init(o_last, 1);
            bar_init(o_last + 8, 1);
            bar_init(q_full, NQ * kTileQ);
            bar_init(o_full, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            sh.value_nan = 0;
            sh.none = 0;
        } else if (tid == 0) {
            sh.none = 1;
        }
        fence_before();
        __syncthreads();
        fence_after();
        if (sh.none) break;
        const uint32_t tmem = sh.tmem;

        const PagePiece &piece = sh.piece;
        const PageSeg &s = piece.s;
        const int head = piece.head, end = sh.seen;
        const int row0 = piece.rt * (int)e.row_tile;
        const int rows = (int)min((int64_t)e.row_tile, (int64_t)s.n * group - row0);
        // tiles of the prefix come first (all of them, or those in front of a request's own)
        const int k0 = piece.k0, pre = s.prefix ? s.len : s.before, pre_tiles = s.prefix ? piece.n_tiles : (int)tiles_of(e, pre);
        // tile t: its first token, and the end of the tokens that it may hold
        auto first_of = [&](int t) { return (k0 + t < pre_tiles ? k0 + t : k0 + t - pre_tiles) * kTileK; };
        auto end_of = [&](int t) { return k0 + t < pre_tiles ? pre : end; };
        const int q_tiles = rows > kTileQ ? 2 : 1;
        // after a wait that ran out the rest of the block's rows are NaN
        const int tiles = sh.gave_up != 0 ? 0 : piece.k1 - piece.k0;
        const int32_t *table = a.pages + (int64_t)s.index * a.pages_stride;
        const int32_t *pre_table = a.prefix_pages + (int64_t)(s.prefix ? (int)s.index : max(s.in, 0)) * a.prefix_stride;
        const int64_t head_off = (int64_t)head * a.pool.s_head;
        const int all_see = s.len - s.n + row0 / group + 1;    // own tokens that every row sees
        // rows see different tokens of tile t
        auto edge = [&](int t) { return k0 + t >= pre_tiles && min(first_of(t) + kTileK, end) > all_see; };

        if (warp < kSoftWarps) {
            // -------------------------------------------------------- softmax
            const int q = warp >> 2, row = (warp & 3) * 32 + lane;      // tile and row of it
            const int in = q * kTileQ + row;
            const bool on = in < rows;
            const int i = on ? (row0 + in) / group : 0, j = on ? row0 + in - i * group : 0;
            const int64_t tok = s.q0 + i;
            const int qh = head * group + j;
            // the scale's sign goes into the queries; a scale of 0 takes zeros
            const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u, keep = a.scale_log2 == 0.0f ? 0u : 0xffffffffu;
            float sc = fabsf(a.scale_log2);
            if (tiles > 0) {
                // A warp brings its 32 rows, neighbouring lanes a row's 16-byte pieces.
                constexpr int PQ = D / 8, AT = PQ <= 8 ? 4 : PQ <= 16 ? 2 : 1, kBatch = 8;
                const int sub = lane / PQ, ch = lane - sub * PQ;
                const long long mine_at = tok * a.q.s_tok + (long long)qh * a.q.s_head;
                const uint32_t live = __ballot_sync(0xffffffffu, on);
                int ex_mine = 127;
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += AT * kBatch) {
                    uint4 u[kBatch];
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int r = r0 + b * AT + sub;
                        const long long from = __shfl_sync(0xffffffffu, mine_at, r & 31);
                        u[b] = make_uint4(0, 0, 0, 0);
                        if (sub < AT && r < 32 && (live >> r & 1)) u[b] = *reinterpret_cast<const uint4 *>(a.q.data + from + ch * 16);
                    }
#pragma unroll
                    for (int b = 0; b < kBatch; ++b) {
                        const int r = r0 + b * AT + sub;
                        uint32_t w[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
                        if (kF8 && !kHalf) {
                            // a bf16 row times 2^(14 - exponent of its largest value); as it is with infinities and NaN
                            uint32_t top = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
                            if (sub < AT) top = __reduce_max_sync(PQ == 32 ? 0xffffffffu : ((1u << (PQ & 31)) - 1u) << (sub * PQ), top);
                            const uint32_t ex = max(top >> 7, 15u);
                            const float up = ex < 255 ? __uint_as_float((268u - ex) << 23) : 1.0f;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float2 f = unpack2<true>(w[k]);
                                w[k] = pack2<false>(f.x * up, f.y * up);
                            }
#pragma unroll
                            for (int k = 0; k < AT; ++k) {           // the row's own thread undoes it
                                const int e_k = __shfl_sync(0xffffffffu, (int)ex, k * PQ & 31);
                                if (lane == r0 + b * AT + k) ex_mine = e_k;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = (w[k] ^ flip) & keep;
                        if (sub < AT && r < 32)
                            sts16(tile_at(base + q * kBytesQ, kBlockQ, (warp & 3) * 32 + r, ch), make_uint4(w[0], w[1], w[2], w[3]));
                    }
                }
                if (kF8 && !kHalf) sc *= ex_mine < 255 ? __uint_as_float((uint32_t)(ex_mine - 14) << 23) : 1.0f;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(q_full);
            }
            sc = fmaxf(sc, 1.2e-38f);       // never 0, so that a masked score of -infinity stays one

            const int own_lim = on ? min(s.len - s.n + i, end - 1) : end - 1;     // sees own tokens 0..that
            const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
            const uint32_t o = mine + 256 + q * D;
            float m = kNoMax, zm = 0.0f, l = 0.0f;    // the maximum (base 2), as a score before its scale, and the sum
            const int my_tiles = q < q_tiles ? tiles : 0;
            for (int t = 0; t < my_tiles; ++t) {
                const uint32_t buf = t & 1, sp = mine + q * 128 + buf * 64;
                const uint32_t half_bar = 16 * q + 8 * buf;
                bar_wait(s_full + half_bar, (t >> 1) & 1, &sh.gave_up);
                __syncwarp();
                fence_after();
                uint32_t y[64];
                tmem_ld32(sp, y);
                tmem_ld32(sp + 32, y + 32);
                const int t0 = first_of(t), lim = k0 + t < pre_tiles ? pre - 1 : own_lim;
                const bool inside = __all_sync(0xffffffffu, t0 + kTileK - 1 <= lim);
                tmem_ld_wait();
                if (!kF8) {
                    const unsigned long long bad = *(volatile unsigned long long *)&sh.bad[t & 7];
                    if (bad != 0) {
#pragma unroll
                        for (int k = 0; k < 64; ++k)
                            if (bad >> k & 1) y[k] = kNanWord;
                    }
                }
                if (!inside) {
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        if (t0 + k > lim) y[k] = 0xff800000u;      // -infinity
                }
                if (!kF8 && edge(t)) {
                    // Rows see different tokens: a value that is not finite would reach all (0 x NaN).  It
                    // leaves the tile, and the rows that see it are put right at the end.
                    const uint32_t st = t % kStages;
                    bar_wait(v_full + 8 * st, (t / kStages) & 1, &sh.gave_up);
#pragma unroll 1
                    for (int i = row; i < (int)kBytesK / 16; i += kTileQ) {
                        if (D % 64 != 0 && i >= (NB - 1) * (int)kBlockK / 16 && ((i ^ i >> 3) & 7) >= D % 64 / 8) continue;   // holds nothing
                        const uint32_t at16 = v_tile + st * kBytesK + i * 16;
                        const uint4 u = lds16(at16);
                        const uint32_t f[4] = {not_finite<kF8, kBf>(u.x), not_finite<kF8, kBf>(u.y), not_finite<kF8, kBf>(u.z), not_finite<kF8, kBf>(u.w)};
                        if ((f[0] | f[1] | f[2] | f[3]) != 0) {
                            sts16(at16, make_uint4(u.x & ~f[0], u.y & ~f[1], u.z & ~f[2], u.w & ~f[3]));
                            sh.value_nan = 1;
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 64; k += 8)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        top[b] = fmaxf(fmaxf(top[b], __uint_as_float(y[k + 2 * b])), __uint_as_float(y[k + 2 * b + 1]));
                const float raw = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                const float most = raw == -INFINITY ? raw : raw * sc - kBits;
                // the maximum moves when it is passed by more than 2^8; then the sums
                // so far, O in tensor memory among them, are scaled down
                float k = 1.0f;
                if (m == kNoMax) {
                    if (most > -INFINITY) {
                        m = most;
                        zm = raw;
                    }
                } else if ((raw - zm) * sc > 8.0f) {
                    k = ex2((zm - raw) * sc);
                    m = most;
                    zm = raw;
                    l *= k;
                }
                __syncwarp();
                if (t > 0 && __any_sync(0xffffffffu, k != 1.0f)) {
                    // The sums of the tile before have to be done: the next scores were begun
                    // after them, and at the end there is a barrier for them.
                    const bool last = t + 1 == my_tiles;
                    bar_wait(last ? o_last + 8 * q : s_full + 16 * q + 8 * (buf ^ 1), last ? 0 : (t + 1) >> 1 & 1, &sh.gave_up);
                    __syncwarp();
                    fence_after();
#pragma unroll 1
                    for (int ch = 0; ch < D / 16; ++ch) {
                        uint32_t z[16];
                        tmem_ld16(o + ch * 16, z);
                        tmem_ld_wait();
#pragma unroll
                        for (int b = 0; b < 16; ++b) z[b] = __float_as_uint(__uint_as_float(z[b]) * k);
                        tmem_st16(o + ch * 16, z);
                    }
                    tmem_st_wait();
                }
                __syncwarp();
                // Differences are taken before the scale: z sc - m in one step (235 us where this takes 238, four chunks of
                // 500 behind 8,192) is off the largest score's own rounding, and from 2^24 on weights pass fp16.
                const float less = m == kNoMax ? 0.0f : -zm;
                const unsigned long long sc2 = pair(__float_as_uint(sc), __float_as_uint(sc));
                const unsigned long long less2 = pair(__float_as_uint(less), __float_as_uint(less));
                const unsigned long long bits2 = pair(__float_as_uint(kBits), __float_as_uint(kBits));
                unsigned long long sum[2] = {0, 0};
#pragma unroll(kF8 ? 1 : 2)
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[16], z[32];
                    if (kF8) {                  // read again: its warps have few registers
                        tmem_ld32(sp + 32 * h, z);
                        tmem_ld_wait();
                        if (!inside) {
#pragma unroll
                            for (int b = 0; b < 32; ++b)
                                if (t0 + 32 * h + b > lim) z[b] = 0xff800000u;
                        }
                    } else {
#pragma unroll
                        for (int b = 0; b < 32; ++b) z[b] = y[32 * (kF8 ? 0 : h) + b];
                    }
#pragma unroll
                    for (int b = 0; b < 32; b += 2) {
                        float2 u = unpair(fma2(add2(pair(z[b], z[b + 1]), less2), sc2, bits2));
                        u.x = ex2(u.x);
                        u.y = ex2(u.y);
                        sum[b >> 1 & 1] = add2(sum[b >> 1 & 1], pair(__float_as_uint(u.x), __float_as_uint(u.y)));
                        p[b / 2] = pack2<kBf>(u.x, u.y);
                    }
                    tmem_st16(sp + h * 16, p);      // over the scores
                }
                const float2 both = unpair(add2(sum[0], sum[1]));
                l += both.x + both.y;
                tmem_st_wait();
                fence_before();
                bar_arrive(p_full + half_bar);
            }
            if (q < q_tiles) {
                if (tiles > 0) bar_wait(o_full, 0, &sh.gave_up);
                __syncwarp();
                fence_after();
                const bool whole = sh.whole != 0, alive = sh.gave_up == 0, spoiled = alive && sh.value_nan != 0;
                const float inv = l != 0.0f ? a.v_scale / l : 0.0f;
                const uint64_t to_row = piece.slot * e.slot_rows + in;
                const long long out_at = tok * a.out.s_tok + (long long)qh * a.out.s_head;
                const uint32_t live = __ballot_sync(0xffffffffu, on);
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    uint32_t y[32];
                    if (tiles > 0) {
                        tmem_ld32(o + ch * 32, y);
                        tmem_ld_wait();
                    }
                    if (on) {
                        if (alive && l == 0.0f)
#pragma unroll
                            for (int b = 0; b < 32; ++b) y[b] = 0;
                        if (!alive)
#pragma unroll
                            for (int b = 0; b < 32; ++b) y[b] = kNanWord;
                        if (spoiled) {
                            // values that are not finite were left out of tiles that rows see in part
                            uint32_t bad = 0;
                            for (int t = max(max(0, k0 - pre_tiles) * kTileK, max(0, all_see) / kTileK * kTileK); t <= own_lim; ++t) {
                                bool wrong;
                                const int64_t off = token_offset(a.pool, table, (uint32_t)t, &wrong);
                                if (wrong) continue;
                                const uint64_t v = a.pool.base[1] + off + head_off + ch * (kF8 ? 32 : 64);
                                for (int b = 0; b < 32; ++b) {
                                    const uint32_t w = kF8 ? *reinterpret_cast<const uint8_t *>(v + b) : *reinterpret_cast<const uint16_t *>(v + 2 * b);
                                    if ((not_finite<kF8, kBf>(w) & (kF8 ? 0xffu : 0xffffu)) != 0) bad |= 1u << b;
                                }
                            }
#pragma unroll
                            for (int b = 0; b < 32; ++b)
                                if (bad >> b & 1) y[b] = kNanWord;
                        }
                    }
                    // through the queries' place in shared memory, so that neighbouring lanes write a row's pieces
                    const uint32_t mine_sm = base + (uint32_t)warp * 4096;
                    __syncwarp();
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t h[4];
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                h[b] = pack2<!kHalf>(__uint_as_float(y[8 * k + 2 * b]) * inv, __uint_as_float(y[8 * k + 2 * b + 1]) * inv);
                            sts16(mine_sm + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
                        }
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = 8 * k + (lane >> 2), c4 = lane & 3;
                            const uint4 w = lds16(mine_sm + r * 64 + ((c4 ^ (r >> 1 & 3)) << 4));
                            const long long to = __shfl_sync(0xffffffffu, out_at, r);
                            if (live >> r & 1) *reinterpret_cast<uint4 *>(a.out.data + to + ch * 64 + c4 * 16) = w;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            sts16(mine_sm + lane * 128 + ((k ^ (lane & 7)) << 4), make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]));
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = 4 * k + (lane >> 3), c8 = lane & 7;
                            const uint4 w = lds16(mine_sm + r * 128 + ((c8 ^ (r & 7)) << 4));
                            if (live >> r & 1) *reinterpret_cast<uint4 *>(e.part_o + (to_row - lane + r) * D + ch * 32 + c8 * 4) = w;
                        }
                    }
                    __syncwarp();
                }
                if (!alive) l = __uint_as_float(kNanWord);
                if (on && whole && a.lse != nullptr)
                    a.lse[tok * a.q_heads + qh] = l != 0.0f ? ((m == kNoMax ? 0.0f : m) + log2f(l)) * 0.693147180559945f : -INFINITY;
                if (on && !whole) *reinterpret_cast<float2 *>(e.part_ml + to_row * 2) = make_float2(m == kNoMax ? 0.0f : m, l);
            }
            fence_before();
        } else if (warp < kSoftWarps + kLoadWarps) {
            // ------------------------------------------------ keys and values
            // Tiles are brought in the order in which the products take them: K0, K1, V0, K2, V1 ...
            if constexpr (!kF8) {
                // The first warp brings keys, the second values, each a tile a step, PV pieces of 16 bytes a token.
                // A lane knows the places of two tokens and hands them round; pages are looked up three
                // tiles ahead.
                constexpr int PV = RB / 16, AT = PV <= 8 ? 4 : PV <= 16 ? 2 : 1;
                const int comp = warp - kSoftWarps, sub = lane / PV, ch = lane - sub * PV;
                const uint32_t full = comp ? v_full : k_full, freed = comp ? v_free : k_free, tile0 = comp ? v_tile : k_tile;
                const uint64_t from = (comp ? a.pool.base[1] : a.pool.base[0]) + head_off + ch * 16;
                auto pages_of = [&](int t, int32_t *pg) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int tk = first_of(t) + 32 * h + lane;
                        pg[h] = t < tiles && tk < end_of(t) ? (k0 + t < pre_tiles ? pre_table : table)[div_T(a.pool, (uint32_t)tk)] : 0;
                    }
                };
                int32_t pg[3][2];
                pages_of(0, pg[0]);
                pages_of(1, pg[1]);
                pages_of(2, pg[2]);
                const uint32_t to0 = (ch >> 3) * kBlockK + sub * 128, swizzle = (ch & 7) ^ sub;
#pragma unroll 1
                for (int t = 0; t < tiles; ++t) {
                        uint32_t where[2], good[2];
                        unsigned long long bads = 0;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int tk = first_of(t) + 32 * h + lane;
                            const bool in = tk < end_of(t), bad = in && (uint32_t)pg[0][h] >= a.pool.P;
                            where[h] = in && !bad ? vector_index(a.pool, (uint32_t)pg[0][h], (uint32_t)tk) : 0;
                            good[h] = __ballot_sync(0xffffffffu, in && !bad);
                            bads |= (unsigned long long)__ballot_sync(0xffffffffu, bad) << (32 * h);
                            pg[0][h] = pg[1][h];
                            pg[1][h] = pg[2][h];
                        }
                        pages_of(t + 3, pg[2]);
                        if (comp == 0 && lane == 0) {
                            *(volatile unsigned long long *)&sh.bad[t & 7] = bads;
                            if (bads != 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_PAGE);
                        }
                        const uint32_t st = t % kStages, tile = tile0 + st * kBytesK + to0;
                        bar_wait(freed + 8 * st, ((t / kStages) & 1) ^ 1, &sh.gave_up);
#pragma unroll
                        for (int it = 0; it < kTileK / AT; ++it) {
                            const int tk = (it * AT & 31) + sub;
                            const uint32_t w = __shfl_sync(0xffffffffu, where[it * AT >> 5], tk);
                            if (sub < AT)
                                copy16(tile + it * AT * 128 + ((swizzle ^ (it * AT & 7)) << 4), from + (uint64_t)w * (uint32_t)RB, good[it * AT >> 5] >> tk & 1);
                        }
                    // arrives when this lane's copies have landed
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full + 8 * st) : "memory");
                }
                asm volatile("cp.async.wait_all;" ::: "memory");     // nothing in flight behind a piece, even if a wait ran out
            } else {
            // fp8 goes through registers.  A thread takes 16 bytes of every kStep-th token of a tile;
            // the first 64 threads look up a token's place each, a tile before it is used, its page another before.
            constexpr int PV = RB / 16, PW = PV <= 4 ? 4 : PV <= 8 ? 8 : PV <= 16 ? 16 : 32, kStep = kLoadThreads / PW, NI = kTileK / kStep;
            static_assert(NI >= 1 && kTileK % kStep == 0, "tokens of a thread");
            const int d = tid - 32 * kSoftWarps, ch = d % PW, tk0 = d / PW;
            const bool idle = ch >= PV;
            auto page_of = [&](int t) {
                const int tk = first_of(t) + d;
                return d < kTileK && t < tiles && tk < end_of(t) ? (k0 + t < pre_tiles ? pre_table : table)[div_T(a.pool, (uint32_t)tk)] : 0;
            };
            auto place = [&](int t, int32_t page) {
                if (d >= kTileK) return;
                const int tk = first_of(t) + d;
                const bool in = t < tiles && tk < end_of(t), bad = in && (uint32_t)page >= a.pool.P;
                sh.place[t & 3][d] = make_uint2(in && !bad ? vector_index(a.pool, (uint32_t)page, (uint32_t)tk) : 0, bad ? 2 : in ? 1 : 0);
                if (bad && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_PAGE);
            };
            int32_t page = page_of(0), page1 = page_of(1);
            place(0, page);
            place(1, page1);
            page = page_of(2);
            const uint64_t from[2] = {a.pool.base[0] + head_off + ch * 16, a.pool.base[1] + head_off + ch * 16};
            auto load_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kLoadThreads) : "memory"); };
            load_sync();
                // the loads of a thread's next keys and values are under way while it converts these
                uint4 raw[2][NI];
                auto fetch = [&](int comp, int t) {
#pragma unroll
                    for (int it = 0; it < NI; ++it) {
                        raw[comp][it] = make_uint4(0, 0, 0, 0);
                        if (idle || t >= tiles) continue;
                        const uint2 w = sh.place[t & 3][tk0 + it * kStep];
                        if (comp == 0 && w.y == 2) raw[comp][it] = make_uint4(~0u, ~0u, ~0u, ~0u);      // NaN
                        if (w.y == 1) raw[comp][it] = *reinterpret_cast<const uint4 *>(from[comp] + (uint64_t)w.x * (uint32_t)RB);
                    }
                };
                auto store = [&](int comp, int t) {
                    const uint32_t st = t % kStages;
                    bar_wait((comp ? v_free : k_free) + 8 * st, ((t / kStages) & 1) ^ 1, &sh.gave_up);
                    const uint32_t tile = (comp ? v_tile : k_tile) + st * kBytesK;
                    const bool look = comp == 1 && edge(t);
                    if (!idle)
#pragma unroll
                        for (int it = 0; it < NI; ++it) {
                            uint32_t w[4] = {raw[comp][it].x, raw[comp][it].y, raw[comp][it].z, raw[comp][it].w};
                            if (look) {
#pragma unroll
                                for (int b = 0; b < 4; ++b) {
                                    const uint32_t f = not_finite<kF8, kBf>(w[b]);
                                    if (f != 0) sh.value_nan = 1;
                                    w[b] &= ~f;
                                }
                            }
                            sts16(tile_at(tile, kBlockK, tk0 + it * kStep, 2 * ch), make_uint4(e4m3x2(w[0]), e4m3x2(w[0] >> 16), e4m3x2(w[1]), e4m3x2(w[1] >> 16)));
                            sts16(tile_at(tile, kBlockK, tk0 + it * kStep, 2 * ch + 1), make_uint4(e4m3x2(w[2]), e4m3x2(w[2] >> 16), e4m3x2(w[3]), e4m3x2(w[3] >> 16)));
                        }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    bar_arrive((comp ? v_full : k_full) + 8 * st);
                };
                fetch(0, 0);
#pragma unroll 1
                for (int t = 0; t <= tiles && tiles > 0; ++t) {
                    if (t < tiles) {
                        store(0, t);
                        fetch(0, t + 1);
                    }
                    if (t > 0) store(1, t - 1);
                    fetch(1, t);
                    place(t + 2, page);
                    page = page_of(t + 3);
                    load_sync();
                }
            }
        } else {
            // -------------------------------------------------------- products
            constexpr uint32_t kScores = idesc(kTileK, false, kBf), kSums = idesc(D, true, kBf);
            const uint32_t one = elected();
            const int n = __shfl_sync(0xffffffffu, tiles, 0), nq = __shfl_sync(0xffffffffu, q_tiles, 0);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            auto wait = [&](uint32_t bar, uint32_t parity) {
                bar_wait(bar, parity, &sh.gave_up);
                __syncwarp();
            };
            auto scores = [&](int q, int t, uint32_t stage) {
                const uint64_t qd = desc(base + q * kBytesQ, 16, 1024), kd = desc(k_tile + stage * kBytesK, 16, 1024);
                const uint32_t to = tm + q * 128 + (t & 1) * 64;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss(to, qd + ((ks >> 2) * kBlockQ + (ks & 3) * 32) / 16, kd + ((ks >> 2) * kBlockK + (ks & 3) * 32) / 16,
                           kScores, ks != 0, one);
                commit(s_full + 16 * q + 8 * (t & 1), one);
            };
            auto sums = [&](int q, int t, uint32_t stage) {
                const uint64_t vd = desc(v_tile + stage * kBytesK, kBlockK, 1024);
                const uint32_t to = tm + 256 + q * D, from = tm + q * 128 + (t & 1) * 64;
#pragma unroll
                for (int ks = 0; ks < kTileK / 16; ++ks)
                    mma_ts(to, from + ks * 8, vd + (ks * 2048) / 16, kSums, t != 0 || ks != 0, one);
            };
            uint32_t ks = 0, kp = 0;        // stage of the keys asked for next, and its parity
            // copies are writes of the generic proxy, which the products' reads have to come after
            auto landed = [&]() {
                if (!kF8) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                fence_after();
            };
            auto keys = [&]() {
                wait(k_full + 8 * ks, kp);
                landed();
            };
            auto next_keys = [&]() {
                commit(k_free + 8 * ks, one);
                if (++ks == (uint32_t)kStages) {
                    ks = 0;
                    kp ^= 1;
                }
            };
            if (n > 0) {
                wait(q_full, 0);
                for (int t = 0; t < 2 && t < n; ++t) {      // both buffers of scores
                    keys();
                    for (int q = 0; q < nq; ++q) scores(q, t, ks);
                    next_keys();
                }
#pragma unroll 2
                for (int t = 0; t < n; ++t) {
                    const uint32_t vs = t % kStages;
                    wait(v_full + 8 * vs, (t / kStages) & 1);
                    landed();
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        if (q >= nq) break;
                        wait(p_full + 16 * q + 8 * (t & 1), (t >> 1) & 1);
                        fence_after();
                        sums(q, t, vs);
                        if (t + 2 < n) {
                            if (q == 0) keys();
                            scores(q, t + 2, ks);       // after the sums that read this buffer
                        } else if (t + 2 == n) {
                            commit(o_last + 8 * q, one);
                        }
                    }
                    if (t + 2 < n) next_keys();
                    commit(v_free + 8 * vs, one);
                }
                commit(o_full, one);
                int never = 0;
                bar_wait(o_full, 0, &never);        // nothing in flight when the barriers are made anew
            }
        }
        __syncwarp();
        fence_before();
        __syncthreads();
        fence_after();
    }
    if (sh.gave_up != 0 && tid == 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_GAVE_UP);
    if (warp == kSoftWarps + kLoadWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem));
}

typedef void(PagesTcFn)(PageAttendArgs);
struct VariantTc {
    uint32_t D;
    bool fp8, fp16;
    PagesTcFn *fn;
    int smem, threads;
};
template <int D, bool kF8, bool kHalf>
constexpr VariantTc variant_tc() {
    return VariantTc{(uint32_t)D, kF8, kHalf, kv_pages_tc_kernel<D, kF8, kHalf>, smem_of(D), threads_of(D, kF8)};
}
#define KVB_PAGES_TC(D) \
    variant_tc<D, false, false>(), variant_tc<D, false, true>(), variant_tc<D, true, false>(), variant_tc<D, true, true>()
const VariantTc kVariantsTc[] = {KVB_PAGES_TC(64), KVB_PAGES_TC(96), KVB_PAGES_TC(128), KVB_PAGES_TC(192), KVB_PAGES_TC(256)};

}  // namespace

cudaError_t launch_pages_tc(const PageAttendArgs &a, uint32_t D, bool fp8, bool fp16, bool pdl, cudaStream_t stream) {
    for (const VariantTc &v : kVariantsTc) {
        if (v.D != D || v.fp8 != fp8 || v.fp16 != fp16) continue;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(a.tc.workers);
        cfg.blockDim = dim3((unsigned)v.threads);
        cfg.dynamicSmemBytes = (size_t)v.smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = pdl ? 1 : 0;
        return cudaLaunchKernelEx(&cfg, v.fn, a);
    }
    return cudaErrorInvalidValue;
}

cudaError_t preload_pages_tc_kernels() {
    cudaFuncAttributes at;
    for (const VariantTc &v : kVariantsTc) {
        cudaError_t e = cudaFuncGetAttributes(&at, (const void *)v.fn);
        if (e == cudaSuccess) e = cudaFuncSetAttribute((const void *)v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute((const void *)v.fn, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kvb
