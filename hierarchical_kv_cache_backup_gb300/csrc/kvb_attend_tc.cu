// kvb_attend_tc.cu -- attention of many new tokens (a prompt chunk) over one
// layer of a 4-bit pool, on the fifth-generation tensor cores.
//
// A block takes 256 query rows (new tokens x the group of one KV head) as two
// tiles of 128, and walks the cached tokens 64 at a time.  Warps have roles:
//   8 warps  unpack keys and values to fp16 in shared memory (swizzled tiles)
//   1 warp   issues tcgen05.mma: scores S = Q K^T and sums O += P V
//   4 + 4    softmax of the two tiles, one row a thread: scores come from tensor
//            memory, probabilities go back there as fp16, the A operand of P V
// Tensor memory holds two buffers of 64 scores a row for each tile (P overwrites
// S) and O0, O1 (D columns each).  With two buffers the scores of the next
// cached tokens are there when a softmax warp is done with the ones before: with one
// buffer of 128, each softmax waited for its own products, 370 us for 2 x 1,000
// new tokens over 8,192 cached ones.
//
// Range.  fp16 operands stay in range by exact powers of two: steps of the keys and
// values of each group of 32 are brought to 2^12 at most by the largest step of the
// request (a kernel that reads the scale words finds it), queries take the key groups'
// powers in exchange, each query row is brought to 2^14..2^15, and probabilities to
// 2^7..2^15 at a row's largest.  That keeps every step's bits where all steps of
// a group are within 2^16 of each other, over all that the request's rows see; a request
// and head where they are not (its small steps would lose bits to a large one that a row may not
// see, or gives no weight) goes to the kernel for few rows, which scales by rows.
// What is rounded: a value once (2^-11; not for fp16 outputs), a probability once
// (2^-11).  Keys are two fp16 parts each, which their products with the queries take
// in turn, for fp16 outputs and where the caller wants the logarithms of the sums:
// with one part (2^-11) a logarithm of few terms is off by 1e-5 of itself, which
// float32 has to show and bf16 outputs do not.  Without them bf16 outputs take one
// part: 2 x 1,000 new tokens over 8,192 cached ones, 282 us with two parts and 229
// with one.
//
// Bound: the products.  A tcgen05.mma of 128 x 64 x 16 with both operands in
// shared memory takes 48 cycles and more where its arithmetic takes 32, since it
// reads 6 KB; a tile of 64 cached tokens has 32 of them and 8 of 128 x 128 x 16 for
// the sums (64 cycles), about 2,050 cycles; traces of one block show 2,400-2,900 a
// tile, the product warp never waiting for the softmax warps.
#include "kvb_tc.h"
#include "kvb_vec.h"
#include "kvb_vec_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kvb {

using namespace tc;

namespace {

constexpr int kTileQ = 128, kTileK = 64;
constexpr int kRowsTc = 2 * kTileQ;
constexpr int kSoftWarps = 8, kUnpackWarps = 8, kUnpackThreads = 32 * kUnpackWarps;
constexpr int kThreadsTc = 32 * (kSoftWarps + kUnpackWarps + 1);
constexpr float kNoMaxTc = -3.0e38f;
// 64 fp16 (128 bytes, swizzled) of every row of a tile
constexpr uint32_t kBlockQ = kTileQ * 128, kBlockK = kTileK * 128;

__host__ __device__ constexpr int blocks_of(int D) { return (D + 63) / 64; }
// Stages of K (of one part or two) and of V.  Two of K: with three the unpacking
// warps run further ahead and the products more slowly (two parts 287 us, 282 with two
// stages; one part 230 and 229); V needs three.
constexpr int kStagesK = 2, kStagesV = 3;
static_assert(kStagesK <= 4 && kStagesV <= 4, "four barriers of each kind");
// fp16 parts of a value: two where the output is fp16, so that only the
// probabilities are rounded before it (300 new tokens over 8,192: error against 64 bits 1.4
// times that of a float32 result rounded once, 1.7 with one part; a bf16 output does not
// show it).
__host__ __device__ constexpr int value_parts(bool half) { return half ? 2 : 1; }
// and of a key: two where the logarithm is wanted or the output is fp16 (300 new tokens over
// 8,192, error against 64 bits 2.4 times that of a float32 result with keys in one part; so
// fp16 outputs are the same bits with and without logarithms).
constexpr int key_parts(bool half, bool lse) { return half || lse ? 2 : 1; }
// Q0, Q1, the stages, and 1 KiB to align
__host__ __device__ constexpr int smem_tc(int D, bool half, int parts) {
    return blocks_of(D) * (int)(2 * kBlockQ + (parts * kStagesK + value_parts(half) * kStagesV) * kBlockK) + 1024;
}

// Place of 16 bytes (8 values from dim 8 chunk) of `row` in a swizzled tile.  The
// values of a chunk stand in the order 0 4 1 5 2 6 3 7 in every tile, as the
// codes unpack: keys and queries agree, and the sums' columns are put right when
// they are read.
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, uint32_t block, uint32_t row, uint32_t chunk) {
    return tile + (chunk >> 3) * block + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// The exponent of a largest step as a power of two (and its inverse); 1 for none.
__device__ __forceinline__ float pow2_of(uint32_t most) {
    return most == 0 ? 1.0f : __uint_as_float(most & 0x7f800000u);
}

// Bits that steps of a group may differ by, and the power of two that the largest is near.
constexpr uint32_t kStepBits = 15;
constexpr float kStepUp = 2048.0f;
// A row's largest probability is taken as 2^7, and may pass that by 2^8 before the maximum moves.
constexpr float kProbBits = 7.0f, kProbDown = 0.0078125f;

struct SharedTc {
    unsigned long long bars[32];
    uint32_t tmem;
    int gave_up, value_nan;
    uint32_t most[2][4];     // largest steps of keys and values, a group each (as bits)
    uint32_t least[2][4];    // and the least that are not 0
};

// The largest and the least steps but 0 (as float bits) of the keys and values that
// kStepTokens tokens of a request hold for one head: [request][part][head][2][4 and 4].
// Together the parts cover what all rows of the request see.

template <int D>
__global__ void __launch_bounds__(256) kv_attend_steps_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int NG = D / 32;
    __shared__ uint32_t all[kStepWords];     // as in a.steps
    asm volatile("griddepcontrol.launch_dependents;");
    const int head = blockIdx.x, part = blockIdx.y, r = blockIdx.z, tid = threadIdx.x;
    if (tid < (int)kStepWords) all[tid] = tid & 4 ? 0xffffffffu : 0u;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    bool bad;
    const Span s = row_span(a.q_start[r], a.q_start[r + 1], a.lens[r], (int)a.tokens, (int)a.max_q,
                            (int)a.max_len, (int)a.group, (int)a.window, 0, (int)(a.max_q * a.group), &bad);
    const int32_t *table = a.pages + (int64_t)r * a.pages_stride;
    const int64_t head_off = (int64_t)head * a.pool.s_head;
    const int t0 = s.lo + part * (int)kStepTokens, t1 = min(s.hi, t0 + (int)kStepTokens);
    uint32_t most[2][NG], least[2][NG];
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i) {
        most[i / NG][i % NG] = 0;
        least[i / NG][i % NG] = 0xffffffffu;
    }
#pragma unroll 4
    for (int t = t0 + tid; t < t1; t += 256) {
        bool wrong;
        const int64_t off = token_offset(a.pool, table, (uint32_t)t, &wrong);
        if (wrong) continue;
#pragma unroll
        for (int comp = 0; comp < 2; ++comp) {
            // four scale words, or fewer and the zeros behind them
            const uint4 u = *reinterpret_cast<const uint4 *>(a.pool.base[comp] + off + head_off + D / 2);
            const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                const uint32_t w = v[gr] & ~15u;
                if (w < 0x7f800000u) most[comp][gr] = max(most[comp][gr], w);
                if (w != 0) least[comp][gr] = min(least[comp][gr], w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i) {
        const uint32_t w = __reduce_max_sync(0xffffffffu, most[i / NG][i % NG]);
        const uint32_t u = __reduce_min_sync(0xffffffffu, least[i / NG][i % NG]);
        if ((tid & 31) == 0) {
            atomicMax(&all[i / NG * 8 + i % NG], w);
            atomicMin(&all[i / NG * 8 + 4 + i % NG], u);
        }
    }
    __syncthreads();
    if (tid < (int)kStepWords)
        a.steps[(((int64_t)r * a.step_parts + part) * a.pool.H + head) * kStepWords + tid] = all[tid];
}

template <int D, bool kHalf, int kParts>
__global__ void __launch_bounds__(kThreadsTc, 1) kv_attend_tc_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int NG = D / 32, NB = blocks_of(D);
    constexpr int kPartsV = value_parts(kHalf);
    constexpr uint32_t kBytesQ = NB * kBlockQ, kBytesK = NB * kBlockK;
    extern __shared__ unsigned char smem_raw[];
    __shared__ SharedTc sh;
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t k_tile = base + 2 * kBytesQ, v_tile = k_tile + kParts * kStagesK * kBytesK;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t bars = smem_u32(sh.bars);
    const uint32_t k_full = bars, v_full = bars + 32, k_free = bars + 64, v_free = bars + 96,
                   s_full = bars + 128, p_full = bars + 160,      // [tile of rows][buffer]
                   o_last = bars + 192, q_full = bars + 208, o_full = bars + 216;

    const int H = (int)a.pool.H, group = (int)a.group;
    // Blocks of whole units first, then those of the units that are cut.
    const bool cut = blockIdx.x >= a.whole_units;
    const uint32_t unit = cut ? a.whole_units + (blockIdx.x - a.whole_units) / a.chunks : blockIdx.x;
    const int ci = cut ? (int)((blockIdx.x - a.whole_units) % a.chunks) : 0;
    const int chunk = cut ? (int)a.chunk : 0x7fffffff;
    const int head = (int)(unit % H);
    // tiles of the last rows see most: they go first
    const int rt = (int)a.row_tiles - 1 - (int)(unit / H % a.row_tiles);
    const int r = (int)(unit / H / a.row_tiles);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    bool bad;
    const Span s = row_span(a.q_start[r], a.q_start[r + 1], a.lens[r], (int)a.tokens, (int)a.max_q,
                            (int)a.max_len, group, (int)a.window, rt, kRowsTc, &bad);
    if (bad && a.status != nullptr && tid == 0 && head == 0) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
    const int row0 = rt * kRowsTc, rows = min(kRowsTc, s.n * group - row0);
    if (rows <= 0) return;
    const int c0 = s.lo + ci * (cut ? chunk : 0), c1 = cut ? min(s.hi, c0 + chunk) : s.hi;
    if (c0 >= c1 && ci > 0) return;
    const bool whole = s.hi - s.lo <= chunk;
    const int q_tiles = rows > kTileQ ? 2 : 1;
    const int tiles = c1 > c0 ? (c1 - c0 + kTileK - 1) / kTileK : 0;
    const int32_t *table = a.pages + (int64_t)r * a.pages_stride;
    const int64_t head_off = (int64_t)head * a.pool.s_head;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            bar_init(k_full + 8 * i, 32 * kUnpackWarps);
            bar_init(v_full + 8 * i, 32 * kUnpackWarps);
            bar_init(k_free + 8 * i, 1);
            bar_init(v_free + 8 * i, 1);
            bar_init(s_full + 8 * i, 1);
            bar_init(p_full + 8 * i, kTileQ);
        }
        bar_init(o_last, 1);
        bar_init(o_last + 8, 1);
        bar_init(q_full, 2 * kTileQ);
        bar_init(o_full, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.gave_up = 0;
        sh.value_nan = 0;
        for (int i = 0; i < 8; ++i) {
            sh.most[i / 4][i % 4] = 0;
            sh.least[i / 4][i % 4] = 0xffffffffu;
        }
    }
    if (warp == kSoftWarps + kUnpackWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;

    // the largest and least step of each group of the request and head
    for (int k = tid; k < (int)(a.step_parts * kStepWords); k += kThreadsTc) {
        const uint32_t w = a.steps[(((int64_t)r * a.step_parts + k / kStepWords) * H + head) * kStepWords + k % kStepWords];
        if ((k & 4) == 0) atomicMax(&sh.most[k >> 3 & 1][k & 3], w);
        else atomicMin(&sh.least[k >> 3 & 1][k & 3], w);
    }
    __syncthreads();
    bool uneven = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w = sh.most[i / 4][i % 4];
        uneven |= w != 0 && (w >> 23) - (sh.least[i / 4][i % 4] >> 23) > kStepBits;
    }
    if (rt == 0 && ci == 0 && tid == 0) a.uneven[(int64_t)r * H + head] = uneven;
    if (uneven) {
        if (warp == kSoftWarps + kUnpackWarps)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
        return;
    }

    if (warp < kSoftWarps) {
        // ------------------------------------------------------------ softmax
        const int q = warp >> 2, row = (warp & 3) * 32 + lane;      // tile and row of it
        const int at = row0 + q * kTileQ + row;                     // row of the request
        const bool on = q * kTileQ + row < rows;
        const int i = on ? at / group : 0, j = on ? at - i * group : 0;
        const int64_t tok = s.q0 + i;
        const int qh = head * group + j;
        // the scale's sign goes into the queries (0 for a scale of 0)
        const float sign = a.scale_log2 < 0.0f ? -1.0f : a.scale_log2 == 0.0f ? 0.0f : 1.0f;
        // this thread's query row, scaled, to shared memory
        float sc;
        {
            const uint64_t src = a.q.data + tok * a.q.s_tok + (int64_t)qh * a.q.s_head;
            // read twice, a group's four runs of 16 bytes under way at once
            auto read = [&](int gr, uint4 *u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = make_uint4(0, 0, 0, 0);
                    if (on) u[i] = *reinterpret_cast<const uint4 *>(src + gr * 64 + i * 16);
                }
            };
            auto value = [&](uint32_t w, int hi) {
                if (kHalf) return __half2float(__ushort_as_half((unsigned short)(hi ? w >> 16 : w & 0xffffu)));
                return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
            };
            float top = 0.0f;
#pragma unroll 2
            for (int gr = 0; gr < NG; ++gr) {
                const float f = pow2_of(sh.most[0][gr]);
                uint4 u[4];
                read(gr, u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(value(w[e / 2], e & 1)) * f);
                }
            }
            if (sign == 0.0f) top = 0.0f;
            // 2^(14 - exponent of top), and its inverse; 1 for infinities and NaN
            const uint32_t ex = max(__float_as_uint(top) >> 23, 15u);
            const float up = ex < 255 ? __uint_as_float((268u - ex) << 23) : 1.0f;
            // never 0, so that a masked score of -infinity stays one
            sc = fmaxf((ex < 255 ? __uint_as_float((ex - 14u) << 23) : 1.0f) * (fabsf(a.scale_log2) / kStepUp), 1.2e-38f);
#pragma unroll 2
            for (int gr = 0; gr < NG; ++gr) {
                const float f = pow2_of(sh.most[0][gr]) * sign;
                uint4 u[4];
                read(gr, u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        h[e] = h2_bits(value(w[e / 2], e & 1) * f * up, value(w[2 + e / 2], e & 1) * f * up);
                    sts16(tile_at(base + q * kBytesQ, kBlockQ, row, gr * 4 + i), make_uint4(h[0], h[1], h[2], h[3]));
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        bar_arrive(q_full);

        const int pos = s.len - s.n + i;
        const int lim = on ? min(pos, c1 - 1) : -1;                 // sees tokens low..lim
        const int low = a.window ? max(0, pos - (int)a.window + 1) : 0;
        const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
        const uint32_t o = mine + 256 + q * D;
        float m = kNoMaxTc, l = 0.0f;
        const int my_tiles = q < q_tiles ? tiles : 0;
        for (int t = 0; t < my_tiles; ++t) {
            const uint32_t buf = t & 1, sp = mine + q * 128 + buf * 64;
            const uint32_t half_bar = 16 * q + 8 * buf;
            bar_wait(s_full + half_bar, (t >> 1) & 1, &sh.gave_up);
            __syncwarp();
            fence_after();
            uint32_t x[64];
            tmem_ld32(sp, x);
            tmem_ld32(sp + 32, x + 32);
            const int t0 = c0 + t * kTileK;
            const bool inside = __all_sync(0xffffffffu, t0 >= low && t0 + kTileK - 1 <= lim);
            tmem_ld_wait();
            if (!inside) {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (t0 + e < low || t0 + e > lim) x[e] = 0xff800000u;      // -infinity
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 64; e += 8)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    top[b] = fmaxf(fmaxf(top[b], __uint_as_float(x[e + 2 * b])), __uint_as_float(x[e + 2 * b + 1]));
            float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            most = most == -INFINITY ? most : most * sc;
            // the maximum moves when it is passed by more than 2^8; then the sums
            // so far, O in tensor memory among them, are scaled down
            float k = 1.0f;
            most -= kProbBits;
            if (m == kNoMaxTc) {
                if (most > -INFINITY) m = most;
            } else if (most > m + 8.0f) {
                k = ex2(m - most);
                m = most;
                l *= k;
            }
            __syncwarp();
            if (t > 0 && __any_sync(0xffffffffu, k != 1.0f)) {
                // The sums of the tile before have to be done: the next scores were begun
                // after them, and at the end there is a barrier for them.
                const bool last = t + 1 == my_tiles;
                bar_wait(last ? o_last + 8 * q : s_full + 16 * q + 8 * (buf ^ 1), last ? 0 : (t + 1) >> 1 & 1,
                         &sh.gave_up);
                __syncwarp();
                fence_after();
#pragma unroll 1
                for (int ch = 0; ch < D / 16; ++ch) {
                    uint32_t y[16];
                    tmem_ld16(o + ch * 16, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * k);
                    tmem_st16(o + ch * 16, y);
                }
                tmem_st_wait();
            }
            __syncwarp();
            const float less = m == kNoMaxTc ? 0.0f : -m;
            const unsigned long long sc2 = pair(__float_as_uint(sc), __float_as_uint(sc));
            const unsigned long long less2 = pair(__float_as_uint(less), __float_as_uint(less));
            unsigned long long sum[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float2 u = unpair(fma2(pair(x[32 * h + e], x[32 * h + e + 1]), sc2, less2));
                    u.x = ex2(u.x);
                    u.y = ex2(u.y);
                    sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], pair(__float_as_uint(u.x), __float_as_uint(u.y)));
                    p[e / 2] = h2_bits(u.x, u.y);
                }
                tmem_st16(sp + h * 16, p);      // over the scores
            }
            const float2 both = unpair(add2(sum[0], sum[1]));
            l += both.x + both.y;
            tmem_st_wait();
            fence_before();
            bar_arrive(p_full + half_bar);
        }
        if (tiles > 0) bar_wait(o_full, 0, &sh.gave_up);
        __syncwarp();
        fence_after();
        const bool alive = sh.gave_up == 0;
        // a value that is not finite: groups of the row's tokens that hold one
        uint32_t nan_groups = alive ? 0u : 0xffu;
        if (alive && sh.value_nan != 0)
            for (int t = max(c0, low); t <= lim; ++t) {
                bool wrong;
                const int64_t off = token_offset(a.pool, table, (uint32_t)t, &wrong);
                if (wrong) continue;
                for (int gr = 0; gr < NG; ++gr)
                    if (*reinterpret_cast<const uint32_t *>(a.pool.base[1] + off + head_off + D / 2 + gr * 4) >=
                        0x7f800000u)
                        nan_groups |= 1u << gr;
            }
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        const int64_t part = ((int64_t)ci * a.tokens + tok) * a.q_heads + qh;
#pragma unroll 1
        for (int ch = 0; ch < NG; ++ch) {
            uint32_t x[32];
            if (tiles > 0) {
                tmem_ld32(o + ch * 32, x);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0;
            }
            if (on) {
                const float f = pow2_of(sh.most[1][ch]) / kStepUp;
                if (nan_groups >> ch & 1)
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = kNanWord;
                if (l == 0.0f && alive)
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = 0;
                if (whole) {
                    const uint64_t dst = a.out.data + tok * a.out.s_tok + (int64_t)qh * a.out.s_head + ch * 64;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            // dims 2 b and 2 b + 1 of the eight
                            const float u = __uint_as_float(x[e + (b < 2 ? 4 * b : 4 * b - 7)]) * inv * f;
                            const float v = __uint_as_float(x[e + (b < 2 ? 4 * b + 2 : 4 * b - 5)]) * inv * f;
                            if (kHalf) {
                                h[b] = h2_bits(u, v);
                            } else {
                                __nv_bfloat162 w = __floats2bfloat162_rn(u, v);
                                h[b] = *reinterpret_cast<uint32_t *>(&w);
                            }
                        }
                        *reinterpret_cast<uint4 *>(dst + e * 2) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                } else {
                    float *dst = a.part_o + part * D + ch * 32;
                    const float fp = f * kProbDown;
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                    {
                        const int k = e / 8 * 8 + (e & 4 ? 1 : 0);
                        *reinterpret_cast<float4 *>(dst + e) =
                            make_float4(__uint_as_float(x[k]) * fp, __uint_as_float(x[k + 2]) * fp,
                                        __uint_as_float(x[k + 4]) * fp, __uint_as_float(x[k + 6]) * fp);
                    }
                }
            }
            __syncwarp();
        }
        if (on && whole && a.lse != nullptr)
            a.lse[tok * a.q_heads + qh] =
                !alive ? __uint_as_float(kNanWord)
                       : l != 0.0f ? ((m == kNoMaxTc ? 0.0f : m) + log2f(l)) * 0.693147180559945f : -INFINITY;
        if (on && !whole)
            *reinterpret_cast<float2 *>(a.part_ml + part * 2) =
                make_float2(m == kNoMaxTc ? 0.0f : m + kProbBits, alive ? l * kProbDown : __uint_as_float(kNanWord));
        fence_before();
    } else if (warp < kSoftWarps + kUnpackWarps) {
        // ------------------------------------------------- unpack to fp16 tiles
        // A thread takes one group of 32 values of every kUnpackThreads / NP-th token
        // of a tile.  As soon as a group is unpacked, the load of its successor in
        // the next tile starts.
        constexpr int NP = NG == 3 ? 4 : NG, kStep = kUnpackThreads / NP;
        constexpr int NI = kTileK > kStep ? kTileK / kStep : 1;
        const int d = tid - 32 * kSoftWarps;
        const int gr = d % NP, tk0 = d / NP;                 // group; tokens tk0 + it * kStep
        const bool idle = gr >= NG || tk0 >= kTileK;
        const float f[2] = {kStepUp / pow2_of(sh.most[0][idle ? 0 : gr]),
                            kStepUp / pow2_of(sh.most[1][idle ? 0 : gr])};
        // Lanes of groups 2 and 3 go through their words two apart from those of 0 and
        // 1, so that 8 lanes' stores meet 8 different places of 16 bytes.
        const bool apart = (gr >> 1 & 1) != 0;
        uint32_t to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = tile_at(0, kBlockK, tk0, gr * 4 + (i ^ (apart ? 2 : 0)));
        int64_t off[NI];
        uint4 code[2][NI];
        uint32_t word[2][NI];
        bool outside = false;
        // A place is looked up in two steps, the page one tile before the offset and
        // that one tile before the loads that use it, so that nothing waits for the
        // page table.
        int32_t page[NI];
        auto token = [&](int it, int t) { return c0 + t * kTileK + tk0 + it * kStep; };
        auto look_up = [&](int it, int t) {
            const int tk = token(it, t);
            page[it] = !idle && tk < c1 ? table[div_T(a.pool, (uint32_t)tk)] : 0;
        };
        auto find = [&](int it, int t) {
            const int tk = token(it, t);
            off[it] = -1;                 // past the end: zeros
            if (!idle && tk < c1) {
                bool wrong;
                off[it] = page_offset(a.pool, (uint32_t)page[it], (uint32_t)tk, &wrong) + head_off;
                if (wrong) off[it] = -2;  // keys NaN
                outside |= wrong;
            }
        };
        auto fetch = [&](int it, int comp) {
            code[comp][it] = make_uint4(0, 0, 0, 0);
            word[comp][it] = off[it] == -2 && comp == 0 ? kNanWord : 0u;
            if (off[it] >= 0) {
                const uint64_t at = a.pool.base[comp] + off[it];
                code[comp][it] = *reinterpret_cast<const uint4 *>(at + gr * 16);
                word[comp][it] = *reinterpret_cast<const uint32_t *>(at + D / 2 + gr * 4);
            }
        };
#pragma unroll
        for (int it = 0; it < NI; ++it) {
            look_up(it, 0);
            find(it, 0);
            fetch(it, 0);
            fetch(it, 1);
            look_up(it, 1);
            find(it, 1);
            look_up(it, 2);
        }
        const __half2 k16 = __half2half2(__ushort_as_half(0x2c00));     // 1/16
        uint32_t ks = 0, kp = 1;              // stage of the keys, and its parity
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
#pragma unroll
            for (int comp = 0; comp < 2; ++comp) {
            const uint32_t vs = t % kStagesV;
            bar_wait(comp ? v_free + 8 * vs : k_free + 8 * ks, comp ? ((t / kStagesV) & 1) ^ 1 : kp, &sh.gave_up);
            const uint32_t tile = comp ? v_tile + vs * (kPartsV * kBytesK) : k_tile + ks * (kParts * kBytesK);
#pragma unroll
            for (int it = 0; it < NI; ++it) {
                uint32_t w = word[comp][it];
                const uint4 u = code[comp][it];
                fetch(it, comp);          // of tile t + 1
                if (comp == 1) {
                    find(it, t + 2);
                    look_up(it, t + 3);
                }
                if (comp == 1 && w >= 0x7f800000u) {
                    w = 0;                // kept out of the products; the softmax warps see to it
                    sh.value_nan = 1;
                }
                // The step as two fp16 parts; a product is rounded once, by the sum with the
                // first part's.  Tiles in two parts: the first has 7 bits, so that its products
                // with code - z are exact, and the second's products go to a tile of their
                // own; products with either err by 2^-19.
                const float step = q4_step(w) * (comp ? f[1] : f[0]);
                const bool split = (comp ? kPartsV : kParts) == 2;
                const float hi = split ? __uint_as_float((__float_as_uint(step) + 0x10000u) & 0xfffe0000u)
                                       : __half2float(__float2half_rn(step));
                const __half2 s1 = __float2half2_rn(hi), s0 = __float2half2_rn(step - hi);
                const uint32_t zz = (w & 15u) * 0x00010001u;
                uint32_t za = zz | 0x64006400u, zb = (zz << 4) | 0xd400d400u;    // 1024 + z, -(64 + z)
                const __half2 z1 = *reinterpret_cast<__half2 *>(&za), z16 = *reinterpret_cast<__half2 *>(&zb);
                const uint32_t cw[4] = {apart ? u.z : u.x, apart ? u.w : u.y, apart ? u.x : u.z,
                                        apart ? u.y : u.w};
                if (!idle)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t v = cw[i] >> 8;
                        uint32_t y[4] = {(cw[i] & 0x000f000fu) | 0x64006400u, (cw[i] & 0x00f000f0u) | 0x64006400u,
                                         (v & 0x000f000fu) | 0x64006400u, (v & 0x00f000f0u) | 0x64006400u};
                        uint32_t y0[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            __half2 x = *reinterpret_cast<__half2 *>(&y[e]);
                            x = e & 1 ? __hfma2(x, k16, z16) : __hsub2(x, z1);    // code - z, exact
                            __half2 low = __hmul2(x, s0), high = split ? __hmul2(x, s1) : __hfma2(x, s1, low);
                            y[e] = *reinterpret_cast<uint32_t *>(&high);
                            y0[e] = *reinterpret_cast<uint32_t *>(&low);
                        }
                        sts16(tile + to[i] + it * kStep * 128, make_uint4(y[0], y[1], y[2], y[3]));
                        if (split)
                            sts16(tile + kBytesK + to[i] + it * kStep * 128, make_uint4(y0[0], y0[1], y0[2], y0[3]));
                    }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            bar_arrive(comp ? v_full + 8 * vs : k_full + 8 * ks);
            }
            if (++ks == kStagesK) {
                ks = 0;
                kp ^= 1;
            }
        }
        if (outside && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_PAGE);
    } else {
        // ------------------------------------------------------------ products
        constexpr uint32_t kScores = idesc(kTileK, false), kSums = idesc(D, true);
        const uint32_t one = elected();
        const int n = __shfl_sync(0xffffffffu, tiles, 0), nq = __shfl_sync(0xffffffffu, q_tiles, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        auto wait = [&](uint32_t bar, uint32_t parity) {
            bar_wait(bar, parity, &sh.gave_up);
            __syncwarp();
        };
        auto scores = [&](int q, int t, uint32_t stage) {
            const uint64_t qd = desc(base + q * kBytesQ, 16, 1024), kd = desc(k_tile + stage * (kParts * kBytesK), 16, 1024);
            const uint32_t to = tm + q * 128 + (t & 1) * 64;
#pragma unroll
            for (int part = 0; part < kParts; ++part)     // of the keys' steps
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss(to, qd + ((ks >> 2) * kBlockQ + (ks & 3) * 32) / 16,
                           kd + (part * kBytesK + (ks >> 2) * kBlockK + (ks & 3) * 32) / 16, kScores,
                           part + ks != 0, one);
            commit(s_full + 16 * q + 8 * (t & 1), one);
        };
        auto sums = [&](int q, int t, uint32_t stage) {
            const uint64_t vd = desc(v_tile + stage * (kPartsV * kBytesK), kBlockK, 1024);
            const uint32_t to = tm + 256 + q * D, from = tm + q * 128 + (t & 1) * 64;
#pragma unroll
            for (int part = 0; part < kPartsV; ++part)
#pragma unroll
                for (int ks = 0; ks < kTileK / 16; ++ks)
                    mma_ts(to, from + ks * 8, vd + (part * kBytesK + ks * 2048) / 16, kSums,
                           t != 0 || part + ks != 0, one);
        };
        uint32_t ks = 0, kp = 0;        // stage of the keys asked for next, and its parity
        auto keys = [&]() {
            wait(k_full + 8 * ks, kp);
            fence_after();
        };
        auto next_keys = [&]() {
            commit(k_free + 8 * ks, one);
            if (++ks == kStagesK) {
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
            // Straight code: a jump back costs this warp an instruction fetch of some 350
            // cycles, since the other warps' code goes through the same caches; four tiles
            // at a time gain nothing more (235, 229 and 230 us for 1, 2 and 4).
#pragma unroll 2
            for (int t = 0; t < n; ++t) {
                // The unpacking warps give the values of a tile before the keys of the next, so
                // keys that have come vouch for them; the last tile has no next.
                const uint32_t vs = t % kStagesV;
                if (t + 1 == n) wait(v_full + 8 * vs, (t / kStagesV) & 1);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
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
            bar_wait(o_full, 0, &never);        // nothing in flight when tensor memory is given back
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (sh.gave_up != 0 && tid == 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_GAVE_UP);
    if (warp == kSoftWarps + kUnpackWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the chunks of the units that were cut: a warp a query row, a lane D / 32
// neighbouring values.
template <int D, bool kHalf>
__global__ void __launch_bounds__(128) kv_attend_join_tc_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int NV = D / 32;
    asm volatile("griddepcontrol.launch_dependents;");
    const int H = (int)a.pool.H, group = (int)a.group, lane = threadIdx.x & 31;
    const uint32_t unit = a.whole_units + blockIdx.x / (kRowsTc / 4);
    const int head = (int)(unit % H), rt = (int)a.row_tiles - 1 - (int)(unit / H % a.row_tiles);
    const int r = (int)(unit / H / a.row_tiles);
    const int row = rt * kRowsTc + (int)(blockIdx.x % (kRowsTc / 4)) * 4 + (threadIdx.x >> 5);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool bad;
    const Span s = row_span(a.q_start[r], a.q_start[r + 1], a.lens[r], (int)a.tokens, (int)a.max_q,
                            (int)a.max_len, group, (int)a.window, rt, kRowsTc, &bad);
    const int n = (s.hi - s.lo + (int)a.chunk - 1) / (int)a.chunk;
    if (row >= s.n * group || n <= 1 || a.uneven[(int64_t)r * H + head] != 0) return;
    const int64_t tok = s.q0 + row / group;
    const int qh = head * group + row % group;
    float top = kNoMaxTc, sum = 0.0f, acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] = 0.0f;
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const int64_t at = ((int64_t)k * a.tokens + tok) * a.q_heads + qh;
        const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + at * 2);
        float x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) x[v] = a.part_o[at * D + v * 32 + lane];
        if (ml.y == 0.0f) continue;
        const float t = fmaxf(top, ml.x), u = ex2(top - t), w = ex2(ml.x - t);
        top = t;
        sum = sum * u + ml.y * w;
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] = acc[v] * u + x[v] * w;
    }
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
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

typedef void(AttendTcFn)(AttendArgs);
struct VariantTc {
    uint32_t D;
    bool fp16;
    int parts;
    AttendTcFn *fn, *steps_fn, *join_fn;
    int smem;
};
template <int D, bool kHalf, int kParts>
constexpr VariantTc variant_tc() {
    return VariantTc{(uint32_t)D, kHalf, kParts, kv_attend_tc_kernel<D, kHalf, kParts>, kv_attend_steps_kernel<D>,
                     kv_attend_join_tc_kernel<D, kHalf>, smem_tc(D, kHalf, kParts)};
}
#define KVB_VARIANTS_TC(D) \
    variant_tc<D, false, 1>(), variant_tc<D, false, 2>(), variant_tc<D, true, 2>()
const VariantTc kVariantsTc[] = {KVB_VARIANTS_TC(64), KVB_VARIANTS_TC(96), KVB_VARIANTS_TC(128)};

}  // namespace

void plan_attend_tc(AttendPlan *p, uint64_t span, uint32_t requests, uint32_t kv_heads, int sms) {
    // A unit is a row tile of one head of one request, and takes an SM for itself.
    // Units that fill the GPU a whole number of times run whole.  What is left
    // over is cut along the cached tokens into the number of chunks that ends
    // soonest: `waves` of blocks of 1/c of the work.  A block begins and ends in the
    // time of about 512 cached tokens (8 us), and writing and joining parts takes that
    // of 1,500: 104 units left over of 8,192 tokens took 115 us whole, 137 cut in four.
    const uint64_t units = (uint64_t)requests * kv_heads * p->row_tiles;
    const uint64_t rest = units % (uint64_t)sms;
    p->rows = kRowsTc;
    p->whole_units = units - rest;
    p->chunk = 0x7fffffffu;
    p->chunks = 1;
    double best = 1e300;
    for (uint64_t c = 1; rest != 0 && c <= 64 && (c == 1 || span / c >= 512); ++c) {
        const uint64_t chunk = (span + c - 1) / c;
        const double waves = (double)((rest * c + sms - 1) / sms);
        const double cost = waves * ((double)chunk + 512.0) + (c > 1 ? 1500.0 : 0.0);
        if (cost < best) {
            best = cost;
            p->chunks = (uint32_t)c;
            p->chunk = (uint32_t)((chunk + kTileK - 1) / kTileK * kTileK);
        }
    }
    if (p->chunks == 1) {
        p->whole_units = units;
        p->chunk = 0x7fffffffu;
    }
}

cudaError_t launch_attend_tc(const AttendArgs &a, uint32_t D, bool fp16, bool pdl, cudaStream_t stream,
                             int *launches) {
    for (const VariantTc &v : kVariantsTc) {
        if (v.D != D || v.fp16 != fp16 || v.parts != key_parts(fp16, a.lse != nullptr)) continue;
        cudaLaunchConfig_t cfg = {};
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = pdl ? 1 : 0;
        cfg.gridDim = dim3(a.pool.H, a.step_parts, a.requests);
        cfg.blockDim = dim3(256);
        cudaError_t e = cudaLaunchKernelEx(&cfg, v.steps_fn, a);
        if (e != cudaSuccess) return e;
        ++*launches;
        const uint32_t units = a.requests * a.pool.H * a.row_tiles;
        cfg.gridDim = dim3(a.whole_units + (units - a.whole_units) * a.chunks);
        cfg.blockDim = dim3(kThreadsTc);
        cfg.dynamicSmemBytes = (size_t)v.smem;
        e = cudaLaunchKernelEx(&cfg, v.fn, a);
        if (e != cudaSuccess) return e;
        ++*launches;
        if (a.chunks > 1) {
            cfg.gridDim = dim3((units - a.whole_units) * (kRowsTc / 4));
            cfg.blockDim = dim3(128);
            cfg.dynamicSmemBytes = 0;
            e = cudaLaunchKernelEx(&cfg, v.join_fn, a);
            if (e == cudaSuccess) ++*launches;
        }
        return e;
    }
    return cudaErrorInvalidValue;
}

cudaError_t preload_attend_tc_kernels() {
    cudaFuncAttributes at;
    for (const VariantTc &v : kVariantsTc) {
        cudaError_t e = cudaFuncGetAttributes(&at, (const void *)v.fn);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute((const void *)v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, (const void *)v.steps_fn);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, (const void *)v.join_fn);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kvb
