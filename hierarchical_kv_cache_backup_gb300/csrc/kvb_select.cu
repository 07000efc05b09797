// kvb_select.cu -- bounds of the keys of each page (kv_bound) and the pages whose bounds
// promise a query most (kv_select).
//
// Mathematics.  For a page and KV head, lo_d <= k_d <= hi_d for all its keys, so q . k is
// at most sum_d max(q_d lo_d, q_d hi_d) = sum over q_d > 0 of q_d hi_d + sum over q_d < 0 of
// q_d lo_d.  Bounds and queries are 8-bit codes in units of a power of two for each 32 dims,
// rounded outwards for bounds: a group's sum is then a whole number below 2^19, exact in any order of
// additions, so that the pages selected do not depend on how the sums are taken, and a page is
// read in half the bytes that 16-bit bounds would take.
#include "kvb_pages.h"
#include "kvb_pages_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

namespace kvb {

namespace {

template <bool kBf>
struct Pair16;
template <>
struct Pair16<true> {
    using T = __nv_bfloat162;
    __device__ static float2 f(T x) { return __bfloat1622float2(x); }
};
template <>
struct Pair16<false> {
    using T = __half2;
    __device__ static float2 f(T x) { return __half22float2(x); }
};

// ------------------------------------------------------------------- kv_bound
//
// A warp takes one page and KV head: 16 bytes of a token a lane, several tokens at once where
// a vector is short, least and largest values two at a time in their own type (fp8 as fp16,
// exact).  Bound: memory, keys read once (four prompts of 32,768 tokens, 8 heads of 128: 36 to 42 us, floor 33.6).
// One page a request is a launch: 3.6 us.
constexpr int kBoundWarps = 8;

template <int D, bool kF8, bool kHalf>
__global__ void __launch_bounds__(kBoundWarps * 32) kv_bound_kernel(const __grid_constant__ BoundArgs a) {
    constexpr bool kBf = !kF8 && !kHalf;
    using P = Pair16<kBf>;
    using T2 = typename P::T;
    constexpr int LT = D / (kF8 ? 16 : 8), AT = 32 / LT;     // lanes of a token, tokens at once
    constexpr int NP = kF8 ? 8 : 4, LG = kF8 ? 2 : 4;        // pairs of a lane, lanes of a group
    constexpr uint32_t kRec = (2 * D + D / 8 + 15) / 16 * 16;
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, H = (int)a.pool.H;
    const int in = lane / LT, piece = lane - in * LT;
    const uint64_t units = (uint64_t)a.requests * a.most_pages * H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (uint64_t u = (uint64_t)blockIdx.x * kBoundWarps + (threadIdx.x >> 5); u < units; u += (uint64_t)gridDim.x * kBoundWarps) {
        const int head = (int)(u % H);
        const uint32_t jr = (uint32_t)(u / H % a.most_pages), r = (uint32_t)(u / H / a.most_pages);
        const int len = a.lens[r], first = a.first != nullptr ? a.first[r] : 0;
        if (len < 0 || len > (int)a.max_len || first < 0 || first > len || len - first > (int)a.max_new) {
            if (jr == 0 && head == 0 && lane == 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
            continue;
        }
        const uint32_t j = div_T(a.pool, (uint32_t)first) + jr;
        const int64_t t0 = (int64_t)j * a.pool.T;
        if (first == len || t0 >= len) continue;
        const int n = (int)min((int64_t)a.pool.T, len - t0);
        const uint32_t page = (uint32_t)a.pages[(int64_t)r * a.pages_stride + j];
        if (page >= a.pool.P) {
            if (head == 0 && lane == 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_PAGE);
            continue;
        }
        T2 lo[NP], hi[NP];
        const uint32_t top = kBf ? 0x7f807f80u : 0x7c007c00u, low = top | 0x80008000u;      // infinities
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            lo[i] = *reinterpret_cast<const T2 *>(&top);
            hi[i] = *reinterpret_cast<const T2 *>(&low);
        }
        const uint64_t from = a.pool.base[0] + (uint64_t)page * a.pool.s_page + (uint64_t)head * a.pool.s_head + piece * 16;
        auto take = [&](const uint4 &w) {
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kF8) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t x;
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((unsigned short)(v[i] >> (16 * h))));
                        const T2 y = *reinterpret_cast<const T2 *>(&x);
                        lo[2 * i + h < NP ? 2 * i + h : 0] = __hmin2_nan(lo[2 * i + h < NP ? 2 * i + h : 0], y);
                        hi[2 * i + h < NP ? 2 * i + h : 0] = __hmax2_nan(hi[2 * i + h < NP ? 2 * i + h : 0], y);
                    }
                } else {
                    const T2 y = *reinterpret_cast<const T2 *>(&v[i]);
                    lo[i] = __hmin2_nan(lo[i], y);
                    hi[i] = __hmax2_nan(hi[i], y);
                }
            }
        };
        if (in < AT) {
            int t = in;
            for (; t + 7 * AT < n; t += 8 * AT) {
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint4 *>(from + (uint64_t)(t + i * AT) * a.pool.s_tok);
#pragma unroll
                for (int i = 0; i < 8; ++i) take(w[i]);
            }
            for (; t < n; t += AT) take(*reinterpret_cast<const uint4 *>(from + (uint64_t)t * a.pool.s_tok));
        }
        // over the tokens that other lanes had
        if (AT > 1) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                T2 l = lo[i], h = hi[i];
#pragma unroll
                for (int s = 1; s < AT; ++s) {
                    const uint32_t lw = __shfl_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&lo[i]), piece + s * LT);
                    const uint32_t hw = __shfl_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&hi[i]), piece + s * LT);
                    l = __hmin2_nan(l, *reinterpret_cast<const T2 *>(&lw));
                    h = __hmax2_nan(h, *reinterpret_cast<const T2 *>(&hw));
                }
                lo[i] = l;
                hi[i] = h;
            }
        }
        float fl[2 * NP], fh[2 * NP];
        uint32_t most = 0;                                   // of the group, as bits: NaN above infinity
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float2 l = P::f(lo[i]), h = P::f(hi[i]);
            fl[2 * i] = l.x;
            fl[2 * i + 1] = l.y;
            fh[2 * i] = h.x;
            fh[2 * i + 1] = h.y;
        }
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i)
            most = max(most, max(__float_as_uint(fl[i]) & 0x7fffffffu, __float_as_uint(fh[i]) & 0x7fffffffu));
#pragma unroll
        for (int d = 1; d < LG; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        float inv;
        const float step = bound_step(most, &inv);
        if (lane < LT) {
            uint8_t *rec = a.bounds + ((uint64_t)page * H + head) * kRec;
            uint32_t wl[NP / 2], wh[NP / 2];
#pragma unroll
            for (int i = 0; i < NP / 2; ++i) {
                wl[i] = wh[i] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int cl = inv != 0.0f ? (int)floorf(__fmul_rn(fl[4 * i + b], inv)) : 0;
                    const int ch = inv != 0.0f ? (int)ceilf(__fmul_rn(fh[4 * i + b], inv)) : 0;
                    wl[i] |= (uint32_t)(cl & 255) << (8 * b);
                    wh[i] |= (uint32_t)(ch & 255) << (8 * b);
                }
            }
            if (kF8) {
                *reinterpret_cast<uint4 *>(rec + 16 * lane) = make_uint4(wl[0], wl[1], wl[2 % (NP / 2)], wl[3 % (NP / 2)]);
                *reinterpret_cast<uint4 *>(rec + D + 16 * lane) = make_uint4(wh[0], wh[1], wh[2 % (NP / 2)], wh[3 % (NP / 2)]);
            } else {
                *reinterpret_cast<uint2 *>(rec + 8 * lane) = make_uint2(wl[0], wl[1]);
                *reinterpret_cast<uint2 *>(rec + D + 8 * lane) = make_uint2(wh[0], wh[1]);
            }
            if (lane % LG == 0) *reinterpret_cast<float *>(rec + 2 * D + lane / LG * 4) = step;
            if (lane < (int)(kRec - 2 * D - D / 8) / 4) *reinterpret_cast<uint32_t *>(rec + 2 * D + D / 8 + lane * 4) = 0;
        }
    }
}

// ------------------------------------------------------------------ kv_select
//
// Scores: a block takes some pages of one query and KV head, a warp 16 pages at a time.  A group of 32 dims is
// the k of one mma.sync m16n8k32 of 8-bit integers: 16 pages by 8 query heads, the codes of the largest
// against the queries' positive ones and of the least against the negative ones into the same sums.  (With
// dp4a, a page's group a lane, 64 instructions stood where 2 do now, at the same time.)  The float terms are
// added in the order of the groups.  Bound: the chain of a warp's instructions, 16 warps an SM, behind the loads
// at a block's beginning.  With the query's values asked for first, 32 requests of up to 1,024 pages went
// from 29.1 to 26.7 us with the picks, and to 25.5 with records handed out by their page's lane; floor 8.1.
constexpr int kScoreWarps = 8, kHeads = 8, kScorePages = 16, kWarpPages = 64;

__host__ __device__ constexpr int record_of(int D) { return (2 * D + D / 8 + 15) / 16 * 16; }
__host__ __device__ constexpr int score_stages(int D) { return D <= 128 ? 3 : 2; }
constexpr int score_smem(int D) { return kScoreWarps * score_stages(D) * kScorePages * record_of(D); }

__device__ __forceinline__ void imma(int *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// 1.5 x 2^23 as a float's bits: added to a whole number below 2^22 it is the bits of the number's float
// but for 1.5 x 2^23.
constexpr int kWhole = 0x4b400000;

template <int D, bool kHalf>
__global__ void __launch_bounds__(kScoreWarps * 32, 2) kv_score_kernel(const __grid_constant__ SelectArgs a) {
    using P = Pair16<!kHalf>;
    constexpr int NG = D / 32, kRec = record_of(D), kStages = score_stages(D), kStage = kScorePages * kRec;
    extern __shared__ __align__(16) uint8_t records[];       // [warp][stage][16] records
    __shared__ int32_t ids[kScoreWarps][kWarpPages];
    __shared__ __align__(16) int8_t code[kHeads][2][D];
    __shared__ float unit[kHeads][NG];
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int chunks = (int)((a.max_pages + a.block_pages - 1) / a.block_pages);
    const int head = (int)blockIdx.x / chunks, p0 = (int)(blockIdx.x % chunks) * (int)a.block_pages;
    const int i = blockIdx.y, r = blockIdx.z;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q0 = a.q_start[r], q1 = a.q_start[r + 1], len = a.lens[r];
    if (q0 < 0 || q1 < q0 || q1 > (int)a.tokens || q1 - q0 > (int)a.max_q || len < 0 || len > (int)a.max_len) return;
    if (i >= q1 - q0) return;
    const int seen = pages_seen(len, q1 - q0, i, a.T);
    if (seen <= (int)a.budget || p0 >= seen) return;
    const int64_t tok = q0 + i;
    const int p1 = min(seen, p0 + (int)a.block_pages);      // block_pages: at most kWarpPages a warp
    const int32_t *table = a.pages + (int64_t)r * a.pages_stride;
    float *scores = a.scores + (tok * a.H + head) * (int64_t)a.max_pages;

    // the query's values, a warp a group of 32 of some head, a lane a value; asked for first, as all that follows waits
    unsigned short x[NG];
    auto values = [&](int h0) {
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            const int h = h0 + (warp + kScoreWarps * k) / NG, gr = (warp + kScoreWarps * k) % NG;
            x[k] = 0;
            if (h < (int)a.group)
                x[k] = *reinterpret_cast<const unsigned short *>(a.q.data + tok * a.q.s_tok + (int64_t)(head * a.group + h) * a.q.s_head + (32 * gr + lane) * 2);
        }
    };
    values(0);

    // A warp takes a run of the block's pages.  It reads their ids at once; records come by cp.async, 16 a stage.
    const int w0 = p0 + warp * ((int)a.block_pages / kScoreWarps), w1 = min(p1, w0 + (int)a.block_pages / kScoreWarps);
#pragma unroll
    for (int k = 0; k < kWarpPages / 32; ++k)
        if (w0 + 32 * k + lane < w1) ids[warp][32 * k + lane] = table[w0 + 32 * k + lane];
    __syncwarp();
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(records) + warp * (kStages * kStage);
    const uint8_t *from = a.bounds + (uint64_t)head * kRec;
    // Codes: neighbouring lanes a record's 16-byte pieces, which its page's lane hands them; steps: a lane a record.
    constexpr int PC = 2 * D / 16, kAtOnce = 32 / PC, kStepPieces = (kRec - 2 * D) / 16;
    static_assert(kStepPieces <= 2, "a half warp a piece");
    const int sub = lane / PC, of = (lane - sub * PC) * 16, tail = 2 * D + (lane >> 4) * 16;
    const uint32_t to = ring + sub * kRec + of, to_tail = ring + (lane & 15) * kRec + tail, row = a.H * (uint32_t)kRec;
    auto copy16 = [](uint32_t smem, const uint8_t *gmem) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
    };
    auto load = [&](int p, int stage) {
        if (p < w1) {
            const uint32_t at = stage * kStage;
            const uint32_t mine = p + (lane & 15) < w1 ? (uint32_t)ids[warp][p - w0 + (lane & 15)] : 0xffffffffu;
#pragma unroll
            for (int k = 0; k < kScorePages / kAtOnce; ++k) {
                const uint32_t page = __shfl_sync(0xffffffffu, mine, (k * kAtOnce + sub) & 15);
                if (sub < kAtOnce && page < a.P) copy16(to + at + k * kAtOnce * kRec, from + (uint64_t)page * row + of);
            }
            if (lane < 16 * kStepPieces && mine < a.P) copy16(to_tail + at, from + (uint64_t)mine * row + tail);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int h0 = 0; h0 < (int)a.group; h0 += kHeads) {
        const int heads = min(kHeads, (int)a.group - h0);
        if (h0 != 0) values(h0);
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) load(w0 + k * kScorePages, k);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NG; ++k) {                       // its codes
            const int h = (warp + kScoreWarps * k) / NG, gr = (warp + kScoreWarps * k) % NG;
            const uint32_t both = (uint32_t)x[k] | (uint32_t)x[k] << 16;
            const float y = P::f(*reinterpret_cast<const typename P::T *>(&both)).x;
            const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(y) & 0x7fffffffu);
            float inv;
            const float step = bound_step(most, &inv);
            const int v = inv != 0.0f ? (int)rintf(__fmul_rn(y, inv)) : 0;
            code[h][0][32 * gr + lane] = (int8_t)max(v, 0);
            code[h][1][32 * gr + lane] = (int8_t)min(v, 0);
            if (lane == 0) unit[h][gr] = step;
        }
        __syncthreads();
        // fragments: head g's codes 4 c .. and 16 + 4 c .. of each group; steps of heads 2 c and 2 c + 1
        uint32_t pos[NG][2], neg[NG][2];
        float t[NG][2];
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                pos[gr][k] = *reinterpret_cast<const uint32_t *>(&code[g][0][32 * gr + 16 * k + 4 * c]);
                neg[gr][k] = *reinterpret_cast<const uint32_t *>(&code[g][1][32 * gr + 16 * k + 4 * c]);
                t[gr][k] = unit[2 * c + k][gr];
            }
        int stage = 0;
        for (int p = w0; p < w1; p += kScorePages) {
            load(p + (kStages - 1) * kScorePages, stage == 0 ? kStages - 1 : stage - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint32_t base = ring + stage * kStage, rows = base + (lane & 15) * kRec + (lane >> 4) * 16;
            const float *step = reinterpret_cast<const float *>(records + (warp * kStages + stage) * kStage + g * kRec + 2 * D);
            float sum[4];
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                uint32_t lo[4], hi[4];
                ldm4(rows + 32 * gr, lo);
                ldm4(rows + D + 32 * gr, hi);
                int dot[4] = {kWhole, kWhole, kWhole, kWhole};
                imma(dot, hi, pos[gr][0], pos[gr][1]);
                imma(dot, lo, neg[gr][0], neg[gr][1]);
                const float s[2] = {step[gr], step[gr + 8 * kRec / 4]};          // of pages g and g + 8
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float term = __fmul_rn(__fsub_rn(__int_as_float(dot[k]), __int_as_float(kWhole)), __fmul_rn(s[k >> 1], t[gr][k & 1]));
                    sum[k] = gr == 0 ? term : __fadd_rn(sum[k], term);
                }
            }
            float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!(fabsf(sum[k]) <= kMostScore)) sum[k] = kMostScore;
                if (2 * c + (k & 1) < heads) best[k >> 1] = fmaxf(best[k >> 1], sum[k]);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                best[k] = fmaxf(best[k], __shfl_xor_sync(0xffffffffu, best[k], 1));
                best[k] = fmaxf(best[k], __shfl_xor_sync(0xffffffffu, best[k], 2));
            }
            const int mine = p + g + 8 * c;                                  // lanes 0 and 1 of a quad write a page each
            if (c < 2 && mine < w1) {
                const bool bad = (uint32_t)ids[warp][mine - w0] >= a.P;
                float x = bad ? -kMostScore : c == 0 ? best[0] : best[1];    // nothing to be found there
                if (h0 != 0) x = fmaxf(x, scores[mine]);
                scores[mine] = x;
                if (bad && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_PAGE);
            }
            __syncwarp();
            if (++stage == kStages) stage = 0;
        }
    }
}

// Picks: a block takes one query and KV head, a thread a run of pages.  The least key that is selected is
// found by a histogram over the range of the keys (so that scores of one size spread over the
// bins); what is in its bin is ranked, key against key, or, if too much, spread over bins again.  A sum
// over the block then says where a thread's picks go, in the order of the pages.  Rows of up to 2,048 pages
// take 256 threads, longer ones 1,024.  Bound: barriers and the latency of shared memory, 8 us for 256 rows of
// up to 1,024 pages.
constexpr int kHeld = 8, kRanked = 256, kShortRow = 2048;

__device__ __forceinline__ unsigned long long scan_up(unsigned long long x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// Keys in the order of the scores.  -0, a negative sum whose steps' product underflows, is 0: the two tie.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
    return u ^ ((u >> 31) != 0 ? 0xffffffffu : 0x80000000u);
}

template <int kPickThreads>
__global__ void __launch_bounds__(kPickThreads) kv_pick_kernel(const __grid_constant__ SelectArgs a) {
    constexpr int kBins = 2 * kPickThreads, kBinBits = kPickThreads == 1024 ? 11 : 9, kWarps = kPickThreads / 32;
    static_assert(kBins == 1 << kBinBits && kRanked <= kPickThreads, "two bins a thread");
    __shared__ uint32_t bins[kBins], ranked[kRanked];
    __shared__ uint32_t sums[kWarps], least_s[kWarps], most_s[kWarps], found[3], listed;
    __shared__ unsigned long long wide[kWarps];
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.x, i = blockIdx.y, r = blockIdx.z;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int q0 = a.q_start[r], q1 = a.q_start[r + 1], len = a.lens[r];
    if (q0 < 0 || q1 < q0 || q1 > (int)a.tokens || q1 - q0 > (int)a.max_q || len < 0 || len > (int)a.max_len) {
        if (tid == 0 && head == 0 && i == 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
        return;
    }
    if (i >= q1 - q0) return;
    const int64_t row = (int64_t)(q0 + i) * a.H + head;
    const int n = pages_seen(len, q1 - q0, i, a.T), budget = (int)a.budget;
    int32_t *picks = a.picks + row * budget;
    if (n <= budget) {
        for (int k = tid; k < budget; k += kPickThreads) picks[k] = k < n ? k : -1;
        return;
    }
    const float *scores = a.scores + row * (int64_t)a.max_pages;
    const int c0 = (int)a.keep_first, c1 = n - (int)a.keep_last;      // candidates [c0, c1); the rest is kept
    uint32_t k = (uint32_t)(budget - c0 - (int)a.keep_last);
    const int per = (n + kPickThreads - 1) / kPickThreads, b0 = tid * per;
    // this thread's run of pages, held in registers where it is short
    uint32_t held[kHeld];
    auto candidate = [&](int p) { return p >= c0 && p < c1; };
    if (per <= kHeld) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) held[j] = j < per && candidate(b0 + j) ? order_key(scores[b0 + j]) : 0u;
    }
    // every page of the run in turn: its number, and its key if it is a candidate (else it is kept)
    auto each = [&](auto &&f) {
        if (per <= kHeld) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
                if (j < per && b0 + j < n) f(b0 + j, held[j], candidate(b0 + j));
        } else {
            for (int p = b0; p < min(n, b0 + per); ++p) f(p, candidate(p) ? order_key(scores[p]) : 0u, candidate(p));
        }
    };
    uint32_t lo = 0xffffffffu, hi = 0;
    each([&](int, uint32_t u, bool c) {
        if (c) {
            lo = min(lo, u);
            hi = max(hi, u);
        }
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        least_s[warp] = lo;
        most_s[warp] = hi;
    }
    if (tid == 0) listed = 0;
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, least_s[lane % kWarps]);
    hi = __reduce_max_sync(0xffffffffu, most_s[lane % kWarps]);
    uint32_t need = k;                                       // of the keys equal to the least one selected
    while (k != 0 && lo != hi) {
        const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);
        bins[tid] = bins[tid + kPickThreads] = 0;
        __syncthreads();
        each([&](int, uint32_t u, bool c) {
            if (c && u >= lo && u <= hi) atomicAdd(&bins[(u - lo) >> shift], 1u);
        });
        __syncthreads();
        // keys in the bins above: thread t looks after the last bins but 2 t and 2 t + 1
        const uint32_t x1 = bins[kBins - 1 - 2 * tid], x0 = bins[kBins - 2 - 2 * tid];
        uint32_t s = x0 + x1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) sums[warp] = s;
        __syncthreads();
        uint32_t before = lane < warp ? sums[lane % kWarps] : 0;
        before = __reduce_add_sync(0xffffffffu, before) + s - x0 - x1;
        if (before < k && before + x1 >= k) {
            found[0] = (uint32_t)(kBins - 1 - 2 * tid);
            found[1] = before;
            found[2] = x1;
        } else if (before + x1 < k && before + x1 + x0 >= k) {
            found[0] = (uint32_t)(kBins - 2 - 2 * tid);
            found[1] = before + x1;
            found[2] = x0;
        }
        __syncthreads();
        const uint32_t bin = found[0], inside = found[2];
        k -= found[1];
        lo += bin << shift;
        hi = min(hi, lo + ((1u << shift) - 1u));
        need = k;
        if (inside == k) {                                   // all of the bin
            need = 0xffffffffu;
            break;
        }
        if (inside <= kRanked && lo != hi) {
            each([&](int, uint32_t u, bool c) {
                if (c && u >= lo && u <= hi) ranked[atomicAdd(&listed, 1u)] = u;
            });
            __syncthreads();
            if (tid < (int)inside) {
                const uint32_t mine = ranked[tid];
                uint32_t above = 0, same = 0;
                for (uint32_t j = 0; j < inside; ++j) {
                    above += ranked[j] > mine;
                    same += ranked[j] == mine;
                }
                if (above < k && above + same >= k) {        // equal keys write the same
                    found[0] = mine;
                    found[1] = k - above;
                }
            }
            __syncthreads();
            lo = found[0];
            need = found[1];
            break;
        }
    }
    if (k == 0) {                                            // the pages that are kept fill the budget
        lo = 0xffffffffu;
        need = 0;
    }
    // key > lo is selected, key == lo for the first `need` of them, and with need without bound all from lo on
    unsigned long long mine = 0;                             // selected, and equal in the high word
    each([&](int, uint32_t u, bool c) {
        if (!c || u > lo) mine += 1;
        else if (u == lo) mine += 1ull << 32;
    });
    const unsigned long long sum = scan_up(mine, lane);
    if (lane == 31) wide[warp] = sum;
    __syncthreads();
    unsigned long long before = sum - mine;
    for (int w = 0; w < warp; ++w) before += wide[w];
    uint32_t gt = (uint32_t)before, eq = (uint32_t)(before >> 32);
    each([&](int p, uint32_t u, bool c) {
        if (!c || u > lo) {
            picks[gt + min(eq, need)] = p;
            ++gt;
        } else if (u == lo) {
            if (eq < need) picks[gt + eq] = p;
            ++eq;
        }
    });
}

typedef void(BoundFn)(BoundArgs);
typedef void(SelectFn)(SelectArgs);
struct BoundVariant {
    uint32_t D;
    bool fp8, fp16;
    BoundFn *fn;
};
struct ScoreVariant {
    uint32_t D;
    bool fp16;
    SelectFn *fn;
    int smem;
};
// fp8 values are the same whatever the queries' type
#define KVB_BOUND(D)                                                                              \
    BoundVariant{D, false, false, kv_bound_kernel<D, false, false>},                              \
        BoundVariant{D, false, true, kv_bound_kernel<D, false, true>}, BoundVariant{D, true, true, kv_bound_kernel<D, true, true>}
#define KVB_SCORE(D) ScoreVariant{D, false, kv_score_kernel<D, false>, score_smem(D)}, ScoreVariant{D, true, kv_score_kernel<D, true>, score_smem(D)}
const BoundVariant kBounds[] = {KVB_BOUND(64), KVB_BOUND(96), KVB_BOUND(128), KVB_BOUND(192), KVB_BOUND(256)};
const ScoreVariant kScores[] = {KVB_SCORE(64), KVB_SCORE(96), KVB_SCORE(128), KVB_SCORE(192), KVB_SCORE(256)};

template <class Args>
cudaError_t launch(void (*fn)(Args), dim3 grid, int threads, cudaStream_t stream, bool pdl, const Args &a, int smem = 0) {
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

cudaError_t launch_bound(const BoundArgs &a, uint32_t D, bool fp8, bool fp16, bool pdl, int sms, cudaStream_t stream) {
    (void)cudaGetLastError();
    for (const BoundVariant &v : kBounds) {
        if (v.D != D || v.fp8 != fp8 || (!fp8 && v.fp16 != fp16)) continue;
        const uint64_t blocks = ((uint64_t)a.requests * a.most_pages * a.pool.H + kBoundWarps - 1) / kBoundWarps;
        return launch(v.fn, dim3((unsigned)std::min<uint64_t>(blocks, (uint64_t)sms * 64)), kBoundWarps * 32, stream, pdl, a);
    }
    return cudaErrorInvalidValue;
}

uint32_t select_block_pages(uint64_t pages, int sms) {
    // Two blocks an SM, all at once, as far as 64 pages a warp go: a block begins with a chain of loads, the
    // request's length, the query's values, the page numbers, records (32 requests of up to 1,024 pages: 38.5 us
    // with blocks of 128 pages, 31.2 of 256, 29.1 of 512; 128 a warp gain nothing more).
    const uint64_t want = pages / (2ull * (uint64_t)sms);
    return (uint32_t)std::min<uint64_t>(kWarpPages * kScoreWarps, std::max<uint64_t>(128, (want + 127) / 128 * 128));
}

cudaError_t launch_select(const SelectArgs &a, uint32_t D, bool fp16, bool pdl, cudaStream_t stream, int *launches) {
    (void)cudaGetLastError();
    for (const ScoreVariant &v : kScores) {
        if (v.D != D || v.fp16 != fp16) continue;
        if (a.max_pages > a.budget) {             // otherwise every page is picked
            const uint32_t chunks = (a.max_pages + a.block_pages - 1) / a.block_pages;
            const cudaError_t e = launch(v.fn, dim3(chunks * a.H, a.max_q, a.requests), kScoreWarps * 32, stream, pdl, a, v.smem);
            if (e != cudaSuccess) return e;
            ++*launches;
        }
        const dim3 grid(a.H, a.max_q, a.requests);
        const cudaError_t e = a.max_pages <= (uint32_t)kShortRow ? launch(kv_pick_kernel<256>, grid, 256, stream, pdl, a)
                                                                 : launch(kv_pick_kernel<1024>, grid, 1024, stream, pdl, a);
        if (e == cudaSuccess) ++*launches;
        return e;
    }
    return cudaErrorInvalidValue;
}

cudaError_t preload_select_kernels() {
    cudaFuncAttributes at;
    for (const BoundVariant &v : kBounds) {
        const cudaError_t e = cudaFuncGetAttributes(&at, (const void *)v.fn);
        if (e != cudaSuccess) return e;
    }
    for (const ScoreVariant &v : kScores) {
        cudaError_t e = cudaFuncGetAttributes(&at, (const void *)v.fn);
        if (e == cudaSuccess) e = cudaFuncSetAttribute((const void *)v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = cudaFuncGetAttributes(&at, (const void *)kv_pick_kernel<256>);
    return e != cudaSuccess ? e : cudaFuncGetAttributes(&at, (const void *)kv_pick_kernel<1024>);
}

}  // namespace kvb
