// kvb_attend.cu -- attention of new tokens over one layer of a 4-bit pool.
//
// Mathematics.  A cached value is (code - z) s with one step s and zero point z
// for each 32 values of a vector (a group g):
//   q . k_t   = sum_g s_tg (q_g . code_tg - z_tg sum q_g)
//   out[dim]  = sum_t (p_t s_tg) code_t[dim] - sum_t (p_t s_tg) z_tg
// The matrix instructions multiply codes and zero points as they are: the
// four bits of a code in the low bits of an fp16 are the subnormal code x 2^-24
// (x 2^-20 four bits higher), exact, and the powers of two go into the queries
// and the last scaling.  Unpacking is one AND a pair of values, and one shift for
// four pairs of keys, three for four of values: the products of an instruction
// are lined up by the exponents of their operands, 2^-14 for all subnormals, and
// what is far below that is lost.  Products with keys share a token and its step;
// those with values do not, and a token whose weight x step is 2^20 times its
// neighbours' would leave them nothing at 2^-24 (64 requests of up to 8,192
// tokens: 3 us of 148).  Steps scale float32 sums on the key side and the probabilities on
// the value side.  p_t = 2^(x_t - m) with a running maximum m.
#include "kvb_vec.h"
#include "kvb_vec_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

namespace kvb {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = 32;        // cached tokens a warp takes at a time
constexpr int kStages = 2;       // tiles in shared memory per warp
constexpr float kNoMax = -3.0e38f;
constexpr int kScaleMost = 100;               // exponents of f: at most this
constexpr float kWeightMost = 32768.0f;       // 2^15: what a weight is kept to, below fp16's 65,504

__host__ __device__ constexpr int vec_bytes(int D) { return (D / 2 + D / 8 + 15) / 16 * 16; }
// Bytes between vectors in shared memory: an odd multiple of 16, so that the 8
// rows of a fragment start 4 banks apart and no load has a bank conflict.
__host__ __device__ constexpr int vec_stride(int D) {
    return vec_bytes(D) / 16 % 2 ? vec_bytes(D) : vec_bytes(D) + 16;
}
__host__ __device__ constexpr int ring_bytes(int D) { return kStages * 2 * kTile * vec_stride(D); }
__host__ __device__ constexpr int merge_floats(int D, int NT) { return 8 * NT * (D + 4); }
__host__ __device__ constexpr int warp_bytes(int D, int NT) {
    return ring_bytes(D) > 4 * merge_floats(D, NT) ? ring_bytes(D) : 4 * merge_floats(D, NT);
}

__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c = a b over 8 values of k, from nothing
__device__ __forceinline__ void mma8(float *c, uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
                 "{%7,%7,%7,%7};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

// Four pairs of codes (nibbles i of both 16-bit halves) as fp16 subnormals: of keys
// code x 2^-24 for i = 0 and 2 and code x 2^-20 for 1 and 3, of values code x 2^-20.
template <bool kValues>
__device__ __forceinline__ void codes4(uint32_t w, uint32_t *p) {
    const uint32_t v = w >> 8;
    p[0] = kValues ? (w << 4) & 0x00f000f0u : w & 0x000f000fu;
    p[1] = w & 0x00f000f0u;
    p[2] = kValues ? (w >> 4) & 0x00f000f0u : v & 0x000f000fu;
    p[3] = v & 0x00f000f0u;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four 8 x 8 blocks of 16-bit values, row i of block b at the address of lane
// 8 b + i: lane (g, c) gets values 2 c and 2 c + 1 of row g, or with kTrans of
// column g the rows 2 c and 2 c + 1.
template <bool kTrans>
__device__ __forceinline__ void blocks4(uint32_t addr, uint32_t *r) {
    if (kTrans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t word_at(uint32_t addr) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(addr) : "memory");
    return w;
}

__device__ __forceinline__ uint4 words_at(uint32_t addr) {
    uint4 w;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(addr) : "memory");
    return w;
}

// two products at a time
__device__ __forceinline__ float2 mul2(float a0, float a1, float b0, float b1) {
    float2 r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
    return r;
}

// 2^e, 0 for e below -126
__device__ __forceinline__ float pow2i(int e) { return e < -126 ? 0.0f : __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t pick(const uint4 &u, int i) {
    return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}

__device__ __forceinline__ void clear(uint4 &u, int i) {
    if (i == 0) u.x = 0;
    else if (i == 1) u.y = 0;
    else if (i == 2) u.z = 0;
    else u.w = 0;
}

__device__ __forceinline__ void copy16(uint32_t smem, uint64_t gmem, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem),
                 "r"(on ? 16 : 0)
                 : "memory");
}

template <int kRows>
__device__ __forceinline__ Span span_of(const AttendArgs &a, int r, int rt, bool *bad) {
    return row_span(a.q_start[r], a.q_start[r + 1], a.lens[r], (int)a.tokens, (int)a.max_q,
                    (int)a.max_len, (int)a.group, (int)a.window, rt, kRows, bad);
}

// --------------------------------------------------------- few rows a request
//
// A block takes one KV head of one request, a tile of 8 NT query rows (new
// tokens x the head's group) and a chunk of the cached tokens; its 8 warps
// take tiles of 32 tokens in turn, each with a private ring in shared memory
// (no barrier in the loop), and join their maxima, sums and accumulators at the
// end.  Cached tokens are the 16-row side of m16n8k16 and query rows its
// 8-column side, so a GQA group of up to 8 heads fills the instruction.
// Scores come out with a token a row; movmatrix turns the probabilities of an
// 8 x 8 block for the second product.
//
// Zero points ride on the matrix instructions too.  Keys: three more values of k
// hold z, against -sum q_g split into three fp16 parts (33 bits).  Values: one
// more 16-row tile holds z of group g in row g, so that its product with the
// rounded probabilities is subtracted at the end and the rounding error of a
// probability acts on (code - z) only.  Zero points stand as z x 2^-18, the most that a
// subnormal holds.
//
// A group of a value that is not finite makes that group of the outputs NaN, for the rows
// that see the token, and nothing else: its step is taken as 0 in the products (0 x NaN would
// reach every group through the zero points' tile and rows whose weight is 0), and the rows
// that see it are marked.
//
// Bound: instructions.  16 tokens of 128 values (2,560 bytes) take 358 a warp
// through both products for 8 query rows, a warp begins and ends with about 1,300; the ALU
// pipe is 57% busy at 2.4 instructions a cycle and SM, 16 warps of 128 registers.  Of
// one request of 131,072 tokens (8 heads, 49.5 us) the part that grows with the tokens
// runs at 5.0 TB/s of 6.8.  Measured and dropped: query fragments in shared memory
// (2% slower), four-warp blocks with 96 registers (5-30% slower), several heads a block for
// NHD pages (20% slower), both halves' exponentials at once for four rows (no change).
template <int D, int NT, bool kHalf, bool kMany>
__device__ __forceinline__ void attend_rows(const AttendArgs &a, int head, int rt, int r, int ci, int chunk,
                                            bool report) {
    constexpr int NG = D / 32;                 // groups of a vector
    constexpr int SV = vec_stride(D), PV = vec_bytes(D) / 16;
    constexpr int kRows = 8 * NT;
    constexpr int WB = warp_bytes(D, NT);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float join_m[kWarps][kRows], join_l[kWarps][kRows];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int32_t *table = a.pages + (int64_t)r * a.pages_stride;
    constexpr int kTurn = kWarps * kTile;      // from a warp's tile to its next

    // Without a window the first tiles' places in the page table are known before the
    // request's length is: their pages are read along with it (a row holds the pages
    // of max_len tokens).  Lane i looks after token i of a tile.
    int32_t page = 0, page1 = 0;
    auto look_up = [&](int t, int end) {
        return t < end ? table[div_T(a.pool, (uint32_t)t)] : 0;
    };
    if (!a.window) {
        const int64_t t = (int64_t)ci * chunk + warp * kTile + lane;
        if (t < (int64_t)a.max_len) page = look_up((int)t, (int)a.max_len);
        if (t + kTurn < (int64_t)a.max_len) page1 = look_up((int)t + kTurn, (int)a.max_len);
    }
    bool bad;
    const Span s = span_of<kRows>(a, r, rt, &bad);
    if (bad && a.status != nullptr && threadIdx.x == 0 && report)
        atomicOr(a.status, KV_STATUS_BAD_LENGTH);
    const int row0 = rt * kRows, rows = min(kRows, s.n * (int)a.group - row0);
    if (rows <= 0) return;
    const int c0 = s.lo + ci * chunk, c1 = min(s.hi, c0 + chunk);
    if (c0 >= c1 && ci > 0) return;
    const bool whole = s.hi - s.lo <= chunk;          // this block sees all the rows see

    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * WB;
    const int group = (int)a.group;
    // Row `row` of the tile as a new token and a head of the group; one new token needs
    // no division.
    auto new_token = [&](int row) { return kMany ? (row0 + row) / group : 0; };

    // the query rows, read while the pages are
    uint4 raw[NT][NG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = 8 * nt + g;
        const bool on = row < rows;
        const int i = on ? new_token(row) : 0, j = on ? row0 + row - i * group : 0;
        const uint64_t src = a.q.data + (int64_t)(s.q0 + i) * a.q.s_tok + (int64_t)(head * group + j) * a.q.s_head;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            raw[nt][gr] = make_uint4(0, 0, 0, 0);
            if (on) raw[nt][gr] = *reinterpret_cast<const uint4 *>(src + (gr * 32 + c * 8) * 2);
        }
    }

    // Tiles are copied 16 bytes a lane, a vector's PV pieces by neighbouring lanes.
    // Lane i knows the place of token i, as a count of vectors, and hands it
    // round.  Page ids are read a tile before they are used.
    constexpr int kAtOnce = 32 / PV;
    const int lane_tok = lane / PV, piece = lane - lane_tok * PV;
    const uint64_t from_k = a.pool.base[0] + (uint64_t)head * a.pool.s_head + piece * 16;
    const uint64_t from_v = a.pool.base[1] + (uint64_t)head * a.pool.s_head + piece * 16;
    const uint32_t to = ring + lane_tok * SV + piece * 16;
    // starts the copy of a tile; returns which of its tokens are in pages outside the pool
    auto load = [&](int stage, int t0, int32_t page) -> uint32_t {
        uint32_t wrong = 0;
        if (t0 < c1) {
            const int t = t0 + lane;
            const bool in = t < c1, bad = in && (uint32_t)page >= a.pool.P, ok = in && !bad;
            const uint32_t at = ok ? vector_index(a.pool, (uint32_t)page, (uint32_t)t) : 0;
            const uint32_t good = __ballot_sync(0xffffffffu, ok);
            wrong = __ballot_sync(0xffffffffu, bad);
            const uint32_t dst = to + stage * (2 * kTile * SV);
#pragma unroll
            for (int k = 0; k < (kTile + kAtOnce - 1) / kAtOnce; ++k) {
                const int tok = k * kAtOnce + lane_tok;
                const uint64_t off = (uint64_t)__shfl_sync(0xffffffffu, at, tok & 31) * (uint32_t)vec_bytes(D);
                if (lane_tok < kAtOnce && (kTile % kAtOnce == 0 || tok < kTile)) {
                    copy16(dst + k * kAtOnce * SV, from_k + off, good >> (tok & 31) & 1);
                    copy16(dst + k * kAtOnce * SV + kTile * SV, from_v + off, good >> (tok & 31) & 1);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return wrong;
    };

    int t0 = c0 + warp * kTile;
    if (a.window) {
        page = look_up(t0 + lane, c1);
        page1 = look_up(t0 + kTurn + lane, c1);
    }
    uint32_t bad_now = load(0, t0, page);
    uint32_t bad_next = load(1, t0 + kTurn, page1);
    page = look_up(t0 + 2 * kTurn + lane, c1);

    // Query rows as B fragments.  Each row is scaled by a power of two that
    // brings its largest value to 2^9..2^10, so that bf16 queries are exact in
    // fp16 (but for values 2^-22 of the row's largest, where 2^-24 is lost); the
    // scores undo it.  Values that meet odd codes are divided by 16.
    uint32_t qf[NT][NG][4], qz[NT][NG];
    float qs[NT][2];
    int lim[NT][2], low[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float x[NG][8], top = 0.0f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            const uint4 u = raw[nt][gr];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (kHalf) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                    x[gr][2 * e] = f.x;
                    x[gr][2 * e + 1] = f.y;
                } else {
                    x[gr][2 * e] = __uint_as_float(w[e] << 16);
                    x[gr][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
                top = fmaxf(top, fmaxf(fabsf(x[gr][2 * e]), fabsf(x[gr][2 * e + 1])));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(9 - exponent of top), and its inverse; 1 for zeros and infinities
        const uint32_t ex = __float_as_uint(top) >> 23;
        const bool scaled = ex >= 10 && ex < 255;
        const float up = scaled ? __uint_as_float((263u - ex) << 23) : 1.0f, up16 = 0.0625f * up;
        const float back = scaled ? __uint_as_float((ex - 9u) << 23) : 1.0f;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            float part[2] = {0.0f, 0.0f};     // those that meet even and odd codes
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y0 = x[gr][e] * (e & 1 ? up16 : up), y1 = x[gr][e + 4] * (e & 1 ? up16 : up);
                qf[nt][gr][e] = half2_bits(y0, y1);
                part[e & 1] += y0 + y1;
            }
            float sum = -0.25f * part[1] - 0.015625f * part[0];      // zero points are z x 2^-18
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const float h0 = __half2float(__float2half_rn(sum));
            const float h1 = __half2float(__float2half_rn(sum - h0));
            qz[nt][gr] = c == 0 ? half2_bits(h0, h1) : c == 1 ? half2_bits(sum - h0 - h1, 0.0f) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            qs[nt][e] = __shfl_sync(0xffffffffu, back, 8 * c + 4 * e) * a.scale_log2 * 16777216.0f;
            const int col = 8 * nt + 2 * c + e;
            const int pos = s.len - s.n + new_token(col);
            lim[nt][e] = min(pos, s.len - 1);
            low[nt][e] = a.window ? pos - (int)a.window + 1 : 0;
        }
    }
    // a tile wholly inside [safe_lo, safe_hi) is seen by every row of the block
    const int safe_hi = kMany ? min(c1, s.len - s.n + new_token(0) + 1) : c1;
    const int safe_lo = kMany && a.window ? s.len - s.n + new_token(rows - 1) - (int)a.window + 1 : 0;

    // lane constants of the fragments' addresses and of the zero points' places
    const uint32_t at_row = ((lane & 15) * SV) + (lane >> 4) * 16;    // rows 0..15, then the next group
    const uint32_t z_mul = c == 0 ? 0x00400040u : c == 1 ? 0x40u : 0u;
    const uint32_t z_group = (g < NG ? g : 0) * 4;

    float o[NG][2][NT][4], oz[NT][4], f[NG][NT][2], m[NT][2], l[NT][2];
    uint32_t nan_groups = 0;      // bit 8 (2 nt + e) + gr: that row's group gr is NaN
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            f[gr][nt][0] = f[gr][nt][1] = __uint_as_float((127u + kScaleMost) << 23);   // set by the first weight that is not 0
#pragma unroll
            for (int e = 0; e < 4; ++e) o[gr][0][nt][e] = o[gr][1][nt][e] = 0.0f;
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) oz[nt][e] = 0.0f;
        m[nt][0] = m[nt][1] = kNoMax;
        l[nt][0] = l[nt][1] = 0.0f;
    }

    auto scale_sums = [&](int gr, int nt, int e, float k) {
        if (g == gr) oz[nt][e] *= k;
        o[gr][0][nt][e] *= k;
        o[gr][0][nt][e + 2] *= k;
        o[gr][1][nt][e] *= k;
        o[gr][1][nt][e + 2] *= k;
    };
    for (int stage = 0; t0 < c1; t0 += kTurn, stage ^= 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const uint32_t ks = ring + stage * (2 * kTile * SV), vs = ks + kTile * SV;

        // scores: x[sub][nt][e] for token 16 sub + g (+ 8 for e >= 2), row 8 nt + 2 c + (e & 1)
        float x[2][NT][4];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            const uint32_t k0 = ks + (16 * sub + g) * SV + D / 2;
            uint4 w0, w1;
            uint32_t kw[4];
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                if (gr % 4 == 0) {
                    w0 = words_at(k0 + gr * 4);
                    w1 = words_at(k0 + 8 * SV + gr * 4);
                }
                if (gr % 2 == 0) blocks4<false>(ks + 16 * sub * SV + gr * 16 + at_row, kw);
                const uint32_t s0 = pick(w0, gr % 4), s1 = pick(w1, gr % 4);
                uint32_t p0[4], p1[4];
                codes4<false>(kw[gr % 2 * 2], p0);
                codes4<false>(kw[gr % 2 * 2 + 1], p1);
                const uint32_t a0[4] = {p0[0], p1[0], p0[1], p1[1]};
                const uint32_t a1[4] = {p0[2], p1[2], p0[3], p1[3]};
                const float d0 = q4_step(s0), d1 = q4_step(s1);
                const uint32_t z0 = (s0 & 15u) * z_mul, z1 = (s1 & 15u) * z_mul;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float acc[4];
                    mma8(acc, z0, z1, qz[nt][gr]);
                    mma(acc, a0, qf[nt][gr][0], qf[nt][gr][1]);
                    mma(acc, a1, qf[nt][gr][2], qf[nt][gr][3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[sub][nt][e] = gr == 0 ? (e < 2 ? d0 : d1) * acc[e]
                                                : x[sub][nt][e] + (e < 2 ? d0 : d1) * acc[e];
                }
            }
        }
        // in units of log2, from the maximum; masked
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[sub][nt][e] = x[sub][nt][e] * qs[nt][e & 1] -
                                    (m[nt][e & 1] == kNoMax ? 0.0f : m[nt][e & 1]);
        if (t0 < safe_lo || t0 + kTile > safe_hi || bad_now != 0) {
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int in = 16 * sub + g + (e >= 2 ? 8 : 0), t = t0 + in;
                        if (bad_now >> in & 1) x[sub][nt][e] = __uint_as_float(kNanWord);
                        if (t >= c1 || (kMany && (t > lim[nt][e & 1] || t < low[nt][e & 1])))
                            x[sub][nt][e] = -INFINITY;
                    }
            if (bad_now != 0 && a.status != nullptr && lane == 0)
                atomicOr(a.status, KV_STATUS_BAD_PAGE);
        }
        // The maximum moves only when a score passes it by more than 2^8: until
        // then probabilities reach up to 2^8, which costs no precision.
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float over = fmaxf(fmaxf(x[0][nt][e], x[0][nt][e + 2]),
                                         fmaxf(x[1][nt][e], x[1][nt][e + 2]));
                move |= over > 8.0f || m[nt][e] == kNoMax;
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float t = fmaxf(fmaxf(x[0][nt][e], x[0][nt][e + 2]),
                                    fmaxf(x[1][nt][e], x[1][nt][e + 2]));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    int rise = 0;                        // of the maximum
                    if (m[nt][e] == kNoMax) {            // nothing seen so far: take it as it is
                        if (t == -INFINITY) continue;
                        m[nt][e] = t;
                    } else {
                        t = ceilf(fmaxf(t, 0.0f));
                        m[nt][e] += t;
                        rise = (int)fminf(t, 1000.0f);
                    }
#pragma unroll
                    for (int sub = 0; sub < 2; ++sub) {
                        x[sub][nt][e] -= t;
                        x[sub][nt][e + 2] -= t;
                    }
                    l[nt][e] *= pow2i(-rise);
                    // The weights' sums stay: f rises by as much as the weights fall.
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        const int most = kScaleMost + 127 - (int)(__float_as_uint(f[gr][nt][e]) >> 23);
                        const int up = min(rise, most);
                        f[gr][nt][e] = __uint_as_float(__float_as_uint(f[gr][nt][e]) + ((uint32_t)up << 23));
                        if (up < rise) scale_sums(gr, nt, e, pow2i(up - rise));
                    }
                }
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[sub][nt][e] = exp2_fast(x[sub][nt][e]);
                    l[nt][e & 1] += x[sub][nt][e];
                }

        // Weights p x step in units of 1/f.  f belongs to one row and group and follows the
        // largest weight that the row has met (it is brought to 2^4..2^5 and may grow to
        // 2^15), so that neither a step that the row does not see nor one that its
        // probability makes small takes bits from the others.
        float most_p[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                most_p[nt][e] = fmaxf(fmaxf(x[0][nt][e], x[0][nt][e + 2]), fmaxf(x[1][nt][e], x[1][nt][e + 2]));
        uint4 vw[2][2][(NG + 3) / 4];
        float bound = 0.0f;           // on the weights of this lane's tokens
        bool not_finite = false;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int q = 0; q < (NG + 3) / 4; ++q) {
                vw[sub][0][q] = words_at(vs + (16 * sub + g) * SV + D / 2 + q * 16);
                vw[sub][1][q] = words_at(vs + (16 * sub + g + 8) * SV + D / 2 + q * 16);
            }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
            auto w = [&](int sub, int k) { return pick(vw[sub][k][gr / 4], gr % 4); };
            const uint32_t top = max(max(w(0, 0), w(0, 1)), max(w(1, 0), w(1, 1)));
            not_finite |= top >= 0x7f800000u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 u = mul2(most_p[nt][0], most_p[nt][1], f[gr][nt][0], f[gr][nt][1]);
                bound = fmaxf(bound, fmaxf(u.x, u.y) * __uint_as_float(top));
            }
        }
        if (__any_sync(0xffffffffu, not_finite)) {
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4 &u = vw[k / 2][k % 2][gr / 4];
                    if (pick(u, gr % 4) >= 0x7f800000u) {
                        clear(u, gr % 4);
                        const int t = t0 + 8 * k + g;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (t < c1 && (!kMany || (t <= lim[nt][e] && t >= low[nt][e])))
                                    nan_groups |= 1u << (8 * (2 * nt + e) + gr);
                    }
                }
            }
        }
        if (__any_sync(0xffffffffu, bound > kWeightMost || not_finite)) {
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = 0.0f;      // the row's largest weight in these tokens
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            t = fmaxf(t, x[k / 2][nt][e + k % 2 * 2] * q4_step(pick(vw[k / 2][k % 2][gr / 4], gr % 4)));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
                        // no branch: one for each row and group takes longer
                        const uint32_t at = __float_as_uint(f[gr][nt][e]) >> 23;
                        const uint32_t to = t * f[gr][nt][e] > kWeightMost ? 258u - min(__float_as_uint(t) >> 23, 254u) : at;
                        scale_sums(gr, nt, e, pow2i((int)to - (int)at));
                        f[gr][nt][e] = __uint_as_float(to << 23);
                    }
            }
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            // zero points of group g: tokens 2 c, 2 c + 1 and the same + 8
            const uint32_t z = vs + (16 * sub + 2 * c) * SV + D / 2 + z_group;
            const uint32_t za = (__byte_perm(word_at(z), word_at(z + SV), 0x5410) & 0x000f000fu) << 6;
            const uint32_t zb = (__byte_perm(word_at(z + 8 * SV), word_at(z + 9 * SV), 0x5410) & 0x000f000fu) << 6;
            uint32_t vc[4];
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                if (gr % 2 == 0) blocks4<true>(vs + 16 * sub * SV + gr * 16 + at_row, vc);
                const float d0 = q4_step(pick(vw[sub][0][gr / 4], gr % 4));
                const float d1 = q4_step(pick(vw[sub][1][gr / 4], gr % 4));
                // fp16 outputs: weights in two fp16 parts, so that only the output is rounded
                // (17 requests of up to 8,906 tokens, 5 heads over 1 of 96: error against 64
                // bits 2.05e-4 as for a float32 plain form, 2.96e-4 with one part; 24
                // requests of 2,000 tokens: heads of 64 19.7 -> 21.5 us, of 256 58 -> 68).
                // A bf16 output does not show it.
                uint32_t b[NT][2], rest[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 u0 = mul2(x[sub][nt][0], x[sub][nt][1], f[gr][nt][0], f[gr][nt][1]);
                    const float2 u1 = mul2(x[sub][nt][2], x[sub][nt][3], f[gr][nt][0], f[gr][nt][1]);
                    const float p[4] = {u0.x * d0, u0.y * d0, u1.x * d1, u1.y * d1};
                    uint32_t h[2] = {half2_bits(p[0], p[1]), half2_bits(p[2], p[3])};
                    b[nt][0] = transpose8x8(h[0]);
                    b[nt][1] = transpose8x8(h[1]);
                    if (kHalf) {
                        const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&h[0]));
                        const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&h[1]));
                        rest[nt][0] = transpose8x8(half2_bits(p[0] - f0.x, p[1] - f0.y));
                        rest[nt][1] = transpose8x8(half2_bits(p[2] - f1.x, p[3] - f1.y));
                    }
                }
                uint32_t p0[4], p1[4];
                codes4<true>(vc[gr % 2 * 2], p0);
                codes4<true>(vc[gr % 2 * 2 + 1], p1);
                const uint32_t a0[4] = {p0[0], p0[1], p1[0], p1[1]};
                const uint32_t a1[4] = {p0[2], p0[3], p1[2], p1[3]};
                const uint32_t az[4] = {g == gr ? za : 0u, 0u, g == gr ? zb : 0u, 0u};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma(o[gr][0][nt], a0, b[nt][0], b[nt][1]);
                    mma(o[gr][1][nt], a1, b[nt][0], b[nt][1]);
                    mma(oz[nt], az, b[nt][0], b[nt][1]);
                    if (kHalf) {
                        mma(o[gr][0][nt], a0, rest[nt][0], rest[nt][1]);
                        mma(o[gr][1][nt], a1, rest[nt][0], rest[nt][1]);
                        mma(oz[nt], az, rest[nt][0], rest[nt][1]);
                    }
                }
            }
        }
        __syncwarp();
        bad_now = bad_next;
        bad_next = load(stage, t0 + kStages * kTurn, page);
        page = look_up(t0 + (kStages + 1) * kTurn + lane, c1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();

    // Join the warps.  A warp's accumulators go to its own ring as [row][D + 4].
    float *mine = reinterpret_cast<float *>(smem + warp * WB);
    if (__any_sync(0xffffffffu, nan_groups != 0)) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) nan_groups |= __shfl_xor_sync(0xffffffffu, nan_groups, d);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float t = l[nt][e];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
            const int row = 8 * nt + 2 * c + e;
            if (g == 0) {
                join_m[warp][row] = m[nt][e];
                join_l[warp][row] = t;
            }
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                // undo f, a power of two, and the subnormals' 2^-20 (2^-18 for zero points)
                const float k = __shfl_sync(0xffffffffu, oz[nt][e], 4 * gr + c) * -262144.0f;
                const float back = __uint_as_float((254u << 23) - __float_as_uint(f[gr][nt][e]));
                float4 v = make_float4(o[gr][0][nt][e] * 1048576.0f + k, o[gr][0][nt][e + 2] * 1048576.0f + k,
                                       o[gr][1][nt][e] * 1048576.0f + k, o[gr][1][nt][e + 2] * 1048576.0f + k);
                v.x *= back;
                v.y *= back;
                v.z *= back;
                v.w *= back;
                if (nan_groups >> (8 * (2 * nt + e) + gr) & 1)
                    v.x = v.y = v.z = v.w = __uint_as_float(kNanWord);
                *reinterpret_cast<float4 *>(mine + row * (D + 4) + gr * 32 + 4 * g) = v;
            }
        }
    __syncthreads();
    const int D4 = D / 4;
    for (int it = threadIdx.x; it < rows * D4; it += kWarps * 32) {
        const int row = it / D4, d4 = it - row * D4;
        float top = kNoMax, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            top = fmaxf(top, join_l[w][row] != 0.0f ? join_m[w][row] : kNoMax);
        float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float lw = join_l[w][row];
            if (lw == 0.0f) continue;          // this warp saw nothing of the row
            const float k = exp2_fast(join_m[w][row] - top);
            const float4 v = *reinterpret_cast<const float4 *>(
                reinterpret_cast<const float *>(smem + w * WB) + row * (D + 4) + d4 * 4);
            sum += lw * k;
            acc.x += v.x * k;
            acc.y += v.y * k;
            acc.z += v.z * k;
            acc.w += v.w * k;
        }
        const int i = new_token(row), j = row0 + row - i * group;
        const int64_t tok = s.q0 + i;
        const int qh = head * (int)a.group + j;
        if (whole) {
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            const uint64_t dst = a.out.data + tok * a.out.s_tok + (int64_t)qh * a.out.s_head + d4 * 8;
            uint2 u;
            if (kHalf) {
                u = make_uint2(half2_bits(acc.x * inv, acc.y * inv), half2_bits(acc.z * inv, acc.w * inv));
            } else {
                __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
                __nv_bfloat162 h1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
                u = make_uint2(*reinterpret_cast<uint32_t *>(&h0), *reinterpret_cast<uint32_t *>(&h1));
            }
            *reinterpret_cast<uint2 *>(dst) = u;
            if (d4 == 0 && a.lse != nullptr)
                a.lse[tok * a.q_heads + qh] =
                    sum != 0.0f ? (top + log2f(sum)) * 0.693147180559945f : -INFINITY;
        } else {
            const int64_t at = ((int64_t)ci * a.tokens + tok) * a.q_heads + qh;
            *reinterpret_cast<float4 *>(a.part_o + at * D + d4 * 4) = acc;
            if (d4 == 0) *reinterpret_cast<float2 *>(a.part_ml + at * 2) = make_float2(top, sum);
        }
    }
}

template <int D, int NT, bool kHalf, bool kMany>
__global__ void __launch_bounds__(kWarps * 32, D * NT <= 128 ? 2 : 1)
    kv_attend_rows_kernel(const __grid_constant__ AttendArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int H = (int)a.pool.H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // every request's first chunk, which is the fullest, before any second one
    attend_rows<D, NT, kHalf, kMany>(a, (int)blockIdx.x % H, (int)blockIdx.x / H, (int)blockIdx.y, (int)blockIdx.z,
                                     (int)a.chunk, blockIdx.x + blockIdx.z == 0);
}

// Requests with many rows whose steps differ too much for the kernel that holds keys
// and values in fp16 (it says so in a.uneven): a block takes row tiles of one head
// and request in turn, each over all its cached tokens.  Blocks of even requests end at once.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kWarps * 32, 1) kv_attend_uneven_kernel(const __grid_constant__ AttendArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int head = (int)blockIdx.x, r = (int)blockIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = (int)min((int64_t)a.q_start[r + 1] - a.q_start[r], (int64_t)a.max_q);
    if (n <= 0 || a.uneven[(int64_t)r * a.pool.H + head] == 0) return;
    for (int rt = (int)blockIdx.z; rt * 16 < n * (int)a.group; rt += (int)gridDim.z) {
        attend_rows<D, 2, kHalf, true>(a, head, rt, r, 0, 1 << 30, false);
        __syncthreads();      // the next tile's copies go where this one's sums stand
    }
}

// Joins the chunks of a row (a query head and token): kW warps a row, each over
// every kW-th chunk, a lane D / 32 values.  Rows of few chunks take one warp, four rows a
// block; with many the parts are too long a chain for one.
template <int D, int kRows, bool kHalf, int kW>
__global__ void __launch_bounds__(128) kv_attend_join_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int NV = D / 32;
    __shared__ float acc_s[kW][D], m_s[kW], l_s[kW];
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int qh = kW == 1 ? blockIdx.x * 4 + warp : blockIdx.x, part = kW == 1 ? 0 : warp;
    const int i = blockIdx.y, r = blockIdx.z;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (qh >= (int)a.q_heads) return;
    bool bad;
    const int j = qh % (int)a.group;
    const Span s = span_of<kRows>(a, r, (i * (int)a.group + j) / kRows, &bad);
    const int n = (s.hi - s.lo + (int)a.chunk - 1) / (int)a.chunk;
    if (i >= s.n || n <= 1) return;
    const int64_t tok = s.q0 + i;
    float top = kNoMax, sum = 0.0f, acc[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) acc[v] = 0.0f;
#pragma unroll 4
    for (int k = part; k < n; k += kW) {
        const int64_t at = ((int64_t)k * a.tokens + tok) * a.q_heads + qh;
        const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + at * 2);
        float x[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) x[v] = a.part_o[at * D + v * 32 + lane];
        if (ml.y == 0.0f) continue;
        const float t = fmaxf(top, ml.x), u = exp2_fast(top - t), w = exp2_fast(ml.x - t);
        top = t;
        sum = sum * u + ml.y * w;
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[v] = acc[v] * u + x[v] * w;
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
        for (int w = 1; w < kW; ++w) {
            if (l_s[w] == 0.0f) continue;
            const float t = fmaxf(top, m_s[w]), u = exp2_fast(top - t), k = exp2_fast(m_s[w] - t);
            top = t;
            sum = sum * u + l_s[w] * k;
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[v] = acc[v] * u + acc_s[w][v * 32 + lane] * k;
        }
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

// ------------------------------------------------------------------ launches

template <typename Fn>
cudaError_t launch(Fn *fn, dim3 grid, int threads, int smem, cudaStream_t stream, bool pdl,
                   const AttendArgs &a) {
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

typedef void(AttendFn)(AttendArgs);
struct Variant {
    uint32_t D, rows;
    bool fp16, many;
    AttendFn *rows_fn, *join_fn, *join4_fn;
    int smem;
};

template <int D, int NT, bool kHalf, bool kMany>
constexpr Variant variant() {
    return Variant{(uint32_t)D, 8u * NT, kHalf, kMany, kv_attend_rows_kernel<D, NT, kHalf, kMany>,
                   kv_attend_join_kernel<D, 8 * NT, kHalf, 1>,
                   kv_attend_join_kernel<D, 8 * NT, kHalf, 4>, kWarps * warp_bytes(D, NT)};
}

#define KVB_VARIANTS(D, NT)                                                                       \
    variant<D, NT, false, false>(), variant<D, NT, true, false>(), variant<D, NT, false, true>(), \
        variant<D, NT, true, true>()
const Variant kVariants[] = {KVB_VARIANTS(64, 1),  KVB_VARIANTS(64, 2),  KVB_VARIANTS(96, 1),
                             KVB_VARIANTS(96, 2),  KVB_VARIANTS(128, 1), KVB_VARIANTS(128, 2),
                             KVB_VARIANTS(192, 1), KVB_VARIANTS(256, 1)};

struct UnevenVariant {
    uint32_t D;
    bool fp16;
    AttendFn *fn;
    int smem;
};
#define KVB_UNEVEN(D)                                                            \
    UnevenVariant{D, false, kv_attend_uneven_kernel<D, false>, kWarps * warp_bytes(D, 2)}, \
        UnevenVariant{D, true, kv_attend_uneven_kernel<D, true>, kWarps * warp_bytes(D, 2)}
const UnevenVariant kUnevenVariants[] = {KVB_UNEVEN(64), KVB_UNEVEN(96), KVB_UNEVEN(128)};

}  // namespace

// Query rows of a request from which the tcgen05 kernel (256 rows a block) is taken.
// 2 / 16 requests of 4,000 tokens, 8 heads of 128, groups of 4, this kernel against that
// one: 64 rows 29.1 against 32.9 / 88 against 97 us, 80 rows 38.3 against 33.9 / 104
// against 98, 256 rows 73 against 44 / 280 against 109.
constexpr uint64_t kManyRows = 80;

AttendPlan plan_attend(uint32_t requests, uint32_t tokens, uint32_t max_q, uint32_t max_len,
                       uint32_t window, uint32_t q_heads, uint32_t kv_heads, uint32_t D, int sms) {
    AttendPlan p{};
    const uint64_t rows = (uint64_t)max_q * (q_heads / kv_heads);
    p.many = D <= 128 && rows >= kManyRows;
    p.rows = p.many ? 256 : rows > 8 && D <= 128 ? 16 : 8;
    p.row_tiles = (uint32_t)((rows + p.rows - 1) / p.rows);
    // the most cached tokens a row tile sees: its queries' windows overlap
    uint64_t span = max_len;
    if (window) span = std::min<uint64_t>(span, (uint64_t)window + p.rows);
    if (p.many) {
        plan_attend_tc(&p, span, requests, kv_heads, sms);
        p.step_parts = step_parts_of(max_len, window, max_q);
        p.step_bytes = ((uint64_t)requests * (p.step_parts * (uint64_t)kStepWords + 1) * kv_heads * sizeof(uint32_t) + 255) /
                       256 * 256;
        p.uneven_blocks = (uint32_t)std::min<uint64_t>(
            (rows + 15) / 16, std::max<uint64_t>(1, 2ull * (uint64_t)sms / ((uint64_t)requests * kv_heads)));
    } else {
        // Cut along the cached tokens into the number of chunks that ends soonest, by a
        // model in tokens of one block: what all blocks read spread over the blocks
        // that fit at once (requests of a batch taken as three quarters of the longest),
        // half a chunk lost at the end when there is more than one wave, never less
        // than a chunk; a block begins and ends in the time of 350 tokens, and parts
        // are joined in that of 500.  64 requests of up to 8,192 tokens and 8 heads, 1 /
        // 2 / 3 chunks: 148 / 148 / 147 us; 32 of them 90 / 86 / 82; 64 of up to 2,048
        // 51 / 58 / 61; 24 of 2,016 of 4 heads of 64, 2 / 3 / 4 chunks: 23.4 / 21.5 / 25.0.
        const uint64_t slots = (uint64_t)sms * (D * (p.rows / 8) <= 128 ? 2 : 1), unit = kWarps * kTile;
        const uint64_t units = std::max<uint64_t>(1, (uint64_t)requests * kv_heads * p.row_tiles);
        const double spread = (requests > 1 ? 0.75 : 1.0) * (double)units * (double)span / (double)slots;
        double best = 1e300;
        for (uint64_t c : {(uint64_t)1, (uint64_t)2, (uint64_t)3, (uint64_t)4, (uint64_t)6, slots / units}) {
            if (c == 0 || (c > 1 && span <= (c - 1) * unit)) continue;
            const uint64_t chunk = std::max<uint64_t>(unit, ((span + c - 1) / c + unit - 1) / unit * unit);
            const uint64_t waves = (units * c + slots - 1) / slots;
            const double cost = std::max(spread + (waves > 1 ? 0.5 * chunk : 0.0), (double)chunk) + 350.0 * waves +
                                (c > 1 ? 500.0 : 0.0);
            if (cost < best) {
                best = cost;
                p.chunk = (uint32_t)chunk;
            }
        }
        p.chunks = (uint32_t)std::max<uint64_t>(1, (span + p.chunk - 1) / p.chunk);
    }
    p.bytes = p.step_bytes;
    if (p.chunks > 1) p.bytes += (uint64_t)p.chunks * tokens * q_heads * (D + 2) * sizeof(float);
    return p;
}

cudaError_t launch_attend_uneven(const AttendArgs &a, const AttendPlan &p, uint32_t D, bool fp16, bool pdl,
                                 cudaStream_t stream) {
    for (const UnevenVariant &v : kUnevenVariants)
        if (v.D == D && v.fp16 == fp16)
            return launch(v.fn, dim3(a.pool.H, a.requests, p.uneven_blocks), kWarps * 32, v.smem, stream, pdl, a);
    return cudaErrorInvalidValue;
}

cudaError_t launch_attend(const AttendArgs &a, const AttendPlan &p, uint32_t D, bool fp16, bool pdl,
                          cudaStream_t stream, int *launches) {
    (void)cudaGetLastError();
    if (p.many) {
        cudaError_t e = launch_attend_tc(a, D, fp16, pdl, stream, launches);
        if (e == cudaSuccess) e = launch_attend_uneven(a, p, D, fp16, pdl, stream);
        if (e == cudaSuccess) ++*launches;
        return e;
    }
    const bool many = a.max_q > 1;
    for (const Variant &v : kVariants) {
        if (v.D != D || v.rows != p.rows || v.fp16 != fp16 || v.many != many) continue;
        const dim3 grid(a.pool.H * p.row_tiles, a.requests, p.chunks);
        cudaError_t e = launch(v.rows_fn, grid, kWarps * 32, v.smem, stream, pdl, a);
        if (e != cudaSuccess) return e;
        ++*launches;
        if (p.chunks > 1) {
            if (p.chunks <= 6)
                e = launch(v.join_fn, dim3((a.q_heads + 3) / 4, a.max_q, a.requests), 128, 0, stream, pdl, a);
            else
                e = launch(v.join4_fn, dim3(a.q_heads, a.max_q, a.requests), 128, 0, stream, pdl, a);
            if (e == cudaSuccess) ++*launches;
        }
        return e;
    }
    return cudaErrorInvalidValue;
}

cudaError_t preload_attend_kernels() {
    cudaFuncAttributes at;
    for (const Variant &v : kVariants) {
        cudaError_t e = cudaFuncGetAttributes(&at, (const void *)v.rows_fn);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute((const void *)v.rows_fn,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, (const void *)v.join_fn);
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, (const void *)v.join4_fn);
        if (e != cudaSuccess) return e;
    }
    for (const UnevenVariant &v : kUnevenVariants) {
        cudaError_t e = cudaFuncGetAttributes(&at, (const void *)v.fn);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute((const void *)v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
        if (e != cudaSuccess) return e;
    }
    return preload_attend_tc_kernels();
}

}  // namespace kvb
