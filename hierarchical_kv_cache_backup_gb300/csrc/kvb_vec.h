// kvb_vec.h -- what the operators on single head vectors share (kv_rotate,
// kv_append, kv_fetch, kv_attend): a layer of a pool as addresses of vectors,
// the 4-bit format's arithmetic, and the kernels' parameter blocks.  The
// functions here also compile as host C++, so that the CPU tests run the very
// address and rounding code that the kernels run.  Not part of the public ABI.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define KVB_HD __host__ __device__ __forceinline__
#else
#define KVB_HD inline
#endif

namespace kvb {

// One layer of a pool.  Vector (page, token t of the page, head h) of component
// c is at base[c] + page * s_page + t * s_tok + h * s_head.  The page term is
// taken in 64 bits: pools pass 4 GiB.
struct PoolLayer {
    uint64_t base[2];    // component 0 (keys) and 1 (values) of this layer
    uint64_t s_page;     // bytes between pages
    uint32_t s_tok;      // bytes between tokens of a page (a page is < 32 GiB / 16)
    uint32_t s_head;     // bytes between heads
    uint32_t T, H, B, P;
    uint32_t v_page, v_tok;    // s_page and s_tok in vectors
    uint32_t t_mul, t_shift;   // division by T (FastDiv's m and s)
};

KVB_HD uint32_t mul_hi32(uint32_t a, uint32_t b) {
#ifdef __CUDA_ARCH__
    return __umulhi(a, b);
#else
    return (uint32_t)(((uint64_t)a * b) >> 32);
#endif
}

KVB_HD uint32_t div_T(const PoolLayer &p, uint32_t n) {
    return (uint32_t)(((uint64_t)mul_hi32(n, p.t_mul) + n) >> p.t_shift);
}

// Offset of the vector of `slot` (head 0) inside a component, or -1 when the
// slot is outside the pool.  The pool has P * T slots, as 64-bit numbers.
KVB_HD int64_t slot_offset(const PoolLayer &p, int64_t slot) {
    if (slot < 0 || slot >= (int64_t)((uint64_t)p.P * p.T)) return -1;
    uint64_t page, t;
    if ((uint64_t)slot >> 32) {
        page = (uint64_t)slot / p.T;
        t = (uint64_t)slot - page * p.T;
    } else {
        page = div_T(p, (uint32_t)slot);
        t = (uint32_t)slot - (uint32_t)page * p.T;
    }
    return (int64_t)(page * p.s_page + t * p.s_tok);
}

// Offset of a request's token t, in page `page` of the pool; -1 (and *wrong) when
// there is no such page.
KVB_HD int64_t page_offset(const PoolLayer &p, uint32_t page, uint32_t t, bool *wrong) {
    *wrong = page >= p.P;
    if (*wrong) return -1;
    return (int64_t)(page * p.s_page + (uint64_t)(t - div_T(p, t) * p.T) * p.s_tok);
}

// The same from the request's row of the page table.
KVB_HD int64_t token_offset(const PoolLayer &p, const int32_t *table, uint32_t t, bool *wrong) {
    return page_offset(p, (uint32_t)table[div_T(p, t)], t, wrong);
}

// The same as a count of vectors, for a page inside the pool.  Every offset is a
// whole number of vectors, and vector_index_fits says that all of them are below 2^32.
KVB_HD uint32_t vector_index(const PoolLayer &p, uint32_t page, uint32_t t) {
    return page * p.v_page + (t - div_T(p, t) * p.T) * p.v_tok;
}

KVB_HD bool vector_index_fits(const PoolLayer &p) {
    return (uint64_t)p.P * (p.s_page / p.B) < (1ull << 32);
}

// What a tile of query rows sees.  Row x of a request is query head x % group
// (of one KV head) of its new token x / group.
struct Span {
    int n, len, q0;      // new tokens, cached tokens, first query token
    int lo, hi;          // cached tokens [lo, hi) that some row of the tile sees
};

// Span of rows [rt * rows, (rt + 1) * rows) of a request with query tokens q0..q1
// and `len` cached tokens.  All three come from device memory and may be
// anything: they are brought into range before they index memory (*bad says
// that they were not).
KVB_HD Span row_span(int q0, int q1, int len, int tokens, int max_q, int max_len, int group,
                     int window, int rt, int rows, bool *bad) {
    Span s;
    const bool out = q0 < 0 || q1 < q0 || q1 > tokens || q1 - q0 > max_q;
    *bad = out || len < 0 || len > max_len;
    s.q0 = out ? 0 : q0;
    s.n = out ? 0 : q1 - q0;
    s.len = len < 0 ? 0 : len > max_len ? max_len : len;
    const int first = rt * rows / group;
    int last = ((rt + 1) * rows - 1) / group;
    if (last > s.n - 1) last = s.n - 1;
    s.hi = s.len - s.n + last + 1;               // at most len
    s.lo = window ? s.len - s.n + first - window + 1 : 0;
    if (s.lo < 0) s.lo = 0;
    if (first >= s.n || s.hi < 0) s.hi = 0;
    if (s.lo > s.hi) s.lo = s.hi;
    return s;
}

// The largest and least steps of a request are found kStepTokens tokens at a time, over all that its
// rows together see (a window and its new tokens, not only what one tile of rows sees).
constexpr uint32_t kStepTokens = 1024;
constexpr uint32_t kStepWords = 16;       // of a part and head: keys' and values' largest and least

KVB_HD uint32_t step_parts_of(uint32_t max_len, uint32_t window, uint32_t max_q) {
    uint64_t span = max_len;
    if (window && (uint64_t)window + max_q - 1 < span) span = (uint64_t)window + max_q - 1;
    const uint32_t parts = (uint32_t)((span + kStepTokens - 1) / kStepTokens);
    return parts != 0 ? parts : 1;
}

// ------------------------------------------------------------ 4-bit format

constexpr uint32_t kGroup = 32;           // values of one scale word
constexpr uint32_t kNanWord = 0x7fc00000u;

#ifdef __CUDA_ARCH__
KVB_HD float f_mul(float a, float b) { return __fmul_rn(a, b); }
KVB_HD float f_sub(float a, float b) { return __fsub_rn(a, b); }
KVB_HD float f_add(float a, float b) { return __fadd_rn(a, b); }
KVB_HD float f_fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
KVB_HD float f_bits(uint32_t u) { return __uint_as_float(u); }
KVB_HD uint32_t u_bits(float f) { return __float_as_uint(f); }
#else
// Host products and sums are kept apart (no contraction into one rounding).
KVB_HD float f_mul(float a, float b) { volatile float r = a * b; return r; }
KVB_HD float f_sub(float a, float b) { volatile float r = a - b; return r; }
KVB_HD float f_add(float a, float b) { volatile float r = a + b; return r; }
KVB_HD float f_fma(float a, float b, float c) { return std::fma(a, b, c); }
KVB_HD float f_bits(uint32_t u) { float f; std::memcpy(&f, &u, 4); return f; }
KVB_HD uint32_t u_bits(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
#endif

// The step s of a group as a float32 with its low four bits clear (0: the
// group is held as zeros), from lo = min(0, x...) and hi = max(0, x...), finite.
KVB_HD uint32_t q4_step_bits(float lo, float hi) {
    const float r15 = f_bits(0x3d888889u);   // 1/15
    const uint32_t b = (u_bits(f_sub(f_mul(hi, r15), f_mul(lo, r15))) + 8u) & ~15u;
    return f_bits(b) < f_bits(0x0d800000u) ? 0u : b;   // under 2^-100: zeros
}

// round(x / s), ties to even, exactly, for |x / s| < 17.  x * inv (inv = 1/s) is
// within a few units in the last place of the quotient, so its rounding r (by
// adding and taking off 1.5 x 2^23) is right or, next to a half-way point, one
// off.  e = x - r s is exact in one fma: it is at most about s/2, and r s and x
// are multiples of 2^-23 s or r is 0.  Where |e| passes s/2, or meets it with r
// odd, r moves by one towards x.
KVB_HD float q4_round(float x, float s, float inv) {
    const float t = f_fma(x, inv, 12582912.0f);
    const float r = f_sub(t, 12582912.0f), h = 0.5f * s;
    const float e = f_fma(-r, s, x), a = fabsf(e);
    const bool odd = (u_bits(t) & 1u) != 0;
    return a > h || (a == h && odd) ? f_add(r, copysignf(1.0f, e)) : r;
}

KVB_HD float q4_zero(float lo, float s, float inv) { return fminf(q4_round(-lo, s, inv), 15.0f); }

// A code as a float.  x >= lo, so that round(x / s) >= -round(-lo / s): never below 0.
KVB_HD float q4_code(float x, float s, float inv, float z) {
    return fminf(f_add(q4_round(x, s, inv), z), 15.0f);
}

// Four codes as 16 bits: their sum below 2^16 is exact.
KVB_HD uint32_t q4_pack(const float *c) {
    return u_bits(f_add(f_fma(f_fma(f_fma(c[3], 16.0f, c[2]), 16.0f, c[1]), 16.0f, c[0]), 8388608.0f)) &
           0xffffu;
}

KVB_HD float q4_step(uint32_t word) { return f_bits(word & ~15u); }

// ------------------------------------------------------- parameter blocks

struct Vecs {
    uint64_t data;
    int64_t s_tok, s_head;    // bytes
};

constexpr int kMaxPairs = 128;

// Turns per position of each pair as 64-bit fractions: the phase of position p
// is p * turns mod 2^64, where integer arithmetic wraps at one whole turn without
// error.  What is left is the fraction's own error, that of a frequency in 53 bits:
// 2^-53 x p x frequency radians (1e-4 at p = 2^40 for a frequency of 1).
struct RotaryK {
    unsigned long long turns[kMaxPairs];
    float gain;
    uint32_t half, style;     // pairs; kv_rotary_style
};

struct VectorArgs {
    Vecs q, q_out, k, v;      // heads of q first, then k, then v
    const int64_t *positions;
    const float *rows_in;
    float *rows_out;
    const int64_t *slots;
    uint32_t *status;
    PoolLayer pool;
    uint32_t tokens, q_heads, kv_heads, D;
    uint32_t half, style;     // half = 0: no rotation
    uint32_t per_block;       // vectors a block handles per token
    uint32_t token_a_warp;    // a warp handles a token by itself
    float k_inv, v_inv;       // E4M3: 1 / scale (append), scale (fetch)
    float sin_sign;
};

struct AttendArgs {
    Vecs q, out;
    float *lse;
    const int32_t *q_start, *lens, *pages;
    int64_t pages_stride;
    float *part_o;            // [chunks][tokens][q_heads][D] partial sums
    float *part_ml;           // [chunks][tokens][q_heads][2] maxima (base 2), sums
    uint32_t *status;
    PoolLayer pool;
    uint32_t requests, tokens, max_q, max_len, q_heads, group;
    uint32_t chunk, chunks;   // cached tokens a block handles; the most of one request
    uint32_t row_tiles;
    uint32_t whole_units;     // many rows: units (row tile, head, request) that are not cut
    uint32_t *steps;          // many rows: [requests][step_parts][H][2][largest 4, least 4] steps
    uint32_t step_parts;
    uint32_t *uneven;         // many rows: [requests][H] 1 where steps differ too much for fp16
    uint32_t window;
    float scale_log2;         // scale * log2(e)
};

}  // namespace kvb
