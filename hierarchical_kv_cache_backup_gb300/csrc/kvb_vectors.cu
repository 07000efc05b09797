// kvb_vectors.cu -- kernels that write and read single head vectors: rotation
// and append (one kernel family) and fetch.  Both are bound by memory: every
// value is read once and written once, the arithmetic hides behind it.
#include "kvb_vec.h"
#include "kvb_vec_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace kvb {

namespace {

constexpr int kThreads = 128;
constexpr uint32_t kTokenAWarp = 4096;   // tokens from which a warp takes one by itself

template <bool kHalf>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    if (kHalf) return __half22float2(*reinterpret_cast<__half2 *>(&u));
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (kHalf) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

template <bool kHalf>
__device__ __forceinline__ void unpack8(uint4 u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<kHalf>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <bool kHalf>
__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack2<kHalf>(x[0], x[1]), pack2<kHalf>(x[2], x[3]), pack2<kHalf>(x[4], x[5]),
                      pack2<kHalf>(x[6], x[7]));
}

template <bool kHalf>
__device__ __forceinline__ float one(uint64_t p) {
    const uint32_t u = *reinterpret_cast<const unsigned short *>(p);
    return unpack2<kHalf>(u).x;
}

// 8 values of one vector in the pool's format.  Q4: the four lanes of a group of
// 32 values are neighbours in the warp (every lane of the warp takes part in
// the exchange; `on` says whether this one stores).
template <int kFormat, bool kHalf>
__device__ __forceinline__ void store8(uint64_t vec, uint32_t chunk, const float *y, uint32_t D,
                                       uint32_t B, float inv_scale, bool on) {
    if (kFormat == 1) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(y[2 * i], inv_scale),
                                                        __fmul_rn(y[2 * i + 1], inv_scale)),
                                            __NV_SATFINITE, __NV_E4M3);
        if (on)
            *reinterpret_cast<uint2 *>(vec + chunk * 8) =
                make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    } else {
        float lo = 0.0f, hi = 0.0f, bad = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, y[i]);
            hi = fmaxf(hi, y[i]);
            bad = __fmaf_rn(y[i], 0.0f, bad);   // NaN once a value is not finite
        }
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, s));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, s));
            bad += __shfl_xor_sync(0xffffffffu, bad, s);
        }
        uint32_t word = bad == 0.0f ? q4_step_bits(lo, hi) : kNanWord, codes = 0;
        if (bad == 0.0f && word != 0) {
            const float s = __uint_as_float(word), inv = __frcp_rn(s);
            const float z = q4_zero(lo, s, inv);
            float c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = q4_code(y[i], s, inv, z);
            codes = q4_pack(c) | q4_pack(c + 4) << 16;
            word |= (uint32_t)z;
        }
        if (on) {
            *reinterpret_cast<uint32_t *>(vec + chunk * 4) = codes;
            if ((chunk & 3) == 0) *reinterpret_cast<uint32_t *>(vec + D / 2 + chunk) = word;
            if (chunk == 0)
                for (uint32_t at = D / 2 + D / 8; at < B; at += 4)
                    *reinterpret_cast<uint32_t *>(vec + at) = 0;
        }
    }
}

// ------------------------------------------------------- rotate and append
//
// With many tokens a warp takes one token and all its vectors (what a token costs
// once -- its slot, cosines and sines -- is then paid once); with few, a block takes
// one token and `per_block` of its vectors.  Queries come first, then keys, then
// values.  A lane owns the same values of every vector that it
// meets, so the token's cosines and sines go to registers once and serve all
// heads.  Vectors never straddle warps, and a warp loads before it stores, so
// a vector may be turned in place.
//
// kPair: a lane owns two runs of 8 values (16 bytes each): in HALF style a run of
// first members and the run of their partners, so that each line is loaded and
// unpacked once; in INTERLEAVED style and past the rotated part, two runs that
// are as far apart.  Four neighbouring lanes still hold the 32 values of a
// 4-bit group when rotated and other part are multiples of 64 values.  Where
// they are not (or not of 16 for the other formats), a lane owns one run and
// reads its partners itself (!kPair).  8,192 tokens of 40 vectors of 128: 31.5
// us (5.5 TB/s, bound by memory), 52 with one run a lane, bound by instructions.
// kFormat: -1 rotate only, else kv_cache_format.  Quantising takes 87 registers where
// it may; seven blocks an SM (72 registers) hide more: append and fetch of 8,192
// tokens 53.7 -> 50 us (the append 38.5, 4.7 TB/s of what it reads and writes, 53% of the ALU pipe).
template <int kFormat, bool kHalf, bool kPair>
__global__ void __launch_bounds__(kThreads, kFormat == 2 ? 7 : 1) kv_vectors_kernel(const __grid_constant__ VectorArgs a,
                                                              const __grid_constant__ RotaryK r) {
    constexpr int kRuns = kPair ? 2 : 1;
    __shared__ __align__(16) float all_rows[kThreads / 32][2][kMaxPairs];
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool alone = a.token_a_warp != 0;           // this warp has a token to itself
    const uint32_t token = alone ? blockIdx.x * (kThreads / 32) + warp : blockIdx.x;
    if (token >= a.tokens) return;
    float(*rows)[kMaxPairs] = all_rows[alone ? warp : 0];
    const uint32_t first = alone ? lane : threadIdx.x, stride = alone ? 32 : kThreads;
    const uint32_t per_vec = a.D / (8 * kRuns), per_warp = 32 / per_vec;
    const uint32_t sub = lane / per_vec, place = lane - sub * per_vec;
    const uint32_t half = a.half, total = a.q_heads + 2 * a.kv_heads;
    // this lane's runs, in units of 8 values
    const uint32_t turned_places = 2 * half / (8 * kRuns);
    const bool turned = kPair ? place < turned_places : place * 8 < 2 * half;
    uint32_t run[kRuns];
    run[0] = kPair && !turned ? 2 * turned_places + (place - turned_places) : place;
    if (kPair) run[kRuns - 1] = run[0] + (turned ? turned_places : per_vec - turned_places);
    asm volatile("griddepcontrol.wait;" ::: "memory");

    int64_t off = -1, slot = -1;
    if (kFormat >= 0) slot = a.slots[token];
    for (uint32_t i = first; i < half; i += stride) {
        float c, s;
        if (kFormat == -1 && a.positions != nullptr) {
            // the phase as a signed 64-bit fraction of a turn, then in half turns
            const unsigned long long p = (unsigned long long)a.positions[token] * r.turns[i];
            const float t = __ll2float_rn((long long)p) * 1.08420217e-19f;   // 2^-63
            sincospif(t, &s, &c);
            c *= r.gain;
            s *= r.gain;
            if (a.rows_out != nullptr && blockIdx.y == 0) {
                float *out = a.rows_out + (uint64_t)token * 2 * half;
                out[i] = c;
                out[half + i] = s;
            }
        } else {
            const float *in = a.rows_in + (uint64_t)token * 2 * half;
            c = in[i];
            s = in[half + i];
        }
        rows[0][i] = c;
        rows[1][i] = kFormat == -1 ? s * a.sin_sign : s;
    }
    if (kFormat >= 0) {
        off = slot_offset(a.pool, slot);
        if (off < 0 && slot != -1 && a.status != nullptr && first == 0 && blockIdx.y == 0)
            atomicOr(a.status, KV_STATUS_BAD_SLOT);
    }
    if (alone)
        __syncwarp();
    else
        __syncthreads();

    // cosines and sines of this lane's values: kPair HALF 8 pairs; kPair
    // INTERLEAVED 4 pairs of each run; else one for each value, signed
    const bool aligned = a.style == 1 || (half & 7) == 0;
    float cs[8], sn[8];
    if (turned) {
        if (kPair) {
            const uint32_t i0 = a.style == 1 ? run[0] * 4 : place * 8;
            const uint32_t i1 = a.style == 1 ? run[kRuns - 1] * 4 : place * 8 + 4;
            *reinterpret_cast<float4 *>(cs) = *reinterpret_cast<const float4 *>(&rows[0][i0]);
            *reinterpret_cast<float4 *>(cs + 4) = *reinterpret_cast<const float4 *>(&rows[0][i1]);
            *reinterpret_cast<float4 *>(sn) = *reinterpret_cast<const float4 *>(&rows[1][i0]);
            *reinterpret_cast<float4 *>(sn + 4) = *reinterpret_cast<const float4 *>(&rows[1][i1]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t d = place * 8 + e;
                cs[e] = 1.0f;
                sn[e] = 0.0f;
                if (d < 2 * half) {
                    const bool second = a.style == 1 ? (d & 1) : d >= half;
                    const uint32_t i = a.style == 1 ? d >> 1 : second ? d - half : d;
                    cs[e] = rows[0][i];
                    sn[e] = second ? rows[1][i] : -rows[1][i];
                }
            }
        }
    }

    // y <- this lane's values of a vector, turned
    auto turn = [&](const uint4 *own, uint64_t src, float(*y)[8]) {
        float x[2][8];
        unpack8<kHalf>(own[0], x[0]);
        unpack8<kHalf>(own[1], x[1]);
        if (kPair && a.style == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[0][e] = __fsub_rn(__fmul_rn(x[0][e], cs[e]), __fmul_rn(x[1][e], sn[e]));
                y[kRuns - 1][e] = __fadd_rn(__fmul_rn(x[0][e], sn[e]), __fmul_rn(x[1][e], cs[e]));
            }
        } else if (kPair) {
#pragma unroll
            for (int k = 0; k < kRuns; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = x[k][2 * e], w = x[k][2 * e + 1];
                    const float c = cs[4 * k + e], s = sn[4 * k + e];
                    y[k][2 * e] = __fsub_rn(__fmul_rn(u, c), __fmul_rn(w, s));
                    y[k][2 * e + 1] = __fadd_rn(__fmul_rn(u, s), __fmul_rn(w, c));
                }
        } else {
            if (a.style == 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[1][e] = x[0][e ^ 1];
            } else if (!aligned) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t d = place * 8 + e;
                    x[1][e] = d < 2 * half ? one<kHalf>(src + (d < half ? d + half : d - half) * 2) : 0.0f;
                }
            }
            // values past the rotated part keep their bits
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[0][e] = place * 8 + e < 2 * half
                              ? __fadd_rn(__fmul_rn(x[0][e], cs[e]), __fmul_rn(x[1][e], sn[e]))
                              : x[0][e];
        }
    };
    auto read = [&](uint4 *own, uint64_t src, bool partners) {
        own[0] = *reinterpret_cast<const uint4 *>(src + run[0] * 16);
        if (kPair)
            own[1] = *reinterpret_cast<const uint4 *>(src + run[kRuns - 1] * 16);
        else if (partners && a.style == 0 && aligned)
            own[1] = *reinterpret_cast<const uint4 *>(
                src + (place * 8 < half ? place * 8 + half : place * 8 - half) * 2);
    };

    // the vectors of this block, or of the token; this warp's first and its step
    const uint32_t lo = alone ? 0 : blockIdx.y * a.per_block;
    const uint32_t hi = alone ? total : min(total, (blockIdx.y + 1) * a.per_block);
    const uint32_t at = alone ? 0 : warp * per_warp, step = alone ? per_warp : per_warp * (kThreads / 32);
    constexpr int kBatch = 2;   // vectors in flight per lane

    const uint32_t q_end = min(hi, a.q_heads);
    if (lo + at < q_end) {
        uint64_t src = a.q.data + (int64_t)token * a.q.s_tok + (int64_t)(lo + at + sub) * a.q.s_head;
        uint64_t dst = a.q_out.data + (int64_t)token * a.q_out.s_tok + (int64_t)(lo + at + sub) * a.q_out.s_head;
        const int64_t src_step = (int64_t)step * a.q.s_head, dst_step = (int64_t)step * a.q_out.s_head;
        for (uint32_t v0 = lo + at; v0 < q_end; v0 += kBatch * step) {
            uint4 own[kBatch][2];
            bool live[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                live[b] = sub < per_warp && v0 + b * step + sub < q_end;
                own[b][0] = own[b][1] = make_uint4(0, 0, 0, 0);
                if (live[b]) read(own[b], src + b * src_step, turned);
            }
            __syncwarp();
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                float y[kRuns][8];
                if (turned && live[b]) turn(own[b], src + b * src_step, y);
                __syncwarp();      // unaligned partners are read by turn()
                if (live[b])
#pragma unroll
                    for (int k = 0; k < kRuns; ++k)
                        *reinterpret_cast<uint4 *>(dst + b * dst_step + run[k] * 16) =
                            turned ? pack8<kHalf>(y[k]) : own[b][k];
            }
            src += kBatch * src_step;
            dst += kBatch * dst_step;
        }
    }
    if (kFormat >= 0 && off >= 0) {
        for (uint32_t v0 = max(lo, a.q_heads) + at; v0 < hi; v0 += kBatch * step) {
            uint4 own[kBatch][2];
            uint64_t src[kBatch], vec[kBatch];
            bool live[kBatch], is_k[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const uint32_t u = v0 + b * step + sub - a.q_heads;
                is_k[b] = u < a.kv_heads;
                live[b] = sub < per_warp && v0 + b * step + sub < hi;
                const uint32_t h = is_k[b] ? u : u - a.kv_heads;
                src[b] = is_k[b] ? a.k.data + (int64_t)token * a.k.s_tok + (int64_t)h * a.k.s_head
                                 : a.v.data + (int64_t)token * a.v.s_tok + (int64_t)h * a.v.s_head;
                vec[b] = (is_k[b] ? a.pool.base[0] : a.pool.base[1]) + (uint64_t)off +
                         (uint64_t)h * a.pool.s_head;
                own[b][0] = own[b][1] = make_uint4(0, 0, 0, 0);
                if (live[b]) read(own[b], src[b], turned && is_k[b]);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (v0 + b * step >= hi) break;        // the whole warp
                const bool to_turn = turned && is_k[b];
                float y[kRuns][8];
                unpack8<kHalf>(own[b][0], y[0]);
                if (kPair) unpack8<kHalf>(own[b][1], y[kRuns - 1]);
                if (to_turn && live[b]) turn(own[b], src[b], y);
                if (kFormat == 0) {
                    if (live[b])
#pragma unroll
                        for (int k = 0; k < kRuns; ++k)
                            *reinterpret_cast<uint4 *>(vec[b] + run[k] * 16) =
                                to_turn ? pack8<kHalf>(y[k]) : own[b][k];
                } else {
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < kRuns; ++k)
                        store8<kFormat, kHalf>(vec[b], run[k], y[k], a.D, a.pool.B,
                                               is_k[b] ? a.k_inv : a.v_inv, live[b]);
                }
            }
        }
    }
}

// -------------------------------------------------------------------- fetch
//
// The same mapping, a lane 8 values of a vector.  Bound by the latency of a token's
// two dependent reads (slot, then vectors): 8,192 tokens of 16 vectors of 128 in 4 bits,
// 12 us.
template <int kFormat, bool kHalf>
__global__ void __launch_bounds__(kThreads) kv_fetch_kernel(const __grid_constant__ VectorArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool alone = a.token_a_warp != 0;
    const uint32_t token = alone ? blockIdx.x * (kThreads / 32) + warp : blockIdx.x;
    if (token >= a.tokens) return;
    const uint32_t per_vec = a.D / 8, per_warp = 32 / per_vec;
    const uint32_t sub = lane / per_vec, chunk = lane - sub * per_vec;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t slot = a.slots[token];
    const int64_t off = slot_offset(a.pool, slot);
    if (off < 0 && slot != -1 && a.status != nullptr && (alone ? lane : threadIdx.x) == 0 && blockIdx.y == 0)
        atomicOr(a.status, KV_STATUS_BAD_SLOT);
    if (sub >= per_warp) return;
    const uint32_t lo = alone ? 0 : blockIdx.y * a.per_block + warp * per_warp;
    const uint32_t end = alone ? 2 * a.kv_heads : min(2 * a.kv_heads, (blockIdx.y + 1) * a.per_block);
    const uint32_t step = alone ? per_warp : per_warp * (kThreads / 32);
#pragma unroll 4
    for (uint32_t v = lo + sub; v < end; v += step) {
        const bool is_k = v < a.kv_heads;
        const uint32_t h = is_k ? v : v - a.kv_heads;
        const Vecs &x = is_k ? a.k : a.v;
        if (x.data == 0) continue;
        const uint64_t vec = a.pool.base[is_k ? 0 : 1] + (uint64_t)off + (uint64_t)h * a.pool.s_head;
        uint4 out = make_uint4(0, 0, 0, 0);
        if (off >= 0) {
            if (kFormat == 0) {
                out = *reinterpret_cast<const uint4 *>(vec + chunk * 16);
            } else {
                float y[8];
                if (kFormat == 1) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(vec + chunk * 8);
                    const float s = is_k ? a.k_inv : a.v_inv;
                    const uint32_t u[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u[i],
                                                                    __NV_E4M3);
                        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&hr));
                        y[2 * i] = __fmul_rn(f.x, s);
                        y[2 * i + 1] = __fmul_rn(f.y, s);
                    }
                } else {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(vec + chunk * 4);
                    const uint32_t word =
                        *reinterpret_cast<const uint32_t *>(vec + a.D / 2 + (chunk & ~3u));
                    // code x 2^-24 as fp16 subnormals; (code - z) s has at most 24 bits, and so
                    // have code x s and z x s: one fma gives it exactly
                    const float s = q4_step(word), less = -(float)(word & 15u) * s;
                    const float s24 = s * 16777216.0f, s20 = s * 1048576.0f;
                    const uint32_t u = w >> 8;
                    const uint32_t p[4] = {w & 0x000f000fu, w & 0x00f000f0u, u & 0x000f000fu, u & 0x00f000f0u};
                    if (s < 1e30f) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 c = __half22float2(*reinterpret_cast<const __half2 *>(&p[i]));
                            y[i] = __fmaf_rn(c.x, i & 1 ? s20 : s24, less);
                            y[i + 4] = __fmaf_rn(c.y, i & 1 ? s20 : s24, less);
                        }
                    } else {        // s x 2^24 would pass float32, or s is NaN
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[i] = __fmul_rn((float)((w >> (4 * i)) & 15u) - (float)(word & 15u), s);
                    }
                }
                out = pack8<kHalf>(y);
            }
        }
        const uint64_t dst = x.data + (int64_t)token * x.s_tok + (int64_t)h * x.s_head;
        *reinterpret_cast<uint4 *>(dst + chunk * 16) = out;
    }
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, cudaStream_t stream, bool pdl, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

typedef void (*VectorsFn)(VectorArgs, RotaryK);   // [format + 1][pair][fp16]
typedef void (*FetchFn)(VectorArgs);
#define KVB_VECTORS(F)                                                        \
    {{kv_vectors_kernel<F, false, false>, kv_vectors_kernel<F, true, false>}, \
     {kv_vectors_kernel<F, false, true>, kv_vectors_kernel<F, true, true>}}
const VectorsFn kVectors[4][2][2] = {KVB_VECTORS(-1), KVB_VECTORS(0), KVB_VECTORS(1), KVB_VECTORS(2)};
const FetchFn kFetch[3][2] = {{kv_fetch_kernel<0, false>, kv_fetch_kernel<0, true>},
                              {kv_fetch_kernel<1, false>, kv_fetch_kernel<1, true>},
                              {kv_fetch_kernel<2, false>, kv_fetch_kernel<2, true>}};

// With tokens enough a warp takes a token (append and fetch of 8,192 tokens 61 ->
// 54 us, of 5,000 28.5 -> 25.9, but of 2,000 19 -> 24); with fewer, a block takes so few of a token's vectors that the blocks fill the
// GPU (its 4 warps take 4 x per_warp at a time; lanes is what a vector takes of a
// warp).  Returns the grid.
dim3 grid_of(VectorArgs *a, uint32_t vectors, uint32_t lanes) {
    const uint32_t at_once = (32 / lanes) * (kThreads / 32);
    uint32_t steps = (vectors + at_once - 1) / at_once;
    if (steps < 1) steps = 1;   // rows of angles alone
    a->token_a_warp = a->tokens >= kTokenAWarp;
    if (a->token_a_warp) return dim3((a->tokens + kThreads / 32 - 1) / (kThreads / 32));
    const uint64_t blocks = (uint64_t)a->tokens * steps;
    uint64_t each = blocks / (152 * 8);
    if (each < 1) each = 1;
    if (each > steps) each = steps;
    a->per_block = (uint32_t)each * at_once;
    const uint32_t y = (vectors + a->per_block - 1) / a->per_block;
    return dim3(a->tokens, y != 0 ? y : 1);
}

}  // namespace

cudaError_t launch_vectors(VectorArgs a, const RotaryK &r, int format, bool fp16, bool pdl,
                           cudaStream_t stream) {
    (void)cudaGetLastError();
    const uint32_t vectors = a.q_heads + 2 * a.kv_heads;
    // two runs a lane where rotated and other part divide into pairs of runs, and, for
    // 4-bit groups, four lanes at a time
    const uint32_t unit = format == KV_CACHE_Q4 ? 64 : 16;
    const bool pair = 2 * a.half % unit == 0 && (a.D - 2 * a.half) % unit == 0;
    const dim3 grid = grid_of(&a, vectors, a.D / (pair ? 16 : 8));
    return launch(kVectors[format + 1][pair][fp16], grid, stream, pdl, a, r);
}

cudaError_t launch_fetch(VectorArgs a, int format, bool fp16, bool pdl, cudaStream_t stream) {
    (void)cudaGetLastError();
    const dim3 grid = grid_of(&a, 2 * a.kv_heads, a.D / 8);
    return launch(kFetch[format][fp16], grid, stream, pdl, a);
}

cudaError_t preload_vector_kernels() {
    cudaFuncAttributes at;
    for (auto &format : kVectors)
        for (auto &row : format)
            for (auto f : row) {
                const cudaError_t e = cudaFuncGetAttributes(&at, (const void *)f);
                if (e != cudaSuccess) return e;
            }
    for (auto &row : kFetch)
        for (auto f : row) {
            const cudaError_t e = cudaFuncGetAttributes(&at, (const void *)f);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

}  // namespace kvb
