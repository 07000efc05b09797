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
// One block takes one token and `per_block` of its vectors (queries, keys and
// values in that order).  A lane owns the same values of every vector that it
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
// reads its partners itself (!kPair).  8,192 tokens of 40 vectors of 128: 52 us
// with one run a lane, bound by instructions.
// kFormat: -1 rotate only, else kv_cache_format.
template <int kFormat, bool kHalf, bool kPair>
__global__ void __launch_bounds__(kThreads) kv_vectors_kernel(const __grid_constant__ VectorArgs a,
                                                              const __grid_constant__ RotaryK r) {
    constexpr int kRuns = kPair ? 2 : 1;
    __shared__ __align__(16) float rows[2][kMaxPairs];
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t token = blockIdx.x;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    for (uint32_t i = threadIdx.x; i < half; i += kThreads) {
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
        if (off < 0 && slot != -1 && a.status != nullptr && threadIdx.x == 0 && blockIdx.y == 0)
            atomicOr(a.status, KV_STATUS_BAD_SLOT);
    }
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

    const uint32_t end = min(total, (blockIdx.y + 1) * a.per_block);
    constexpr int kBatch = 2;   // vectors in flight per lane
    for (uint32_t v0 = blockIdx.y * a.per_block + warp * per_warp; v0 < end;
         v0 += kBatch * per_warp * (kThreads / 32)) {
        uint4 own[kBatch][2];   // this lane's runs; !kPair: its run and the partners
        uint64_t src[kBatch];
        bool live[kBatch], turn[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const uint32_t v = v0 + b * per_warp * (kThreads / 32) + sub;
            const bool is_q = v < a.q_heads, is_k = !is_q && v < a.q_heads + a.kv_heads;
            live[b] = sub < per_warp && v < end && (is_q || off >= 0);
            turn[b] = live[b] && turned && (is_q || is_k);
            const Vecs &x = is_q ? a.q : is_k ? a.k : a.v;
            const uint32_t h = is_q ? v : is_k ? v - a.q_heads : v - a.q_heads - a.kv_heads;
            src[b] = x.data + (int64_t)token * x.s_tok + (int64_t)h * x.s_head;
            own[b][0] = own[b][1] = make_uint4(0, 0, 0, 0);
            if (live[b]) {
                own[b][0] = *reinterpret_cast<const uint4 *>(src[b] + run[0] * 16);
                if (kPair) own[b][1] = *reinterpret_cast<const uint4 *>(src[b] + run[kRuns - 1] * 16);
            }
            if (!kPair && turn[b] && a.style == 0 && aligned)
                own[b][1] = *reinterpret_cast<const uint4 *>(
                    src[b] + (place * 8 < half ? place * 8 + half : place * 8 - half) * 2);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const uint32_t v = v0 + b * per_warp * (kThreads / 32) + sub;
            const bool is_q = v < a.q_heads;
            float y[kRuns][8];
            const bool need = turn[b] || (kFormat > 0 && live[b] && !is_q);
            if (need) {
                float x[2][8];
                unpack8<kHalf>(own[b][0], x[0]);
                unpack8<kHalf>(own[b][1], x[1]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y[0][e] = x[0][e];
                    if (kPair) y[kRuns - 1][e] = x[1][e];
                }
                if (turn[b]) {
                    if (kPair && a.style == 0) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            y[0][e] = __fsub_rn(__fmul_rn(x[0][e], cs[e]), __fmul_rn(x[1][e], sn[e]));
                            y[kRuns - 1][e] = __fadd_rn(__fmul_rn(x[0][e], sn[e]),
                                                        __fmul_rn(x[1][e], cs[e]));
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
                                x[1][e] = d < 2 * half
                                              ? one<kHalf>(src[b] + (d < half ? d + half : d - half) * 2)
                                              : 0.0f;
                            }
                        }
                        // values past the rotated part keep their bits
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (place * 8 + e < 2 * half)
                                y[0][e] = __fadd_rn(__fmul_rn(x[0][e], cs[e]), __fmul_rn(x[1][e], sn[e]));
                    }
                }
            }
            __syncwarp();
            const bool is_k = !is_q && v < a.q_heads + a.kv_heads;
            if (live[b] && (is_q || kFormat == 0)) {
                uint64_t dst;
                if (is_q) {
                    dst = a.q_out.data + (int64_t)token * a.q_out.s_tok + (int64_t)v * a.q_out.s_head;
                } else {
                    const uint32_t h = is_k ? v - a.q_heads : v - a.q_heads - a.kv_heads;
                    dst = a.pool.base[is_k ? 0 : 1] + (uint64_t)off + (uint64_t)h * a.pool.s_head;
                }
#pragma unroll
                for (int k = 0; k < kRuns; ++k)
                    *reinterpret_cast<uint4 *>(dst + run[k] * 16) = turn[b] ? pack8<kHalf>(y[k])
                                                                            : own[b][k];
            }
            // a warp of queries only has nothing to hold
            if (kFormat > 0 && __any_sync(0xffffffffu, live[b] && !is_q)) {
                const uint32_t h = is_k ? v - a.q_heads : v - a.q_heads - a.kv_heads;
                const uint64_t vec = a.pool.base[is_k ? 0 : 1] + (uint64_t)off +
                                     (uint64_t)h * a.pool.s_head;
                if (!need)
#pragma unroll
                    for (int k = 0; k < kRuns; ++k)
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[k][e] = 0.0f;
#pragma unroll
                for (int k = 0; k < kRuns; ++k)
                    store8<kFormat, kHalf>(vec, run[k], y[k], a.D, a.pool.B, is_k ? a.k_inv : a.v_inv,
                                           live[b] && !is_q);
            }
        }
    }
}

// -------------------------------------------------------------------- fetch
//
// The same mapping: one block takes one token, a lane 8 values of a vector.
template <int kFormat, bool kHalf>
__global__ void __launch_bounds__(kThreads) kv_fetch_kernel(const __grid_constant__ VectorArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t token = blockIdx.x;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t per_vec = a.D / 8, per_warp = 32 / per_vec;
    const uint32_t sub = lane / per_vec, chunk = lane - sub * per_vec;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t slot = a.slots[token];
    const int64_t off = slot_offset(a.pool, slot);
    if (off < 0 && slot != -1 && a.status != nullptr && threadIdx.x == 0 && blockIdx.y == 0)
        atomicOr(a.status, KV_STATUS_BAD_SLOT);
    if (sub >= per_warp) return;
    const uint32_t end = min(2 * a.kv_heads, (blockIdx.y + 1) * a.per_block);
#pragma unroll 2
    for (uint32_t v = blockIdx.y * a.per_block + warp * per_warp + sub; v < end;
         v += per_warp * (kThreads / 32)) {
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
                    const float s = q4_step(word), z = (float)(word & 15u);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = __fmul_rn((float)((w >> (4 * i)) & 15u) - z, s);
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

// Vectors a block takes: all of a token's when there are tokens enough to fill
// the GPU, else so few that the blocks do (a block's 4 warps take
// 4 x per_warp at a time; lanes is what a vector takes of a warp).
uint32_t per_block_of(uint32_t tokens, uint32_t vectors, uint32_t lanes) {
    const uint32_t at_once = (32 / lanes) * (kThreads / 32);
    uint32_t steps = (vectors + at_once - 1) / at_once;
    if (steps < 1) steps = 1;   // rows of angles alone
    const uint64_t blocks = (uint64_t)tokens * steps;
    uint64_t each = blocks / (152 * 8);
    if (each < 1) each = 1;
    if (each > steps) each = steps;
    return (uint32_t)each * at_once;
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
    a.per_block = per_block_of(a.tokens, vectors, a.D / (pair ? 16 : 8));
    const uint32_t blocks = (vectors + a.per_block - 1) / a.per_block;
    const dim3 grid(a.tokens, blocks != 0 ? blocks : 1);   // no vectors: the rows alone
    return launch(kVectors[format + 1][pair][fp16], grid, stream, pdl, a, r);
}

cudaError_t launch_fetch(VectorArgs a, int format, bool fp16, bool pdl, cudaStream_t stream) {
    (void)cudaGetLastError();
    a.per_block = per_block_of(a.tokens, 2 * a.kv_heads, a.D / 8);
    const dim3 grid(a.tokens, (2 * a.kv_heads + a.per_block - 1) / a.per_block);
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
