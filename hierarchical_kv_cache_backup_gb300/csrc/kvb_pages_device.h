// kvb_pages_device.h -- device code that the two attention kernels over 16-bit and fp8 pages share.
#pragma once

#include "kvb.h"
#include "kvb_pages.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace kvb {

// two fp8 values as fp16, exact
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)w));
    return r;
}
template <bool kBf>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (kBf) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}
template <bool kBf>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (kBf) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
// which 16-bit or fp8 values of a word are not finite, as a mask of their bits
template <bool kF8, bool kBf>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    if (kF8) return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
    const uint32_t e = kBf ? 0x7f807f80u : 0x7c007c00u;
    return __vcmpeq2(w & e, e);
}

// Up to this many segments a warp finds its worker's first tile by itself.
constexpr uint32_t kWarpSegs = 128;

__device__ __forceinline__ unsigned long long scan_add(unsigned long long x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// A warp sums tiles and units of all segments and finds the segment of `worker`'s first tile;
// with `record` it writes the sums before each segment to the workspace, for the join, and
// reports what is out of range.  Returns the tiles of a worker, *total the tiles of all (0 where
// the units pass the workspace's room).
__device__ __forceinline__ unsigned long long warp_share(const PageAttendArgs &a, const PageEngine &e, uint32_t worker, bool record,
                                                         PageCursor *start, unsigned long long *total) {
    const int lane = threadIdx.x & 31;
    const uint32_t n = seg_count(a, e);
    unsigned long long all_t = 0, all_u = 0, t = 0, u = 0;
    auto segment = [&](uint32_t s, bool report) {
        t = u = 0;
        if (s >= n) return;
        const PageSeg g = seg_at(a, e, s);
        t = seg_tiles(a, e, g);
        u = t != 0 ? (unsigned long long)row_tiles(a, e, g) * a.pool.H : 0;
        if (g.bad && report && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
    };
    for (uint32_t s0 = 0; s0 < n; s0 += 32) {
        segment(s0 + lane, record);
        all_t += t;
        all_u += u;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        all_t += __shfl_xor_sync(0xffffffffu, all_t, d);
        all_u += __shfl_xor_sync(0xffffffffu, all_u, d);
    }
    if (record && lane == 0) {
        e.seg_tiles[n] = all_t;
        e.seg_units[n] = all_u;
        if (all_u > e.units && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
    }
    if (all_u > e.units) all_t = 0;
    *total = all_t;
    const unsigned long long share = share_of(all_t, e.workers), x = worker * share;
    unsigned long long before_t = 0, before_u = 0;
    for (uint32_t s0 = 0; s0 < n; s0 += 32) {
        if (n > 32) segment(s0 + lane, false);
        const unsigned long long it = scan_add(t, lane), iu = scan_add(u, lane);
        const unsigned long long bt = before_t + it - t, bu = before_u + iu - u;
        if (record && s0 + lane < n) {
            e.seg_tiles[s0 + lane] = bt;
            e.seg_units[s0 + lane] = bu;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, x >= bt && x < bt + t);
        if (in != 0) {
            const int l = __ffs(in) - 1;
            start->tiles = __shfl_sync(0xffffffffu, bt, l);
            start->units = __shfl_sync(0xffffffffu, bu, l);
            start->seg = s0 + l;
            if (!record) break;
        }
        before_t += __shfl_sync(0xffffffffu, it, 31);
        before_u += __shfl_sync(0xffffffffu, iu, 31);
    }
    return share;
}

// The same over a block, for any number of segments and the block's workers, worker0 and the
// next; worker 0's block records.
template <int kThreads>
__device__ __forceinline__ unsigned long long share_out(const PageAttendArgs &a, const PageEngine &e, uint32_t worker0,
                                                        uint32_t workers_here, PageCursor *starts, unsigned long long *total) {
    constexpr int kW = kThreads / 32;
    __shared__ unsigned long long sums[2][kW];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t n = seg_count(a, e);
    unsigned long long share = 0, all_t = 0;
    for (int pass = 0; pass < 2; ++pass) {
        unsigned long long run_t = 0, run_u = 0;
        for (uint32_t s0 = 0; s0 < n; s0 += kThreads) {
            const uint32_t s = s0 + tid;
            unsigned long long t = 0, u = 0;
            if (s < n) {
                const PageSeg g = seg_at(a, e, s);
                t = seg_tiles(a, e, g);
                u = t != 0 ? (unsigned long long)row_tiles(a, e, g) * a.pool.H : 0;
                if (g.bad && pass == 0 && worker0 == 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
            }
            unsigned long long it = t, iu = u;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned long long xt = __shfl_up_sync(0xffffffffu, it, d), xu = __shfl_up_sync(0xffffffffu, iu, d);
                if (lane >= d) {
                    it += xt;
                    iu += xu;
                }
            }
            __syncthreads();
            if (lane == 31) {
                sums[0][warp] = it;
                sums[1][warp] = iu;
            }
            __syncthreads();
            unsigned long long bt = run_t, bu = run_u;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                if (w < warp) {
                    bt += sums[0][w];
                    bu += sums[1][w];
                }
                run_t += sums[0][w];
                run_u += sums[1][w];
            }
            if (pass == 1 && s < n) {
                const unsigned long long before = bt + it - t;
                for (uint32_t k = 0; k < workers_here; ++k) {
                    const unsigned long long x = (worker0 + k) * share;
                    if (x >= before && x < before + t) starts[k] = PageCursor{before, bu + iu - u, s};
                }
                if (worker0 == 0) {
                    e.seg_tiles[s] = before;
                    e.seg_units[s] = bu + iu - u;
                }
            }
        }
        all_t = run_u > e.units ? 0 : run_t;
        share = share_of(all_t, e.workers);
        if (run_u > e.units && worker0 == 0 && tid == 0 && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
        if (pass == 1 && worker0 == 0 && tid == 0) {
            e.seg_tiles[n] = run_t;
            e.seg_units[n] = run_u;
        }
    }
    __syncthreads();
    *total = all_t;
    return share;
}

}  // namespace kvb
