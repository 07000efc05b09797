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

__device__ __forceinline__ unsigned long long scan_add(unsigned long long x, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// Groups that are out of range, where no segment of their own tells (a block's threads, one of all blocks).
__device__ __forceinline__ void report_groups(const PageAttendArgs &a) {
    if (!a.joined || a.status == nullptr) return;
    for (uint32_t g = threadIdx.x; g < a.groups; g += blockDim.x)
        if (prefix_seg(a, g).bad) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
}

// Fills a block's table of the call's segments: one thread a segment, one sum over four warps.  Block 0
// (`record`) writes what comes before each segment to the workspace, for the join, and reports what
// is out of range.  The table is there for all threads when it returns.
__device__ __forceinline__ void fill_table(const PageAttendArgs &a, const PageEngine &e, bool record, PageTableSpace &t) {
    __shared__ unsigned long long sums[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t n = seg_count(a, e);
    unsigned long long x = 0, sum = 0;           // tiles, and units in the high word
    if (record) report_groups(a);
    if (tid < (int)kPlanSegs) {
        if (tid < (int)n) {
            const PageSeg s = seg_at(a, e, tid);
            const uint64_t tiles = seg_tiles(a, e, s);
            x = pack_work(e, tiles, seg_units(a, e, s, tiles));
            put_seg(t.seg + tid * kSegWords, s);
            if (s.bad && record && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
        }
        sum = scan_add(x, lane);
        if (lane == 31) sums[warp] = sum;
    }
    __syncthreads();
    if (tid < (int)kPlanSegs) {
        for (int w = 0; w < warp; ++w) sum += sums[w];
        t.tiles[tid + 1] = (uint32_t)sum;
        t.units[tid + 1] = sum >> 32;
        if (tid == 0) t.tiles[0] = t.units[0] = 0;
        if (record && tid < (int)n) {
            if (!e.whole) {
                e.seg_tiles[tid + 1] = (uint32_t)sum;
                e.seg_units[tid + 1] = sum >> 32;
                if (tid == 0) e.seg_tiles[0] = e.seg_units[0] = 0;
            }
            if (tid + 1 == (int)n && (sum >> 32) > e.units && a.status != nullptr) atomicOr(a.status, KV_STATUS_BAD_LENGTH);
        }
    }
    __syncthreads();
}

// The table of a call, and a worker's run from *x to *x1, of tiles or whole units (nothing where the units pass the workspace's room).
__device__ __forceinline__ PageTable table_and_share(const PageAttendArgs &a, const PageEngine &e, bool record, uint32_t worker,
                                                     PageTableSpace &space, unsigned long long *x, unsigned long long *x1) {
    PageTable t{e.seg_tiles, e.seg_units, e.seg_table};
    if (e.small) {
        fill_table(a, e, record, space);
        t = PageTable{space.tiles, space.units, space.seg};
    }
    const uint32_t n = seg_count(a, e);
    const unsigned long long units = t.units[n], total = units > e.units ? 0 : e.whole ? units : t.tiles[n];
    const unsigned long long share = e.whole ? 1 : share_of(total, e.workers);
    *x = worker * share;
    *x1 = min(total, *x + share);
    return t;
}

}  // namespace kvb
