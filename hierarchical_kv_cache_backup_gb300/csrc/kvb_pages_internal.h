// kvb_pages_internal.h -- host entry points of the kernels on 16-bit and fp8 pages.
#pragma once

#include "kvb.h"
#include "kvb_internal.h"
#include "kvb_pages.h"

namespace kvb {

// How attention over 16-bit and fp8 pages cuts a call, and its workspace.
struct PagePlan {
    PageEngine rows, tc;      // pointers are offsets from the workspace's start
    uint64_t bytes;
    bool wide_join;           // a row may have many pieces
    uint32_t join_heads;      // rows that a warp of the join takes in turn
    bool joined;              // units of own tokens take the prefix too
};
PagePlan plan_pages(uint32_t requests, uint32_t tokens, uint32_t max_q, uint32_t max_len, uint32_t groups,
                    uint32_t max_group, uint32_t max_prefix, uint32_t budget, uint32_t T, uint32_t q_heads,
                    uint32_t kv_heads, uint32_t D, bool fp8, int sms);
cudaError_t launch_pages(const PageAttendArgs &a, const PagePlan &p, uint32_t D, bool fp8, bool fp16, bool pdl,
                         cudaStream_t stream, int *launches);
cudaError_t preload_pages_kernels();
// The kernel on tcgen05: query rows of its units, cached tokens of its tiles.
uint32_t pages_tc_rows(uint32_t D, uint64_t rows);
uint32_t pages_tc_shift();
cudaError_t launch_pages_tc(const PageAttendArgs &a, uint32_t D, bool fp8, bool fp16, bool pdl, cudaStream_t stream);
cudaError_t preload_pages_tc_kernels();

cudaError_t launch_bound(const BoundArgs &a, uint32_t D, bool fp8, bool fp16, bool pdl, int sms, cudaStream_t stream);
cudaError_t launch_select(const SelectArgs &a, uint32_t D, bool fp16, bool pdl, cudaStream_t stream, int *launches);
uint32_t select_block_pages(uint64_t pages, int sms);
cudaError_t preload_select_kernels();

}  // namespace kvb
