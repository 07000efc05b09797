// kvb_pages_internal.h -- host entry points of the kernels on 16-bit and fp8 pages.
#pragma once

#include "kvb.h"
#include "kvb_internal.h"
#include "kvb_pages.h"
#include "kvb_pages_plan.h"

namespace kvb {

// Blocks of the kernel for few rows that an SM holds (set when the kernels are loaded).
uint32_t pages_blocks(uint32_t D, bool fp8);
cudaError_t launch_pages(const PageAttendArgs &a, const PagePlan &p, uint32_t D, bool fp8, bool fp16, bool pdl,
                         cudaStream_t stream, int *launches);
cudaError_t preload_pages_kernels();
cudaError_t launch_pages_tc(const PageAttendArgs &a, uint32_t D, bool fp8, bool fp16, bool pdl, cudaStream_t stream);
cudaError_t preload_pages_tc_kernels();

cudaError_t launch_bound(const BoundArgs &a, uint32_t D, bool fp8, bool fp16, bool pdl, int sms, cudaStream_t stream);
cudaError_t launch_select(const SelectArgs &a, uint32_t D, bool fp16, bool pdl, cudaStream_t stream, int *launches);
uint32_t select_block_pages(uint64_t pages, int sms);
cudaError_t preload_select_kernels();

}  // namespace kvb
