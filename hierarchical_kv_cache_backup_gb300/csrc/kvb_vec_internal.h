// kvb_vec_internal.h -- host entry points of the head-vector kernels, and what
// the engine (kvb_api.cpp) gives their C ABI (kvb_vec.cpp).
#pragma once

#include "kvb.h"
#include "kvb_internal.h"
#include "kvb_vec.h"

namespace kvb {

cudaError_t launch_vectors(VectorArgs a, const RotaryK &r, int format, bool fp16, bool pdl,
                           cudaStream_t stream);
cudaError_t launch_fetch(VectorArgs a, int format, bool fp16, bool pdl, cudaStream_t stream);
cudaError_t preload_vector_kernels();

// How kv_attend cuts a call: cached tokens a block takes and the most blocks
// along the tokens of one request, query rows a block takes, and workspace.
struct AttendPlan {
    uint32_t rows, row_tiles, chunk, chunks;
    bool many;             // the kernel for many query rows (kvb_attend_tc.cu)
    uint64_t whole_units;  // many: units that are not cut
    uint32_t step_parts;   // many: parts of a request whose steps are looked over apart
    uint64_t step_bytes;   // workspace of those, and of what they find, at its start
    uint32_t uneven_blocks;// many: blocks a head and request for those whose steps differ too much
    uint64_t bytes;        // workspace in all
};
AttendPlan plan_attend(uint32_t requests, uint32_t tokens, uint32_t max_q, uint32_t max_len,
                       uint32_t window, uint32_t q_heads, uint32_t kv_heads, uint32_t D, int sms);
cudaError_t launch_attend(const AttendArgs &a, const AttendPlan &p, uint32_t D, bool fp16, bool pdl,
                          cudaStream_t stream, int *launches);
cudaError_t preload_attend_kernels();
void plan_attend_tc(AttendPlan *p, uint64_t span, uint32_t requests, uint32_t kv_heads, int sms);
// What launch_attend_tc leaves to the kernel for few rows (a.uneven).
cudaError_t launch_attend_uneven(const AttendArgs &a, const AttendPlan &p, uint32_t D, bool fp16, bool pdl,
                                 cudaStream_t stream);
cudaError_t launch_attend_tc(const AttendArgs &a, uint32_t D, bool fp16, bool pdl, cudaStream_t stream,
                             int *launches);
cudaError_t preload_attend_tc_kernels();

// Handle checks of one operator call on a pool (CLOSED / STALE) and its device
// made ready; vec_begin ends a run of overlapped restores on `stream`.
struct VecPool {
    kv_layout layout;
    uint64_t base[2];      // component bases of the layer
    uint64_t s_page;
    int device, sms;
    bool pdl;
};
int vec_enter_pool(const void *pool_handle, uint32_t layer, VecPool *out);
void vec_begin(int device, void *stream);
int vec_enter_device(int device, void *stream, bool *pdl);
int vec_cuda_error(cudaError_t e, const char *what);
void vec_count(int launches);

}  // namespace kvb
