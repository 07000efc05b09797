// kvb_vec.cpp -- C ABI of the operators on single head vectors: kv_rotary_*,
// kv_rotate, kv_append, kv_fetch, kv_attend, kv_attend_shared, kv_bound, kv_select,
// kv_attend_selected.  Checks of arguments, frequencies, and the launch of each
// call; the kernels are in kvb_vectors.cu, kvb_attend.cu, kvb_pages.cu and
// kvb_select.cu.
#include "kvb.h"
#include "kvb_internal.h"
#include "kvb_pages_internal.h"
#include "kvb_vec.h"
#include "kvb_vec_internal.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <new>
#include <unordered_map>

using namespace kvb;

namespace {

kv_status fail(kv_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return (kv_status)set_last_error(st, buf);
}

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr uint32_t kMaxDim = 256;

std::mutex g_rot_mu;
std::unordered_map<uint64_t, RotaryK> g_rotary;
uint64_t g_next_rotary = 1;

bool find_rotary(kv_rotary h, RotaryK *out) {
    std::lock_guard<std::mutex> lk(g_rot_mu);
    auto it = g_rotary.find((uint64_t)(uintptr_t)h);
    if (it == g_rotary.end()) return false;
    *out = it->second;
    return true;
}

// Device pointers of a call: device memory (not host memory that happens to be
// reachable) of the call's device.
kv_status on_device(const void *p, const char *name, int device) {
    cudaPointerAttributes at;
    const cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, name);
    if ((at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) ||
        (at.type == cudaMemoryTypeDevice && at.device != device))
        return fail(KV_ERR_INVALID_ARG, "%s (%p) is not device memory of device %d", name, p, device);
    return KV_OK;
}

kv_status check_vecs(const kv_vecs &v, const char *name) {
    if (v.data == nullptr) return fail(KV_ERR_INVALID_ARG, "%s is NULL", name);
    if (v.token_stride < 0 || v.head_stride < 0)
        return fail(KV_ERR_INVALID_ARG, "%s has a negative stride (%lld, %lld)", name,
                    (long long)v.token_stride, (long long)v.head_stride);
    if ((uintptr_t)v.data % 16 != 0 || v.token_stride % 8 != 0 || v.head_stride % 8 != 0)
        return fail(KV_ERR_ALIGNMENT, "%s (%p, strides %lld and %lld) does not start every vector on "
                    "a 16-byte boundary", name, v.data, (long long)v.token_stride,
                    (long long)v.head_stride);
    return KV_OK;
}

Vecs vecs(const kv_vecs &v) {
    return Vecs{(uint64_t)(uintptr_t)v.data, v.token_stride * 2, v.head_stride * 2};
}

kv_status check_dim(uint32_t head_dim, uint32_t dtype) {
    if (head_dim == 0 || head_dim % 8 != 0 || head_dim > kMaxDim)
        return fail(KV_ERR_INVALID_ARG, "head_dim %u is not a multiple of 8 in 8..256", head_dim);
    if (dtype > KV_FP16) return fail(KV_ERR_INVALID_ARG, "unknown dtype %u", dtype);
    return KV_OK;
}

#define TRY(expr)                          \
    do {                                   \
        const kv_status st_ = (expr);      \
        if (st_ != KV_OK) return st_;      \
    } while (0)

kv_status head_bytes(uint32_t format, uint32_t D, uint32_t *out) {
    const uint32_t unit = format == KV_CACHE_SAME ? 8 : format == KV_CACHE_E4M3 ? 16 : 32;
    if (format > KV_CACHE_Q4) return fail(KV_ERR_INVALID_ARG, "unknown cache format %u", format);
    if (D == 0 || D % unit != 0 || D > kMaxDim)
        return fail(KV_ERR_LAYOUT, "head_dim %u: cache format %u takes multiples of %u up to %u", D,
                    format, unit, kMaxDim);
    *out = format == KV_CACHE_SAME ? 2 * D
         : format == KV_CACHE_E4M3 ? D : (D / 2 + D / 8 + 15) / 16 * 16;
    return KV_OK;
}

// The layer's addresses, once the layout is known to hold vectors of the format.
kv_status pool_layer(const VecPool &p, uint32_t format, uint32_t head_dim, PoolLayer *out) {
    const kv_layout &l = p.layout;
    uint32_t B = 0;
    TRY(head_bytes(format, head_dim, &B));
    if (l.num_comps != 2)
        return fail(KV_ERR_LAYOUT, "the pool has %u components: keys and values are wanted",
                    l.num_comps);
    if (l.head_bytes != B)
        return fail(KV_ERR_LAYOUT, "the pool's head vectors have %u bytes; format %u of head_dim %u "
                    "has %u", l.head_bytes, format, head_dim, B);
    const uint64_t row = (uint64_t)(l.heads == KV_HND ? l.page_tokens : l.num_heads) * B;
    if (row >= (1ull << 32) || (uint64_t)l.num_pages > 0x7fffffffull || l.page_tokens > 0x7fffffffu)
        return fail(KV_ERR_LAYOUT, "page geometry too large for vector addressing");
    PoolLayer r{};
    r.base[0] = p.base[0];
    r.base[1] = p.base[1];
    r.s_page = p.s_page;
    r.s_tok = l.heads == KV_HND ? B : (uint32_t)row;
    r.s_head = l.heads == KV_HND ? (uint32_t)row : B;
    r.T = l.page_tokens;
    r.H = l.num_heads;
    r.B = B;
    r.P = l.num_pages;
    r.v_page = (uint32_t)(r.s_page / B);
    r.v_tok = r.s_tok / B;
    const FastDiv d = make_fastdiv(l.page_tokens);
    r.t_mul = d.m;
    r.t_shift = d.s;
    *out = r;
    return KV_OK;
}

struct Guard {
    int prev = -1;
    explicit Guard(int d) {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev == d || cudaSetDevice(d) != cudaSuccess) prev = -1;
    }
    ~Guard() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

// Below 2^-128 a scale's inverse is infinite, and zeros would be held as NaN.
kv_status scales(uint32_t format, float k, float v) {
    if (format != KV_CACHE_E4M3) return KV_OK;
    for (const float s : {k, v})
        if (!(s > 0.0f) || !std::isfinite(s) || !std::isfinite(1.0f / s))
            return fail(KV_ERR_INVALID_ARG, "k_scale %g and v_scale %g must be above 0 and finite, and so their inverses", k, v);
    return KV_OK;
}

// A window longer than any request hides nothing.
uint32_t window_of(const kv_attend_args *a) { return std::min(a->window, 1u << 30); }

// What plan_attend and the kernels need of a block, without its pointers.
kv_status check_attend(const kv_attend_args *a, const VecPool &p, PoolLayer *layer) {
    TRY(check_dim(a->head_dim, a->dtype));
    if (a->reserved[0] != 0 || a->reserved[1] != 0)
        return fail(KV_ERR_INVALID_ARG, "reserved members must be 0");
    if (a->head_dim != 64 && a->head_dim != 96 && a->head_dim != 128 && a->head_dim != 192 &&
        a->head_dim != 256)
        return fail(KV_ERR_LAYOUT, "head_dim %u: attention takes 64, 96, 128, 192 and 256", a->head_dim);
    TRY(pool_layer(p, KV_CACHE_Q4, a->head_dim, layer));
    if (!vector_index_fits(*layer))
        return fail(KV_ERR_LAYOUT, "the pool's pages span 2^32 head vectors or more");
    if (a->q_heads == 0 || a->q_heads % layer->H != 0)
        return fail(KV_ERR_INVALID_ARG, "%u query heads are not a multiple of the pool's %u", a->q_heads,
                    layer->H);
    if (a->q_heads > 65535 || a->requests > 65535 || a->max_q > 65535)
        return fail(KV_ERR_INVALID_ARG, "requests %u, max_q %u and q_heads %u: 65535 at most each",
                    a->requests, a->max_q, a->q_heads);
    // the kernels count rows, tokens and places in 32 bits with room to add
    if (a->tokens > 0x7fffffffu || a->max_len > (1u << 30) ||
        (uint64_t)a->max_q * (a->q_heads / layer->H) > (1u << 30))
        return fail(KV_ERR_INVALID_ARG, "tokens %u, max_len %u or max_q %u (of %u heads a KV head) too large",
                    a->tokens, a->max_len, a->max_q, a->q_heads / layer->H);
    if (a->max_q > a->tokens)
        return fail(KV_ERR_INVALID_ARG, "max_q %u is more than all %u query tokens", a->max_q, a->tokens);
    if (!std::isfinite(a->scale)) return fail(KV_ERR_INVALID_ARG, "scale is not finite");
    return KV_OK;
}

constexpr uint32_t kMostTokens = 1u << 29;     // of a request, or of a prefix

kv_status check_wide_dim(uint32_t head_dim, const char *what) {
    if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192 && head_dim != 256)
        return fail(KV_ERR_LAYOUT, "head_dim %u: %s takes 64, 96, 128, 192 and 256", head_dim, what);
    return KV_OK;
}

// Counts that the operators on 16-bit and fp8 pages share.
kv_status check_counts(uint32_t requests, uint32_t tokens, uint32_t max_q, uint32_t max_len, uint32_t q_heads,
                       uint32_t H, uint32_t T) {
    if (T > (1u << 20)) return fail(KV_ERR_LAYOUT, "pages of %u tokens: 2^20 at most", T);
    if (H > 65535) return fail(KV_ERR_LAYOUT, "%u KV heads: 65535 at most", H);
    if (q_heads == 0 || q_heads % H != 0)
        return fail(KV_ERR_INVALID_ARG, "%u query heads are not a multiple of the pool's %u", q_heads, H);
    if (q_heads > 65535 || requests > 65535 || max_q > 65535)
        return fail(KV_ERR_INVALID_ARG, "requests %u, max_q %u and q_heads %u: 65535 at most each", requests,
                    max_q, q_heads);
    if (tokens > 0x7fffffffu || max_len > kMostTokens || (uint64_t)max_q * (q_heads / H) > (1u << 30) ||
        (uint64_t)tokens * (q_heads / H) > (1u << 30))
        return fail(KV_ERR_INVALID_ARG, "tokens %u, max_len %u or max_q %u (of %u heads a KV head) too large",
                    tokens, max_len, max_q, q_heads / H);
    if (max_q > tokens)
        return fail(KV_ERR_INVALID_ARG, "max_q %u is more than all %u query tokens", max_q, tokens);
    return KV_OK;
}

kv_status check_table(const void *pages, int64_t stride, uint32_t rows, uint32_t max_len, uint32_t T, const char *name) {
    if (pages == nullptr && max_len != 0) return fail(KV_ERR_INVALID_ARG, "%s is NULL", name);
    const uint64_t entries = ((uint64_t)max_len + T - 1) / T;
    if (stride < 0 || (rows > 1 && (uint64_t)stride < entries))
        return fail(KV_ERR_INVALID_ARG, "the stride of %s, %lld, is less than the %llu pages of %u tokens", name,
                    (long long)stride, (unsigned long long)entries, max_len);
    return KV_OK;
}

kv_status check_space(const void *workspace, uint64_t have, uint64_t need) {
    if (need != 0 && workspace == nullptr)
        return fail(KV_ERR_INVALID_ARG, "workspace is NULL; %llu bytes are needed", (unsigned long long)need);
    if (have < need)
        return fail(KV_ERR_OUT_OF_RANGE, "workspace of %llu bytes; %llu are needed", (unsigned long long)have,
                    (unsigned long long)need);
    if ((uintptr_t)workspace % 16 != 0) return fail(KV_ERR_ALIGNMENT, "the workspace is not 16-byte aligned");
    return KV_OK;
}

// kv_attend_shared and kv_attend_selected as one: a selected call has no groups, a shared one no budget.
struct PagesCall {
    kv_attend_shared_args a;
    const int32_t *picks;
    uint32_t budget;
};

PagesCall shared_call(const kv_attend_shared_args *a) { return PagesCall{*a, nullptr, 0}; }

PagesCall selected_call(const kv_attend_selected_args *s) {
    PagesCall c{};
    kv_attend_shared_args &a = c.a;
    a.q = s->q;
    a.out = s->out;
    a.lse = s->lse;
    a.q_start = s->q_start;
    a.lens = s->lens;
    a.pages = s->pages;
    a.pages_stride = s->pages_stride;
    a.workspace = s->workspace;
    a.workspace_bytes = s->workspace_bytes;
    a.status = s->status;
    a.requests = s->requests;
    a.tokens = s->tokens;
    a.max_q = s->max_q;
    a.max_len = s->max_len;
    a.q_heads = s->q_heads;
    a.head_dim = s->head_dim;
    a.dtype = s->dtype;
    a.format = s->format;
    a.layer = s->layer;
    a.scale = s->scale;
    a.k_scale = s->k_scale;
    a.v_scale = s->v_scale;
    a.reserved = s->reserved;
    c.picks = s->picks;
    c.budget = s->budget;
    return c;
}

bool empty_call(const kv_attend_shared_args &a) { return a.requests == 0 || a.tokens == 0 || a.max_q == 0; }

// What the plan and the kernels need of a block, without its pointers.
kv_status check_pages(const PagesCall &c, bool selected, const VecPool &p, PoolLayer *layer, PagePlan *plan) {
    const kv_attend_shared_args &a = c.a;
    TRY(check_dim(a.head_dim, a.dtype));
    if (a.reserved != 0) return fail(KV_ERR_INVALID_ARG, "reserved members must be 0");
    TRY(check_wide_dim(a.head_dim, "attention"));
    if (a.format != KV_CACHE_SAME && a.format != KV_CACHE_E4M3)
        return fail(KV_ERR_INVALID_ARG, "format %u: SAME and E4M3 pages are taken (Q4 by kv_attend)", a.format);
    TRY(pool_layer(p, a.format, a.head_dim, layer));
    if (!vector_index_fits(*layer) || (a.format == KV_CACHE_SAME && (uint64_t)layer->P * layer->v_page > 0x7fffffffull))
        return fail(KV_ERR_LAYOUT, "the pool's pages span too many head vectors (2^31 of 16-bit values, 2^32 of fp8)");
    TRY(check_counts(a.requests, a.tokens, a.max_q, a.max_len, a.q_heads, layer->H, layer->T));
    if (a.groups > 65535 || a.max_prefix > kMostTokens)
        return fail(KV_ERR_INVALID_ARG, "groups %u or max_prefix %u too large", a.groups, a.max_prefix);
    if (selected && (c.budget == 0 || c.budget > (1u << 24)))
        return fail(KV_ERR_INVALID_ARG, "budget %u is not in 1..2^24", c.budget);
    TRY(scales(a.format, a.k_scale, a.v_scale));
    const float scale = a.scale * (a.format == KV_CACHE_E4M3 ? a.k_scale : 1.0f) * 1.44269504088896340736f;
    if (!std::isfinite(scale)) return fail(KV_ERR_INVALID_ARG, "scale (with k_scale) is not finite");
    *plan = PagePlan{};
    if (!empty_call(a))
        *plan = plan_pages(a.requests, a.tokens, a.max_q, a.max_len, a.groups, std::min(a.max_group, a.tokens), a.max_prefix, c.budget,
                           layer->T, a.q_heads, layer->H, a.head_dim, a.format == KV_CACHE_E4M3, p.sms,
                           pages_blocks(a.head_dim, a.format == KV_CACHE_E4M3));
    if (!plan_counts_fit(*plan, a.max_q, a.max_len, std::min(a.max_group, a.tokens), a.max_prefix, c.budget, layer->T, a.q_heads, layer->H))
        return fail(KV_ERR_INVALID_ARG, "tokens %u, max_q %u, max_len %u, max_group %u, max_prefix %u and budget %u make too much work",
                    a.tokens, a.max_q, a.max_len, a.max_group, a.max_prefix, c.budget);
    return KV_OK;
}

kv_status pages_workspace(kv_pool pool, const PagesCall &c, bool selected, uint64_t *out) {
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, c.a.layer, &p));
    PoolLayer layer;
    PagePlan plan;
    TRY(check_pages(c, selected, p, &layer, &plan));
    *out = plan.bytes;
    return KV_OK;
}

void at_workspace(PageEngine *e, void *workspace) {
    const uint64_t w = (uint64_t)(uintptr_t)workspace;
    e->part_o = (float *)((uint64_t)(uintptr_t)e->part_o + w);
    e->part_ml = (float *)((uint64_t)(uintptr_t)e->part_ml + w);
    e->seg_tiles = (uint64_t *)((uint64_t)(uintptr_t)e->seg_tiles + w);
    e->seg_units = (uint64_t *)((uint64_t)(uintptr_t)e->seg_units + w);
    e->seg_table = (int32_t *)((uint64_t)(uintptr_t)e->seg_table + w);
}

kv_status attend_pages(kv_pool pool, const PagesCall &c, bool selected, void *stream) {
    const kv_attend_shared_args &a = c.a;
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, a.layer, &p));
    PageAttendArgs k{};
    PagePlan plan;
    TRY(check_pages(c, selected, p, &k.pool, &plan));
    if (empty_call(a)) return KV_OK;
    TRY(check_vecs(a.q, "q"));
    TRY(check_vecs(a.out, "out"));
    if (a.q_start == nullptr || a.lens == nullptr)
        return fail(KV_ERR_INVALID_ARG, "q_start or lens is NULL");
    TRY(check_table(a.pages, a.pages_stride, a.requests, a.max_len, k.pool.T, "pages"));
    if (a.groups != 0) {
        if (a.group_start == nullptr || a.prefix_lens == nullptr)
            return fail(KV_ERR_INVALID_ARG, "group_start or prefix_lens is NULL");
        TRY(check_table(a.prefix_pages, a.prefix_stride, a.groups, a.max_prefix, k.pool.T, "prefix_pages"));
    }
    if (selected && c.picks == nullptr) return fail(KV_ERR_INVALID_ARG, "picks is NULL");
    const void *words[] = {a.q_start, a.lens, a.pages, a.lse, a.status, a.group_start, a.prefix_lens, a.prefix_pages, c.picks};
    for (const void *w : words)
        if ((uintptr_t)w % 4 != 0)
            return fail(KV_ERR_ALIGNMENT, "arrays of 32-bit words must be 4-byte aligned (%p is not)", w);
    TRY(check_space(a.workspace, a.workspace_bytes, plan.bytes));
    TRY(on_device(a.q.data, "q", p.device));
    TRY(on_device(a.out.data, "out", p.device));
    TRY(on_device(a.q_start, "q_start", p.device));
    TRY(on_device(a.lens, "lens", p.device));
    if (a.pages != nullptr) TRY(on_device(a.pages, "pages", p.device));
    if (a.lse != nullptr) TRY(on_device(a.lse, "lse", p.device));
    if (a.status != nullptr) TRY(on_device(a.status, "status", p.device));
    if (selected) TRY(on_device(c.picks, "picks", p.device));
    if (a.groups != 0) {
        TRY(on_device(a.group_start, "group_start", p.device));
        TRY(on_device(a.prefix_lens, "prefix_lens", p.device));
        if (a.prefix_pages != nullptr) TRY(on_device(a.prefix_pages, "prefix_pages", p.device));
    }
    if (plan.bytes != 0) TRY(on_device(a.workspace, "workspace", p.device));
    Guard guard(p.device);
    vec_begin(p.device, stream);
    k.q = vecs(a.q);
    k.out = vecs(a.out);
    k.lse = a.lse;
    k.q_start = a.q_start;
    k.lens = a.lens;
    k.pages = a.pages;
    k.pages_stride = a.pages_stride;
    k.group_start = a.group_start;
    k.prefix_lens = a.prefix_lens;
    k.prefix_pages = a.prefix_pages;
    k.prefix_stride = a.prefix_stride;
    k.picks = c.picks;
    k.budget = c.budget;
    k.status = a.status;
    k.requests = a.requests;
    k.tokens = a.tokens;
    k.max_q = a.max_q;
    k.max_len = a.max_len;
    k.groups = a.groups;
    k.max_group = std::min(a.max_group, a.tokens);
    k.max_prefix = a.max_prefix;
    k.q_heads = a.q_heads;
    k.group = a.q_heads / k.pool.H;
    const bool fp8 = a.format == KV_CACHE_E4M3;
    k.scale_log2 = a.scale * (fp8 ? a.k_scale : 1.0f) * 1.44269504088896340736f;
    k.v_scale = fp8 ? a.v_scale : 1.0f;
    k.join_heads = plan.join_heads;
    k.joined = plan.joined;
    k.rows = plan.rows;
    k.tc = plan.tc;
    at_workspace(&k.rows, a.workspace);
    at_workspace(&k.tc, a.workspace);
    int launches = 0;
    const cudaError_t e = launch_pages(k, plan, a.head_dim, fp8, a.dtype == KV_FP16, p.pdl, (cudaStream_t)stream,
                                       &launches);
    vec_count(launches);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, "launch of the attention kernels");
    return KV_OK;
}

kv_status check_select(const kv_select_args *a, const VecPool &p, SelectArgs *k, uint64_t *need) {
    TRY(check_dim(a->head_dim, a->dtype));
    if (a->reserved[0] != 0 || a->reserved[1] != 0)
        return fail(KV_ERR_INVALID_ARG, "reserved members must be 0");
    TRY(check_wide_dim(a->head_dim, "selection"));
    const kv_layout &l = p.layout;
    TRY(check_counts(a->requests, a->tokens, a->max_q, a->max_len, a->q_heads, l.num_heads, l.page_tokens));
    if (a->budget == 0 || a->budget > (1u << 24))
        return fail(KV_ERR_INVALID_ARG, "budget %u is not in 1..2^24", a->budget);
    if (a->keep_first > a->budget || a->keep_last > a->budget - a->keep_first)
        return fail(KV_ERR_INVALID_ARG, "keep_first %u and keep_last %u are more than the budget of %u", a->keep_first,
                    a->keep_last, a->budget);
    k->T = l.page_tokens;
    k->P = l.num_pages;
    k->H = l.num_heads;
    k->max_pages = (a->max_len + l.page_tokens - 1) / l.page_tokens;
    const uint64_t rows = (uint64_t)a->tokens * l.num_heads;
    if (k->max_pages != 0 && rows > (1ull << 58) / k->max_pages)
        return fail(KV_ERR_INVALID_ARG, "tokens %u and max_len %u make too many scores", a->tokens, a->max_len);
    k->block_pages = select_block_pages(rows * k->max_pages, p.sms);
    const uint64_t chunks = (k->max_pages + k->block_pages - 1) / k->block_pages;
    if (chunks * l.num_heads > 0x7fffffffull)
        return fail(KV_ERR_INVALID_ARG, "max_len %u makes too many blocks", a->max_len);
    *need = k->max_pages > a->budget ? rows * k->max_pages * sizeof(float) : 0;
    return KV_OK;
}

}  // namespace

extern "C" {

kv_status kv_cache_head_bytes(uint32_t format, uint32_t head_dim, uint32_t *out) {
    if (out == nullptr) return fail(KV_ERR_INVALID_ARG, "output pointer is NULL");
    return head_bytes(format, head_dim, out);
}

kv_status kv_rotary_create(const kv_rotary_desc *d, kv_rotary *out) {
    if (d == nullptr || out == nullptr) return fail(KV_ERR_INVALID_ARG, "descriptor or output is NULL");
    if (d->reserved != 0) return fail(KV_ERR_INVALID_ARG, "reserved members must be 0");
    const uint32_t R = d->rot_dim;
    if (R < 2 || R % 2 != 0 || R > 2 * kMaxPairs)
        return fail(KV_ERR_INVALID_ARG, "rot_dim %u is not an even number in 2..%d", R, 2 * kMaxPairs);
    if (d->style > KV_ROTARY_INTERLEAVED || d->scaling > KV_ROTARY_BANDS)
        return fail(KV_ERR_INVALID_ARG, "unknown style %u or scaling %u", d->style, d->scaling);
    if (!(d->base > 1.0) || !std::isfinite(d->base))
        return fail(KV_ERR_INVALID_ARG, "base %g must be finite and above 1", d->base);
    if (!(d->gain >= 0.0) || !std::isfinite((float)d->gain))   // cosines and sines are float32
        return fail(KV_ERR_INVALID_ARG, "gain %g must be a finite float32 and not negative", d->gain);
    const uint32_t sc = d->scaling;
    if (sc != KV_ROTARY_PLAIN && (!(d->factor >= 1.0) || !std::isfinite(d->factor)))
        return fail(KV_ERR_INVALID_ARG, "factor %g must be finite and at least 1", d->factor);
    if (sc == KV_ROTARY_NTK && R < 4) return fail(KV_ERR_INVALID_ARG, "NTK scaling needs rot_dim >= 4");
    if ((sc == KV_ROTARY_YARN || sc == KV_ROTARY_BANDS) &&
        (!(d->slow > 0.0) || !(d->fast > d->slow) || !std::isfinite(d->fast) || d->original_len < 1))
        return fail(KV_ERR_INVALID_ARG, "YARN and BANDS need 0 < slow (%g) < fast (%g) and "
                    "original_len >= 1", d->slow, d->fast);
    const double len = (double)d->original_len;
    double base = d->base, lo = 0.0, hi = 0.0, gain = d->gain > 0.0 ? d->gain : 1.0;
    if (sc == KV_ROTARY_NTK) base *= std::pow(d->factor, (double)R / (R - 2));
    if (sc == KV_ROTARY_YARN) {
        auto pair_of = [&](double turns) { return R * std::log(len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
        lo = std::max(0.0, std::floor(pair_of(d->fast)));
        hi = std::min((double)R - 1.0, std::ceil(pair_of(d->slow)));
        if (d->gain == 0.0) gain = 0.1 * std::log(d->factor) + 1.0;
    }
    RotaryK r{};
    r.half = R / 2;
    r.style = d->style;
    r.gain = (float)gain;
    for (uint32_t i = 0; i < r.half; ++i) {
        double f = std::pow(base, -2.0 * i / R);
        if (sc == KV_ROTARY_LINEAR) f /= d->factor;
        if (sc == KV_ROTARY_YARN) {
            const double t = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
            f = f / d->factor * t + f * (1.0 - t);
        }
        if (sc == KV_ROTARY_BANDS) {
            const double t = (len * f / kTwoPi - d->slow) / (d->fast - d->slow);
            const double k = std::min(1.0, std::max(0.0, t));
            f = f / d->factor * (1.0 - k) + f * k;
        }
        // f <= 1 radian, so a turn's fraction is below 1; 2^64 x 0.16 fits
        r.turns[i] = (unsigned long long)std::ldexp(f / kTwoPi, 64);
    }
    try {
        std::lock_guard<std::mutex> lk(g_rot_mu);
        const uint64_t id = g_next_rotary++;
        g_rotary.emplace(id, r);
        *out = (kv_rotary)(uintptr_t)id;
    } catch (const std::bad_alloc &) {
        return fail(KV_ERR_NO_MEMORY, "out of host memory");
    }
    return KV_OK;
}

kv_status kv_rotary_close(kv_rotary rotary) {
    std::lock_guard<std::mutex> lk(g_rot_mu);
    if (g_rotary.erase((uint64_t)(uintptr_t)rotary) == 0)
        return fail(KV_ERR_CLOSED, "rotary handle is closed or unknown");
    return KV_OK;
}

kv_status kv_rotate(kv_rotary rotary, const kv_rotate_args *a, void *stream) {
    RotaryK r;
    if (a == nullptr || rotary == nullptr)
        return fail(KV_ERR_INVALID_ARG, "rotary handle or argument block is NULL");
    if (!find_rotary(rotary, &r)) return fail(KV_ERR_CLOSED, "rotary handle is closed or unknown");
    if (a->reserved != 0 || (a->flags & ~KV_ROTATE_INVERSE) != 0)
        return fail(KV_ERR_INVALID_ARG, "unknown flags 0x%x, or reserved members not 0", a->flags);
    TRY(check_dim(a->head_dim, a->dtype));
    if (a->head_dim < 2 * r.half)
        return fail(KV_ERR_INVALID_ARG, "head_dim %u is less than rot_dim %u", a->head_dim, 2 * r.half);
    if (a->tokens > 0x7fffffffu || a->heads > 65535)
        return fail(KV_ERR_INVALID_ARG, "too many tokens (%u) or heads (%u)", a->tokens, a->heads);
    if (a->tokens == 0 || (a->heads == 0 && a->rows_out == nullptr)) return KV_OK;
    if (a->heads != 0) {
        TRY(check_vecs(a->x, "x"));
        TRY(check_vecs(a->out, "out"));
        if (a->x.data == a->out.data && (a->x.token_stride != a->out.token_stride ||
                                         a->x.head_stride != a->out.head_stride))
            return fail(KV_ERR_INVALID_ARG, "out is x with other strides");
    }
    if ((a->positions == nullptr) == (a->rows_in == nullptr))
        return fail(KV_ERR_INVALID_ARG, "exactly one of positions and rows_in is wanted");
    if (a->rows_out != nullptr && a->positions == nullptr)
        return fail(KV_ERR_INVALID_ARG, "rows_out needs positions");
    if (a->rows_out != nullptr && (uintptr_t)a->rows_out % 16 != 0)
        return fail(KV_ERR_ALIGNMENT, "rows_out is not 16-byte aligned");
    if (a->rows_in != nullptr && (uintptr_t)a->rows_in % 16 != 0)
        return fail(KV_ERR_ALIGNMENT, "rows_in is not 16-byte aligned");
    if ((uintptr_t)a->positions % 8 != 0) return fail(KV_ERR_ALIGNMENT, "positions are not 8-byte aligned");
    cudaPointerAttributes at;
    const void *lead = a->positions != nullptr ? (const void *)a->positions : (const void *)a->rows_in;
    const cudaError_t e = cudaPointerGetAttributes(&at, lead);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, "cudaPointerGetAttributes");
    const int device = at.device;
    TRY(on_device(lead, "positions or rows_in", device));
    if (a->heads != 0) {
        TRY(on_device(a->x.data, "x", device));
        TRY(on_device(a->out.data, "out", device));
    }
    if (a->rows_out != nullptr) TRY(on_device(a->rows_out, "rows_out", device));
    Guard guard(device);
    bool pdl = true;
    TRY((kv_status)vec_enter_device(device, stream, &pdl));
    VectorArgs k{};
    k.q = vecs(a->x);
    k.q_out = vecs(a->out);
    k.positions = a->positions;
    k.rows_in = a->rows_in;
    k.rows_out = a->rows_out;
    k.tokens = a->tokens;
    k.q_heads = a->heads;
    k.D = a->head_dim;
    k.half = r.half;
    k.style = r.style;
    k.sin_sign = a->flags & KV_ROTATE_INVERSE ? -1.0f : 1.0f;
    const cudaError_t le = launch_vectors(k, r, -1, a->dtype == KV_FP16, pdl, (cudaStream_t)stream);
    if (le != cudaSuccess) return (kv_status)vec_cuda_error(le, "launch of the rotation kernel");
    vec_count(1);
    return KV_OK;
}

kv_status kv_append(kv_pool pool, kv_rotary rotary, const kv_append_args *a, void *stream) {
    if (a == nullptr) return fail(KV_ERR_INVALID_ARG, "argument block is NULL");
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, a->layer, &p));
    RotaryK r{};
    if (rotary != nullptr && !find_rotary(rotary, &r))
        return fail(KV_ERR_CLOSED, "rotary handle is closed or unknown");
    if (a->reserved[0] != 0 || a->reserved[1] != 0)
        return fail(KV_ERR_INVALID_ARG, "reserved members must be 0");
    TRY(check_dim(a->head_dim, a->dtype));
    if (a->head_dim < 2 * r.half)
        return fail(KV_ERR_INVALID_ARG, "head_dim %u is less than rot_dim %u", a->head_dim, 2 * r.half);
    VectorArgs k{};
    TRY(pool_layer(p, a->format, a->head_dim, &k.pool));
    TRY(scales(a->format, a->k_scale, a->v_scale));
    const bool with_q = a->q.data != nullptr;
    if (a->tokens > 0x7fffffffu || a->q_heads > 65535 || k.pool.H > 65535)
        return fail(KV_ERR_INVALID_ARG, "too many tokens (%u) or heads (%u, %u)", a->tokens, a->q_heads,
                    k.pool.H);
    if (a->tokens == 0) return KV_OK;
    TRY(check_vecs(a->k, "k"));
    TRY(check_vecs(a->v, "v"));
    if (a->slots == nullptr) return fail(KV_ERR_INVALID_ARG, "slots is NULL");
    if ((uintptr_t)a->slots % 8 != 0 || (uintptr_t)a->rows % 16 != 0 || (uintptr_t)a->status % 4 != 0)
        return fail(KV_ERR_ALIGNMENT, "slots, rows and status must be 8-, 16- and 4-byte aligned");
    if ((rotary != nullptr) != (a->rows != nullptr))
        return fail(KV_ERR_INVALID_ARG, "rows and a rotary handle go together");
    if (with_q) {
        if (rotary == nullptr) return fail(KV_ERR_INVALID_ARG, "q needs a rotary handle");
        TRY(check_vecs(a->q, "q"));
        TRY(check_vecs(a->q_out, "q_out"));
        if (a->q.data == a->q_out.data && (a->q.token_stride != a->q_out.token_stride ||
                                           a->q.head_stride != a->q_out.head_stride))
            return fail(KV_ERR_INVALID_ARG, "q_out is q with other strides");
    }
    TRY(on_device(a->k.data, "k", p.device));
    TRY(on_device(a->v.data, "v", p.device));
    TRY(on_device(a->slots, "slots", p.device));
    if (a->rows != nullptr) TRY(on_device(a->rows, "rows", p.device));
    if (a->status != nullptr) TRY(on_device(a->status, "status", p.device));
    if (with_q) {
        TRY(on_device(a->q.data, "q", p.device));
        TRY(on_device(a->q_out.data, "q_out", p.device));
    }
    Guard guard(p.device);
    vec_begin(p.device, stream);
    k.k = vecs(a->k);
    k.v = vecs(a->v);
    if (with_q) {
        k.q = vecs(a->q);
        k.q_out = vecs(a->q_out);
        k.q_heads = a->q_heads;
    }
    k.rows_in = a->rows;
    k.slots = a->slots;
    k.status = a->status;
    k.tokens = a->tokens;
    k.kv_heads = k.pool.H;
    k.D = a->head_dim;
    k.half = r.half;
    k.style = r.style;
    k.k_inv = 1.0f / a->k_scale;
    k.v_inv = 1.0f / a->v_scale;
    k.sin_sign = 1.0f;
    const cudaError_t e = launch_vectors(k, r, (int)a->format, a->dtype == KV_FP16, p.pdl,
                                         (cudaStream_t)stream);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, "launch of the append kernel");
    vec_count(1);
    return KV_OK;
}

kv_status kv_fetch(kv_pool pool, const kv_fetch_args *a, void *stream) {
    if (a == nullptr) return fail(KV_ERR_INVALID_ARG, "argument block is NULL");
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, a->layer, &p));
    if (a->reserved != 0) return fail(KV_ERR_INVALID_ARG, "reserved members must be 0");
    TRY(check_dim(a->head_dim, a->dtype));
    VectorArgs k{};
    TRY(pool_layer(p, a->format, a->head_dim, &k.pool));
    TRY(scales(a->format, a->k_scale, a->v_scale));
    if (a->tokens > 0x7fffffffu || k.pool.H > 65535)
        return fail(KV_ERR_INVALID_ARG, "too many tokens (%u) or heads (%u)", a->tokens, k.pool.H);
    if (a->tokens == 0 || (a->k.data == nullptr && a->v.data == nullptr)) return KV_OK;
    if (a->k.data != nullptr) TRY(check_vecs(a->k, "k"));
    if (a->v.data != nullptr) TRY(check_vecs(a->v, "v"));
    if (a->slots == nullptr) return fail(KV_ERR_INVALID_ARG, "slots is NULL");
    if ((uintptr_t)a->slots % 8 != 0 || (uintptr_t)a->status % 4 != 0)
        return fail(KV_ERR_ALIGNMENT, "slots and status must be 8- and 4-byte aligned");
    if (a->k.data != nullptr) TRY(on_device(a->k.data, "k", p.device));
    if (a->v.data != nullptr) TRY(on_device(a->v.data, "v", p.device));
    TRY(on_device(a->slots, "slots", p.device));
    if (a->status != nullptr) TRY(on_device(a->status, "status", p.device));
    Guard guard(p.device);
    vec_begin(p.device, stream);
    k.k = vecs(a->k);
    k.v = vecs(a->v);
    k.slots = a->slots;
    k.status = a->status;
    k.tokens = a->tokens;
    k.kv_heads = k.pool.H;
    k.D = a->head_dim;
    k.k_inv = a->k_scale;
    k.v_inv = a->v_scale;
    const cudaError_t e = launch_fetch(k, (int)a->format, a->dtype == KV_FP16, p.pdl,
                                       (cudaStream_t)stream);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, "launch of the fetch kernel");
    vec_count(1);
    return KV_OK;
}

kv_status kv_attend_workspace(kv_pool pool, const kv_attend_args *a, uint64_t *out) {
    if (a == nullptr || out == nullptr)
        return fail(KV_ERR_INVALID_ARG, "argument block or output pointer is NULL");
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, a->layer, &p));
    PoolLayer layer;
    TRY(check_attend(a, p, &layer));
    *out = 0;
    if (a->requests != 0 && a->tokens != 0 && a->max_q != 0)
        *out = plan_attend(a->requests, a->tokens, a->max_q, a->max_len, window_of(a), a->q_heads, layer.H,
                           a->head_dim, p.sms).bytes;
    return KV_OK;
}

kv_status kv_attend(kv_pool pool, const kv_attend_args *a, void *stream) {
    if (a == nullptr) return fail(KV_ERR_INVALID_ARG, "argument block is NULL");
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, a->layer, &p));
    AttendArgs k{};
    TRY(check_attend(a, p, &k.pool));
    if (a->requests == 0 || a->tokens == 0 || a->max_q == 0) return KV_OK;
    TRY(check_vecs(a->q, "q"));
    TRY(check_vecs(a->out, "out"));
    if (a->q_start == nullptr || a->lens == nullptr)
        return fail(KV_ERR_INVALID_ARG, "q_start or lens is NULL");
    if (a->pages == nullptr && a->max_len != 0) return fail(KV_ERR_INVALID_ARG, "pages is NULL");
    const uint64_t entries = ((uint64_t)a->max_len + k.pool.T - 1) / k.pool.T;
    if (a->pages_stride < 0 || (a->requests > 1 && (uint64_t)a->pages_stride < entries))
        return fail(KV_ERR_INVALID_ARG, "pages_stride %lld is less than the %llu pages of max_len %u",
                    (long long)a->pages_stride, (unsigned long long)entries, a->max_len);
    if ((uintptr_t)a->q_start % 4 != 0 || (uintptr_t)a->lens % 4 != 0 || (uintptr_t)a->pages % 4 != 0 ||
        (uintptr_t)a->lse % 4 != 0 || (uintptr_t)a->status % 4 != 0 || (uintptr_t)a->workspace % 16 != 0)
        return fail(KV_ERR_ALIGNMENT, "q_start, lens, pages, lse and status must be 4-byte and the "
                    "workspace 16-byte aligned");
    const AttendPlan plan = plan_attend(a->requests, a->tokens, a->max_q, a->max_len, window_of(a),
                                        a->q_heads, k.pool.H, a->head_dim, p.sms);
    if ((uint64_t)plan.row_tiles * plan.chunks * k.pool.H * (plan.many ? a->requests : 1) > 0x7fffffffull ||
        plan.step_parts > 65535 || plan.chunks > 65535)
        return fail(KV_ERR_INVALID_ARG, "max_q %u and max_len %u make too many blocks", a->max_q,
                    a->max_len);
    if (plan.bytes != 0 && a->workspace == nullptr)
        return fail(KV_ERR_INVALID_ARG, "workspace is NULL; %llu bytes are needed",
                    (unsigned long long)plan.bytes);
    if (a->workspace_bytes < plan.bytes)
        return fail(KV_ERR_OUT_OF_RANGE, "workspace of %llu bytes; %llu are needed",
                    (unsigned long long)a->workspace_bytes, (unsigned long long)plan.bytes);
    TRY(on_device(a->q.data, "q", p.device));
    TRY(on_device(a->out.data, "out", p.device));
    TRY(on_device(a->q_start, "q_start", p.device));
    TRY(on_device(a->lens, "lens", p.device));
    if (a->pages != nullptr) TRY(on_device(a->pages, "pages", p.device));
    if (a->lse != nullptr) TRY(on_device(a->lse, "lse", p.device));
    if (a->status != nullptr) TRY(on_device(a->status, "status", p.device));
    if (plan.bytes != 0) TRY(on_device(a->workspace, "workspace", p.device));
    Guard guard(p.device);
    vec_begin(p.device, stream);
    k.q = vecs(a->q);
    k.out = vecs(a->out);
    k.lse = a->lse;
    k.q_start = a->q_start;
    k.lens = a->lens;
    k.pages = a->pages;
    k.pages_stride = a->pages_stride;
    k.status = a->status;
    k.requests = a->requests;
    k.tokens = a->tokens;
    k.max_q = a->max_q;
    k.max_len = a->max_len;
    k.q_heads = a->q_heads;
    k.group = a->q_heads / k.pool.H;
    k.chunk = plan.chunk;
    k.chunks = plan.chunks;
    k.row_tiles = plan.row_tiles;
    k.window = window_of(a);
    k.scale_log2 = a->scale * 1.44269504088896340736f;
    k.whole_units = (uint32_t)plan.whole_units;
    k.steps = (uint32_t *)a->workspace;
    k.step_parts = plan.step_parts;
    k.uneven = k.steps + (uint64_t)a->requests * plan.step_parts * k.pool.H * kStepWords;
    if (plan.bytes != 0) {
        k.part_o = (float *)((char *)a->workspace + plan.step_bytes);
        k.part_ml = k.part_o + (uint64_t)plan.chunks * a->tokens * a->q_heads * a->head_dim;
    }
    int launches = 0;
    const cudaError_t e = launch_attend(k, plan, a->head_dim, a->dtype == KV_FP16, p.pdl,
                                        (cudaStream_t)stream, &launches);
    vec_count(launches);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, "launch of the attention kernel");
    return KV_OK;
}

kv_status kv_attend_shared_workspace(kv_pool pool, const kv_attend_shared_args *a, uint64_t *out) {
    if (a == nullptr || out == nullptr)
        return fail(KV_ERR_INVALID_ARG, "argument block or output pointer is NULL");
    return pages_workspace(pool, shared_call(a), false, out);
}

kv_status kv_attend_shared(kv_pool pool, const kv_attend_shared_args *a, void *stream) {
    if (a == nullptr) return fail(KV_ERR_INVALID_ARG, "argument block is NULL");
    return attend_pages(pool, shared_call(a), false, stream);
}

kv_status kv_attend_selected_workspace(kv_pool pool, const kv_attend_selected_args *a, uint64_t *out) {
    if (a == nullptr || out == nullptr)
        return fail(KV_ERR_INVALID_ARG, "argument block or output pointer is NULL");
    return pages_workspace(pool, selected_call(a), true, out);
}

kv_status kv_attend_selected(kv_pool pool, const kv_attend_selected_args *a, void *stream) {
    if (a == nullptr) return fail(KV_ERR_INVALID_ARG, "argument block is NULL");
    return attend_pages(pool, selected_call(a), true, stream);
}

kv_status kv_bound_bytes(uint32_t head_dim, uint32_t *out) {
    if (out == nullptr) return fail(KV_ERR_INVALID_ARG, "output pointer is NULL");
    TRY(check_wide_dim(head_dim, "kv_bound"));
    *out = record_bytes(head_dim);
    return KV_OK;
}

kv_status kv_bound(kv_pool pool, const kv_bound_args *a, void *stream) {
    if (a == nullptr) return fail(KV_ERR_INVALID_ARG, "argument block is NULL");
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, a->layer, &p));
    TRY(check_dim(a->head_dim, a->dtype));
    if (a->reserved != 0) return fail(KV_ERR_INVALID_ARG, "reserved members must be 0");
    TRY(check_wide_dim(a->head_dim, "kv_bound"));
    if (a->format != KV_CACHE_SAME && a->format != KV_CACHE_E4M3)
        return fail(KV_ERR_INVALID_ARG, "format %u: SAME and E4M3 pages are taken", a->format);
    BoundArgs k{};
    TRY(pool_layer(p, a->format, a->head_dim, &k.pool));
    if (k.pool.T > (1u << 20)) return fail(KV_ERR_LAYOUT, "pages of %u tokens: 2^20 at most", k.pool.T);
    if (a->requests > 65535 || a->max_len > kMostTokens || a->max_new > a->max_len)
        return fail(KV_ERR_INVALID_ARG, "requests %u, max_len %u or max_new %u too large", a->requests, a->max_len,
                    a->max_new);
    if (a->requests == 0 || a->max_new == 0) return KV_OK;
    if (a->bounds == nullptr || a->lens == nullptr)
        return fail(KV_ERR_INVALID_ARG, "bounds or lens is NULL");
    TRY(check_table(a->pages, a->pages_stride, a->requests, a->max_len, k.pool.T, "pages"));
    if ((uintptr_t)a->bounds % 16 != 0 || (uintptr_t)a->lens % 4 != 0 || (uintptr_t)a->first % 4 != 0 ||
        (uintptr_t)a->pages % 4 != 0 || (uintptr_t)a->status % 4 != 0)
        return fail(KV_ERR_ALIGNMENT, "bounds must be 16-byte, lens, first, pages and status 4-byte aligned");
    TRY(on_device(a->bounds, "bounds", p.device));
    TRY(on_device(a->lens, "lens", p.device));
    if (a->first != nullptr) TRY(on_device(a->first, "first", p.device));
    TRY(on_device(a->pages, "pages", p.device));
    if (a->status != nullptr) TRY(on_device(a->status, "status", p.device));
    Guard guard(p.device);
    vec_begin(p.device, stream);
    k.bounds = (uint8_t *)a->bounds;
    k.lens = a->lens;
    k.first = a->first;
    k.pages = a->pages;
    k.pages_stride = a->pages_stride;
    k.status = a->status;
    k.requests = a->requests;
    k.max_len = a->max_len;
    k.max_new = a->max_new;
    k.most_pages = (a->max_new - 1 + k.pool.T - 1) / k.pool.T + 1;
    const cudaError_t e = launch_bound(k, a->head_dim, a->format == KV_CACHE_E4M3, a->dtype == KV_FP16, p.pdl, p.sms,
                                       (cudaStream_t)stream);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, "launch of the bounds kernel");
    vec_count(1);
    return KV_OK;
}

kv_status kv_select_workspace(kv_pool pool, const kv_select_args *a, uint64_t *out) {
    if (a == nullptr || out == nullptr)
        return fail(KV_ERR_INVALID_ARG, "argument block or output pointer is NULL");
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, 0, &p));
    SelectArgs k{};
    return check_select(a, p, &k, out);
}

kv_status kv_select(kv_pool pool, const kv_select_args *a, void *stream) {
    if (a == nullptr) return fail(KV_ERR_INVALID_ARG, "argument block is NULL");
    VecPool p;
    TRY((kv_status)vec_enter_pool(pool, 0, &p));
    SelectArgs k{};
    uint64_t need = 0;
    TRY(check_select(a, p, &k, &need));
    if (a->requests == 0 || a->tokens == 0 || a->max_q == 0) return KV_OK;
    TRY(check_vecs(a->q, "q"));
    if (a->q_start == nullptr || a->lens == nullptr || a->picks == nullptr || a->bounds == nullptr)
        return fail(KV_ERR_INVALID_ARG, "q_start, lens, picks or bounds is NULL");
    TRY(check_table(a->pages, a->pages_stride, a->requests, a->max_len, k.T, "pages"));
    if ((uintptr_t)a->bounds % 16 != 0 || (uintptr_t)a->q_start % 4 != 0 || (uintptr_t)a->lens % 4 != 0 ||
        (uintptr_t)a->pages % 4 != 0 || (uintptr_t)a->picks % 4 != 0 || (uintptr_t)a->status % 4 != 0)
        return fail(KV_ERR_ALIGNMENT, "bounds must be 16-byte, q_start, lens, pages, picks and status 4-byte aligned");
    TRY(check_space(a->workspace, a->workspace_bytes, need));
    TRY(on_device(a->bounds, "bounds", p.device));
    TRY(on_device(a->q.data, "q", p.device));
    TRY(on_device(a->q_start, "q_start", p.device));
    TRY(on_device(a->lens, "lens", p.device));
    if (a->pages != nullptr) TRY(on_device(a->pages, "pages", p.device));
    TRY(on_device(a->picks, "picks", p.device));
    if (a->status != nullptr) TRY(on_device(a->status, "status", p.device));
    if (need != 0) TRY(on_device(a->workspace, "workspace", p.device));
    Guard guard(p.device);
    vec_begin(p.device, stream);
    k.bounds = (const uint8_t *)a->bounds;
    k.q = vecs(a->q);
    k.q_start = a->q_start;
    k.lens = a->lens;
    k.pages = a->pages;
    k.pages_stride = a->pages_stride;
    k.picks = a->picks;
    k.scores = (float *)a->workspace;
    k.status = a->status;
    k.requests = a->requests;
    k.tokens = a->tokens;
    k.max_q = a->max_q;
    k.max_len = a->max_len;
    k.q_heads = a->q_heads;
    k.group = a->q_heads / k.H;
    k.budget = a->budget;
    k.keep_first = a->keep_first;
    k.keep_last = a->keep_last;
    int launches = 0;
    const cudaError_t e = launch_select(k, a->head_dim, a->dtype == KV_FP16, p.pdl, (cudaStream_t)stream, &launches);
    vec_count(launches);
    if (e != cudaSuccess) return (kv_status)vec_cuda_error(e, "launch of the selection kernels");
    return KV_OK;
}

}  // extern "C"
