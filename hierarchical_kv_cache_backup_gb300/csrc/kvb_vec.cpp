// kvb_vec.cpp -- C ABI of the operators on single head vectors: kv_rotary_*,
// kv_rotate, kv_append, kv_fetch, kv_attend.  Checks of arguments, frequencies,
// and the launch of each call; the kernels are in kvb_vectors.cu and
// kvb_attend.cu.
#include "kvb.h"
#include "kvb_internal.h"
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

}  // extern "C"
