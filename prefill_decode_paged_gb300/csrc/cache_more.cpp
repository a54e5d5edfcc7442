// cache_more.cpp -- host side of the decode cache's further calls: validation ahead of their launches.
#include <math.h>

#include <initializer_list>
#include <utility>

#include "cache.h"

namespace {

bool multiples(int64_t of, std::initializer_list<int64_t> xs) {
    for (int64_t x : xs)
        if (x % of != 0) return false;
    return true;
}
bool negative(std::initializer_list<int64_t> xs) {
    for (int64_t x : xs)
        if (x < 0) return true;
    return false;
}
// Rows of `row` entries (or bytes), `outer` by `inner` of them, do not overlap.
bool disjoint_rows(int64_t outer, int64_t outer_stride, int64_t inner, int64_t inner_stride, int64_t row) {
    if (outer <= 1) outer_stride = INT64_MAX;
    if (inner <= 1) inner_stride = INT64_MAX;
    if (outer_stride < inner_stride) {
        std::swap(outer, inner);
        std::swap(outer_stride, inner_stride);
    }
    if (inner > 1 && inner_stride < row) return false;
    return outer <= 1 || (__int128)outer_stride >= (inner > 1 ? (__int128)(inner - 1) * inner_stride : 0) + row;
}
// No C++ exception crosses the ABI.
template <typename F>
kvr_status guarded(F launch) {
    try {
        return launch();
    } catch (...) {
        return KVR_ERR_NOMEM;
    }
}
// The same for calls that write rows or weights: an eviction chooses by a first launch what a second moves, and no
// other thread's call may change it between them on their stream.
template <typename F>
kvr_status together(const kvc_cache *c, F launch) {
    return guarded([&] {
        std::lock_guard<std::mutex> lock(c->use);
        return launch();
    });
}
int64_t address(const void *p) { return (int64_t)(uintptr_t)p; }

}  // namespace

extern "C" kvr_status kv_cache_append_at(const kvc_cache *c, int32_t layer, const kvc_append *a,
                                         const int32_t *angles, void *stream) {
    const kvr_status st = kvc_check_append(c, layer, a);
    if (st != KVR_OK) return st;
    if (address(angles) % 4 != 0) return KVR_ERR_ALIGNMENT;
    if (!kvc_on_device(c)) return KVR_ERR_INVALID_ARG;
    if (a->num_tokens == 0) return KVR_OK;
    return together(c, [&] { return kvc_append_at_launch(c, layer, a, angles, stream); });
}

kvr_status kvc_check_scoring(const kvc_cache *c, const kvc_scoring &s) {
    if (!(s.cap >= 0.0f) || !std::isfinite(s.cap) || s.reserved != 0) return KVR_ERR_INVALID_ARG;
    // (so that it and its reciprocal are numbers of fp32, times log2 e as well)
    if (s.cap > 0.0f && (s.cap < 0x1p-100f || s.cap > 0x1p100f)) return KVR_ERR_UNSUPPORTED;
    if (address(s.slopes) % 4 != 0) return KVR_ERR_ALIGNMENT;
    return c->latent() && (s.cap > 0.0f || s.slopes != nullptr) ? KVR_ERR_UNSUPPORTED : KVR_OK;
}

extern "C" kvr_status kv_cache_attend_scored(const kvc_cache *c, int32_t layer, const kvc_attend *a,
                                             const kvc_scoring *scoring, void *stream) {
    if (scoring == nullptr) return kv_cache_attend(c, layer, a, stream);
    kvr_status st = kvc_check_attend(c, layer, a);
    if (st == KVR_OK) st = kvc_check_scoring(c, *scoring);
    if (st != KVR_OK) return st;
    if (scoring->cap == 0.0f && scoring->slopes == nullptr) return kv_cache_attend(c, layer, a, stream);
    if (!kvc_on_device(c)) return KVR_ERR_INVALID_ARG;
    if (a->num_requests == 0) return KVR_OK;
    return guarded([&] { return kvc_attend_scored_launch(c, layer, a, scoring, stream); });
}

extern "C" kvr_status kv_cache_weigh(const kvc_cache *c, int32_t layer, const kvc_weigh *a, void *stream) {
    if (c == nullptr || a == nullptr) return KVR_ERR_INVALID_ARG;
    const kvc_desc &d = c->d;
    if (layer < 0 || layer >= d.num_layers) return KVR_ERR_LAYER_RANGE;
    if (d.query_heads < 1 || c->latent()) return KVR_ERR_UNSUPPORTED;
    if (a->num_requests < 0 || a->num_requests > d.max_requests || a->num_new < 1 || a->num_new > d.max_new ||
        a->window < 0 || (a->add != 0 && a->add != 1) || a->reserved != 0 || a->weights_width < 0 ||
        !std::isfinite(a->scale) || !kvc_ok_table(a->table) || a->table.rows < a->num_requests)
        return KVR_ERR_INVALID_ARG;
    if (!kvc_type_fits(c, a->dtype)) return KVR_ERR_UNSUPPORTED;
    // positions are 32-bit: a table row must not describe more of them
    if ((int64_t)a->table.width * d.block_size > (int64_t)INT32_MAX - KVC_MAX_REQUESTS)
        return KVR_ERR_UNSUPPORTED;
    if (a->num_requests > 0 && (a->lengths == nullptr || a->q == nullptr || a->lse == nullptr ||
                                (a->weights == nullptr && a->weights_width > 0)))
        return KVR_ERR_INVALID_ARG;
    if (negative({a->q_request_stride, a->q_token_stride, a->q_head_stride, a->weights_request_stride,
                  a->weights_head_stride}))
        return KVR_ERR_INVALID_ARG;
    // (each head's weights are written by blocks of its own)
    if (!disjoint_rows(a->num_requests, a->weights_request_stride, d.kv_heads, a->weights_head_stride,
                       a->weights_width))
        return KVR_ERR_POOL_OVERLAP;
    if (!multiples(4, {address(a->lengths), address(a->lse), address(a->weights)}) ||
        !multiples(16, {address(a->q), a->q_request_stride, a->q_token_stride, a->q_head_stride}))
        return KVR_ERR_ALIGNMENT;
    const kvr_status st = kvc_check_scoring(c, a->scoring);
    if (st != KVR_OK) return st;
    if (!kvc_on_device(c)) return KVR_ERR_INVALID_ARG;
    if (a->num_requests == 0) return KVR_OK;
    return together(c, [&] { return kvc_weigh_launch(c, layer, a, stream); });
}

extern "C" kvr_status kv_cache_evict(const kvc_cache *c, int32_t layer, const kvc_evict *a, void *stream) {
    if (c == nullptr || a == nullptr) return KVR_ERR_INVALID_ARG;
    const kvc_desc &d = c->d;
    if (layer < 0 || layer >= d.num_layers) return KVR_ERR_LAYER_RANGE;
    if (c->latent()) return KVR_ERR_UNSUPPORTED;
    if (a->num_requests < 0 || a->keep < 1 || a->recent < 0 || a->recent > a->keep || a->reserved != 0 ||
        a->weights_width < 0 || !kvc_ok_table(a->table) || a->table.rows < a->num_requests ||
        !kvc_ok_table(a->into) || (a->into.ids != nullptr && a->into.rows < a->num_requests))
        return KVR_ERR_INVALID_ARG;
    // (no table at all means in place; one without entries is a mistake that would rewrite the requests' own blocks)
    if (a->num_requests > 0 && a->into.ids == nullptr &&
        (a->into.rows != 0 || a->into.width != 0 || a->into.stride != 0))
        return KVR_ERR_INVALID_ARG;
    // a table in another form of the same memory would be neither in place nor apart
    if (a->into.ids != nullptr && a->into.ids == a->table.ids &&
        (a->into.width != a->table.width || (a->num_requests > 1 && a->into.stride != a->table.stride)))
        return KVR_ERR_INVALID_ARG;
    // positions are 32-bit: a table row must not describe more of them
    for (const kvc_table *t : {&a->table, &a->into})
        if ((int64_t)t->width * d.block_size > (int64_t)INT32_MAX - KVC_MAX_REQUESTS) return KVR_ERR_UNSUPPORTED;
    if (a->num_requests > KVC_MAX_REQUESTS || a->weights_width > INT32_MAX - KVC_MAX_REQUESTS ||
        a->keep > INT32_MAX - KVC_MAX_REQUESTS)
        return KVR_ERR_UNSUPPORTED;
    if (a->num_requests > 0 && (a->lengths == nullptr || a->kept == nullptr ||
                                (a->weights_width > 0 && (a->weights == nullptr || a->weights_out == nullptr))))
        return KVR_ERR_INVALID_ARG;
    if (negative({a->weights_request_stride, a->weights_head_stride, a->out_request_stride, a->out_head_stride}))
        return KVR_ERR_INVALID_ARG;
    if (a->weights == a->weights_out && (a->weights_request_stride != a->out_request_stride ||
                                         a->weights_head_stride != a->out_head_stride))
        return KVR_ERR_INVALID_ARG;
    // (each head's weights are written by blocks of its own)
    if (!disjoint_rows(a->num_requests, a->out_request_stride, d.kv_heads, a->out_head_stride, a->weights_width))
        return KVR_ERR_POOL_OVERLAP;
    if (!multiples(4, {address(a->lengths), address(a->weights), address(a->weights_out), address(a->kept)}))
        return KVR_ERR_ALIGNMENT;
    if (!kvc_on_device(c)) return KVR_ERR_INVALID_ARG;
    if (a->num_requests == 0) return KVR_OK;
    return together(c, [&] { return kvc_evict_launch(c, layer, a, stream); });
}

extern "C" kvr_status kv_cache_read(const kvc_cache *c, int32_t layer, const kvc_read *a, void *stream) {
    if (c == nullptr || a == nullptr) return KVR_ERR_INVALID_ARG;
    if (layer < 0 || layer >= c->d.num_layers) return KVR_ERR_LAYER_RANGE;
    if (a->num_tokens < 0 || !kvc_ok_table(a->table)) return KVR_ERR_INVALID_ARG;
    if (a->num_tokens > 0 && (a->requests == nullptr || a->positions == nullptr || a->k == nullptr ||
                              (a->v == nullptr) != c->latent()))
        return KVR_ERR_INVALID_ARG;
    if (!kvc_type_fits(c, a->dtype)) return KVR_ERR_UNSUPPORTED;
    if (negative({a->k_token_stride, a->k_head_stride, a->v_token_stride, a->v_head_stride}))
        return KVR_ERR_INVALID_ARG;
    if (!multiples(4, {address(a->requests), address(a->positions)}) ||
        !multiples(16, {address(a->k), address(a->v), a->k_token_stride, a->k_head_stride,
                        a->v_token_stride, a->v_head_stride}))
        return KVR_ERR_ALIGNMENT;
    // (each row is written by threads of its own)
    const int32_t H = c->d.kv_heads, row = 2 * c->d.head_dim;
    if (a->num_tokens > 0 &&
        (!disjoint_rows(a->num_tokens, a->k_token_stride, H, a->k_head_stride, row) ||
         (!c->latent() && !disjoint_rows(a->num_tokens, a->v_token_stride, H, a->v_head_stride, row))))
        return KVR_ERR_POOL_OVERLAP;
    if (!kvc_on_device(c)) return KVR_ERR_INVALID_ARG;
    if (a->num_tokens == 0) return KVR_OK;
    return guarded([&] { return kvc_read_launch(c, layer, a, stream); });
}
