// cache_read.cu -- tokens' keys and values out of a paged pool, as 16-bit rows.
//
// The inverse of append, for what works on contiguous rows: attention of a new prompt over a cached prefix, or a
// cache that moves to another type of pool. 16-bit pools are copied, codes become code * block scale * s, exact up
// to the product with s, which is fp32 and rounded once. A thread takes 16 elements of each of a block's tokens
// at a time. Bound by HBM with many tokens (a 4-bit row is 0.56 bytes read for 2 written an element), by the
// launch and then position, block id and row, one after another, with few.
#include "cache.h"

namespace {

using namespace kvc;

struct ReadArgs {
    KvcPlane k_plane, v_plane;
    const unsigned char *k_block_scales, *v_block_scales;
    unsigned char *k, *v;
    int64_t k_token, k_head, v_token, v_head;
    const int32_t *requests, *positions;
    KvcSlots slots;
    const float *k_scale, *v_scale;
    uint32_t *flags;
    int32_t H, tokens;
    KvrDiv units;             // of 16 elements, of a row
};

constexpr int MOST_THREADS = 256;

// Where a token's rows begin in a plane, in bytes; -1: nowhere.
__device__ __forceinline__ int64_t slot_of(const ReadArgs &a, int32_t pos, int32_t req, uint32_t *bad) {
    if (pos < 0) return -1;
    const uint32_t entry = a.slots.block.div((uint32_t)pos);
    if (req < 0 || req >= a.slots.rows) {
        *bad |= KVC_FLAG_REQUEST;
        return -1;
    }
    if (entry >= (uint32_t)a.slots.width) {
        *bad |= KVC_FLAG_POSITION;
        return -1;
    }
    const int32_t id = __ldg(a.slots.ids + (int64_t)req * a.slots.stride + entry);
    const int32_t off = pos - (int32_t)(entry * a.slots.block.d);
    if (id < 0 || id >= a.slots.num_blocks) {
        *bad |= KVC_FLAG_BLOCK;
        return -1;
    }
    return id * a.k_plane.block_stride + off * a.k_plane.token_stride;
}

// 16 elements of a pool as they lie there, and as 16-bit numbers.
template <int POOL>
struct Raw {
    uint4 w[POOL == KVR_DTYPE_FP8_E4M3 || POOL == KVC_DTYPE_E2M1 ? 1 : 2];
    uint32_t scale;

    __device__ __forceinline__ void load(const unsigned char *row, const unsigned char *scales, int32_t j) {
        if constexpr (POOL == KVC_DTYPE_E2M1) {
            const uint2 c = __ldg((const uint2 *)(row + 8 * j));
            w[0].x = c.x, w[0].y = c.y;
            scale = __ldg(scales + j);
        } else if constexpr (POOL == KVR_DTYPE_FP8_E4M3) {
            w[0] = __ldg((const uint4 *)(row + 16 * j));
        } else {
            w[0] = __ldg((const uint4 *)(row + 32 * j));
            w[1] = __ldg((const uint4 *)(row + 32 * j) + 1);
        }
    }
    // `s`: the plane's scale
    template <bool F16>
    __device__ __forceinline__ void store(unsigned char *to, float s, bool some) const {
        uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        uint32_t *o = (uint32_t *)out;
        if (!some) {
        } else if constexpr (POOL == KVC_DTYPE_E2M1) {
            uint32_t h[8];
            e2m1_to_f16x2(w[0].x, h);
            e2m1_to_f16x2(w[0].y, h + 4);
            const float by = widen2<true>(e4m3_to_f16x2(scale)).x;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = widen2<true>(h[i]);
                o[i] = narrow2<F16>(f.x * by * s, f.y * by * s);
            }
        } else if constexpr (POOL == KVR_DTYPE_FP8_E4M3) {
            const uint32_t c[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = widen2<true>(e4m3_to_f16x2(i % 2 == 0 ? c[i / 2] : c[i / 2] >> 16));
                o[i] = narrow2<F16>(f.x * s, f.y * s);
            }
        } else {
            out[0] = w[0], out[1] = w[1];
        }
        *(uint4 *)to = out[0];
        *(uint4 *)(to + 16) = out[1];
    }
};

template <int POOL, bool F16, int TOKENS>
__global__ void __launch_bounds__(MOST_THREADS) read_kernel(ReadArgs a) {
    constexpr bool CODES = POOL == KVR_DTYPE_FP8_E4M3 || POOL == KVC_DTYPE_E2M1;
    wait_for_previous();
    let_next_start();
    const int64_t first = (int64_t)blockIdx.x * TOKENS;
    int32_t pos[TOKENS], req[TOKENS];
#pragma unroll
    for (int k = 0; k < TOKENS; ++k) {
        const bool some = first + k < a.tokens;
        pos[k] = some ? __ldg(a.positions + first + k) : -1;
        req[k] = some ? __ldg(a.requests + first + k) : 0;
    }
    int64_t slot[TOKENS];                    // -1: zeros
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < TOKENS; ++k) slot[k] = slot_of(a, pos[k], req[k], &bad);
    if (bad != 0 && threadIdx.x == 0) atomicOr(a.flags, bad);
    const int32_t n = a.H * (int32_t)a.units.d;
    // (a key's unit and its value's by one thread: the same offsets)
    for (int32_t t = threadIdx.x; t < n; t += blockDim.x) {
        const int32_t row = (int32_t)a.units.div((uint32_t)t), j = t - row * (int32_t)a.units.d;
        const int64_t head = row * a.k_plane.head_stride;
        const bool values = a.v != nullptr;
        Raw<POOL> key[TOKENS], value[TOKENS];
#pragma unroll
        for (int k = 0; k < TOKENS; ++k) {
            const int64_t at = slot[k] + head;
            if (slot[k] >= 0) key[k].load(a.k_plane.base + at, a.k_block_scales + at / 8, j);
            if (slot[k] >= 0 && values) value[k].load(a.v_plane.base + at, a.v_block_scales + at / 8, j);
        }
        const float ks = CODES ? __ldg(a.k_scale + row) : 1.0f;
        const float vs = CODES && values ? __ldg(a.v_scale + row) : 1.0f;
        unsigned char *k_to = a.k + first * a.k_token + row * a.k_head + 32 * j;
        unsigned char *v_to = a.v + first * a.v_token + row * a.v_head + 32 * j;
#pragma unroll
        for (int k = 0; k < TOKENS; ++k) {
            if (first + k >= a.tokens) break;
            key[k].template store<F16>(k_to, ks, slot[k] >= 0);
            if (values) value[k].template store<F16>(v_to, vs, slot[k] >= 0);
            k_to += a.k_token, v_to += a.v_token;
        }
    }
}

// Few tokens: a block each. Many: two to a block, so that their chains of waits go side by side (41931
// tokens of 16 rows of 4 bits 40 us; four 44, one 52).
template <int POOL, bool F16>
kvr_status go(ReadArgs &a, int sms, void *stream) {
    const int64_t n = (int64_t)a.H * a.units.d, rounds = (n + MOST_THREADS - 1) / MOST_THREADS;
    const int threads = (int)((n + 32 * rounds - 1) / (32 * rounds)) * 32;
    if (a.tokens > 16 * sms)
        return kvc_launch(read_kernel<POOL, F16, 2>, a, dim3((unsigned)(a.tokens / 2 + a.tokens % 2)), threads, 0, stream);
    return kvc_launch(read_kernel<POOL, F16, 1>, a, dim3((unsigned)a.tokens), threads, 0, stream);
}

}  // namespace

kvr_status kvc_read_launch(const kvc_cache *c, int32_t layer, const kvc_read *p, void *stream) {
    ReadArgs a = {};
    a.H = c->d.kv_heads;
    a.k_plane = c->plane(layer, 0);
    a.k_scale = c->scale_of(layer, 0);
    a.k_block_scales = c->block_scales(layer, 0);
    if (!c->latent()) {
        a.v_plane = c->plane(layer, 1);
        a.v_scale = c->scale_of(layer, 1);
        a.v_block_scales = c->block_scales(layer, 1);
    }
    a.k = (unsigned char *)p->k, a.v = (unsigned char *)p->v;
    a.k_token = p->k_token_stride, a.k_head = p->k_head_stride;
    a.v_token = p->v_token_stride, a.v_head = p->v_head_stride;
    a.requests = p->requests;
    a.positions = p->positions;
    a.slots = c->slots(p->table);
    a.flags = c->ws.flags;
    a.units = kvr_make_div((uint32_t)c->d.head_dim / 16);
    a.tokens = p->num_tokens;
    const bool f16 = p->dtype == KVC_DTYPE_F16;
    if (c->d.dtype == KVC_DTYPE_E2M1)
        return f16 ? go<KVC_DTYPE_E2M1, true>(a, c->sm_count, stream)
                   : go<KVC_DTYPE_E2M1, false>(a, c->sm_count, stream);
    if (c->d.dtype == KVR_DTYPE_FP8_E4M3)
        return f16 ? go<KVR_DTYPE_FP8_E4M3, true>(a, c->sm_count, stream)
                   : go<KVR_DTYPE_FP8_E4M3, false>(a, c->sm_count, stream);
    return go<KVR_DTYPE_BF16, false>(a, c->sm_count, stream);      // (16-bit rows are copied, whichever they are)
}
