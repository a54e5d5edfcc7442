// cache_read.cu -- tokens' keys and values out of a paged pool, as 16-bit rows.
//
// The inverse of append, for what works on contiguous rows: attention of a new prompt over a cached prefix, or a
// cache that moves to another type of pool. 16-bit pools are copied, codes become code * block scale * s, exact up
// to the product with s, which is fp32 and rounded once. One block does one token; a thread takes 16 elements
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
    int32_t H, comps;
    KvrDiv units;             // of 16 elements, of a row
};

constexpr int MOST_THREADS = 256;

template <int POOL, bool F16>
__global__ void __launch_bounds__(MOST_THREADS) read_kernel(ReadArgs a) {
    wait_for_previous();
    let_next_start();
    const int64_t token = blockIdx.x;
    const int32_t pos = __ldg(a.positions + token), req = __ldg(a.requests + token);
    int64_t slot = -1;                       // the token's slot in a plane, in bytes; -1: zeros
    if (pos >= 0) {
        const uint32_t entry = a.slots.block.div((uint32_t)pos);
        uint32_t bad = 0;
        if (req < 0 || req >= a.slots.rows) {
            bad = KVC_FLAG_REQUEST;
        } else if (entry >= (uint32_t)a.slots.width) {
            bad = KVC_FLAG_POSITION;
        } else {
            const int32_t id = __ldg(a.slots.ids + (int64_t)req * a.slots.stride + entry);
            const int32_t off = pos - (int32_t)(entry * a.slots.block.d);
            if (id < 0 || id >= a.slots.num_blocks)
                bad = KVC_FLAG_BLOCK;
            else
                slot = id * a.k_plane.block_stride + off * a.k_plane.token_stride;
        }
        if (bad != 0 && threadIdx.x == 0) atomicOr(a.flags, bad);
    }
    const int32_t n = a.comps * a.H * (int32_t)a.units.d;
    for (int32_t t = threadIdx.x; t < n; t += blockDim.x) {
        int32_t row = (int32_t)a.units.div((uint32_t)t);
        const int32_t j = t - row * (int32_t)a.units.d;
        const bool value = row >= a.H;
        if (value) row -= a.H;
        const unsigned char *base = (value ? a.v_plane : a.k_plane).base;
        const int64_t at = slot + row * a.k_plane.head_stride;
        unsigned char *to = (value ? a.v + token * a.v_token + row * a.v_head
                                   : a.k + token * a.k_token + row * a.k_head) + 32 * j;
        uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (slot >= 0) {
            if constexpr (POOL == KVR_DTYPE_FP8_E4M3 || POOL == KVC_DTYPE_E2M1) {
                const float s = __ldg((value ? a.v_scale : a.k_scale) + row);
                uint32_t h[8], *o = (uint32_t *)out;
                float by = s;
                if constexpr (POOL == KVC_DTYPE_E2M1) {
                    const uint2 w = __ldg((const uint2 *)(base + at + 8 * j));
                    const uint32_t b = __ldg((value ? a.v_block_scales : a.k_block_scales) + at / 8 + j);
                    e2m1_to_f16x2(w.x, h);
                    e2m1_to_f16x2(w.y, h + 4);
                    const float scale = widen2<true>(e4m3_to_f16x2(b)).x;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = widen2<true>(h[i]);
                        o[i] = narrow2<F16>(f.x * scale * by, f.y * scale * by);
                    }
                } else {
                    const uint4 w = __ldg((const uint4 *)(base + at + 16 * j));
                    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = widen2<true>(e4m3_to_f16x2(i % 2 == 0 ? c[i / 2] : c[i / 2] >> 16));
                        o[i] = narrow2<F16>(f.x * by, f.y * by);
                    }
                }
            } else {
                out[0] = __ldg((const uint4 *)(base + at + 32 * j));
                out[1] = __ldg((const uint4 *)(base + at + 32 * j) + 1);
            }
        }
        *(uint4 *)to = out[0];
        *(uint4 *)(to + 16) = out[1];
    }
}

}  // namespace

kvr_status kvc_read_launch(const kvc_cache *c, int32_t layer, const kvc_read *p, void *stream) {
    ReadArgs a = {};
    a.comps = c->d.num_components, a.H = c->d.kv_heads;
    a.k_plane = c->plane(layer, 0);
    a.k_scale = c->scale_of(layer, 0);
    a.k_block_scales = c->block_scales(layer, 0);
    if (a.comps == 2) {
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
    const int64_t n = (int64_t)a.comps * a.H * a.units.d, rounds = (n + MOST_THREADS - 1) / MOST_THREADS;
    const int threads = (int)((n + 32 * rounds - 1) / (32 * rounds)) * 32;
    const bool f16 = p->dtype == KVC_DTYPE_F16;
    const auto kernel =
        c->d.dtype == KVC_DTYPE_E2M1
            ? (f16 ? read_kernel<KVC_DTYPE_E2M1, true> : read_kernel<KVC_DTYPE_E2M1, false>)
        : c->d.dtype == KVR_DTYPE_FP8_E4M3
            ? (f16 ? read_kernel<KVR_DTYPE_FP8_E4M3, true> : read_kernel<KVR_DTYPE_FP8_E4M3, false>)
            : read_kernel<KVR_DTYPE_BF16, false>;       // (16-bit rows are copied, whichever they are)
    return kvc_launch(kernel, a, dim3((unsigned)p->num_tokens), threads, 0, stream);
}
