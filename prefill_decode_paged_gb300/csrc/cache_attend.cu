// cache_attend.cu -- attention of a request's newest tokens over its paged cache.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "cache_attend.cuh"

namespace {

using namespace kvc;

struct SimpleArgs {
    KvcPlane k_plane, v_plane;
    KvcSlots slots;
    const int32_t *lengths;
    const unsigned char *q;
    unsigned char *out;
    float *lse;
    int64_t q_request, q_token, q_head, out_request, out_token, out_head;
    const float *k_scale, *v_scale;
    uint32_t *flags;
    int32_t requests, m, Hq, H, G, D, V, window, f16, pool;
    float scale;
};

__device__ __forceinline__ float elem(const unsigned char *p, int32_t type, int i) {
    if (type == KVR_DTYPE_FP8_E4M3) return widen2<true>(e4m3_to_f16x2(p[i])).x;
    const uint32_t w = ((const unsigned short *)p)[i];
    return type == KVC_DTYPE_F16 ? widen2<true>(w).x : widen2<false>(w).x;
}

// One warp a query row: lanes over the row's elements, one key after another.
__global__ void __launch_bounds__(128) attend_simple(SimpleArgs a) {
    wait_for_previous();
    const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= (int64_t)a.requests * a.m * a.Hq) return;
    const int32_t hq = (int32_t)(row % a.Hq), i = (int32_t)(row / a.Hq % a.m),
                  r = (int32_t)(row / a.Hq / a.m), h = hq / a.G;
    int32_t len = a.lengths[r];
    const int32_t most = a.slots.width * (int32_t)a.slots.block.d;
    if (len < 0 || len > most) {
        if (lane == 0) atomicOr(a.flags, KVC_FLAG_LENGTH);
        len = len < 0 ? 0 : most;
    }
    const int32_t p = len - a.m + i;
    const int32_t first = a.window > 0 ? max(0, p - a.window + 1) : 0;
    const unsigned char *q = a.q + r * a.q_request + i * a.q_token + hq * a.q_head;
    float qv[18], acc[18];
    const float f = a.scale * (a.k_scale ? a.k_scale[h] : 1.0f);
#pragma unroll
    for (int e = 0; e < 18; ++e) {
        qv[e] = e * 32 + lane < a.D ? elem(q, a.f16 ? KVC_DTYPE_F16 : KVR_DTYPE_BF16, e * 32 + lane) : 0.0f;
        acc[e] = 0.0f;
    }
    float top = -INFINITY, total = 0.0f;
    for (int32_t j = first; j <= p; ++j) {
        const uint32_t entry = a.slots.block.div((uint32_t)j);
        const int32_t id = a.slots.ids[(int64_t)r * a.slots.stride + entry];
        if (id < 0 || id >= a.slots.num_blocks) {
            if (lane == 0) atomicOr(a.flags, KVC_FLAG_BLOCK);
            continue;
        }
        const int32_t off = j - (int32_t)(entry * a.slots.block.d);
        const unsigned char *k = a.k_plane.base + id * a.k_plane.block_stride +
                                 off * a.k_plane.token_stride + h * a.k_plane.head_stride;
        const unsigned char *v = a.v_plane.base + id * a.v_plane.block_stride +
                                 off * a.v_plane.token_stride + h * a.v_plane.head_stride;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 18; ++e)
            if (e * 32 + lane < a.D) s += qv[e] * elem(k, a.pool, e * 32 + lane);
        for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(~0u, s, o);
        s *= f;
        const float next = fmaxf(top, s);
        const float shrink = __expf(top - next), w = __expf(s - next);
        total = total * shrink + w;
        top = next;
#pragma unroll
        for (int e = 0; e < 18; ++e)
            if (e * 32 + lane < a.V)
                acc[e] = acc[e] * shrink + w * elem(v, a.pool, e * 32 + lane);
    }
    const float inv = total > 0.0f ? (a.v_scale ? a.v_scale[h] : 1.0f) / total : 0.0f;
    unsigned char *out = a.out + r * a.out_request + i * a.out_token + hq * a.out_head;
#pragma unroll
    for (int e = 0; e < 18; ++e)
        if (e * 32 + lane < a.V) {
            const uint32_t w = a.f16 ? narrow2<true>(acc[e] * inv, 0.0f) : narrow2<false>(acc[e] * inv, 0.0f);
            ((unsigned short *)out)[e * 32 + lane] = (unsigned short)w;
        }
    if (a.lse != nullptr && lane == 0) a.lse[row] = total > 0.0f ? top + logf(total) : -INFINITY;
}

AttendPick pick(const kvc_desc &d, int32_t M) {
    return d.dtype == KVR_DTYPE_FP8_E4M3 ? attend_pick_e4m3(d.head_dim, M)
           : d.dtype == KVC_DTYPE_F16    ? attend_pick_f16(d.head_dim, M)
                                         : attend_pick_bf16(d.head_dim, M);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

kvr_status simple_launch(const kvc_cache *c, int32_t layer, const kvc_attend *p, void *stream) {
    SimpleArgs a = {};
    a.k_plane = c->plane(layer, 0);
    a.v_plane = c->latent() ? a.k_plane : c->plane(layer, 1);
    a.k_scale = c->scale_of(layer, 0);
    a.v_scale = c->scale_of(layer, c->latent() ? 0 : 1);
    a.slots = c->slots(p->table);
    a.lengths = p->lengths;
    a.q = (const unsigned char *)p->q;
    a.out = (unsigned char *)p->out;
    a.lse = p->lse;
    a.q_request = p->q_request_stride, a.q_token = p->q_token_stride, a.q_head = p->q_head_stride;
    a.out_request = p->out_request_stride, a.out_token = p->out_token_stride;
    a.out_head = p->out_head_stride;
    a.flags = c->ws.flags;
    a.requests = p->num_requests, a.m = p->num_new, a.Hq = c->d.query_heads, a.H = c->d.kv_heads;
    a.G = a.Hq / a.H, a.D = c->d.head_dim, a.V = c->d.value_dim, a.window = p->window;
    a.f16 = p->dtype == KVC_DTYPE_F16, a.pool = c->d.dtype, a.scale = p->scale;
    const int64_t rows = (int64_t)a.requests * a.m * a.Hq;
    return kvc_launch(attend_simple, a, dim3((unsigned)((rows + 3) / 4)), 128, 0, stream);
}

}  // namespace

// Each block leaves at most two parts of jobs: the one it begins in and the one it ends in.
size_t kvc_attend_partial_bytes(const kvc_desc &d, int32_t sm_count) {
    if (d.num_components == 1) return 0;
    size_t rows = 0;
    for (int32_t M : {8, 16, 32}) rows = std::max(rows, (size_t)pick(d, M).rp);
    return (size_t)sm_count * 2 * 2 * rows * (size_t)(d.head_dim + 2) * sizeof(float);
}

size_t kvc_attend_jobs(const kvc_desc &d) {
    const int64_t M = (int64_t)d.max_new * (d.query_heads / d.kv_heads);
    return (size_t)d.max_requests * d.kv_heads * (size_t)ceil_div(M, 8);
}

kvr_status kvc_attend_setup(const kvc_cache *c) {
    if (c->latent()) return KVR_OK;
    for (int32_t M : {8, 16, 32}) {
        const AttendPick p = pick(c->d, M);
        if (cudaFuncSetAttribute(p.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)p.smem(KVC_MAX_REQUESTS)) != cudaSuccess) {
            cudaGetLastError();
            return KVR_ERR_CUDA;
        }
    }
    return KVR_OK;
}

kvr_status kvc_attend_launch(const kvc_cache *c, int32_t layer, const kvc_attend *p, void *stream) {
    if (c->latent()) return simple_launch(c, layer, p, stream);
    AttendArgs a = {};
    a.k_plane = c->plane(layer, 0);
    a.v_plane = c->plane(layer, 1);
    a.k_scale = c->scale_of(layer, 0);
    a.v_scale = c->scale_of(layer, 1);
    a.slots = c->slots(p->table);
    a.lengths = p->lengths;
    a.q = (const unsigned char *)p->q;
    a.out = (unsigned char *)p->out;
    a.lse = p->lse;
    a.q_request = p->q_request_stride, a.q_token = p->q_token_stride, a.q_head = p->q_head_stride;
    a.out_request = p->out_request_stride, a.out_token = p->out_token_stride;
    a.out_head = p->out_head_stride;
    a.partial = c->ws.partial;
    a.arrived = c->ws.arrived;
    a.flags = c->ws.flags;
    a.requests = p->num_requests, a.m = p->num_new, a.H = c->d.kv_heads;
    a.G = c->d.query_heads / a.H, a.D = c->d.head_dim, a.window = p->window;
    a.f16 = p->dtype == KVC_DTYPE_F16, a.scale = p->scale;
    a.group = kvr_make_div((uint32_t)a.G);
    const int32_t M = a.m * a.G;
    const AttendPick k = pick(c->d, M);
    a.chunks = (int32_t)ceil_div(M, k.rp);
    // most units of a job; the kernel counts a job of every request in 32 bits
    const int64_t most = ceil_div((int64_t)p->table.width * c->d.block_size, k.unit) + 1;
    if (most * a.requests > INT32_MAX) return KVR_ERR_UNSUPPORTED;
    const size_t smem = k.smem(a.requests);
    // an SM has 228 KB, of which each block takes 1 KB for itself
    const int64_t resident = std::min<int64_t>(k.blocks, (228 << 10) / (int64_t)(smem + 1024));
    const int64_t grid = std::min<int64_t>(resident * kvc_stream_sms(c, stream),
                                           most * a.requests * a.H * a.chunks);
    return kvc_launch(k.kernel, a, dim3((unsigned)grid), ATTEND_THREADS, smem, stream);
}
