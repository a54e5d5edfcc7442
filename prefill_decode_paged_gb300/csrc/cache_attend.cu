// cache_attend.cu -- attention of a request's newest tokens over its paged cache.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "cache_attend.cuh"
#include "cache_latent.h"

namespace {

using namespace kvc;

AttendPick pick(const kvc_desc &d, int32_t M) {
    return d.dtype == KVR_DTYPE_FP8_E4M3 ? attend_pick_e4m3(d.head_dim, M)
           : d.dtype == KVC_DTYPE_F16    ? attend_pick_f16(d.head_dim, M)
                                         : attend_pick_bf16(d.head_dim, M);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Each block leaves at most two parts of jobs: the one it begins in and the one it ends in.
size_t kvc_attend_partial_bytes(const kvc_desc &d, int32_t sm_count) {
    if (d.num_components == 1) return kvc_latent_partial_bytes(sm_count);
    size_t rows = 0;
    for (int32_t M : {8, 16, 32}) rows = std::max(rows, (size_t)pick(d, M).rp);
    return (size_t)sm_count * 2 * 2 * rows * (size_t)(d.head_dim + 2) * sizeof(float);
}

size_t kvc_attend_jobs(const kvc_desc &d) {
    if (d.num_components == 1) return 2 * ((size_t)d.max_requests + 1);   // latents: units and parts before each request
    const int64_t M = (int64_t)d.max_new * (d.query_heads / d.kv_heads);
    return (size_t)d.max_requests * d.kv_heads * (size_t)ceil_div(M, 8);
}

kvr_status kvc_attend_setup(kvc_cache *c) {
    if (c->latent()) return kvc_latent_setup(c);
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
    if (c->latent()) return kvc_latent_launch(c, layer, p, stream);
    AttendArgs a = {};
    a.k_plane = c->plane(layer, 0);
    a.v_plane = c->plane(layer, 1);
    a.k_scale = c->scale_of(layer, 0);
    a.v_scale = c->scale_of(layer, 1);
    a.split = {c->slots(p->table), p->lengths, c->ws.flags, p->num_requests, p->num_new, p->window};
    a.q = (const unsigned char *)p->q;
    a.out = (unsigned char *)p->out;
    a.lse = p->lse;
    a.q_request = p->q_request_stride, a.q_token = p->q_token_stride, a.q_head = p->q_head_stride;
    a.out_request = p->out_request_stride, a.out_token = p->out_token_stride;
    a.out_head = p->out_head_stride;
    a.partial = c->ws.partial;
    a.arrived = c->ws.arrived;
    a.m = p->num_new, a.H = c->d.kv_heads, a.G = c->d.query_heads / a.H, a.D = c->d.head_dim;
    a.f16 = p->dtype == KVC_DTYPE_F16, a.scale = p->scale;
    a.group = kvr_make_div((uint32_t)a.G);
    const int32_t M = a.m * a.G;
    const AttendPick k = pick(c->d, M);
    a.chunks = (int32_t)ceil_div(M, k.rp);
    // most units of a job; the kernel counts those of all jobs in 32 bits
    const int64_t most = ceil_div((int64_t)p->table.width * c->d.block_size, k.unit) + 1;
    const int64_t all = most * p->num_requests * a.H * a.chunks;
    if (all > INT32_MAX) return KVR_ERR_UNSUPPORTED;
    const size_t smem = k.smem(p->num_requests);
    // an SM has 228 KB, of which each block takes 1 KB for itself
    const int64_t resident = std::min<int64_t>(k.blocks, (228 << 10) / (int64_t)(smem + 1024));
    const int64_t grid = std::min<int64_t>(resident * kvc_stream_sms(c, stream), all);
    a.by_chunks = kvr_make_div((uint32_t)a.chunks);
    a.shape = make_cut_shape(p->num_requests, a.H * a.chunks, (int32_t)grid, SLACK);
    return kvc_launch(k.kernel, a, dim3((unsigned)grid), ATTEND_THREADS, smem, stream);
}
