// cache_weigh.cu -- how much attention the cached keys got: instances and launch.
#include "cache_weigh.cuh"

#include <limits.h>

#include <algorithm>

namespace {

using namespace kvc;

WeighPick pick(const kvc_desc &d, int32_t M) {
    return d.dtype == KVR_DTYPE_FP8_E4M3 ? weigh_pick_e4m3(d.head_dim, M)
           : d.dtype == KVC_DTYPE_E2M1   ? weigh_pick_e2m1(d.head_dim, M)
           : d.dtype == KVC_DTYPE_F16    ? weigh_pick_f16(d.head_dim, M)
                                         : weigh_pick_bf16(d.head_dim, M);
}

}  // namespace

kvr_status kvc_weigh_setup(kvc_cache *c) {
    for (int32_t M : {8, 16, 32, 64}) {
        const WeighPick p = pick(c->d, M);
        if (cudaFuncSetAttribute(p.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)p.smem(KVC_MAX_REQUESTS)) != cudaSuccess) {
            cudaGetLastError();
            return KVR_ERR_CUDA;
        }
    }
    return KVR_OK;
}

kvr_status kvc_weigh_launch(const kvc_cache *c, int32_t layer, const kvc_weigh *p, void *stream) {
    WeighArgs a = {};
    a.k_plane = c->plane(layer, 0);
    a.k_scale = c->scale_of(layer, 0);
    a.k_block_scales = c->block_scales(layer, 0);
    a.split = {c->slots(p->table), p->lengths, c->ws.flags, p->num_requests, p->num_new, p->window};
    a.q = (const unsigned char *)p->q;
    a.lse = p->lse;
    a.weights = p->weights;
    a.q_request = p->q_request_stride, a.q_token = p->q_token_stride, a.q_head = p->q_head_stride;
    a.w_request = p->weights_request_stride, a.w_head = p->weights_head_stride;
    a.width = p->weights_width, a.add = p->add;
    a.m = p->num_new, a.H = c->d.kv_heads, a.G = c->d.query_heads / a.H, a.D = c->d.head_dim;
    a.f16 = p->dtype == KVC_DTYPE_F16, a.scale = p->scale;
    a.scoring = make_scoring(&p->scoring);
    a.group = kvr_make_div((uint32_t)a.G);
    const int32_t M = a.m * a.G;
    const WeighPick k = pick(c->d, M);
    a.chunks = (M + k.rp - 1) / k.rp;
    // most units of a job; the kernel counts those of all jobs in 32 bits
    const int64_t most = ((int64_t)p->table.width * c->d.block_size + k.unit - 1) / k.unit + 1;
    const int64_t all = most * p->num_requests * a.H;
    if (all > INT32_MAX) return KVR_ERR_UNSUPPORTED;
    const size_t smem = k.smem(p->num_requests);
    // an SM has 228 KB, of which each block takes 1 KB for itself
    const int64_t resident = std::min<int64_t>(k.blocks, (228 << 10) / (int64_t)(smem + 1024));
    const int64_t grid = std::min<int64_t>(resident * kvc_stream_sms(c, stream), all);
    a.by_heads = kvr_make_div((uint32_t)a.H);
    a.parts = (int32_t)(k.abreast ? std::max<int64_t>(1, grid / a.H) : grid);
    a.shape = make_cut_shape(p->num_requests, k.abreast ? 1 : a.H, a.parts, 0);
    return kvc_launch(k.kernel, a, dim3((unsigned)(k.abreast ? a.parts * a.H : grid)), ATTEND_THREADS, smem, stream);
}
