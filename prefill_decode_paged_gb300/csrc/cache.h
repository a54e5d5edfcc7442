// cache.h -- what the decode-side cache's host code and kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>
#include <vector>

#include "kv_cache.h"
#include "kvr_index.h"

#define KVC_LATENT_DIM 576
#define KVC_LATENT_VALUES 512

// One plane (layer, component) of a pool: slot (b, t, h) starts at
// base + b * block_stride + t * token_stride + h * head_stride.
struct KvcPlane {
    unsigned char *base;
    int64_t block_stride, token_stride, head_stride;
};

// A block table and what turns a position into a slot of the pool.
struct KvcSlots {
    const int32_t *ids;
    int64_t stride;
    int32_t rows, width;
    int32_t num_blocks;
    KvrDiv block;
};

// Where the attention calls of a cache keep what their parts hand to one another.
struct KvcWorkspace {
    unsigned char *mem;       // one allocation
    size_t bytes;
    float *scales;            // [L][C][H] (E4M3 pools)
    float *partial;           // attend: accumulators of key ranges that another part finishes
    uint32_t *arrived;        // attend: parts of a job that are done, zero between launches; latents:
                              // units and parts before each request, from the products to the join
    uint32_t *flags;          // KVC_FLAG_* found by the kernels
};

struct kvc_cache {
    kvc_desc d = {};
    std::vector<uint64_t> base;       // [L][C]
    std::vector<float> scales;        // [L][C][H]
    int64_t block_stride = 0, token_stride = 0, head_stride = 0;
    int64_t row_bytes = 0;
    int64_t span = 0;                 // bytes from a plane's base to its end
    KvrDiv block = {};
    KvcWorkspace ws = {};
    std::vector<CUtensorMap> maps;    // copy-engine maps of the planes, two a layer
    int32_t piece = 0;                // tokens of a map's box; 0: there are no maps
    int device = 0;
    int sm_count = 0;
    mutable std::mutex use;           // held over the two launches of an attention over latents

    KvcPlane plane(int32_t layer, int32_t comp) const {
        return {(unsigned char *)(uintptr_t)base[(size_t)layer * d.num_components + comp],
                block_stride, token_stride, head_stride};
    }
    KvcSlots slots(const kvc_table &t) const {
        return {t.ids, t.stride, t.rows, t.width, (int32_t)d.num_blocks, block};
    }
    const float *scale_of(int32_t layer, int32_t comp) const {
        return ws.scales == nullptr
                   ? nullptr
                   : ws.scales + ((size_t)layer * d.num_components + comp) * d.kv_heads;
    }
    bool latent() const { return d.num_components == 1; }
};

inline int kvc_elem_bytes(int32_t dtype) { return dtype == KVR_DTYPE_FP8_E4M3 ? 1 : 2; }

// SMs that a launch on `stream` may use (sm_stream.cpp tells a green context's).
int32_t kvr_stream_green_sms(void *stream);
inline int kvc_stream_sms(const kvc_cache *c, void *stream) {
    const int32_t green = kvr_stream_green_sms(stream);
    return green > 0 && green < c->sm_count ? green : c->sm_count;
}

// One launch on `stream` whose kernel may start before the kernel ahead of it has finished: it
// waits (griddepcontrol.wait) before it touches global memory.
template <typename Args>
inline kvr_status kvc_launch(void (*kernel)(Args), const Args &a, dim3 grid, int threads,
                             size_t smem, void *stream, int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess) return KVR_OK;
    cudaGetLastError();
    return KVR_ERR_CUDA;
}

// cache.cpp: a copy-engine map of a plane of `es`-byte elements, `dims` from the innermost on,
// byte strides of the others (0 where the extent is 1), swizzled in lines of 128 or 64 bytes.
// False if the driver has none for it.
bool kvc_make_map(CUtensorMap *map, int es, int rank, uint64_t base, int64_t row_bytes,
                  const uint64_t *dims, const int64_t *strides, const uint32_t *box, int line);

// cache_attend.cu, cache_latent.cu: the launches behind kv_cache_attend(), and what they want
// of the workspace. (`setup` runs once a cache: shared memory limits of the kernels.)
kvr_status kvc_attend_launch(const kvc_cache *c, int32_t layer, const kvc_attend *a, void *stream);
size_t kvc_attend_partial_bytes(const kvc_desc &d, int32_t sm_count);
size_t kvc_attend_jobs(const kvc_desc &d);
kvr_status kvc_attend_setup(kvc_cache *c);
// cache_append.cu
kvr_status kvc_append_launch(const kvc_cache *c, int32_t layer, const kvc_append *a, void *stream);

#if defined(__CUDACC__)

namespace kvc {

__device__ __forceinline__ void wait_for_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The two halves of a 32-bit word as fp32 (exact), and back with one rounding each.
template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
    if (F16) {
        float2 f;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
            "cvt.f32.f16 %1, h;\n\t}"
            : "=f"(f.x), "=f"(f.y)
            : "r"(w));
        return f;
    }
    return make_float2(bf16_lo(w), bf16_hi(w));
}
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    uint32_t w;
    if (F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// Two E4M3 codes (the low one first) as f16x2: exact, a NaN code gives a NaN.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two_codes) {
    uint32_t h2;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(h2)
        : "r"(two_codes));
    return h2;
}

}  // namespace kvc

#endif
