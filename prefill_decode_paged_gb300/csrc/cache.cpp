// cache.cpp -- host side of the decode cache: validation, workspace, rotation tables.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <vector>

#include "cache.h"
#include "device_free.h"

namespace {

bool mul_fits(std::initializer_list<int64_t> xs, int64_t *out) {
    __int128 p = 1;
    for (int64_t x : xs) {
        p *= x;
        if (p > (__int128)INT64_MAX) return false;
    }
    *out = (int64_t)p;
    return true;
}

// The slots of a view must not overlap, for appends write them: sorted by stride, each
// dimension of extent > 1 steps over the whole extent of the smaller ones.
bool slots_are_disjoint(int64_t N, int64_t bs, int64_t B, int64_t ts, int64_t H, int64_t hs,
                        int64_t row) {
    std::vector<std::pair<int64_t, int64_t>> dims;   // (stride, extent)
    if (N > 1) dims.push_back({bs, N});
    if (B > 1) dims.push_back({ts, B});
    if (H > 1) dims.push_back({hs, H});
    std::sort(dims.begin(), dims.end());
    __int128 inner = row;
    for (const auto &dm : dims) {
        if ((__int128)dm.first < inner) return false;
        inner += (__int128)(dm.second - 1) * dm.first;
    }
    return true;
}

kvr_status build(const kvc_desc *desc, kvc_cache *c) {
    if (desc == nullptr) return KVR_ERR_INVALID_ARG;
    c->d = *desc;
    kvc_desc &d = c->d;
    const int32_t L = d.num_layers, C = d.num_components, H = d.kv_heads, D = d.head_dim;
    if (L < 1 || (C != 1 && C != 2) || H < 1 || D < 1 || d.block_size < 1 || d.num_blocks < 1 ||
        d.value_dim < 0 || (d.per_head != 0 && d.per_head != 1) || d.query_heads < 0)
        return KVR_ERR_INVALID_ARG;
    if (d.dtype != KVR_DTYPE_BF16 && d.dtype != KVC_DTYPE_F16 && d.dtype != KVR_DTYPE_FP8_E4M3 &&
        d.dtype != KVC_DTYPE_E2M1)
        return KVR_ERR_UNSUPPORTED;
    const bool four = d.dtype == KVC_DTYPE_E2M1;
    if (four && (C != 2 || D % 64 != 0)) return KVR_ERR_UNSUPPORTED;
    if (d.num_blocks > INT32_MAX || (int64_t)L * C > (int64_t)1 << 26) return KVR_ERR_UNSUPPORTED;
    if (d.value_dim == 0) d.value_dim = C == 1 ? KVC_LATENT_VALUES : D;
    if (C == 1) {
        if (H != 1 || D != KVC_LATENT_DIM || d.value_dim != KVC_LATENT_VALUES)
            return KVR_ERR_UNSUPPORTED;
        if (d.dtype == KVR_DTYPE_FP8_E4M3 && d.query_heads > 0) return KVR_ERR_UNSUPPORTED;
    } else if (D % 16 != 0 || D > 256 || d.value_dim != D) {
        return KVR_ERR_UNSUPPORTED;
    }
    if (d.query_heads > 0) {
        if (d.query_heads % H != 0 || d.max_requests < 1 || d.max_new < 1)
            return KVR_ERR_INVALID_ARG;
        if (d.max_requests > KVC_MAX_REQUESTS || d.query_heads > 4096 || d.max_new > 4096)
            return KVR_ERR_UNSUPPORTED;
    }
    const int64_t row = kvc_row_bytes(d.dtype, D);
    c->row_bytes = row;
    c->block = kvr_make_div((uint32_t)d.block_size);

    c->scales.clear();
    if (d.dtype == KVR_DTYPE_FP8_E4M3 || four) {
        if (d.scales == nullptr && !four) return KVR_ERR_INVALID_ARG;
        for (int64_t v = 0; v < (int64_t)L * C; ++v)
            for (int32_t h = 0; h < H; ++h) {
                const float s = d.scales == nullptr ? 1.0f : d.scales[d.per_head ? v * H + h : v];
                if (!(s > 0.0f) || !std::isfinite(s)) return KVR_ERR_INVALID_ARG;
                c->scales.push_back(s);
            }
    } else if (d.scales != nullptr) {
        return KVR_ERR_INVALID_ARG;
    }

    c->base.assign((size_t)L * C, 0);
    if (d.layout == nullptr) {
        if (d.pool == nullptr) return KVR_ERR_INVALID_ARG;
        if ((uintptr_t)d.pool % 16 != 0) return KVR_ERR_ALIGNMENT;
        c->head_stride = row;
        c->token_stride = H * row;
        int64_t plane = 0, total = 0;
        if (!mul_fits({d.block_size, H, row}, &c->block_stride) ||
            !mul_fits({d.num_blocks, c->block_stride}, &plane) || !mul_fits({plane, L, C}, &total))
            return KVR_ERR_UNSUPPORTED;
        c->span = plane;
        for (size_t v = 0; v < c->base.size(); ++v)
            c->base[v] = (uint64_t)(uintptr_t)d.pool + v * (uint64_t)plane;
        if (four) {
            if (total > INT64_MAX - total / 8 ||
                (uint64_t)(uintptr_t)d.pool > UINT64_MAX - (uint64_t)(total + total / 8))
                return KVR_ERR_UNSUPPORTED;
            for (size_t v = 0; v < c->base.size(); ++v)
                c->block_scale_base.push_back((uint64_t)(uintptr_t)d.pool + (uint64_t)total +
                                              v * (uint64_t)(plane / 8));
        }
    } else {
        const kvr_layout &lay = *d.layout;
        if (lay.bases == nullptr || lay.block_stride < 0 || lay.token_stride < 0 ||
            lay.head_stride < 0)
            return KVR_ERR_INVALID_ARG;
        // a stride counts only where its dimension has more than one position
        c->block_stride = d.num_blocks > 1 ? lay.block_stride : 0;
        c->token_stride = d.block_size > 1 ? lay.token_stride : 0;
        c->head_stride = H > 1 ? lay.head_stride : 0;
        const int64_t step = four ? (D % 128 == 0 ? 64 : 32) : 16;
        if (c->block_stride % step != 0 || c->token_stride % step != 0 || c->head_stride % step != 0)
            return KVR_ERR_ALIGNMENT;
        int64_t a = 0, b = 0, h = 0;
        if (!mul_fits({d.num_blocks - 1, c->block_stride}, &a) ||
            !mul_fits({(int64_t)d.block_size - 1, c->token_stride}, &b) ||
            !mul_fits({(int64_t)H - 1, c->head_stride}, &h) ||
            (__int128)a + b + h + row > (__int128)INT64_MAX)
            return KVR_ERR_UNSUPPORTED;
        c->span = a + b + h + row;
        for (size_t v = 0; v < c->base.size(); ++v) {
            if (lay.bases[v] == nullptr) return KVR_ERR_INVALID_ARG;
            if ((uintptr_t)lay.bases[v] % 16 != 0) return KVR_ERR_ALIGNMENT;
            c->base[v] = (uint64_t)(uintptr_t)lay.bases[v];
        }
        for (size_t v = c->base.size(); four && v < 2 * c->base.size(); ++v) {
            if (lay.bases[v] == nullptr) return KVR_ERR_INVALID_ARG;
            if ((uintptr_t)lay.bases[v] % 16 != 0) return KVR_ERR_ALIGNMENT;
            c->block_scale_base.push_back((uint64_t)(uintptr_t)lay.bases[v]);
        }
        if (!slots_are_disjoint(d.num_blocks, c->block_stride, d.block_size, c->token_stride, H,
                                c->head_stride, row))
            return KVR_ERR_POOL_OVERLAP;
    }
    for (uint64_t b : c->base)
        if (b > UINT64_MAX - (uint64_t)c->span) return KVR_ERR_UNSUPPORTED;
    for (uint64_t b : c->block_scale_base)
        if (b > UINT64_MAX - (uint64_t)(c->span / 8)) return KVR_ERR_UNSUPPORTED;
    // host pointers of the caller's that are not needed any more
    d.layout = nullptr;
    d.scales = nullptr;
    return KVR_OK;
}

size_t aligned(size_t n) { return (n + 255) / 256 * 256; }

// The workspace's parts, one after another; `at` NULL only counts.
size_t place(const kvc_cache &c, int32_t sm_count, unsigned char *at, KvcWorkspace *ws) {
    size_t off = 0;
    auto put = [&](size_t bytes) {
        unsigned char *p = at == nullptr ? nullptr : at + off;
        off += aligned(bytes);
        return p;
    };
    KvcWorkspace w = {};
    w.flags = (uint32_t *)put(sizeof(uint32_t));
    w.scales = (float *)put(c.scales.size() * sizeof(float));
    if (c.scales.empty()) w.scales = nullptr;
    if (c.d.query_heads > 0) {
        w.arrived = (uint32_t *)put(kvc_attend_jobs(c.d) * sizeof(uint32_t));
        w.partial = (float *)put(kvc_attend_partial_bytes(c.d, sm_count));
    }
    w.mem = at;
    w.bytes = off;
    if (ws != nullptr) *ws = w;
    return off;
}

// A plane's first and last byte must be memory that device `dev` can access.
kvr_status check_plane(uint64_t base, int64_t span, int dev) {
    const unsigned char *ends[2] = {(const unsigned char *)(uintptr_t)base,
                                    (const unsigned char *)(uintptr_t)(base + (uint64_t)span - 1)};
    for (const unsigned char *q : ends) {
        cudaPointerAttributes at;
        if (cudaPointerGetAttributes(&at, q) != cudaSuccess) {
            cudaGetLastError();
            return KVR_ERR_POOL_ADDRESS;
        }
        const bool ok = at.type == cudaMemoryTypeDevice ? at.device == dev
                        : at.type == cudaMemoryTypeManaged
                            ? true
                            : at.type == cudaMemoryTypeHost && at.devicePointer == (const void *)q;
        if (!ok) return KVR_ERR_POOL_ADDRESS;
    }
    return KVR_OK;
}

bool aligned16(std::initializer_list<int64_t> xs) {
    for (int64_t x : xs)
        if (x % 16 != 0) return false;
    return true;
}

}  // namespace

bool kvc_on_device(const kvc_cache *c) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

bool kvc_ok_table(const kvc_table &t) {
    return t.rows >= 0 && t.width >= 0 && t.stride >= 0 &&
           (t.ids != nullptr || t.rows == 0 || t.width == 0) && (uintptr_t)t.ids % 4 == 0;
}

bool kvc_type_fits(const kvc_cache *c, int32_t dtype) {
    return c->d.dtype == KVR_DTYPE_FP8_E4M3 || c->d.dtype == KVC_DTYPE_E2M1
               ? dtype == KVR_DTYPE_BF16 || dtype == KVC_DTYPE_F16
               : dtype == c->d.dtype;
}

bool kvc_make_map(CUtensorMap *map, int es, int rank, uint64_t base, int64_t row_bytes,
                  const uint64_t *dims, const int64_t *strides, const uint32_t *box, int line) {
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, CUDART_VERSION,
                                         cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || p == nullptr) {
        cudaGetLastError();
        return false;
    }
    cuuint64_t extents[5], steps[4];
    cuuint32_t boxes[5], ones[5];
    for (int i = 0; i < rank; ++i) {
        extents[i] = dims[i];
        boxes[i] = box[i];
        ones[i] = 1;
        // (a stride of an extent of 1 is not used, but may not be zero)
        if (i > 0) steps[i - 1] = (cuuint64_t)(strides[i - 1] > 0 ? strides[i - 1] : row_bytes);
    }
    return reinterpret_cast<Encode>(p)(
               map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
               (cuuint32_t)rank, (void *)(uintptr_t)base, extents, steps, boxes, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" kvr_status kv_cache_workspace_bytes(const kvc_desc *desc, int32_t sm_count,
                                               int64_t *bytes) {
    if (bytes == nullptr || sm_count < 1) return KVR_ERR_INVALID_ARG;
    try {
        kvc_cache c;
        const kvr_status st = build(desc, &c);
        if (st != KVR_OK) return st;
        *bytes = (int64_t)place(c, sm_count, nullptr, nullptr);
        return KVR_OK;
    } catch (...) {
        return KVR_ERR_NOMEM;
    }
}

extern "C" kvr_status kv_cache_create(const kvc_desc *desc, kvc_cache **out) {
    if (out == nullptr) return KVR_ERR_INVALID_ARG;
    *out = nullptr;
    kvc_cache *c = new (std::nothrow) kvc_cache();
    if (c == nullptr) return KVR_ERR_NOMEM;
    kvr_status st;
    try {
        st = build(desc, c);
        if (st == KVR_OK &&
            (cudaGetDevice(&c->device) != cudaSuccess ||
             cudaDeviceGetAttribute(&c->sm_count, cudaDevAttrMultiProcessorCount, c->device) !=
                 cudaSuccess)) {
            cudaGetLastError();
            st = KVR_ERR_CUDA;
        }
        for (size_t v = 0; st == KVR_OK && v < c->base.size(); ++v)
            st = check_plane(c->base[v], c->span, c->device);
        for (size_t v = 0; st == KVR_OK && v < c->block_scale_base.size(); ++v)
            st = check_plane(c->block_scale_base[v], c->span / 8, c->device);
        if (st == KVR_OK && c->d.query_heads > 0) st = kvc_attend_setup(c);
        if (st == KVR_OK) {
            const size_t bytes = place(*c, c->sm_count, nullptr, nullptr);
            void *mem = nullptr;
            if (cudaMalloc(&mem, bytes) != cudaSuccess) {
                cudaGetLastError();
                st = KVR_ERR_NOMEM;
            } else {
                place(*c, c->sm_count, (unsigned char *)mem, &c->ws);
                // zeroed up to the partial results: the flags and the counters start at zero
                const size_t head = c->ws.partial != nullptr
                                        ? (size_t)((unsigned char *)c->ws.partial - c->ws.mem)
                                        : bytes;
                if (cudaMemset(mem, 0, head) != cudaSuccess ||
                    (!c->scales.empty() &&
                     cudaMemcpy(c->ws.scales, c->scales.data(), c->scales.size() * sizeof(float),
                                cudaMemcpyHostToDevice) != cudaSuccess) ||
                    cudaDeviceSynchronize() != cudaSuccess) {
                    cudaGetLastError();
                    cudaFree(mem);
                    st = KVR_ERR_CUDA;
                }
            }
        }
    } catch (...) {
        st = KVR_ERR_NOMEM;
    }
    if (st != KVR_OK) {
        delete c;
        return st;
    }
    *out = c;
    return KVR_OK;
}

extern "C" void kv_cache_destroy(kvc_cache *cache) {
    if (cache == nullptr) return;
    kvr_device_free(cache->ws.mem);
    delete cache;
}

kvr_status kvc_check_append(const kvc_cache *c, int32_t layer, const kvc_append *a) {
    if (c == nullptr || a == nullptr) return KVR_ERR_INVALID_ARG;
    const kvc_desc &d = c->d;
    if (layer < 0 || layer >= d.num_layers) return KVR_ERR_LAYER_RANGE;
    if (a->num_tokens < 0 || a->reserved != 0 || a->q_heads < 0 || !kvc_ok_table(a->table) ||
        (a->flags & ~(KVC_INTERLEAVED | KVC_ROTATE_LAST)) != 0)
        return KVR_ERR_INVALID_ARG;
    if (a->num_tokens > 0 && (a->requests == nullptr || a->positions == nullptr ||
                              a->k == nullptr || (a->v == nullptr) != c->latent()))
        return KVR_ERR_INVALID_ARG;
    if (!kvc_type_fits(c, a->dtype)) return KVR_ERR_UNSUPPORTED;
    if ((uintptr_t)a->requests % 4 != 0 || (uintptr_t)a->positions % 4 != 0 ||
        !aligned16({(int64_t)(uintptr_t)a->k, (int64_t)(uintptr_t)a->v, a->k_token_stride,
                    a->k_head_stride, a->v_token_stride, a->v_head_stride}))
        return KVR_ERR_ALIGNMENT;
    if (a->k_token_stride < 0 || a->k_head_stride < 0 || a->v_token_stride < 0 ||
        a->v_head_stride < 0)
        return KVR_ERR_INVALID_ARG;
    if (a->rotary != nullptr) {
        if (a->rotary_dim < 1 || a->rotary_rows < 1) return KVR_ERR_INVALID_ARG;
        if (a->rotary_dim % 16 != 0 || a->rotary_dim > d.head_dim) return KVR_ERR_UNSUPPORTED;
        if ((uintptr_t)a->rotary % 16 != 0) return KVR_ERR_ALIGNMENT;
    }
    if (a->q_heads > 0) {
        if (a->rotary == nullptr || a->q_dim < 1) return KVR_ERR_INVALID_ARG;
        if (a->num_tokens > 0 && (a->q == nullptr || a->q_out == nullptr))
            return KVR_ERR_INVALID_ARG;
        if (a->q_dim < a->rotary_dim || (a->q_dim - a->rotary_dim) % 16 != 0 ||
            a->q_dim > KVC_LATENT_DIM || a->q_heads > 4096)
            return KVR_ERR_UNSUPPORTED;
        if (a->q_token_stride < 0 || a->q_head_stride < 0 || a->q_out_token_stride < 0 ||
            a->q_out_head_stride < 0)
            return KVR_ERR_INVALID_ARG;
        if (!aligned16({(int64_t)(uintptr_t)a->q, (int64_t)(uintptr_t)a->q_out, a->q_token_stride,
                        a->q_head_stride, a->q_out_token_stride, a->q_out_head_stride}))
            return KVR_ERR_ALIGNMENT;
    }
    // (two threads share a group of 16 elements: rotated ones come in whole pairs of threads)
    if (d.dtype == KVC_DTYPE_E2M1 && ((a->rotary != nullptr && a->rotary_dim % 32 != 0) ||
                                      (a->q_heads > 0 && a->q_dim % 32 != 0)))
        return KVR_ERR_UNSUPPORTED;
    return KVR_OK;
}

extern "C" kvr_status kv_cache_append(const kvc_cache *c, int32_t layer, const kvc_append *a,
                                      void *stream) {
    const kvr_status st = kvc_check_append(c, layer, a);
    if (st != KVR_OK) return st;
    if (!kvc_on_device(c)) return KVR_ERR_INVALID_ARG;
    if (a->num_tokens == 0) return KVR_OK;
    try {
        std::lock_guard<std::mutex> lock(c->use);
        return kvc_append_launch(c, layer, a, stream);
    } catch (...) {
        return KVR_ERR_NOMEM;
    }
}

kvr_status kvc_check_attend(const kvc_cache *c, int32_t layer, const kvc_attend *a) {
    if (c == nullptr || a == nullptr) return KVR_ERR_INVALID_ARG;
    const kvc_desc &d = c->d;
    if (layer < 0 || layer >= d.num_layers) return KVR_ERR_LAYER_RANGE;
    if (d.query_heads < 1) return KVR_ERR_UNSUPPORTED;
    if (a->num_requests < 0 || a->num_requests > d.max_requests || a->num_new < 1 ||
        a->num_new > d.max_new || a->window < 0 || a->reserved != 0 || !std::isfinite(a->scale) ||
        !kvc_ok_table(a->table) || a->table.rows < a->num_requests)
        return KVR_ERR_INVALID_ARG;
    if (!kvc_type_fits(c, a->dtype)) return KVR_ERR_UNSUPPORTED;
    // positions are 32-bit: a table row must not describe more of them
    if ((int64_t)a->table.width * d.block_size > (int64_t)INT32_MAX - KVC_MAX_REQUESTS)
        return KVR_ERR_UNSUPPORTED;
    if (a->num_requests > 0 && (a->lengths == nullptr || a->q == nullptr || a->out == nullptr))
        return KVR_ERR_INVALID_ARG;
    if (a->q_request_stride < 0 || a->q_token_stride < 0 || a->q_head_stride < 0 ||
        a->out_request_stride < 0 || a->out_token_stride < 0 || a->out_head_stride < 0)
        return KVR_ERR_INVALID_ARG;
    if ((uintptr_t)a->lengths % 4 != 0 || (uintptr_t)a->lse % 4 != 0 ||
        !aligned16({(int64_t)(uintptr_t)a->q, (int64_t)(uintptr_t)a->out, a->q_request_stride,
                    a->q_token_stride, a->q_head_stride, a->out_request_stride,
                    a->out_token_stride, a->out_head_stride}))
        return KVR_ERR_ALIGNMENT;
    return KVR_OK;
}

extern "C" kvr_status kv_cache_attend(const kvc_cache *c, int32_t layer, const kvc_attend *a,
                                      void *stream) {
    const kvr_status st = kvc_check_attend(c, layer, a);
    if (st != KVR_OK) return st;
    if (!kvc_on_device(c)) return KVR_ERR_INVALID_ARG;
    if (a->num_requests == 0) return KVR_OK;
    try {
        // Latents take two launches that hand the workspace over: another host thread's must not
        // come between them on the stream.
        std::unique_lock<std::mutex> lock(c->use, std::defer_lock);
        if (c->latent()) lock.lock();
        return kvc_attend_launch(c, layer, a, stream);
    } catch (...) {
        return KVR_ERR_NOMEM;
    }
}

extern "C" kvr_status kv_cache_status(const kvc_cache *cache, uint32_t *flags) {
    if (flags != nullptr) *flags = 0;
    if (cache == nullptr) return KVR_ERR_INVALID_ARG;
    // the cache's device is waited for, whichever is current
    int current = -1;
    if (cudaGetDevice(&current) != cudaSuccess ||
        (current != cache->device && cudaSetDevice(cache->device) != cudaSuccess)) {
        cudaGetLastError();
        return KVR_ERR_CUDA;
    }
    uint32_t word = 0;
    const bool ok =
        cudaDeviceSynchronize() == cudaSuccess &&
        cudaMemcpy(&word, cache->ws.flags, sizeof(word), cudaMemcpyDeviceToHost) == cudaSuccess &&
        cudaMemset(cache->ws.flags, 0, sizeof(word)) == cudaSuccess &&
        cudaDeviceSynchronize() == cudaSuccess;
    if (!ok) cudaGetLastError();
    if (current != cache->device) cudaSetDevice(current);
    if (!ok) return KVR_ERR_CUDA;
    if (flags != nullptr) *flags = word;
    return word != 0 ? KVR_ERR_DEVICE_BOUNDS : KVR_OK;
}

extern "C" kvr_status kv_cache_rotary_table(float *out, int32_t rows, int32_t rotary_dim,
                                            double base, const kvc_scaling *sc) {
    if (out == nullptr || rows < 1 || rotary_dim < 2 || rotary_dim % 2 != 0 || !(base > 1.0) ||
        !std::isfinite(base))
        return KVR_ERR_INVALID_ARG;
    const int32_t kind = sc == nullptr ? (int32_t)KVC_SCALE_NONE : sc->kind;
    if (kind < KVC_SCALE_NONE || kind > KVC_SCALE_BANDS) return KVR_ERR_UNSUPPORTED;
    const bool parts = kind == KVC_SCALE_RAMP || kind == KVC_SCALE_BANDS;
    if (kind != KVC_SCALE_NONE && (!(sc->factor >= 1.0) || !std::isfinite(sc->factor)))
        return KVR_ERR_INVALID_ARG;
    if (parts && (sc->original < 1 || !(sc->beta_slow > 0.0) || !(sc->beta_fast > sc->beta_slow) ||
                  !std::isfinite(sc->beta_fast)))
        return KVR_ERR_INVALID_ARG;
    if (kind == KVC_SCALE_RAMP && (!(sc->magnitude >= 0.0) || !std::isfinite(sc->magnitude)))
        return KVR_ERR_INVALID_ARG;
    if (kind == KVC_SCALE_BASE && rotary_dim < 4) return KVR_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    const int32_t half = rotary_dim / 2;
    double m = 1.0;
    try {
        std::vector<double> w((size_t)half);
        if (kind == KVC_SCALE_BASE)
            base *= pow(sc->factor, (double)rotary_dim / (rotary_dim - 2));
        for (int32_t i = 0; i < half; ++i) w[i] = pow(base, -2.0 * i / rotary_dim);
        if (kind == KVC_SCALE_LINEAR)
            for (double &x : w) x /= sc->factor;
        if (parts) {
            // the pair index at which a pair turns `turns` times over the original length
            auto index = [&](double turns) {
                return rotary_dim * log(sc->original / (turns * two_pi)) / (2.0 * log(base));
            };
            double lo = floor(index(sc->beta_fast)), hi = ceil(index(sc->beta_slow));
            lo = std::max(lo, 0.0);
            hi = std::min(hi, (double)rotary_dim - 1.0);
            if (hi <= lo) hi = lo + 0.001;
            for (int32_t i = 0; i < half; ++i) {
                double keep;   // the share of w[i] that stays as it is
                if (kind == KVC_SCALE_RAMP) {
                    keep = 1.0 - (i - lo) / (hi - lo);
                } else {
                    const double turns = sc->original * w[i] / two_pi;
                    keep = (turns - sc->beta_slow) / (sc->beta_fast - sc->beta_slow);
                }
                keep = std::min(1.0, std::max(0.0, keep));
                w[i] = w[i] * keep + w[i] / sc->factor * (1.0 - keep);
            }
            if (kind == KVC_SCALE_RAMP)
                m = sc->magnitude > 0.0 ? sc->magnitude : 1.0 + 0.1 * log(sc->factor);
        }
        for (int64_t p = 0; p < rows; ++p) {
            float *row = out + p * rotary_dim;
            for (int32_t i = 0; i < half; ++i) {
                row[i] = (float)(m * cos((double)p * w[i]));
                row[half + i] = (float)(m * sin((double)p * w[i]));
            }
        }
    } catch (...) {
        return KVR_ERR_NOMEM;
    }
    return KVR_OK;
}
