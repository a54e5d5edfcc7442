// cache_more_host_check.cpp -- test harness: the host side of the cache's further calls on a CUDA runtime of its own
// making.
//
// Linked with cache.cpp and cache_more.cpp; defines the runtime calls that they make, and the launches behind
// their calls, as stand-ins that record what they are asked, so that host threads and refusals can be played through
// without a GPU.
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <chrono>
#include <thread>

#include "cache.h"

namespace {
std::atomic<int> moving{0}, mixed{0}, launches{0};
unsigned char memory[1 << 24];

void pause_for(int us) { std::this_thread::sleep_for(std::chrono::microseconds(us)); }
// A call of one launch that writes what an eviction reads or moves.
kvr_status write_once() {
    if (moving != 0) ++mixed;
    pause_for(20);
    ++launches;
    return KVR_OK;
}
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaPointerGetAttributes(struct cudaPointerAttributes *at, const void *) {
    *at = {};
    at->type = cudaMemoryTypeDevice, at->device = 0;
    return cudaSuccess;
}
cudaError_t cudaMalloc(void **p, size_t bytes) {
    return bytes <= sizeof memory ? (*p = memory, cudaSuccess) : cudaErrorMemoryAllocation;
}
cudaError_t cudaFree(void *) { return cudaSuccess; }
cudaError_t cudaThreadExchangeStreamCaptureMode(enum cudaStreamCaptureMode *) { return cudaSuccess; }
cudaError_t cudaMemset(void *, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void *, const void *, size_t, enum cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *) {
    return cudaErrorUnknown;
}
}

size_t kvc_attend_partial_bytes(const kvc_desc &, int32_t) { return 4096; }
size_t kvc_attend_jobs(const kvc_desc &) { return 16; }
kvr_status kvc_attend_setup(kvc_cache *) { return KVR_OK; }
kvr_status kvc_attend_launch(const kvc_cache *, int32_t, const kvc_attend *, void *) { return ++launches, KVR_OK; }
kvr_status kvc_attend_scored_launch(const kvc_cache *, int32_t, const kvc_attend *, const kvc_scoring *, void *) {
    return ++launches, KVR_OK;
}
kvr_status kvc_read_launch(const kvc_cache *, int32_t, const kvc_read *, void *) { return ++launches, KVR_OK; }
kvr_status kvc_append_launch(const kvc_cache *, int32_t, const kvc_append *, void *) { return write_once(); }
kvr_status kvc_append_at_launch(const kvc_cache *, int32_t, const kvc_append *, const int32_t *, void *) {
    return write_once();
}
kvr_status kvc_weigh_launch(const kvc_cache *, int32_t, const kvc_weigh *, void *) { return write_once(); }
// Two steps that belong together, with time in between for another thread's.
kvr_status kvc_evict_launch(const kvc_cache *, int32_t, const kvc_evict *, void *) {
    if (moving.fetch_add(1) != 0) ++mixed;
    pause_for(100);
    --moving;
    ++launches;
    return KVR_OK;
}

#define REQUIRE(x)                             \
    do {                                       \
        if (!(x)) {                            \
            printf("%d: %s\n", __LINE__, #x);  \
            return 1;                          \
        }                                      \
    } while (0)

#define AT(type) ((type *)(uintptr_t)0x4000)     // somewhere on the device

static int make_cache(kvc_cache **c) {
    kvc_desc d = {};
    d.num_layers = 1, d.num_components = 2, d.kv_heads = 2, d.head_dim = 64, d.dtype = KVR_DTYPE_BF16;
    d.block_size = 16, d.num_blocks = 4, d.pool = AT(void), d.query_heads = 4, d.max_requests = 4, d.max_new = 1;
    return kv_cache_create(&d, c);
}

static kvc_table a_table() {
    kvc_table t = {};
    t.ids = AT(const int32_t), t.stride = 3, t.rows = 2, t.width = 3;
    return t;
}
static kvc_evict an_eviction() {
    kvc_evict e = {};
    e.num_requests = 2, e.keep = 20, e.recent = 4, e.weights_width = 48;
    e.lengths = AT(const int32_t), e.table = a_table();
    e.weights = e.weights_out = AT(float), e.kept = AT(int32_t);
    e.weights_request_stride = e.out_request_stride = 96, e.weights_head_stride = e.out_head_stride = 48;
    return e;
}
static kvc_weigh a_weighing() {
    kvc_weigh w = {};
    w.num_requests = 2, w.num_new = 1, w.dtype = KVR_DTYPE_BF16, w.scale = 1.0f, w.add = 1;
    w.lengths = AT(const int32_t), w.table = a_table(), w.q = AT(void), w.lse = AT(float), w.weights = AT(float);
    w.q_request_stride = 512, w.q_head_stride = 128;
    w.weights_request_stride = 96, w.weights_head_stride = 48, w.weights_width = 48;
    return w;
}
static kvc_append an_append() {
    kvc_append a = {};
    a.num_tokens = 2, a.dtype = KVR_DTYPE_BF16, a.requests = a.positions = AT(const int32_t), a.table = a_table();
    a.k = a.v = AT(void), a.k_token_stride = a.v_token_stride = 256, a.k_head_stride = a.v_head_stride = 128;
    return a;
}

// Host threads that evict, weigh and append with one cache: nothing that writes weights or rows comes between an
// eviction's two steps.
static int threads() {
    kvc_cache *c;
    REQUIRE(make_cache(&c) == KVR_OK);
    const kvc_evict e = an_eviction();
    const kvc_weigh w = a_weighing();
    const kvc_append a = an_append();
    std::atomic<int> wrong{0};
    std::thread of[5];
    for (int i = 0; i < 5; ++i)
        of[i] = std::thread([&, i] {
            for (int k = 0; k < 50; ++k) {
                const kvr_status st = i < 2    ? kv_cache_evict(c, 0, &e, nullptr)
                                      : i == 2 ? kv_cache_weigh(c, 0, &w, nullptr)
                                      : i == 3 ? kv_cache_append(c, 0, &a, nullptr)
                                               : kv_cache_append_at(c, 0, &a, AT(const int32_t), nullptr);
                if (st != KVR_OK) ++wrong;
            }
        });
    for (auto &t : of) t.join();
    REQUIRE(wrong == 0 && launches == 250);
    REQUIRE(mixed == 0);
    kv_cache_destroy(c);
    return 0;
}

// What an eviction goes into: no table at all is in place, an empty one is refused.
static int into() {
    kvc_cache *c;
    REQUIRE(make_cache(&c) == KVR_OK);
    kvc_evict e = an_eviction();
    REQUIRE(kv_cache_evict(c, 0, &e, nullptr) == KVR_OK && launches == 1);
    e.into = a_table();
    REQUIRE(kv_cache_evict(c, 0, &e, nullptr) == KVR_OK && launches == 2);
    for (int what = 0; what < 3; ++what) {
        e.into = {};
        (what == 0 ? e.into.rows : e.into.width) = what == 2 ? 0 : 3;      // (no columns; no rows)
        if (what == 2) e.into.stride = 3;
        REQUIRE(kv_cache_evict(c, 0, &e, nullptr) == KVR_ERR_INVALID_ARG && launches == 2);
    }
    // of no requests nothing is asked
    e.num_requests = 0, e.into.width = 3;
    REQUIRE(kv_cache_evict(c, 0, &e, nullptr) == KVR_OK && launches == 2);
    kv_cache_destroy(c);
    return 0;
}

// Where read writes: rows that overlap one another are refused, whichever input has them.
static int overlap() {
    kvc_cache *c;
    REQUIRE(make_cache(&c) == KVR_OK);
    kvc_read good = {};
    good.num_tokens = 3, good.dtype = KVR_DTYPE_BF16, good.requests = good.positions = AT(const int32_t);
    good.table = a_table(), good.k = good.v = AT(void);
    good.k_token_stride = good.v_token_stride = 256, good.k_head_stride = good.v_head_stride = 128;
    // [T][H][D], wider rows, [H][T][D], and one token's strides of zero
    const int64_t fits[][3] = {{3, 256, 128}, {3, 768, 128}, {3, 128, 384}, {1, 0, 128}, {0, 0, 0}};
    // all tokens at one place, all heads, rows within one another, heads that reach the next token
    const int64_t bad[][3] = {{3, 0, 128}, {3, 256, 0}, {3, 112, 1024}, {3, 256, 112}, {3, 240, 128}, {3, 128, 240}};
    for (int which = 0; which < 2; ++which) {
        auto with = [&](const int64_t s[3]) {
            kvc_read r = good;
            r.num_tokens = (int32_t)s[0];
            (which == 0 ? r.k_token_stride : r.v_token_stride) = s[1];
            (which == 0 ? r.k_head_stride : r.v_head_stride) = s[2];
            return kv_cache_read(c, 0, &r, nullptr);
        };
        for (const auto &s : fits) REQUIRE(with(s) == KVR_OK);
        const int before = launches;
        for (const auto &s : bad) REQUIRE(with(s) == KVR_ERR_POOL_OVERLAP);
        REQUIRE(launches == before);
    }
    kv_cache_destroy(c);
    return 0;
}

int main(int argc, char **argv) {
    if (argc > 1 && strcmp(argv[1], "overlap") == 0) return overlap();
    if (argc > 1 && strcmp(argv[1], "into") == 0) return into();
    if (argc > 1 && strcmp(argv[1], "threads") == 0) return threads();
    return 2;
}
