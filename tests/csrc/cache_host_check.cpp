// cache_host_check.cpp -- test harness: the decode cache's host code on a CUDA runtime of its own making.
//
// Includes cache.cpp and defines the few runtime calls that it makes, and the launches behind its
// calls, as stand-ins that record what they are asked, so that devices, host threads and failures can
// be played through without a GPU.
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <chrono>
#include <thread>

#include "cache.cpp"

namespace {
std::atomic<int> current{0};             // the current device (one for all threads here)
std::atomic<int> inside{0}, overlaps{0}, launches{0};
int synced = -1, failing = 0;
uint32_t flags_word = 0;
unsigned char memory[1 << 24];
}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int *d) { return *d = current, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return current = d, cudaSuccess; }
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
cudaError_t cudaMemset(void *p, int, size_t bytes) {
    if (bytes == sizeof(uint32_t)) flags_word = 0;
    return cudaSuccess;
}
cudaError_t cudaMemcpy(void *to, const void *from, size_t bytes, enum cudaMemcpyKind kind) {
    if (kind == cudaMemcpyDeviceToHost) memcpy(to, &flags_word, bytes);
    return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() { return synced = current, failing ? cudaErrorUnknown : cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *) {
    return cudaErrorUnknown;
}
}

size_t kvc_attend_partial_bytes(const kvc_desc &, int32_t) { return 4096; }
size_t kvc_attend_jobs(const kvc_desc &) { return 16; }
kvr_status kvc_attend_setup(kvc_cache *) { return KVR_OK; }
kvr_status kvc_append_launch(const kvc_cache *, int32_t, const kvc_append *, void *) { return KVR_OK; }
// Two steps that belong together, with time in between for another thread's.
kvr_status kvc_attend_launch(const kvc_cache *, int32_t, const kvc_attend *, void *) {
    if (inside.fetch_add(1) != 0) ++overlaps;
    std::this_thread::sleep_for(std::chrono::microseconds(200));
    --inside;
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

static int latent_cache(kvc_cache **c) {
    kvc_desc d = {};
    d.num_layers = d.num_components = d.kv_heads = 1;
    d.head_dim = 576, d.dtype = KVR_DTYPE_BF16, d.block_size = 16, d.num_blocks = 4;
    d.pool = (void *)0x1000000, d.query_heads = 16, d.max_requests = 2, d.max_new = 1;
    return kv_cache_create(&d, c);
}

// Host threads that attend with one cache: the steps of their calls do not mix.
static int threads() {
    kvc_cache *c;
    REQUIRE(latent_cache(&c) == KVR_OK);
    kvc_attend a = {};
    a.num_requests = a.num_new = 1, a.dtype = KVR_DTYPE_BF16, a.scale = 1.0f;
    a.lengths = (const int32_t *)64, a.q = (const void *)64, a.out = (void *)64;
    a.table.ids = (const int32_t *)64, a.table.stride = a.table.rows = a.table.width = 1;
    std::atomic<int> wrong{0};
    std::thread of[4];
    for (auto &t : of)
        t = std::thread([&] {
            for (int k = 0; k < 50; ++k)
                if (kv_cache_attend(c, 0, &a, nullptr) != KVR_OK) ++wrong;
        });
    for (auto &t : of) t.join();
    REQUIRE(wrong == 0 && launches == 200);
    REQUIRE(overlaps == 0);
    kv_cache_destroy(c);
    return 0;
}

// Status under another current device: the cache's own is waited for, the current one stays.
static int device() {
    kvc_cache *c;
    REQUIRE(latent_cache(&c) == KVR_OK);
    for (int now : {0, 1, 3}) {
        current = now;
        flags_word = KVC_FLAG_LENGTH | KVC_FLAG_BLOCK, synced = -1, failing = 0;
        uint32_t flags = 7;
        REQUIRE(kv_cache_status(c, &flags) == KVR_ERR_DEVICE_BOUNDS);
        REQUIRE(flags == (KVC_FLAG_LENGTH | KVC_FLAG_BLOCK) && flags_word == 0);
        REQUIRE(synced == 0 && current == now);
        REQUIRE(kv_cache_status(c, nullptr) == KVR_OK && current == now);
        flags_word = KVC_FLAG_POSITION, failing = 1, flags = 7;
        REQUIRE(kv_cache_status(c, &flags) == KVR_ERR_CUDA);
        REQUIRE(flags == 0 && flags_word == KVC_FLAG_POSITION && current == now);
    }
    current = 0;
    kv_cache_destroy(c);
    return 0;
}

int main(int argc, char **argv) {
    if (argc > 1 && strcmp(argv[1], "threads") == 0) return threads();
    if (argc > 1 && strcmp(argv[1], "device") == 0) return device();
    return 2;
}
