/*
 * kv_cache.h -- C ABI of what a decode instance does with the KV it was handed: append the
 * new tokens' keys and values, and attend to the cache.
 *
 * A cache is ONE shard pool of a decode side as kv_relayout.h describes it,
 *   [num_layers][num_components][num_blocks][block_size][kv_heads][head_dim],
 * or any strided view of one (kvr_layout); kv_heads is the shard's own head count. Components:
 * 2 = keys then values, 1 = a latent plane whose rows are the keys and whose first value_dim
 * elements are the values (MLA, one head).
 *
 * Step inputs (lengths, positions, block tables) are DEVICE arrays, so that a step can be
 * enqueued, or captured in a CUDA graph, without the host knowing them. They cannot be checked
 * on the host; the kernels check every request index, position, length and block id that they
 * use. What is out of range is neither read nor written (keys and values of a block id out of
 * range count as zeros, a length out of range as the nearest that is in range), it sets a flag, and
 * kv_cache_status() returns KVR_ERR_DEVICE_BOUNDS with the flags.
 *
 * Launch calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default stream),
 * allocate nothing, never synchronize, and report launch errors only. The current device must
 * be the cache's device (KVR_ERR_INVALID_ARG otherwise). The attention calls of one cache share
 * its workspace: calls on different streams must be ordered by the caller (or use a second
 * cache of the same pool). Host threads may call with one cache at once: what a call enqueues
 * stays together. Every launch is ordered after the work before it on `stream`.
 * No C++ exception crosses this ABI.
 */
#ifndef KV_CACHE_H_
#define KV_CACHE_H_

#include <stdint.h>

#include "kv_relayout.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types: kvr_dtype's KVR_DTYPE_BF16 (1) and KVR_DTYPE_FP8_E4M3 (2), and IEEE half. */
#define KVC_DTYPE_F16 3

/* Most requests of one attention call. */
#define KVC_MAX_REQUESTS 2048

/* Flags of kv_cache_status(). */
#define KVC_FLAG_REQUEST 1u    /* append: a request index outside the block table's rows */
#define KVC_FLAG_POSITION 2u   /* append: a position beyond the block table or the rotation table */
#define KVC_FLAG_LENGTH 4u     /* attend: a negative length, or one beyond the block table */
#define KVC_FLAG_BLOCK 8u      /* a block id outside [0, num_blocks) */
#define KVC_FLAG_TIMEOUT 16u   /* a wait inside a kernel gave up (a defect of the library) */

typedef struct kvc_desc {
    int32_t num_layers;        /* L >= 1 */
    int32_t num_components;    /* 2 (keys, values) or 1 (latent) */
    int32_t kv_heads;          /* H >= 1 heads of this shard (1 for a latent) */
    int32_t head_dim;          /* D: a multiple of 16, at most 256; a latent: 576 */
    int32_t value_dim;         /* a latent's values: 512; otherwise D (0 = these) */
    int32_t dtype;             /* element type of the pool; a latent's is a 16-bit one to attend */
    int32_t block_size;        /* B >= 1 tokens of a block */
    int32_t per_head;          /* 0: a scale per (layer, component); 1: per head too */
    int64_t num_blocks;        /* N >= 1 */
    void *pool;                /* device, 16-byte aligned (ignored with a layout) */
    const kvr_layout *layout;  /* NULL: the standard layout; else bases [L * C], byte strides */
    const float *scales;       /* host [L][C] or [L][C][H], E4M3 pools only (required there):
                                  positive, finite; copied */
    int32_t query_heads;       /* Hq: a multiple of H (0: this cache only appends) */
    int32_t max_requests;      /* most requests of an attention call, 1..KVC_MAX_REQUESTS */
    int32_t max_new;           /* most newest tokens of a request that attend at once, >= 1 */
} kvc_desc;

typedef struct kvc_cache kvc_cache;

/*
 * Validate *desc (KVR_ERR_INVALID_ARG, _UNSUPPORTED, _ALIGNMENT, _POOL_OVERLAP for a layout
 * whose slots overlap), check that the pool is memory the current device can access
 * (_POOL_ADDRESS), and allocate the device workspace of its calls. *out is the new cache, or
 * NULL on failure. The workspace (kv_cache_workspace_bytes()) is 256 bytes where query_heads is 0; for
 * attention on 152 SMs it is 40 MB over latents and 5 to 10 MB over keys and values, whatever the pool's
 * size and layers: caches of many shards on one device that only append need not reserve it.
 */
kvr_status kv_cache_create(const kvc_desc *desc, kvc_cache **out);
/* Frees the workspace like cudaFree(); allowed while a stream is being captured. */
void kv_cache_destroy(kvc_cache *cache);

/* Bytes of the device workspace that kv_cache_create() allocates (host only, no CUDA call;
 * sm_count: the device's SMs). Validates *desc like it, but for the pool's memory. */
kvr_status kv_cache_workspace_bytes(const kvc_desc *desc, int32_t sm_count, int64_t *bytes);

/* A block table on the device: row r holds the physical blocks of request r, entry k those of
 * its tokens [k * B, (k + 1) * B). */
typedef struct kvc_table {
    const int32_t *ids;        /* device [rows][width] */
    int64_t stride;            /* entries between rows, >= 0 (rows may overlap: one row for all
                                  requests has a stride of 0) */
    int32_t rows;
    int32_t width;
} kvc_table;

/*
 * Rotation of positions. A head row has `dim` elements, of which the first `rotary_dim` (or,
 * with KVC_ROTATE_LAST, the last) are rotated: pair i of them, (a, b), becomes
 *   (a cos - b sin, b cos + a sin),  cos = table[p][i], sin = table[p][rotary_dim / 2 + i]
 * for a token at position p. Pairs are (x[i], x[i + rotary_dim / 2]), or with
 * KVC_INTERLEAVED (x[2 i], x[2 i + 1]). Products and sums are fp32 and rounded once, to the
 * type that is stored.
 */
#define KVC_INTERLEAVED 1u
#define KVC_ROTATE_LAST 2u

/*
 * Append tokens to layer `layer`. Token t belongs to request requests[t] (a row of the block
 * table) and goes to position p = positions[t]: block ids[requests[t]][p / B], slot p % B. A
 * negative position marks padding: nothing of that token is written. Keys (or latents)
 * are rotated, values are not; rows are stored in the pool's type. An E4M3 pool stores
 * E4M3(x * fl32(1 / s)), nearest-even, saturating at +-448, of the rotated fp32 value x (a NaN
 * gives a NaN code).
 * The queries, where given, are rotated into q_out (which may be q itself).
 * Requirements: k, v, q of `dtype` (the pool's type if that has 16 bits), rows contiguous,
 * every address and stride a multiple of 16 bytes; rotary_dim a multiple of 16, at most both
 * row lengths; q_dim a multiple of 16, at most 576. Two tokens of one call must not have the same slot; k, v and q must not overlap the
 * pool.
 */
typedef struct kvc_append {
    int32_t num_tokens;        /* >= 0 */
    int32_t dtype;             /* KVR_DTYPE_BF16 or KVC_DTYPE_F16: type of k, v, q, q_out */
    const int32_t *requests;   /* device [num_tokens] */
    const int32_t *positions;  /* device [num_tokens] */
    kvc_table table;
    const void *k;             /* device [num_tokens][H][D] */
    const void *v;             /* device [num_tokens][H][D]; NULL for a latent */
    int64_t k_token_stride, k_head_stride;     /* bytes */
    int64_t v_token_stride, v_head_stride;
    const float *rotary;       /* device [rotary_rows][rotary_dim]: cosines, then sines; NULL: none */
    int32_t rotary_rows, rotary_dim;
    uint32_t flags;            /* KVC_INTERLEAVED, KVC_ROTATE_LAST */
    int32_t q_heads;           /* 0: no queries */
    int32_t q_dim;
    int32_t reserved;          /* 0 */
    const void *q;             /* device [num_tokens][q_heads][q_dim] */
    void *q_out;
    int64_t q_token_stride, q_head_stride;
    int64_t q_out_token_stride, q_out_head_stride;
} kvc_append;

kvr_status kv_cache_append(const kvc_cache *cache, int32_t layer, const kvc_append *args,
                           void *stream);

/*
 * Attention of the newest `num_new` tokens of each request over layer `layer`. lengths[r]
 * counts the request's cached tokens, the newest included (append them first). Query i of
 * request r is the token at position p = lengths[r] - num_new + i; it sees the keys at
 * positions j <= p and, with window > 0, j > p - window. Query head g attends to key head
 * g / (Hq / H). With x_j = scale * q . k_j over the keys it sees,
 *   out = sum_j exp(x_j - lse) v_j,   lse = log sum_j exp(x_j)   (natural logarithm).
 * A query that sees nothing (p < 0) gives out = 0 and lse = -infinity. What the cache holds at
 * places that no query of the request sees (beyond its length, or below its newest tokens'
 * windows) is never used, NaN included, and table entries of blocks that hold such places only
 * are not looked at; a NaN or an infinity in a value at a place that only some of a request's
 * newest tokens see may reach the others.
 * Weights below 2^-24 of a row's largest count as zero where the cache holds f16 or E4M3. Before they
 * meet the values, weights count with 15 bits or more over bf16 and f16 keys and values and under at most
 * 32 rows (num_new Hq) of latents, with those of an f16 over E4M3, and with those of the pool's type
 * under more rows of latents; sums are fp32.
 * Requirements: q and out of `dtype` (the pool's type if that has 16 bits), rows contiguous,
 * every address and stride a multiple of 16 bytes; lse NULL or [R][num_new][Hq], contiguous.
 */
typedef struct kvc_attend {
    int32_t num_requests;      /* 0..max_requests */
    int32_t num_new;           /* 1..max_new */
    int32_t dtype;
    int32_t window;            /* 0: none */
    float scale;               /* finite */
    int32_t reserved;          /* 0 */
    const int32_t *lengths;    /* device [num_requests] */
    kvc_table table;           /* rows >= num_requests */
    const void *q;             /* device [num_requests][num_new][Hq][D] */
    void *out;                 /* device [num_requests][num_new][Hq][value_dim] */
    float *lse;
    int64_t q_request_stride, q_token_stride, q_head_stride;          /* bytes */
    int64_t out_request_stride, out_token_stride, out_head_stride;
} kvc_attend;

kvr_status kv_cache_attend(const kvc_cache *cache, int32_t layer, const kvc_attend *args,
                           void *stream);

/* Waits for the cache's device (which need not be the current one), reads and clears the flags
 * of what the kernels found out of range:
 * KVR_OK with *flags = 0, or KVR_ERR_DEVICE_BOUNDS with the KVC_FLAG_* bits. */
kvr_status kv_cache_status(const kvc_cache *cache, uint32_t *flags);

/*
 * Fill a rotation table on the host: out[p][i] = m cos(p w_i), out[p][rotary_dim / 2 + i] =
 * m sin(p w_i), computed in fp64 and rounded once, for positions [0, rows). Without scaling
 * (NULL) w_i = base^(-2 i / rotary_dim) and m = 1. For contexts longer than the `original`
 * length that a model was trained at:
 *   KVC_SCALE_LINEAR: w_i / factor (positions interpolated);
 *   KVC_SCALE_BASE: base * factor^(rotary_dim / (rotary_dim - 2)) in place of base;
 *   KVC_SCALE_RAMP: pairs that turn more than beta_fast times over the original length keep
 *     w_i, those that turn less than beta_slow times take w_i / factor, with a linear ramp
 *     over the pair index between; m = magnitude (0 means 1 + 0.1 ln factor);
 *   KVC_SCALE_BANDS: as KVC_SCALE_RAMP with the ramp linear in the number of turns.
 */
typedef enum kvc_scaling_kind {
    KVC_SCALE_NONE = 0,
    KVC_SCALE_LINEAR = 1,
    KVC_SCALE_BASE = 2,
    KVC_SCALE_RAMP = 3,
    KVC_SCALE_BANDS = 4
} kvc_scaling_kind;

typedef struct kvc_scaling {
    int32_t kind;
    int32_t original;          /* RAMP, BANDS: the original length, >= 1 */
    double factor;             /* >= 1 */
    double beta_fast, beta_slow;   /* RAMP, BANDS: 0 < beta_slow < beta_fast */
    double magnitude;          /* RAMP: m, 0 for the rule above */
} kvc_scaling;

kvr_status kv_cache_rotary_table(float *out, int32_t rows, int32_t rotary_dim, double base,
                                 const kvc_scaling *scaling);

#ifdef __cplusplus
}
#endif
#endif /* KV_CACHE_H_ */
