// cache_evict.cu -- which of a head's cached tokens stay, by their weights, and their rows moved together.
//
// Select. Of n tokens the `recent` newest stay, and of the others the `need` = keep - recent of the largest
// weights: those above the need-th largest, T, and of those equal to it the lowest slots. A cluster of blocks has
// a head; each block a contiguous share of its weights, held in shared memory. T comes digit by digit (11, 11 and
// 10 bits of the weights as ordered integers): each block counts its weights that fit the digits so far, every
// block adds all blocks' counts up and so finds the same digit, with one barrier of the cluster a digit. Then each
// warp counts what stays of its share, and writes those slots where the shares before it end. A few
// thousand weights are read once: barriers and shared memory bound it, not HBM.
//
// Move. Row i of the kept goes to slot i, which is not after its own. Into other blocks, rows in any
// order by any block. In place, slot i may still hold a row that has to go further down; it is the source of
// a row i' <= i. A cluster has a head, goes up the kept rows in rounds of a few rows a block, and each
// round's rows are all in registers before any of them is stored (one barrier of the cluster a round; the
// next round's are asked for before that, as no store of this round reaches slots of rows behind it).
#include <cooperative_groups.h>

#include <algorithm>

#include "cache.h"

namespace {

using namespace kvc;
namespace cg = cooperative_groups;

constexpr int SELECT_THREADS = 512, SELECT_WARPS = SELECT_THREADS / 32;
constexpr int BINS = 2048;
constexpr int HELD = 4096;         // weights that a block holds in shared memory; those beyond are read each time
constexpr int MOVE_THREADS = 256;
constexpr int UNITS = 8;           // 16-byte units of a thread at a time
constexpr int WORDS = 9;           // words of a row besides: its weight, and block scales of 4-bit rows (2 D / 64)

struct EvictArgs {
    KvcSlots from, into;
    KvcPlane k_plane, v_plane;
    unsigned char *k_block_scales, *v_block_scales;
    const int32_t *lengths;
    const float *weights;
    float *weights_out;
    int32_t *kept;                 // [requests][H][keep]
    uint32_t *flags;
    int64_t w_request, w_head, out_request, out_head;
    int32_t requests, H, width, keep, recent;
    int32_t rows;                  // of a round (or block)
    int32_t chunks;                // blocks of a head, into other blocks
    int32_t words;                 // besides a row's units
    KvrDiv by_heads, by_chunks, by_units, by_words;
};

// A request's cached tokens. A length out of range counts as the nearest in range.
__device__ __forceinline__ int32_t tokens_of(const EvictArgs &a, int32_t r, uint32_t *bad) {
    const int32_t n = __ldg(a.lengths + r);
    const int32_t most = min(a.width, a.from.width * (int32_t)a.from.block.d);
    if (n >= 0 && n <= most) return n;
    *bad = KVC_FLAG_LENGTH;
    return n < 0 ? 0 : most;
}

// Weights as integers of the same order: -0 as 0, NaN above all.
__device__ __forceinline__ uint32_t ordered(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(SELECT_THREADS) select_kernel(EvictArgs a) {
    __shared__ uint32_t held[HELD];
    __shared__ uint32_t hist[2][BINS];
    __shared__ uint32_t scan[SELECT_WARPS][2];
    __shared__ uint32_t found[2], own[2];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int32_t blocks = (int32_t)cluster.num_blocks(), part = (int32_t)cluster.block_rank();
    const int32_t head = (int32_t)blockIdx.x / blocks;
    const int32_t r = (int32_t)a.by_heads.div((uint32_t)head), h = head - r * a.H;
    wait_for_previous();
    let_next_start();
    uint32_t bad = 0;
    const int32_t n = tokens_of(a, r, &bad);
    if (bad != 0 && h == 0 && part == 0 && tid == 0) atomicOr(a.flags, bad);
    int32_t *kept = a.kept + (int64_t)head * a.keep;
    // (every block of the cluster goes the same way here and below)
    if (n <= a.keep) {
        for (int32_t i = part * SELECT_THREADS + tid; i < n; i += blocks * SELECT_THREADS) kept[i] = i;
        return;
    }
    const int32_t old = n - a.recent, need = a.keep - a.recent;
    for (int32_t i = part * SELECT_THREADS + tid; i < a.recent; i += blocks * SELECT_THREADS)
        kept[need + i] = old + i;
    if (need == 0) return;

    const float *weights = a.weights + r * a.w_request + h * a.w_head;
    const int32_t share = (old + blocks - 1) / blocks;
    const int32_t j0 = min(old, part * share), size = min(old, j0 + share) - j0;
    auto key = [&](int32_t i) -> uint32_t { return i < HELD ? held[i] : ordered(weights[j0 + i]); };
    for (int i = tid; i < BINS; i += SELECT_THREADS) hist[0][i] = 0;
    for (int32_t i = tid; i < min(size, HELD); i += SELECT_THREADS) held[i] = ordered(weights[j0 + i]);

    uint32_t known = 0, mask = 0;        // T's digits so far, and which bits they are
    uint32_t left = (uint32_t)need;      // of the weights that fit them, how many stay
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
        uint32_t *count = hist[pass & 1];
        __syncthreads();
        for (int32_t i = tid; i < size; i += SELECT_THREADS) {
            const uint32_t k = key(i);
            if ((k & mask) == known) atomicAdd(count + (k >> shift & (uint32_t)(bins - 1)), 1u);
        }
        cluster.sync();
        // (what the others read last of the other array, they read before this barrier)
        for (int i = tid; i < BINS; i += SELECT_THREADS) hist[pass & 1 ^ 1][i] = 0;
        // a thread's bins, from the top down: their counts over all blocks
        constexpr int PER = BINS / SELECT_THREADS;
        uint32_t c[PER], sum = 0;
        const int first = BINS - PER * (tid + 1);          // lowest of its bins
#pragma unroll
        for (int e = 0; e < PER; ++e) c[e] = 0;
        for (int32_t b = 0; b < blocks; ++b) {
            const uint4 v = *(const uint4 *)(cluster.map_shared_rank(count, b) + first);
            c[0] += v.x, c[1] += v.y, c[2] += v.z, c[3] += v.w;
        }
        static_assert(PER == 4, "");
#pragma unroll
        for (int e = 0; e < PER; ++e) sum += c[e];
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t y = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp][0] = incl;
        __syncthreads();
        uint32_t above = incl - sum;
        for (int w = 0; w < warp; ++w) above += scan[w][0];
        if (above < left && left <= above + sum) {
#pragma unroll
            for (int e = PER - 1; e >= 0; --e) {
                if (above < left && left <= above + c[e]) {
                    found[0] = (uint32_t)(first + e);
                    found[1] = left - above;
                }
                above += c[e];
            }
        }
        __syncthreads();
        known |= found[0] << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        left = found[1];
    }

    // a warp's share of the block's: how many are above T, and how many equal it
    const int32_t run = (size + SELECT_WARPS - 1) / SELECT_WARPS;
    const int32_t i0 = min(size, warp * run), i1 = min(size, i0 + run);
    uint32_t above = 0, same = 0;
    for (int32_t i = i0 + lane; i < i1; i += 32) {
        const uint32_t k = key(i);
        above += k > known;
        same += k == known;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        above += __shfl_xor_sync(~0u, above, o);
        same += __shfl_xor_sync(~0u, same, o);
    }
    if (lane == 0) scan[warp][0] = above, scan[warp][1] = same;
    __syncthreads();
    if (tid < 2) {
        uint32_t t = 0;
        for (int w = 0; w < SELECT_WARPS; ++w) t += scan[w][tid];
        own[tid] = t;
    }
    cluster.sync();
    above = same = 0;
    for (int32_t b = 0; b < part; ++b) {
        const uint32_t *o = cluster.map_shared_rank(own, b);
        above += o[0];
        same += o[1];
    }
    for (int w = 0; w < warp; ++w) above += scan[w][0], same += scan[w][1];
    for (int32_t i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? key(i + lane) : 0u;
        const bool gt = i + lane < i1 && k > known, eq = i + lane < i1 && k == known;
        const uint32_t gts = __ballot_sync(~0u, gt), eqs = __ballot_sync(~0u, eq);
        const uint32_t before = (1u << lane) - 1u;
        const uint32_t g = above + __popc(gts & before), e = same + __popc(eqs & before);
        if (gt || (eq && e < left)) kept[g + min(e, left)] = j0 + i + lane;
        above += __popc(gts);
        same += __popc(eqs);
    }
    cluster.sync();                      // no block leaves while others read its counts
}

// Where slot j of request r is in a plane, in bytes; -1: nowhere.
__device__ __forceinline__ int64_t offset_of(const EvictArgs &a, const KvcSlots &s, int32_t r, int32_t h, int32_t j,
                                             uint32_t *bad) {
    const uint32_t entry = s.block.div((uint32_t)j);
    const int32_t in = j - (int32_t)(entry * s.block.d);
    if (entry >= (uint32_t)s.width) {
        *bad |= KVC_FLAG_LENGTH;
        return -1;
    }
    const int32_t id = __ldg(s.ids + (int64_t)r * s.stride + entry);
    if (id < 0 || id >= s.num_blocks) {
        *bad |= KVC_FLAG_BLOCK;
        return -1;
    }
    return id * a.k_plane.block_stride + in * a.k_plane.token_stride + h * a.k_plane.head_stride;
}

// A round's rows: from where and to where (equal: nothing to move), and their weights' places.
struct Round {
    int64_t from[MOVE_THREADS], to[MOVE_THREADS];
    int32_t slot[MOVE_THREADS];
};

// What a thread holds of a round.
struct Held {
    uint4 unit[UNITS];
    uint32_t word[WORDS];
};

template <bool FOUR>
struct Mover {
    const EvictArgs &a;
    const Round &rd;
    const float *weights;
    float *weights_out;
    int32_t i0, count;                   // the round's first row, and how many it has

    // 16-byte unit `u` of the round: its row, and its offset there (both planes of it)
    __device__ __forceinline__ void unit(int32_t u, int32_t *row, int32_t *off, bool *value) const {
        *row = (int32_t)a.by_units.div((uint32_t)u);
        const int32_t c = u - *row * (int32_t)a.by_units.d, half = (int32_t)a.by_units.d / 2;
        *value = c >= half;
        *off = 16 * (c - (*value ? half : 0));
    }
    // word `u`: of the weight (0), or of the block scales
    __device__ __forceinline__ void word(int32_t u, int32_t *row, int32_t *c) const {
        *row = FOUR ? (int32_t)a.by_words.div((uint32_t)u) : u;
        *c = u - *row * a.words;
    }
    __device__ __forceinline__ unsigned char *scales(int32_t c, int64_t at) const {
        const int32_t half = (a.words - 1) / 2;
        return c <= half ? a.k_block_scales + at / 8 + 4 * (c - 1)
                         : a.v_block_scales + at / 8 + 4 * (c - 1 - half);
    }
    __device__ __forceinline__ void load(Held &x) const {
        const int32_t units = count * (int32_t)a.by_units.d;
#pragma unroll
        for (int e = 0; e < UNITS; ++e) {
            const int32_t u = e * MOVE_THREADS + (int32_t)threadIdx.x;
            if (u < units) {
                int32_t row, off;
                bool value;
                unit(u, &row, &off, &value);
                const int64_t from = rd.from[row];
                if (from >= 0 && rd.to[row] >= 0)
                    x.unit[e] = *(const uint4 *)((value ? a.v_plane : a.k_plane).base + from + off);
            }
        }
        const int32_t words = count * (FOUR ? a.words : 1);
#pragma unroll
        for (int e = 0; e < (FOUR ? WORDS : 1); ++e) {
            const int32_t u = e * MOVE_THREADS + (int32_t)threadIdx.x;
            if (u < words) {
                int32_t row, c;
                word(u, &row, &c);
                if (!FOUR || c == 0)
                    x.word[e] = __float_as_uint(weights[rd.slot[row]]);
                else if (rd.from[row] >= 0 && rd.to[row] >= 0)
                    x.word[e] = *(const uint32_t *)scales(c, rd.from[row]);
            }
        }
    }
    __device__ __forceinline__ void store(const Held &x) const {
        const int32_t units = count * (int32_t)a.by_units.d;
#pragma unroll
        for (int e = 0; e < UNITS; ++e) {
            const int32_t u = e * MOVE_THREADS + (int32_t)threadIdx.x;
            if (u < units) {
                int32_t row, off;
                bool value;
                unit(u, &row, &off, &value);
                const int64_t to = rd.to[row];
                if (to >= 0 && rd.from[row] >= 0)
                    *(uint4 *)((value ? a.v_plane : a.k_plane).base + to + off) = x.unit[e];
            }
        }
        const int32_t words = count * (FOUR ? a.words : 1);
#pragma unroll
        for (int e = 0; e < (FOUR ? WORDS : 1); ++e) {
            const int32_t u = e * MOVE_THREADS + (int32_t)threadIdx.x;
            if (u < words) {
                int32_t row, c;
                word(u, &row, &c);
                if (!FOUR || c == 0)
                    weights_out[i0 + row] = __uint_as_float(x.word[e]);
                else if (rd.to[row] >= 0 && rd.from[row] >= 0)
                    *(uint32_t *)scales(c, rd.to[row]) = x.word[e];
            }
        }
    }
};

// Rows [i0, i0 + count) of the kept: their places. By all threads; a barrier has to follow.
__device__ __forceinline__ void place_rows(const EvictArgs &a, Round &rd, const int32_t *kept, int32_t r, int32_t h,
                                           int32_t i0, int32_t count, uint32_t *bad) {
    if ((int32_t)threadIdx.x < count) {
        const int32_t j = kept[i0 + threadIdx.x];
        const int64_t from = offset_of(a, a.from, r, h, j, bad);
        const int64_t to = offset_of(a, a.into, r, h, i0 + (int32_t)threadIdx.x, bad);
        // (a row that is where it goes stays there)
        rd.from[threadIdx.x] = from == to ? -1 : from;
        rd.to[threadIdx.x] = to;
        rd.slot[threadIdx.x] = j;
    }
}

// Into other blocks.
template <bool FOUR>
__global__ void __launch_bounds__(MOVE_THREADS, 4) copy_kernel(EvictArgs a) {
    __shared__ Round rd;
    const int32_t head = (int32_t)a.by_chunks.div(blockIdx.x), chunk = (int32_t)blockIdx.x - head * a.chunks;
    const int32_t r = (int32_t)a.by_heads.div((uint32_t)head), h = head - r * a.H;
    wait_for_previous();
    let_next_start();
    uint32_t bad = 0;
    const int32_t n = tokens_of(a, r, &bad), total = min(n, a.keep);
    bad = 0;                             // (told by the kernel before)
    float *out = a.weights_out + r * a.out_request + h * a.out_head;
    for (int32_t j = total + chunk * MOVE_THREADS + (int32_t)threadIdx.x; j < n; j += a.chunks * MOVE_THREADS)
        out[j] = 0.0f;
    const int32_t i0 = chunk * a.rows, count = min(a.rows, total - i0);
    if (count <= 0) return;
    place_rows(a, rd, a.kept + (int64_t)head * a.keep, r, h, i0, count, &bad);
    if (bad != 0) atomicOr(a.flags, bad);
    __syncthreads();
    const Mover<FOUR> mv = {a, rd, a.weights + r * a.w_request + h * a.w_head, out, i0, count};
    Held x;
    mv.load(x);
    mv.store(x);
}

// In place.
template <bool FOUR>
__global__ void __launch_bounds__(MOVE_THREADS, 2) gather_kernel(EvictArgs a) {
    __shared__ Round rounds[2];
    cg::cluster_group cluster = cg::this_cluster();
    const int32_t blocks = (int32_t)cluster.num_blocks(), part = (int32_t)cluster.block_rank();
    const int32_t head = (int32_t)blockIdx.x / blocks;
    const int32_t r = (int32_t)a.by_heads.div((uint32_t)head), h = head - r * a.H;
    wait_for_previous();
    let_next_start();
    uint32_t bad = 0;
    const int32_t n = tokens_of(a, r, &bad), total = min(n, a.keep);
    bad = 0;                             // (told by the kernel before)
    const int32_t *kept = a.kept + (int64_t)head * a.keep;
    const float *weights = a.weights + r * a.w_request + h * a.w_head;
    float *out = a.weights_out + r * a.out_request + h * a.out_head;
    const int32_t step = blocks * a.rows, count_of = (total + step - 1) / step;
    auto rows_of = [&](int32_t k) { return max(0, min(a.rows, total - (k * step + part * a.rows))); };
    Held x;
    if (count_of > 0) {
        place_rows(a, rounds[0], kept, r, h, part * a.rows, rows_of(0), &bad);
        __syncthreads();
        const Mover<FOUR> mv = {a, rounds[0], weights, out, part * a.rows, rows_of(0)};
        mv.load(x);
    }
    for (int32_t k = 0; k < count_of; ++k) {
        const int32_t i0 = k * step + part * a.rows;
        Held next;
        if (k + 1 < count_of) {
            place_rows(a, rounds[(k + 1) & 1], kept, r, h, i0 + step, rows_of(k + 1), &bad);
            __syncthreads();
            const Mover<FOUR> mv = {a, rounds[(k + 1) & 1], weights, out, i0 + step, rows_of(k + 1)};
            mv.load(next);
        }
        cluster.sync();                  // all of this round's rows are held
        const Mover<FOUR> mv = {a, rounds[k & 1], weights, out, i0, rows_of(k)};
        mv.store(x);
        __syncthreads();
        x = next;
    }
    if (bad != 0) atomicOr(a.flags, bad);
    // (every source of a row has been read)
    for (int32_t j = total + part * MOVE_THREADS + (int32_t)threadIdx.x; j < n; j += blocks * MOVE_THREADS)
        out[j] = 0.0f;
}

}  // namespace

kvr_status kvc_evict_launch(const kvc_cache *c, int32_t layer, const kvc_evict *p, void *stream) {
    EvictArgs a = {};
    const int32_t H = c->d.kv_heads;
    const bool four = c->d.dtype == KVC_DTYPE_E2M1;
    const bool other = p->into.ids != nullptr && p->into.ids != p->table.ids;
    a.from = c->slots(p->table);
    a.into = c->slots(other ? p->into : p->table);
    a.k_plane = c->plane(layer, 0);
    a.v_plane = c->plane(layer, 1);
    a.k_block_scales = c->block_scales(layer, 0);
    a.v_block_scales = c->block_scales(layer, 1);
    a.lengths = p->lengths;
    a.weights = p->weights;
    a.weights_out = p->weights_out;
    a.kept = p->kept;
    a.flags = c->ws.flags;
    a.w_request = p->weights_request_stride, a.w_head = p->weights_head_stride;
    a.out_request = p->out_request_stride, a.out_head = p->out_head_stride;
    a.requests = p->num_requests, a.H = H, a.width = p->weights_width;
    a.keep = p->keep, a.recent = p->recent;
    const int32_t units = (int32_t)(2 * c->row_bytes / 16);
    a.words = four ? 1 + 2 * (c->d.head_dim / 64) : 1;
    a.rows = std::max(1, std::min(MOVE_THREADS, UNITS * MOVE_THREADS / units));
    a.by_heads = kvr_make_div((uint32_t)H);
    a.by_units = kvr_make_div((uint32_t)units);
    a.by_words = kvr_make_div((uint32_t)a.words);
    const int64_t heads = (int64_t)p->num_requests * H;
    const int32_t sms = kvc_stream_sms(c, stream);
    const int64_t longest = std::min<int64_t>(p->weights_width, (int64_t)p->table.width * c->d.block_size);
    // blocks of a cluster: as many as keep the SMs busy and have something to do
    auto cluster_of = [&](int64_t each) {
        int32_t blocks = 1;
        while (blocks < 8 && heads * blocks * 2 <= 2 * (int64_t)sms && (longest + blocks - 1) / blocks > each) blocks *= 2;
        return blocks;
    };
    const int32_t choose = cluster_of(2048);
    a.chunks = (int32_t)std::max<int64_t>(1, (std::min<int64_t>(longest, p->keep) + a.rows - 1) / a.rows);
    a.by_chunks = kvr_make_div((uint32_t)a.chunks);
    if (heads * 8 > INT32_MAX || heads * a.chunks > INT32_MAX) return KVR_ERR_UNSUPPORTED;
    kvr_status st = kvc_launch(select_kernel, a, dim3((unsigned)(heads * choose)), SELECT_THREADS, 0, stream, choose);
    if (st != KVR_OK) return st;
    if (other && p->weights_out != p->weights)
        return kvc_launch(four ? copy_kernel<true> : copy_kernel<false>, a, dim3((unsigned)(heads * a.chunks)),
                          MOVE_THREADS, 0, stream);
    const int32_t blocks = cluster_of(a.rows);
    return kvc_launch(four ? gather_kernel<true> : gather_kernel<false>, a, dim3((unsigned)(heads * blocks)),
                      MOVE_THREADS, 0, stream, blocks);
}
