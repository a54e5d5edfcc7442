// cache_evict.cu -- which of a head's cached tokens stay, by their weights, and their rows moved together.
//
// Select. Of n tokens the `recent` newest stay, and of the others the `need` = keep - recent of the largest
// weights: those above the need-th largest, T, and of those equal to it the lowest slots. A cluster of blocks has
// a head; each block a contiguous share of its weights, each warp of that, held in registers. T comes digit by digit (8
// bits of the weights as ordered integers): each block counts its weights that fit the digits so far and sends the
// counts to all, every block adds them up and so finds the same digit, with one barrier of the cluster a digit. From
// the same counts it knows what stays of the blocks before it; each warp counts what stays of its own share and
// writes those slots where the shares before it end. The weights are read once: barriers bound it, not HBM. (Digits of
// 11 bits are one barrier fewer, but eight times the counts between blocks: 44 us where 8 bits took 17, 16 heads of
// 32768 weights. Counts fetched after the barrier, weights in shared memory: 41 us with the rows, now 38.)
//
// Move. Row i of the kept goes to slot i, which is not after its own. Into other blocks, rows in any
// order by any block. In place, slot i may still hold a row that has to go further down; it is the source of
// a row i' <= i. A cluster has a head, goes up the kept rows in rounds of a few rows a block, and each
// round's rows are all in registers before any of them is stored (one barrier of the cluster a round; the
// next ones are asked for before that, as no store reaches slots of rows behind its own).
//
// Measured, into other blocks: 16 requests of 2000 to 8192 tokens cut to 2048, 8 heads of 128 in bf16 (274 MB) 56 us, of
// which select 12; 4 of 32768 to 8192, 4 heads, 38 us, select 13. Rows move at 5.9 TB/s. In place 82 and 73 us: a head
// is one cluster of 8 blocks at most, and each round waits for its loads and for the slowest block (stalls: barrier,
// fence; in the second 128 blocks for 152 SMs, HBM at 19 % of its nominal rate). In 4 bits 33 and 28 us into other
// blocks, 50 and 47 in place (floors 11.8 and 6.2: select and the chains of waits of short rows; the in-place
// kernel spills 92 bytes a thread under its limit of 128 registers).
#include <cooperative_groups.h>

#include <algorithm>

#include "cache.h"

namespace {

using namespace kvc;
namespace cg = cooperative_groups;

constexpr int SELECT_THREADS = 512, SELECT_WARPS = SELECT_THREADS / 32;
constexpr int BINS = 256;
constexpr int MOST_BLOCKS = 8;     // of a cluster
constexpr int SHARE = 2048;        // weights of a block, above which a head gets another, while there is room for it
constexpr int HELD = 8;            // weights that a thread holds; those beyond are read each time
constexpr int COPY_THREADS = 128, MOVE_THREADS = 256;
constexpr int MOST_CLEARING = 1 << 20;   // blocks of a head that clear weights behind what stays, into other blocks
constexpr int UNITS = 8;           // 16-byte units of a thread at a time
constexpr int WORDS = 9;           // words of a thread besides: a weight, and block scales of 4-bit rows

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
    int32_t step_rows, step_units; // what as many units as a block has threads are
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

// The sum of what the warps before this one have left in `scan`.
__device__ __forceinline__ uint32_t before_warp(const uint32_t (*scan)[2], int which) {
    static_assert(SELECT_WARPS <= 32, "");
    const int lane = threadIdx.x % 32;
    return __reduce_add_sync(~0u, lane < (int)threadIdx.x / 32 ? scan[lane][which] : 0u);
}

template <int BLOCKS>
__global__ void __launch_bounds__(SELECT_THREADS) select_kernel(EvictArgs a) {
    __shared__ uint32_t hist[BINS];
    __shared__ uint32_t all[2][BLOCKS][BINS];              // all blocks' counts, as each sends its own
    __shared__ uint32_t scan[SELECT_WARPS][2];
    __shared__ uint32_t found[5];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    constexpr int blocks = BLOCKS;
    const int32_t part = BLOCKS > 1 ? (int32_t)cluster.block_rank() : 0;
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
        for (Share s(0, n, part * SELECT_THREADS + tid, blocks * SELECT_THREADS); s.more(); s.next()) kept[s.at()] = s.at();
        return;
    }
    const int32_t old = n - a.recent, need = a.keep - a.recent;
    // (written last: a barrier of the cluster waits for stores before it)
    auto newest = [&] {
        for (Share s(0, a.recent, part * SELECT_THREADS + tid, blocks * SELECT_THREADS); s.more(); s.next())
            kept[need + s.at()] = old + s.at();
    };
    if (need == 0) {
        newest();
        return;
    }

    if (BLOCKS > 1) cluster.barrier_arrive();              // (that the others have begun; waited for below)
    const float *weights = a.weights + r * a.w_request + h * a.w_head;
    const int32_t share = (old + blocks - 1) / blocks;
    const int32_t j0 = min(old, part * share), size = min(old, j0 + share) - j0;
    // a warp's part of the block's share; its lanes' weights, those beyond what registers hold read each time
    const int32_t run = (size + SELECT_WARPS - 1) / SELECT_WARPS;
    const int32_t i0 = min(size, warp * run), i1 = min(size, i0 + run);
    uint32_t held[HELD];
#pragma unroll
    for (int t = 0; t < HELD; ++t) {
        const int32_t i = i0 + 32 * t + lane;
        held[t] = i < i1 ? ordered(weights[j0 + i]) : 0u;
    }
    // f(i, key, whether there is one) for each; warps stay whole
    auto each = [&](auto f) {
#pragma unroll
        for (int t = 0; t < HELD; ++t)
            if (i0 + 32 * t < i1) f(i0 + 32 * t + lane, held[t], i0 + 32 * t + lane < i1);
        for (int32_t i = i0 + 32 * HELD; i < i1; i += 32) {
            const bool some = i + lane < i1;
            f(i + lane, some ? ordered(weights[j0 + i + lane]) : 0u, some);
        }
    };
    if (tid < BINS) hist[tid] = 0;

    uint32_t known = 0, mask = 0;        // T's digits so far, and which bits they are
    uint32_t left = (uint32_t)need;      // of the weights that fit them, how many stay
    uint32_t lower_above = 0, lower_same = 0;   // of the blocks before this one: above T, and equal
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        uint32_t(*counts)[BINS] = all[pass & 1];
        __syncthreads();
        each([&](int32_t, uint32_t k, bool some) {
            if (some && (k & mask) == known) atomicAdd(hist + (k >> shift & 255u), 1u);
        });
        __syncthreads();
        if (BLOCKS > 1 && pass == 0) cluster.barrier_wait();
        // (what the others read of this array, two digits ago, they read before the barrier of the last)
        static_assert(SELECT_THREADS >= BINS && BINS % 32 == 0, "");
        if (tid < BINS) {
            const uint32_t c = hist[tid];
            hist[tid] = 0;
            if (BLOCKS > 1) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) *cluster.map_shared_rank(&counts[part][tid], b) = c;
            } else {
                counts[0][tid] = c;
            }
        }
        if (BLOCKS > 1)
            cluster.sync();
        else
            __syncthreads();
        // a thread's bin, from the top down: its count over all blocks, and over those before this one
        const int bin = BINS - 1 - tid;
        uint32_t sum = 0, lower = 0, sums = 0, lowers = 0;
        if (tid < BINS) {
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                const uint32_t c = counts[b][bin];
                sum += c;
                lower += b < part ? c : 0u;
            }
            sums = sum, lowers = lower;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t y = __shfl_up_sync(~0u, sums, o), z = __shfl_up_sync(~0u, lowers, o);
                if (lane >= o) sums += y, lowers += z;
            }
            if (lane == 31) scan[warp][0] = sums, scan[warp][1] = lowers;
        }
        __syncthreads();
        if (tid < BINS) {
            const uint32_t above = sums - sum + before_warp(scan, 0);
            const uint32_t lower_before = lowers - lower + before_warp(scan, 1);
            if (above < left && left <= above + sum) {
                found[0] = (uint32_t)bin;
                found[1] = left - above;
                found[2] = sum;
                found[3] = lower_before;
                found[4] = lower;
            }
        }
        __syncthreads();
        known |= found[0] << shift;
        mask |= 255u << shift;
        left = found[1];
        lower_above += found[3];
        lower_same = found[4];
        if (left == found[2]) break;     // all that fit stay, whatever follows (the same in every block)
    }

    // of the warp's: how many are above T, and how many equal it
    uint32_t above = 0, same = 0;
    each([&](int32_t, uint32_t k, bool some) {
        above += some && (k & mask) > known;
        same += some && (k & mask) == known;
    });
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        above += __shfl_xor_sync(~0u, above, o);
        same += __shfl_xor_sync(~0u, same, o);
    }
    if (lane == 0) scan[warp][0] = above, scan[warp][1] = same;
    __syncthreads();
    above = lower_above + before_warp(scan, 0), same = lower_same + before_warp(scan, 1);
    each([&](int32_t i, uint32_t k, bool some) {
        const bool gt = some && (k & mask) > known, eq = some && (k & mask) == known;
        const uint32_t gts = __ballot_sync(~0u, gt), eqs = __ballot_sync(~0u, eq);
        const uint32_t before = (1u << lane) - 1u;
        const uint32_t g = above + __popc(gts & before), e = same + __popc(eqs & before);
        if (gt || (eq && e < left)) kept[g + min(e, left)] = j0 + i;
        above += __popc(gts);
        same += __popc(eqs);
    });
    newest();
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

// A round's rows: from where (-1: nothing to move) and to where, and the slots that they had.
template <int THREADS>
struct Round {
    int64_t from[THREADS], to[THREADS];
    int32_t slot[THREADS];
};

// What a thread holds of a round.
template <bool FOUR>
struct Held {
    uint4 unit[UNITS];
    uint32_t word[FOUR ? WORDS : 1];
};

// A round's rows between memory and the threads' registers.
template <int THREADS, bool FOUR>
struct Mover {
    const EvictArgs &a;
    const Round<THREADS> &rd;
    const float *weights;
    float *weights_out;
    int32_t i0, count;                   // the round's first row, and how many it has

    // Each of the thread's 16-byte units: f(e, row, plane, offset in the row). A row's units are its key's, then
    // its value's; a thread's are THREADS apart.
    template <typename F>
    __device__ __forceinline__ void units(F f) const {
        const int32_t of_row = (int32_t)a.by_units.d, half = of_row / 2;
        int32_t row = (int32_t)a.by_units.div(threadIdx.x), c = (int32_t)threadIdx.x - row * of_row;
#pragma unroll
        for (int e = 0; e < UNITS; ++e) {
            if (row < count) {
                const bool value = c >= half;
                f(e, row, (value ? a.v_plane : a.k_plane).base, 16 * (c - (value ? half : 0)));
            }
            row += a.step_rows, c += a.step_units;
            if (c >= of_row) c -= of_row, ++row;
        }
    }
    // The same of its words of block scales: f(e, row, plane, offset in the row's).
    template <typename F>
    __device__ __forceinline__ void words(F f) const {
#pragma unroll
        for (int e = 0; e < WORDS - 1; ++e) {
            const int32_t u = e * THREADS + (int32_t)threadIdx.x, row = (int32_t)a.by_words.div((uint32_t)u);
            const int32_t c = u - row * (int32_t)a.by_words.d, half = (int32_t)a.by_words.d / 2;
            if (row < count) f(e, row, c >= half ? a.v_block_scales : a.k_block_scales, 4 * (c >= half ? c - half : c));
        }
    }
    __device__ __forceinline__ void load(Held<FOUR> &x) const {
        units([&](int e, int32_t row, const unsigned char *plane, int32_t off) {
            const int64_t from = rd.from[row];
            if (from >= 0) x.unit[e] = *(const uint4 *)(plane + from + off);
        });
        if ((int32_t)threadIdx.x < count) x.word[0] = __float_as_uint(weights[rd.slot[threadIdx.x]]);
        if constexpr (FOUR)
            words([&](int e, int32_t row, const unsigned char *plane, int32_t off) {
                const int64_t from = rd.from[row];
                if (from >= 0) x.word[1 + e] = *(const uint32_t *)(plane + from / 8 + off);
            });
    }
    __device__ __forceinline__ void store(const Held<FOUR> &x) const {
        units([&](int e, int32_t row, unsigned char *plane, int32_t off) {
            if (rd.from[row] >= 0) *(uint4 *)(plane + rd.to[row] + off) = x.unit[e];
        });
        if ((int32_t)threadIdx.x < count) weights_out[i0 + threadIdx.x] = __uint_as_float(x.word[0]);
        if constexpr (FOUR)
            words([&](int e, int32_t row, unsigned char *plane, int32_t off) {
                if (rd.from[row] >= 0) *(uint32_t *)(plane + rd.to[row] / 8 + off) = x.word[1 + e];
            });
    }
};

// Rows [i0, i0 + count) of the kept: their places. By all threads; a barrier has to follow.
template <int THREADS>
__device__ __forceinline__ void place_rows(const EvictArgs &a, Round<THREADS> &rd, const int32_t *kept, int32_t r,
                                           int32_t h, int32_t i0, int32_t count, uint32_t *bad) {
    if ((int32_t)threadIdx.x < count) {
        const int32_t j = kept[i0 + threadIdx.x];
        const int64_t from = offset_of(a, a.from, r, h, j, bad);
        const int64_t to = offset_of(a, a.into, r, h, i0 + (int32_t)threadIdx.x, bad);
        // (a row that is where it goes stays there)
        rd.from[threadIdx.x] = from == to || to < 0 ? -1 : from;
        rd.to[threadIdx.x] = to;
        rd.slot[threadIdx.x] = j;
    }
}

// Into other blocks. Small blocks, many on an SM: each begins with a chain of waits (length, kept slots, block
// ids, rows), which the others' rows cover.
template <bool FOUR>
__global__ void __launch_bounds__(COPY_THREADS, 8) copy_kernel(EvictArgs a) {
    __shared__ Round<COPY_THREADS> rd;
    const int32_t head = (int32_t)a.by_chunks.div(blockIdx.x), chunk = (int32_t)blockIdx.x - head * a.chunks;
    const int32_t r = (int32_t)a.by_heads.div((uint32_t)head), h = head - r * a.H;
    wait_for_previous();
    let_next_start();
    uint32_t bad = 0;
    const int32_t n = tokens_of(a, r, &bad), total = min(n, a.keep);
    bad = 0;                             // (told by the kernel before)
    float *out = a.weights_out + r * a.out_request + h * a.out_head;
    // (a head of 2^28 tokens has so many blocks that not all of their threads can be counted in 32 bits)
    const int32_t clearing = min(a.chunks, MOST_CLEARING);
    if (chunk < clearing)
        for (Share s(total, n, chunk * COPY_THREADS + (int32_t)threadIdx.x, clearing * COPY_THREADS); s.more(); s.next())
            out[s.at()] = 0.0f;
    const int32_t i0 = chunk * a.rows, count = min(a.rows, total - i0);
    if (count <= 0) return;
    place_rows(a, rd, a.kept + (int64_t)head * a.keep, r, h, i0, count, &bad);
    if (bad != 0) atomicOr(a.flags, bad);
    __syncthreads();
    const Mover<COPY_THREADS, FOUR> mv = {a, rd, a.weights + r * a.w_request + h * a.w_head, out, i0, count};
    Held<FOUR> x;
    mv.load(x);
    mv.store(x);
}

// In place.
template <bool FOUR>
__global__ void __launch_bounds__(MOVE_THREADS, 2) gather_kernel(EvictArgs a) {
    __shared__ Round<MOVE_THREADS> rounds[2];
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
    Held<FOUR> x;
    if (count_of > 0) {
        place_rows(a, rounds[0], kept, r, h, part * a.rows, rows_of(0), &bad);
        __syncthreads();
        const Mover<MOVE_THREADS, FOUR> mv = {a, rounds[0], weights, out, part * a.rows, rows_of(0)};
        mv.load(x);
    }
    for (int32_t k = 0; k < count_of; ++k) {
        const int32_t i0 = k * step + part * a.rows;
        Held<FOUR> next;
        if (k + 1 < count_of) {
            place_rows(a, rounds[(k + 1) & 1], kept, r, h, i0 + step, rows_of(k + 1), &bad);
            __syncthreads();
            const Mover<MOVE_THREADS, FOUR> mv = {a, rounds[(k + 1) & 1], weights, out, i0 + step, rows_of(k + 1)};
            mv.load(next);
        }
        cluster.sync();                  // all of these rows are held
        const Mover<MOVE_THREADS, FOUR> mv = {a, rounds[k & 1], weights, out, i0, rows_of(k)};
        mv.store(x);
        __syncthreads();
        x = next;
    }
    if (bad != 0) atomicOr(a.flags, bad);
    // (every source of a row has been read)
    for (Share s(total, n, part * MOVE_THREADS + (int32_t)threadIdx.x, blocks * MOVE_THREADS); s.more(); s.next())
        out[s.at()] = 0.0f;
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
    const bool apart = other && p->weights_out != p->weights;
    const int32_t units = (int32_t)(2 * c->row_bytes / 16), threads = apart ? COPY_THREADS : MOVE_THREADS;
    // (block scales: 2 D / 64 words a row, as many as its units or fewer)
    a.rows = std::max(1, std::min(threads, UNITS * threads / units));
    a.step_rows = threads / units;
    a.step_units = threads % units;
    a.by_heads = kvr_make_div((uint32_t)H);
    a.by_units = kvr_make_div((uint32_t)units);
    a.by_words = kvr_make_div((uint32_t)std::max(1, 2 * (c->d.head_dim / 64)));
    const int64_t heads = (int64_t)p->num_requests * H;
    const int32_t sms = kvc_stream_sms(c, stream);
    const int64_t longest = std::min<int64_t>(p->weights_width, (int64_t)p->table.width * c->d.block_size);
    // blocks of a cluster: as many as keep the SMs busy and have something to do
    auto cluster_of = [&](int64_t each, int64_t resident) {
        int32_t blocks = 1;
        while (blocks < MOST_BLOCKS && heads * blocks * 2 <= resident * sms && (longest + blocks - 1) / blocks > each)
            blocks *= 2;
        return blocks;
    };
    const int32_t choose = cluster_of(SHARE, 2);
    a.chunks = (int32_t)std::max<int64_t>(1, (std::min<int64_t>(longest, p->keep) + a.rows - 1) / a.rows);
    a.by_chunks = kvr_make_div((uint32_t)a.chunks);
    if (heads * 8 > INT32_MAX || heads * a.chunks > INT32_MAX) return KVR_ERR_UNSUPPORTED;
    const auto select = choose == 1   ? select_kernel<1>
                        : choose == 2 ? select_kernel<2>
                        : choose == 4 ? select_kernel<4> : select_kernel<8>;
    kvr_status st = kvc_launch(select, a, dim3((unsigned)(heads * choose)), SELECT_THREADS, 0, stream, choose);
    if (st != KVR_OK) return st;
    if (apart)
        return kvc_launch(four ? copy_kernel<true> : copy_kernel<false>, a, dim3((unsigned)(heads * a.chunks)),
                          COPY_THREADS, 0, stream);
    const int32_t blocks = cluster_of(a.rows, 2);
    return kvc_launch(four ? gather_kernel<true> : gather_kernel<false>, a, dim3((unsigned)(heads * blocks)),
                      MOVE_THREADS, 0, stream, blocks);
}
