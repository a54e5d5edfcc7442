// cache_latent.cu -- attention of a request's newest tokens over its paged latents (tcgen05).
//
// A latent row is 576 elements: it is the key of all query heads, and its first 512 elements are
// the value. The R = m Hq rows of a request (in passes of 128) meet each latent once: 2 x 1088
// flops a row and latent against its 1152 bytes. With 128 rows that is 242 flops a byte, close
// to what the card has (278), so both HBM and the tensor cores have to be kept busy; with 16 rows
// it is HBM alone, and the 128-row products cost nothing that is missed.
//
// Why a cluster of two. O is 128 x 512 in fp32, all of an SM's 512 columns of tensor memory, and
// leaves no room for S. So two SMs share a tile of KT keys, each with HALF OF THE ELEMENTS (256
// of the value and 32 of the rest): each loads its half of every latent, and nothing twice; each
// computes the partial S = Q K^T of its half and sends it to the other through distributed
// shared memory (16 KB a tile); each adds the two halves in the same way, so both hold the same
// softmax, and multiplies P with its 256 value elements. No product and no load is done twice;
// the exponentials are.
//
// Tensor memory: O [128 x 256] fp32 in columns 0-255; Q, 288 16-bit elements a row, in 144
// columns, where the products read it as operand A (from shared memory it would take 72 KB of it
// and cost more of its bandwidth than all of K); three S of KT = 32 columns, and one P of 16:
// all 512. What a tile waits for is the way from its S to its P, through the other SM and
// back, so the number of S under way counts for more than their size: tiles of 64 keys, which
// leave room for one S, took 210 us where these take 165; 48 keys with P over S 540; a second P,
// with part of Q in shared memory instead, 181.
//
// Shared memory: a ring of 9 tiles' halves (18 KB each), and three times the half of S that the
// other SM sends. A tile is laid out in 128-byte rows of 64 elements (swizzled), which serve as
// the K-major operand of S and as the MN-major operand of O. Tiles come by the copy engine, in
// boxes of a block's tokens, where blocks are multiples of 8 tokens that divide a tile or are
// divided by it; a request's last, partial tile, a window's first, and all tiles of other block sizes,
// come row by row by 16-byte cp.async, with zeros for the rows that no query sees. (By cp.async alone the load
// and store units were what the kernel waited for.)
//
// Warps: two times 4 of softmax (one thread a row; every second tile), 4 that send S to the other
// SM, 4 of loads, 2 that issue the products of S and 1 those of O, 1 that tells the other SM what
// it may send over. One tile's softmax takes its 4 warps about 1700 cycles, and HBM wants a tile
// in 780, so one set is too few; a third (177 us) only shares the SM's issue slots with the
// others. A tile's softmax needs of the one before only what P is relative to, which goes through
// shared memory as soon as it is known. O is rescaled only when a row's maximum outgrows by 2^20
// (f16: 2^8) the one that its P is relative to, which hardly happens after the first tiles of a
// job: powers of two cost no precision in P, O and the sums.
//
// Numbers: S, maxima, sums, O and all joins are fp32. With more than 32 rows P is rounded once to the
// pool's 16-bit type for its product: a second product for what is left of it reads V again, and its
// columns of tensor memory leave room for two S instead of three (181 -> 221 us for 64 requests of 1024 to
// 16384 latents under 128 heads, L2 cold). Up to 32 rows (FINE) most of the 128 are free, and as many of
// them take what is left: rows r and r + FINE hold the same query, so both get the same S, maxima and P, bit
// for bit; one enters P cut to 16 bits into the product, the other the rest, and their O are added at the
// end: 15 bits of P count over bf16. Errors against 64 bits (2-norm, relative) are 0.0016 to 0.0017 then, those
// of 32-bit sums rounded to bf16, instead of 0.0019 to 0.0026 (f16 0.00021, 0.00022 to 0.00026). Up to 16 rows
// both are a warp's, and it costs the cutting and 16 shuffles a piece of O; up to 32, a second warp of
// softmax and of sending, and O's way from one warp to the other: one request of 4096, 16 heads 14.0 ->
// 14.6 us, 4 of 32768 40.7 -> 41.9, 64 of 8192 112 -> 116; 32 rows: 9 of 5 to 6001 19.9 -> 21.1, 64 of 8192 117 ->
// 122. (By a second product 64 of 8192 under 16 heads took 15 % more. 33 to 64 rows could be done the same way,
// but would then keep all four warps busy, as 128 do: 53.4 instead of 44 us for 4 of 32768.)
//
// Every wait ends: after two seconds it gives up and flags KVC_FLAG_TIMEOUT, and its warp goes to
// the end of the kernel, as the others do for want of it.
//
// Measured, with the join: 64 requests of 1024 to 16384 latents, 128 heads, bf16 (528,481
// latents, 627 MB and 147 GFLOP): 162 us, 3.9 TB/s and 0.91 PFLOP/s, 57 % of what HBM alone would
// allow; 64 of 8192 (622 MB) 149 us. A tile of 32 keys comes through in about 1000 cycles. No unit is
// busy for all of them (tensor cores 40 %, shared memory about 75 %: 85 KB of boxes, operands and S a
// tile); from S to P's product a tile is under way for some 5000, most of it in the products, where
// S of two tiles and O of a third take turns, and in the exchange. Each change of job costs about 8 us of 262 KB of
// partial results and an empty pipe, and the join 5 us. One request of 4096 latents with 16 heads: 14.6 us, its fill,
// four tiles and the join one after another.
#include <math.h>

#include <algorithm>

#include <cuda.h>

#include "cache_latent.h"
#include "cache_split.cuh"

namespace {

using namespace kvc;

constexpr int KT = 32;                    // keys of a tile
constexpr int ROWS = 128;                 // query rows of a pass
constexpr int HALF = 256, REST = 32;      // value elements and others of an SM
constexpr int STAGES = 9;                 // tiles in the ring
constexpr int SBUF = 3;                   // halves of S at a time, own and received
constexpr int CHUNK = KT * 128;           // 64 elements of each key
constexpr int STAGE = 4 * CHUNK + KT * 64;
constexpr int XBUF = ROWS * KT * 4;
// warps: softmax of every second tile (2 x 4), sending, loading (4 each); products of S of even
// tiles, of odd tiles, of O; telling
constexpr int SOFT = 2, SEND = 4 * SOFT, LOAD = SEND + 4, KEYS = LOAD + 4, VALS = KEYS + 2,
              TELL = VALS + 1, WARPS = TELL + 1, THREADS = 32 * WARPS;
constexpr int OFF_XBUF = STAGES * STAGE, OFF_BARS = OFF_XBUF + SBUF * XBUF, OFF_TOPS = OFF_BARS + 768,
              OFF_SUMS = OFF_TOPS + SOFT * ROWS * 8,
              OFF_AHEAD = OFF_SUMS + 2 * SOFT * ROWS * 4,
              OFF_PREFIX = OFF_AHEAD + 4 * (AHEAD_MOST + 4);
constexpr uint32_t COL_O = 0, COL_Q = 256, COL_S = 400, COL_P = COL_S + SBUF * KT;
static_assert(COL_P + KT / 2 <= 512, "tensor memory");
constexpr int VALUES = KVC_LATENT_VALUES;
// floats of one part's results: [element / 4][row][4], then (max, sum) a row
constexpr size_t SLOT = (size_t)ROWS * VALUES + 2 * ROWS;

// barriers, in 8-byte words after OFF_BARS
// (a wait tells a phase from the one before only; where more may be under way there are more
// barriers: O_DONE has 4, and S_FREE twice as many as there are S)
enum { K_FULL = 0, K_EMPTY = K_FULL + STAGES, S_FULL = K_EMPTY + STAGES, S_FREE = S_FULL + SBUF,
       X_FULL = S_FREE + 2 * SBUF, X_EMPTY = X_FULL + SBUF, X_READ = X_EMPTY + SBUF,
       P_FULL = X_READ + SBUF, O_DONE = P_FULL + 2, Q_FULL = O_DONE + 4, O_FREE, SUMS,
       DRAIN, REST_FULL = DRAIN + 3, REST_READ = REST_FULL + 2 * SOFT, BARS = REST_READ + 2 * SOFT };
constexpr int OFF_TMEM = BARS * 8, OFF_SCRATCH = OFF_TMEM + 16;
static_assert(OFF_SCRATCH + 4 * WARPS <= 768, "the words after the barriers");

struct LatentArgs {
    CUtensorMap values, rest;  // the plane's rows in pieces of `piece` tokens (piece 0: no such map)
    KvcPlane plane;
    int32_t piece;
    SplitArgs split;
    const unsigned char *q;
    unsigned char *out;
    float *lse;
    int64_t q_request, q_token, q_head, out_request, out_token, out_head;
    float *partial;
    int32_t *prefix, *ahead;  // [requests + 1], what the first block counted, for the join
    int32_t m, Hq, chunks, parts;
    KvrDiv heads;             // by Hq
    CutShape shape;
    float scale;
};

// -- barriers -------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// the same barrier of the other SM of the cluster
__device__ __forceinline__ void bar_arrive_remote(uint32_t remote) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
__device__ __forceinline__ uint32_t remote_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Waits for the phase of `parity`, in turns of a microsecond and for about two seconds at most.
__device__ __forceinline__ uint32_t wait_for(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
                 "AGAIN:\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
                 "@p bra OUT;\n\t"
                 "add.u32 n, n, 1;\n\t"
                 "setp.lt.u32 p, n, 2000000;\n\t"
                 "@p bra AGAIN;\n\t"
                 "setp.ne.u32 p, n, n;\n"
                 "OUT:\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done;
}
// Each lane's row's maximum after a tile, and telling it. One 64-bit word holds both, so no barrier
// has to order two stores; a wait by barrier costs both sides ten times as much.
__device__ __forceinline__ void tell_top(uint32_t tops, uint32_t tile, float top) {
    const uint64_t word = (uint64_t)(tile + 1) << 32 | __float_as_uint(top);
    asm volatile("st.volatile.shared.b64 [%0], %1;" ::"r"(tops + tile % SOFT * (ROWS * 8)), "l"(word)
                 : "memory");
}
__device__ __forceinline__ bool top_after(uint32_t tops, uint32_t tile, float *top, uint32_t *flags) {
    uint64_t word = 0;
    for (uint32_t n = 0; n < (1u << 24); ++n) {
        asm volatile("ld.volatile.shared.b64 %0, [%1];"
                     : "=l"(word)
                     : "r"(tops + tile % SOFT * (ROWS * 8))
                     : "memory");
        if (__all_sync(~0u, (uint32_t)(word >> 32) == tile + 1)) {
            *top = __uint_as_float((uint32_t)word);
            return true;
        }
    }
    atomicOr(flags, KVC_FLAG_TIMEOUT);
    return false;
}
// For a warp, whose lanes go on together with the same answer: false, and a flag, if it gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t *flags) {
    const bool done = __all_sync(~0u, wait_for(bar, parity));
    if (!done) atomicOr(flags, KVC_FLAG_TIMEOUT);
    return done;
}

// -- tensor memory and products ---------------------------------------------------

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tm_load16(uint32_t v[16], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
                 "%10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]),
                   "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t v[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, "
                 "%10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                 "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
                 "r"(v[14]), "r"(v[15])
                 : "memory");
}
// D (+)= A B with A in tensor memory, B in shared memory: two steps of 16 elements, A's 8 columns
// apart, B's `step` times 16 bytes; four such. (One statement, so that an operand is one addition.)
__device__ __forceinline__ void product2(uint32_t d, uint32_t a, uint64_t b, uint32_t step, uint32_t idesc,
                                         uint32_t add) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 b1;\n\t.reg .b32 a1;\n\t"
                 "setp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
                 "add.u32 a1, %1, 8;\n\tadd.u64 b1, %2, %3;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "l"((uint64_t)step), "r"(idesc), "r"(add)
                 : "memory");
}
__device__ __forceinline__ void product4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
                 "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
                 "add.u64 b1, %2, 2;\n\tadd.u64 b2, %2, 4;\n\tadd.u64 b3, %2, 6;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(add)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

// a box of the pool's plane by the copy engine; its bytes count at `bar`
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int32_t element,
                                         int32_t token, int32_t block, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
                 "l"(map), "r"(element), "r"(token), "r"(block), "r"(bar)
                 : "memory");
}

// Shared-memory operand: start, leading and stride offsets in bytes; layout 2 = 128-byte
// swizzle, 4 = 64-byte swizzle. (A shared address of a cluster holds the rank above its 18 bits.)
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride,
                                            uint32_t layout) {
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | ((uint64_t)layout << 61);
}

// fp32 accumulation of 16-bit operands: type (0 f16, 1 bf16) of both, B transposed (MN-major), N
__host__ __device__ constexpr uint32_t idesc(bool bf16, bool mn_major, uint32_t n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
           ((mn_major ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((ROWS >> 4) << 24);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two fp32 numbers in one register pair, and what is done to both at once
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t d) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
    return f;
}
__device__ __forceinline__ uint64_t splat2(float f) {
    return pack2(__float_as_uint(f), __float_as_uint(f));
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    return d;
}
// s[0..1] = (s[0..1] + (x, y)) * sc: the same on both SMs, whose halves change places
__device__ __forceinline__ void scaled_sum(uint32_t *s, float x, float y, uint64_t sc2) {
    uint64_t d = add2(pack2(s[0], s[1]), pack2(__float_as_uint(x), __float_as_uint(y)));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(sc2));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(s[0]), "=r"(s[1]) : "l"(d));
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
    return d;
}

// Two weights cut to 16 bits, or what that leaves of them, cut: less is -1 in both halves for the rest, else
// 0. (That the rest may be zero, which an infinite value would not stand, is no matter for latents: a row
// with an infinite value has an infinite key.)
template <bool F16>
__device__ __forceinline__ uint32_t first_or_rest2(float lo, float hi, uint64_t less) {
    uint64_t cut;
    if (F16) {
        uint32_t w;
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
        const float2 f = widen2<true>(w);
        cut = pack2(__float_as_uint(f.x), __float_as_uint(f.y));
    } else {
        cut = pack2(__float_as_uint(lo) & 0xFFFF0000u, __float_as_uint(hi) & 0xFFFF0000u);
    }
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(cut), "l"(less), "l"(pack2(__float_as_uint(lo), __float_as_uint(hi))));
    const float2 f = unpack2(d);
    uint32_t w;
    if (F16)
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f.y), "f"(f.x));
    else
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f.y), "f"(f.x));
    return w;
}

// Units (tiles) that a change of job costs (cache_split.cuh). Parts
// within jobs took (us) 37.6 where equal ones took 41.7 (8 requests of 8192 latents, 128 heads), 25.3
// for 28.8 (2 of 8192), 21.3 for 23.0 (9 of up to 6001, 32 rows); groups 10 above the equal parts 39.9
// for 34.7 (19 of 4096, 64 heads).
constexpr int SLACK = 8;
__device__ __forceinline__ Cut cut_of(const LatentArgs &a, const int32_t *prefix) {
    return Cut(prefix[a.split.requests] * a.chunks, a.shape);
}

// -- the kernel -------------------------------------------------------------------

// How far (as a power of two) P may exceed 1 before O is rescaled. bf16 P and fp32 sums reach further
// than is of use: with logits of 5 (in powers of two) standard deviation 8 takes 186 us where 16 to
// 40 take 162, and O of values up to 2^100 has to stay finite. f16 P ends at 2^16.
template <bool F16>
constexpr float GROWTH_OF = F16 ? 8.0f : 20.0f;

// FINE (16 or 32, 0: not so): rows r and r + FINE of the products are the same query; P of the first is
// the 16-bit number next below the weight, P of the second what is left of it, and O of the two is added.
template <bool F16, int FINE>
__global__ void __launch_bounds__(THREADS, 1) latent_kernel(const __grid_constant__ LatentArgs a) {
    constexpr float GROWTH = GROWTH_OF<F16>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t smem0 = smem_addr(smem), bars = smem0 + OFF_BARS;
    int32_t *prefix = (int32_t *)(smem + OFF_PREFIX), *ahead = (int32_t *)(smem + OFF_AHEAD);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint32_t rank;
    asm("mov.u32 %0, %cluster_ctarank;" : "=r"(rank));
    auto bar = [&](int which) { return bars + 8 * which; };
    auto wait = [&](uint32_t b, uint32_t parity) { return warp_wait(b, parity, a.split.flags); };

    if (warp == KEYS) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         bars + OFF_TMEM)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            bar_init(bar(K_FULL + i), a.piece > 0 ? 1 : 32);   // the loading warp or its threads
            bar_init(bar(K_EMPTY + i), 1);
        }
        for (int i = 0; i < SBUF; ++i) {
            bar_init(bar(S_FULL + i), 1);
            bar_init(bar(S_FREE + i), 8);         // softmax and sending warps
            bar_init(bar(S_FREE + SBUF + i), 8);
            bar_init(bar(X_FULL + i), 2);         // both halves of S: the product, the other SM's bytes
            bar_init(bar(X_EMPTY + i), 1);        // its telling warp
            bar_init(bar(X_READ + i), 4);         // the softmax warps
        }
        for (int i = 0; i < 2; ++i) bar_init(bar(P_FULL + i), 4);
        for (int i = 0; i < 4; ++i) bar_init(bar(O_DONE + i), 1);
        bar_init(bar(Q_FULL), 4);
        bar_init(bar(O_FREE), SEND);
        bar_init(bar(SUMS), SEND);
        bar_init(bar(DRAIN), 1);
        bar_init(bar(DRAIN + 1), 1);
        bar_init(bar(DRAIN + 2), 1);
        for (int i = 0; i < 2 * SOFT; ++i) bar_init(bar(REST_FULL + i), 1), bar_init(bar(REST_READ + i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < SOFT * ROWS; i += THREADS) ((uint64_t *)(smem + OFF_TOPS))[i] = 0;
    wait_for_previous();
    let_next_start();
    unit_prefix<KT>(a.split, KT, prefix, (int32_t *)(smem + OFF_BARS + OFF_SCRATCH));
    const Cut cut = cut_of(a, prefix);
    if (warp == KEYS && cut.group > 0) cut.count(prefix, a.split.requests, ahead);
    __syncwarp();
    fence_before();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    fence_after();
    const uint32_t tmem = *(volatile uint32_t *)(smem + OFF_BARS + OFF_TMEM);

    if (blockIdx.x == 0)
        for (int32_t r = tid; r <= a.split.requests; r += THREADS) {
            a.prefix[r] = prefix[r];
            if (cut.group > 0) a.ahead[r] = ahead[r];
        }
    const int32_t part = blockIdx.x / 2;
    int32_t x, x_end;
    int32_t known = cut.units_of(part, prefix, ahead, a.shape, &x, &x_end);
    const int32_t M = a.m * a.Hq;

    // a thread's query row in a segment: lane of tensor memory, row of the pass
    const int row = tid % ROWS;
    const uint32_t lanes = tmem + ((uint32_t)(row & ~31) << 16);
    struct Query {
        int32_t token, hq;
        bool mine;
    };
    auto query_of = [&](const Segment &seg) -> Query {
        const int32_t rho = seg.job * ROWS + (FINE > 0 ? row % (FINE > 0 ? FINE : 1) : row);
        const int32_t token = (int32_t)a.heads.div((uint32_t)rho);
        return {token, rho - token * a.Hq, rho < M};
    };
    // Warps of 32 rows that a segment has rows for. The others of softmax and sending only keep
    // step: what lies in their lanes of tensor memory is read by nobody. (4 requests of 32768
    // latents, 16 heads: 40.7 us, and 45.5 with all at work.)
    auto live_warps = [&](const Segment &seg) {
        return FINE > 0 ? FINE / 16 : min(ROWS / 32, (M - seg.job * ROWS + 31) / 32);
    };
    const bool second = FINE > 0 && (row / (FINE > 0 ? FINE : 1)) % 2 == 1;      // of what is left of P

    if (warp < SEND) {
        // ---- softmax of every second tile ----
        const uint32_t group = warp / 4;
        const uint64_t sc2 = splat2(a.scale * 1.4426950408889634f);
        const uint64_t less = splat2(second ? -1.0f : 0.0f);
        // what a row's P is relative to after a tile: (maximum, tile + 1) by tile % SOFT and row. One
        // 64-bit word, so that whoever sees the number sees its maximum too
        const uint32_t tops = smem0 + OFF_TOPS + row * 8;
        float *sums = (float *)(smem + OFF_SUMS);     // [2][SOFT][ROWS]
        uint32_t it = 0, segments = 0;            // tiles and segments so far
        uint32_t handed = 0;                      // pieces of O from second rows to first ones
        bool ok = true;
        while (ok && x < x_end) {
            const Segment seg = segment_at(x, x_end, prefix, a.shape, known);
            known = -1;
            const uint32_t n = (uint32_t)(seg.u1 - seg.u0);
            x += n;
            uint32_t bad = 0;
            const Span sp = span_of(a.split, seg.r, KT, &bad);
            const Query query = query_of(seg);
            const bool live = (int)(warp % 4) < live_warps(seg);
            const int32_t end = sp.n - a.m + query.token + 1;
            const int32_t seen_all = sp.n - a.m + 1;
            const int32_t seen_from = a.split.window > 0 ? sp.n - a.split.window : 0;
            // the row's sum of P over these warps' tiles, relative to 2^ref
            float ref = -INFINITY, sum = 0.0f;

            for (uint32_t k = (group + SOFT - it % SOFT) % SOFT; k < n; k += SOFT) {
                const uint32_t i = it + k, sb = i % SBUF;
                const float4 *from = (const float4 *)(smem + OFF_XBUF + sb * XBUF) + row;
                uint32_t s[KT];
                if (!(ok = wait(bar(X_FULL + sb), (i / SBUF) & 1))) break;
                if (!live) {
                    if (lane == 0) bar_arrive(bar(S_FREE + i % (2 * SBUF))), bar_arrive(bar(X_READ + sb));
                    if (i > 0 && !(ok = wait(bar(O_DONE + ((i - 1) & 3)), ((i - 1) >> 2) & 1))) break;
                    if (lane == 0) bar_arrive(bar(P_FULL + (i & 1)));
                    continue;
                }
                fence_after();
#pragma unroll
                for (int e = 0; e < KT / 16; ++e) tm_load16(s + 16 * e, lanes + COL_S + sb * KT + 16 * e);
                float4 other[KT / 4];
#pragma unroll
                for (int e = 0; e < KT / 4; ++e) other[e] = from[e * ROWS];
                wait_ld();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(S_FREE + i % (2 * SBUF)));
#pragma unroll
                for (int e = 0; e < KT / 4; ++e) {
                    scaled_sum(s + 4 * e, other[e].x, other[e].y, sc2);
                    scaled_sum(s + 4 * e + 2, other[e].z, other[e].w, sc2);
                }
                __syncwarp();
                if (lane == 0) bar_arrive(bar(X_READ + sb));
                const int32_t j0 = sp.lo + (seg.u0 + (int32_t)k) * KT;
                if (j0 + KT > seen_all || j0 < seen_from) {
#pragma unroll
                    for (int e = 0; e < KT; ++e)
                        if (j0 + e >= end || (a.split.window > 0 && j0 + e < window_from(end, a.split.window)))
                            s[e] = 0xFF800000u;   // -infinity
                }
                float best = -INFINITY, more = -INFINITY;
#pragma unroll
                for (int e = 0; e < KT; e += 4) {
                    best = max3(best, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    more = max3(more, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
                }
                best = fmaxf(best, more);
                // what P and O are relative to: as the tile before left it, or more
                float top = best;                 // O starts from a segment's first tile
                if (k > 0) {
                    if (!(ok = top_after(tops, i - 1, &top, a.split.flags))) break;
                    if (__any_sync(~0u, best > top + GROWTH)) {
                        const float next = fmaxf(top, best);
                        const float shrink = next == top ? 1.0f : ex2(top - next);
                        top = next;
                        if (!(ok = wait(bar(O_DONE + ((i - 1) & 3)), ((i - 1) >> 2) & 1))) break;
                        fence_after();
#pragma unroll 1
                        for (int c = 0; c < HALF; c += 16) {
                            uint32_t w[16];
                            tm_load16(w, lanes + COL_O + c);
                            wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = __float_as_uint(__uint_as_float(w[e]) * shrink);
                            tm_store16(lanes + COL_O + c, w);
                        }
                        wait_st();
                    }
                }
                tell_top(tops, i, top);
                if (top != ref) sum *= ref == -INFINITY ? 0.0f : ex2(ref - top);
                ref = top;
                const uint64_t minus = splat2(top == -INFINITY ? 0.0f : -top);
                uint32_t p[KT / 2];
                uint64_t add = 0;                 // two sums
#pragma unroll
                for (int e = 0; e < KT / 2; ++e) {
                    const float2 d = unpack2(add2(pack2(s[2 * e], s[2 * e + 1]), minus));
                    const float p0 = ex2(d.x), p1 = ex2(d.y);
                    add = add2(add, pack2(__float_as_uint(p0), __float_as_uint(p1)));
                    p[e] = FINE > 0 ? first_or_rest2<F16>(p0, p1, less) : narrow2<F16>(p0, p1);
                }
                const float2 both = unpack2(add);
                sum += both.x + both.y;
                // the product before has read the P that this one goes over
                if (i > 0 && !(ok = wait(bar(O_DONE + ((i - 1) & 3)), ((i - 1) >> 2) & 1))) break;
                tm_store16(lanes + COL_P, p);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(P_FULL + (i & 1)));
            }
            if (!ok) break;
            it += n;

            // the segment's maximum and sum, then its O: each set of warps has its share of the
            // columns
            const uint32_t last = it - 1;
            float top = -INFINITY;
            if (live && !(ok = top_after(tops, last, &top, a.split.flags))) break;
            if (top != ref) sum *= ref == -INFINITY ? 0.0f : ex2(ref - top);
            float *all_sums = sums + (segments & 1) * SOFT * ROWS;
            all_sums[group * ROWS + row] = sum;
            __syncwarp();
            if (lane == 0) bar_arrive(bar(SUMS));
            if (!(ok = wait(bar(SUMS), segments & 1))) break;
            sum = 0.0f;
#pragma unroll
            for (int g = 0; g < SOFT; ++g) sum += all_sums[g * ROWS + row];
            ++segments;
            if (!(ok = wait(bar(O_DONE + (last & 3)), (last >> 2) & 1))) break;
            fence_after();

            const bool whole = seg.u0 == 0 && seg.u1 == seg.units, mine = query.mine && !second;
            const bool some = sum > 0.0f || sum != sum;
            const float inv = some ? 1.0f / sum : 0.0f;
            float *slot = a.partial + (size_t)(2 * part + (seg.u0 == 0 ? 1 : 0)) * SLOT;
            unsigned char *out = a.out + seg.r * a.out_request + query.token * a.out_token +
                                 query.hq * a.out_head + rank * (HALF * 2);
            constexpr int PIECE = FINE == 32 ? 32 : 16;      // columns at a time
#pragma unroll 1
            for (int c = group * PIECE; live && c < HALF; c += SOFT * PIECE) {
                uint32_t w[PIECE];
#pragma unroll
                for (int e = 0; e < PIECE; e += 16) tm_load16(w + e, lanes + COL_O + c + e);
                wait_ld();
                if (FINE == 16)                       // the second rows' O to the first's, 16 lanes away
#pragma unroll
                    for (int e = 0; e < PIECE; ++e)
                        w[e] = __float_as_uint(__uint_as_float(w[e]) +
                                               __uint_as_float(__shfl_xor_sync(~0u, w[e], 16)));
                if (FINE == 32) {
                    // the second rows' O to the first's, through where rows 64 to 127 of S would come
                    const uint32_t buf = 2 * group + handed % 2, turn = handed / 2;
                    float4 *at = (float4 *)(smem + OFF_XBUF + group * XBUF) + 64 + handed % 2 * 32 + lane;
                    ++handed;
                    if (second) {
                        if (turn > 0 && !(ok = wait(bar(REST_READ + buf), (turn - 1) & 1))) break;
#pragma unroll
                        for (int e = 0; e < PIECE / 4; ++e)
                            at[e * ROWS] = *(const float4 *)((const float *)w + 4 * e);
                        __syncwarp();
                        if (lane == 0) bar_arrive(bar(REST_FULL + buf));
                        continue;
                    }
                    if (!(ok = wait(bar(REST_FULL + buf), turn & 1))) break;
#pragma unroll
                    for (int e = 0; e < PIECE / 4; ++e) {
                        const float4 v = at[e * ROWS];
                        w[4 * e] = __float_as_uint(__uint_as_float(w[4 * e]) + v.x);
                        w[4 * e + 1] = __float_as_uint(__uint_as_float(w[4 * e + 1]) + v.y);
                        w[4 * e + 2] = __float_as_uint(__uint_as_float(w[4 * e + 2]) + v.z);
                        w[4 * e + 3] = __float_as_uint(__uint_as_float(w[4 * e + 3]) + v.w);
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar(REST_READ + buf));
                }
                if (mine && whole) {
#pragma unroll
                    for (int e = 0; e < PIECE; ++e) {
                        const float v = __uint_as_float(w[e]);
                        w[e] = some ? __float_as_uint(v * inv) : 0u;
                    }
#pragma unroll
                    for (int e = 0; e < PIECE / 8; ++e) {
                        uint4 v;
                        const float *f = (const float *)w + 8 * e;
                        v.x = narrow2<F16>(f[0], f[1]), v.y = narrow2<F16>(f[2], f[3]);
                        v.z = narrow2<F16>(f[4], f[5]), v.w = narrow2<F16>(f[6], f[7]);
                        *(uint4 *)(out + c * 2 + e * 16) = v;
                    }
                } else if (mine) {
                    float4 *to = (float4 *)slot + (size_t)((rank * HALF + c) / 4) * ROWS + row;
#pragma unroll
                    for (int e = 0; e < PIECE / 4; ++e)
                        __stcg(to + e * ROWS, *(const float4 *)((const float *)w + 4 * e));
                }
                __syncwarp();
            }
            if (FINE == 32 && !ok) break;
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(O_FREE));
            if (mine && rank == 0 && group == 0) {
                if (whole) {
                    if (a.lse != nullptr)
                        a.lse[((int64_t)seg.r * a.m + query.token) * a.Hq + query.hq] =
                            some ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
                } else {
                    __stcg((float2 *)(slot + (size_t)ROWS * VALUES) + row, make_float2(top, sum));
                }
            }
        }
    } else if (warp < LOAD) {
        // ---- sending: this SM's half of S to the other; and a segment's q to tensor memory ----
        const uint32_t x_remote = remote_addr(smem0 + OFF_XBUF, rank ^ 1u) + row * 16;
        const uint32_t bars_remote = remote_addr(bars, rank ^ 1u);
        uint32_t it = 0;
        bool ok = true;
        while (ok && x < x_end) {
            const Segment seg = segment_at(x, x_end, prefix, a.shape, known);
            known = -1;
            const uint32_t n = (uint32_t)(seg.u1 - seg.u0);
            x += n;
            // (S of every tile so far was waited for below: no product reads the q before)
            const Query query = query_of(seg);
            const unsigned char *q = a.q + seg.r * a.q_request + query.token * a.q_token +
                                     query.hq * a.q_head;
            const unsigned char *first = q + rank * (HALF * 2), *rest = q + (VALUES + rank * REST) * 2;
            const bool live = (int)(warp % 4) < live_warps(seg);
#pragma unroll 3
            for (int k = 0; k < 9 && live; ++k) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (query.mine) v = __ldg((const uint4 *)(k < 8 ? first + k * 64 : rest) + e);
                    w[4 * e] = v.x, w[4 * e + 1] = v.y, w[4 * e + 2] = v.z, w[4 * e + 3] = v.w;
                }
                __syncwarp();
                tm_store16(lanes + COL_Q + 16 * k, w);
            }
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(Q_FULL));
            for (uint32_t k = 0; k < n; ++k, ++it) {
                const uint32_t sb = it % SBUF, ph = (it / SBUF) & 1;
                if (!(ok = wait(bar(X_EMPTY + sb), ph ^ 1))) break;
                if (!(ok = wait(bar(S_FULL + sb), ph))) break;
                if (!live) {
                    if (lane == 0) bar_arrive(bar(S_FREE + it % (2 * SBUF)));
                    continue;
                }
                fence_after();
                uint32_t s[KT];
#pragma unroll
                for (int e = 0; e < KT / 16; ++e) tm_load16(s + 16 * e, lanes + COL_S + sb * KT + 16 * e);
                wait_ld();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(bar(S_FREE + it % (2 * SBUF)));
#pragma unroll
                for (int e = 0; e < KT / 4; ++e)
                    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], "
                                 "{%1, %2, %3, %4}, [%5];" ::"r"(x_remote + sb * XBUF + e * ROWS * 16),
                                 "r"(s[4 * e]), "r"(s[4 * e + 1]), "r"(s[4 * e + 2]), "r"(s[4 * e + 3]),
                                 "r"(bars_remote + 8 * (X_FULL + sb))
                                 : "memory");
            }
        }
        // Nothing is on its way to an SM that may leave: what this warp sent last has been read. (A warp
        // that gave up has waited for two seconds since it sent anything.)
        for (uint32_t i = it > SBUF ? it - SBUF : 0; ok && i < it; ++i)
            ok = wait(bar(X_EMPTY + i % SBUF), (i / SBUF) & 1);
    } else if (warp == TELL) {
        // ---- telling the other SM what it may send over: its arrival takes some hundred cycles,
        // which the softmax warps do not have ----
        const uint32_t bars_remote = remote_addr(bars, rank ^ 1u);
        uint32_t it = 0;
        bool ok = true;
        while (ok && x < x_end) {
            const Segment seg = segment_at(x, x_end, prefix, a.shape, known);
            known = -1;
            x += seg.u1 - seg.u0;
            for (int32_t u = seg.u0; u < seg.u1; ++u, ++it) {
                if (!(ok = wait(bar(X_READ + it % SBUF), (it / SBUF) & 1))) break;
                if (lane == 0) bar_arrive_remote(bars_remote + 8 * (X_EMPTY + it % SBUF));
                __syncwarp();
            }
        }
    } else if (warp < KEYS) {
        // ---- loads: warp w of 4 has every fourth tile ----
        uint32_t leader;
        asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(leader));
        const uint32_t w = warp - LOAD;
        static_assert(KT == 32, "a lane's number is its key");
        uint32_t it = 0, bad = 0;
        bool ok = true;
        const unsigned char *src = a.plane.base;
        while (ok && x < x_end) {
            const Segment seg = segment_at(x, x_end, prefix, a.shape, known);
            known = -1;
            const uint32_t n = (uint32_t)(seg.u1 - seg.u0);
            x += n;
            const Span sp = span_of(a.split, seg.r, KT, &bad);
            const int32_t *table = a.split.slots.ids + (int64_t)seg.r * a.split.slots.stride;
            // tiles of which all keys are seen come in boxes, if there are any: [full, whole)
            const int32_t full = sp.first > sp.lo ? 1 : 0;
            const int32_t whole = a.piece > 0 ? min(seg.u1, (sp.n - sp.lo) / KT) : 0;
            auto boxed = [&](int32_t u) { return u >= full && u < whole; };
            const int32_t pieces = a.piece > 0 ? KT / a.piece : 0;
            // the block id that this lane looks up for tile u: of box piece `lane`, or of its key.
            // It is asked for a turn ahead and not looked at before.
            auto position = [&](int32_t u) -> int32_t {
                if (boxed(u)) return lane < pieces ? sp.lo + u * KT + lane * a.piece : -1;
                const int32_t j = sp.lo + u * KT + lane;
                return u < seg.u1 && j >= sp.first && j < sp.n ? j : -1;
            };
            auto look_up = [&](int32_t j) -> int32_t {
                return j < 0 ? 0 : __ldg(table + a.split.slots.block.div((uint32_t)j));
            };
            uint32_t k = (w - it) & 3;
            int32_t next = look_up(position(seg.u0 + (int32_t)k));
            for (; k < n; k += 4) {
                const int32_t u = seg.u0 + (int32_t)k;
                const uint32_t i = it + k, stage = i % STAGES;
                int32_t id = next;
                next = look_up(position(u + 4));
                if (!(ok = wait(bar(K_EMPTY + stage), (i / STAGES + 1) & 1))) break;
                const uint32_t base = smem0 + stage * STAGE, filled = bar(K_FULL + stage);
                const int32_t j = position(u);
                const bool there = j >= 0 && id >= 0 && id < a.split.slots.num_blocks;
                if (j >= 0 && !there) bad |= KVC_FLAG_BLOCK;
                const int32_t token =
                    max(j, 0) - (int32_t)(a.split.slots.block.div((uint32_t)max(j, 0)) * a.split.slots.block.d);
                if (boxed(u)) {
                    if (!there) id = a.split.slots.num_blocks;    // past the last: zeros
                    if (leader)
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(filled),
                                     "r"(STAGE)
                                     : "memory");
                    for (int piece = 0; piece < pieces; ++piece) {
                        const int32_t block = __shfl_sync(~0u, id, piece);
                        const int32_t first = __shfl_sync(~0u, token, piece);
                        if (leader) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                load_box(base + c * CHUNK + piece * a.piece * 128, &a.values,
                                         (int32_t)rank * HALF + c * 64, first, block, filled);
                            load_box(base + 4 * CHUNK + piece * a.piece * 64, &a.rest,
                                     VALUES + (int32_t)rank * REST, first, block, filled);
                        }
                    }
                    __syncwarp();
                    continue;
                }
                const int64_t slot = there ? id * a.plane.block_stride + (int64_t)token * a.plane.token_stride : -1;
                // values: 32 pieces of 16 bytes a key, one key at a time
#pragma unroll 8
                for (int row = 0; row < KT; ++row) {
                    const int64_t off = __shfl_sync(~0u, slot, row);
                    const int64_t at = off >= 0 ? off + rank * (HALF * 2) + lane * 16 : 0;
                    const uint32_t dst = base + (lane / 8) * CHUNK + row * 128 + (((lane % 8) ^ (row & 7)) << 4);
                    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst),
                                 "l"(src + at), "r"(off >= 0 ? 16 : 0)
                                 : "memory");
                }
                // the rest: 4 pieces a key, 8 keys at a time
#pragma unroll
                for (int r0 = 0; r0 < KT; r0 += 8) {
                    const int64_t off = __shfl_sync(~0u, slot, r0 + lane / 4);
                    const uint32_t row = r0 + lane / 4, c = lane % 4;
                    const int64_t at = off >= 0 ? off + (VALUES + rank * REST) * 2 + c * 16 : 0;
                    const uint32_t dst = base + 4 * CHUNK + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                                 "l"(src + at), "r"(off >= 0 ? 16 : 0)
                                 : "memory");
                }
                if (a.piece > 0) {
                    // a request's last tile, or a window's first
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) bar_arrive(filled);
                } else {
                    // arrives when this thread's copies so far have
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(filled) : "memory");
                }
            }
            it += n;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // What was asked for has to come, whatever the other warps gave up: the last tiles here (no
        // later one has gone over them); where this warp gave up itself, whatever is under way.
        for (uint32_t i = it > STAGES ? it - STAGES : 0; ok && i < it; ++i)
            if ((i & 3) == w) wait_for(bar(K_FULL + i % STAGES), (i / STAGES) & 1);
        if (!ok)
            for (uint32_t i = 0; i < STAGES; ++i) wait_for(bar(K_FULL + i), 0), wait_for(bar(K_FULL + i), 1);
        if (bad != 0) atomicOr(a.split.flags, bad);
    } else {
        // ---- products, S by two warps and O by another, so that none waits for what another
        // waits for. A warp runs as one, which keeps operand descriptors in uniform registers, and
        // one elected lane issues ----
        uint32_t leader;
        asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(leader));
        const uint32_t tm = __shfl_sync(~0u, tmem, 0), ring = __shfl_sync(~0u, smem0, 0);
        constexpr uint32_t ID_S = idesc(!F16, false, KT), ID_O = idesc(!F16, true, HALF);
        uint32_t it = 0, segments = 0;
        bool ok = true;
        while (ok && x < x_end) {
            const Segment seg = segment_at(x, x_end, prefix, a.shape, known);
            known = -1;
            const uint32_t n = (uint32_t)(seg.u1 - seg.u0);
            x += n;
            if (warp < VALS) {
                ok = wait(bar(Q_FULL), segments++ & 1);
                for (uint32_t k = (it ^ warp) & 1; ok && k < n; k += 2) {
                    const uint32_t i = it + k, sb = i % SBUF, stage = i % STAGES;
                    if (!(ok = wait(bar(K_FULL + stage), (i / STAGES) & 1))) break;
                    // the S that this one goes over has been read
                    const uint32_t over = i - SBUF;
                    if (i >= SBUF && !(ok = wait(bar(S_FREE + over % (2 * SBUF)), (over / (2 * SBUF)) & 1)))
                        break;
                    fence_after();
                    // rows that came through the generic proxy; the products read through the async one
                    if (a.piece == 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    const uint32_t base = __shfl_sync(~0u, ring + stage * STAGE, 0);
                    const uint32_t s_col = __shfl_sync(~0u, tm + COL_S + sb * KT, 0);
                    if (leader) {
                        const uint64_t first = operand(base, 16, 1024, 2);
#pragma unroll
                        for (int e = 0; e < HALF / 64; ++e)
                            product4(s_col, tm + COL_Q + 32 * e, first + e * (CHUNK / 16), ID_S, e > 0);
                        static_assert(REST == 32, "");
                        product2(s_col, tm + COL_Q + HALF / 2, operand(base + 4 * CHUNK, 16, 512, 4), 2, ID_S, 1);
                        commit(bar(S_FULL + sb));
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                                         bar(X_FULL + sb)),
                                     "r"(live_warps(seg) * (32 * KT * 4))
                                     : "memory");
                        commit(bar(X_FULL + sb));
                    }
                    __syncwarp();
                }
            } else {
                for (uint32_t k = 0; ok && k < n; ++k) {
                    const uint32_t i = it + k, b = i & 1, stage = i % STAGES;
                    // O of the segment before has been read
                    if (k == 0 && segments++ > 0 && !(ok = wait(bar(O_FREE), segments & 1))) break;
                    if (!(ok = wait(bar(P_FULL + b), (i >> 1) & 1))) break;
                    fence_after();
                    const uint32_t base = __shfl_sync(~0u, ring + stage * STAGE, 0);
                    const uint32_t p_col = __shfl_sync(~0u, tm + COL_P, 0);
                    if (leader) {
                        product2(tm + COL_O, p_col, operand(base, CHUNK, 1024, 2), 2048 / 16, ID_O, k > 0);
                        commit(bar(K_EMPTY + stage));
                        commit(bar(O_DONE + (i & 3)));
                    }
                    __syncwarp();
                }
            }
            it += n;
        }
        // nothing that was issued outlives the block's memory, whatever gave up above
        if (leader) commit(bar(DRAIN + (warp - KEYS)));
        __syncwarp();
        wait_for(bar(DRAIN + (warp - KEYS)), 0);
    }

    // both SMs stay until neither has anything under way to the other (S that was sent: above)
    __syncwarp();
    fence_before();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    fence_after();
    if (warp == KEYS)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// -- joining the parts ------------------------------------------------------------

constexpr int JOIN_ROWS = 4, JOIN_COLS = 32, JOIN_SET = JOIN_ROWS * JOIN_COLS;
constexpr int JOIN_GRID = VALUES / 4 / JOIN_COLS, JOIN_RESIDENT = 1024;   // of an SM's threads
constexpr int PARTS_MOST = 128;           // clusters of the attention kernel

// One block a job, 4 of its rows and 128 of their elements: the parts' accumulators weighted by
// their maxima, in an order that depends on the lengths alone. Jobs that one part did whole are
// not touched. (Four rows' pieces of 16 bytes are two whole sectors; small blocks, so that 16 rows
// are still 16 blocks.) It is the latency of few loads that it waits for, so the statistics of
// all parts are asked for at once, the first accumulators before they are there, and SETS sets of
// threads take every SETS-th part: as many as the SMs hold at once, and as have two parts each.
// With 1, 2, 4 and 8 sets the whole attention took (us, * the choice) 20.8, 17.0, 14.6, 13.8* for
// one request of 4096 latents and 16 heads; 59.7, 46.2, 39.0, 36.1* for one of 65536 and 128
// heads; 57.6, 54.8*, 55.7, 63.1 for 4 of 32768; 41.9*, 45.1, 53.9, 78.5 for 16 of 4096.
//
// With many jobs of few parts each it is bound by its instructions (77 % of the issue slots), most of
// which come before the first product. So where at most 3 parts are to be expected and the
// blocks are still 4 an SM, one takes all 512 elements (ALL): 166.8 -> 162.9 us for 64 requests of 1024 to
// 16384 latents, 60.6 -> 59.2 for 32 of 4096 (with 9 parts a job it would be 37.5 -> 43.9).
template <bool F16, int SETS, bool ALL>
__global__ void __launch_bounds__(JOIN_SET * SETS) latent_join(const __grid_constant__ LatentArgs a) {
    // parts and 4-element columns that a thread asks for at a time
    constexpr int AHEAD = ALL ? 2 : SETS == 1 ? 4 : 8, PIECES = ALL ? JOIN_GRID : 1;
    static_assert(!ALL || SETS == 1, "");
    __shared__ float weights[PARTS_MOST][JOIN_ROWS];   // a part's share of a row; below 0: has none
    __shared__ float2 warp_stat[JOIN_SET * SETS / 32][JOIN_ROWS];
    __shared__ float4 sums[SETS > 1 ? SETS - 1 : 1][JOIN_SET];   // (PIECES is 1)
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, set = tid / JOIN_SET;
    const int jr = tid % JOIN_ROWS;
    wait_for_previous();
    let_next_start();
    const Cut cut = cut_of(a, a.prefix);
    const int32_t M = a.m * a.Hq, groups = (min(M, ROWS) + JOIN_ROWS - 1) / JOIN_ROWS;
    const int32_t jg = blockIdx.x / groups, r = jg / a.chunks, job = jg - r * a.chunks;
    const int32_t row = (blockIdx.x % groups) * JOIN_ROWS + jr;
    const int32_t rho = job * ROWS + row;
    const int32_t e4 = blockIdx.y * JOIN_COLS + tid % JOIN_SET / JOIN_ROWS;     // 4 elements
    const int32_t before = a.prefix[r], units = a.prefix[r + 1] - before;
    const int32_t first = before * a.chunks + job * units;
    int32_t c0, n;
    cut.parts_of(r, job, first, units, a.ahead, a.shape, &c0, &n);
    if (n == 1) return;
    const bool mine = rho < M;
    auto slot = [&](int32_t c) { return a.partial + (size_t)(2 * (c0 + c) + (c == 0 ? 1 : 0)) * SLOT; };

    float4 p[AHEAD][PIECES];
    auto ask = [&](int32_t c1) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (mine && c1 + k * SETS < n) {
                const float4 *from = (const float4 *)slot(c1 + k * SETS) + (size_t)e4 * ROWS + row;
#pragma unroll
                for (int i = 0; i < PIECES; ++i) p[k][i] = __ldcg(from + i * JOIN_COLS * ROWS);
            }
    };
    // one part and row a thread: (max, sum), then the rows' maxima and sums over all parts
    constexpr int TURN = JOIN_SET * SETS / JOIN_ROWS, TURNS = (PARTS_MOST + TURN - 1) / TURN;
    float2 ml[TURNS];
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
        const int32_t c = tid / JOIN_ROWS + k * TURN;
        ml[k] = make_float2(-INFINITY, 0.0f);
        if (mine && c < n) ml[k] = __ldcg((const float2 *)(slot(c) + (size_t)ROWS * VALUES) + row);
    }
    ask(set);
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int k = 0; k < TURNS; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
    for (int o = JOIN_ROWS; o < 32; o *= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
    if (lane < JOIN_ROWS) warp_stat[warp][jr].x = m;
    __syncthreads();
    for (int w = 0; w < JOIN_SET * SETS / 32; ++w) m = fmaxf(m, warp_stat[w][jr].x);
#pragma unroll
    for (int k = 0; k < TURNS; ++k) {
        const int32_t c = tid / JOIN_ROWS + k * TURN;
        const bool some = !(ml[k].x == -INFINITY && ml[k].y == 0.0f);
        const float f = ml[k].x == -INFINITY ? 0.0f : ex2(ml[k].x - m);
        if (some) l += f * ml[k].y;
        if (c < n) weights[c][jr] = some ? f : -1.0f;
    }
#pragma unroll
    for (int o = JOIN_ROWS; o < 32; o *= 2) l += __shfl_xor_sync(~0u, l, o);
    if (lane < JOIN_ROWS) warp_stat[warp][jr].y = l;
    __syncthreads();

    float4 v[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) v[i] = make_float4(0, 0, 0, 0);
    for (int32_t c1 = set; c1 < n; c1 += AHEAD * SETS) {
        if (c1 != set) ask(c1);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int32_t c = c1 + k * SETS;
            const float f = c < n && mine ? weights[c][jr] : -1.0f;
            if (f < 0.0f) continue;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                v[i].x += f * p[k][i].x, v[i].y += f * p[k][i].y;
                v[i].z += f * p[k][i].z, v[i].w += f * p[k][i].w;
            }
        }
    }
    if (SETS > 1) {
        if (set > 0) sums[set - 1][tid % JOIN_SET] = v[0];
        __syncthreads();
        if (set > 0) return;
        for (int k = 0; k < SETS - 1; ++k) {
            const float4 w = sums[k][tid];
            v[0].x += w.x, v[0].y += w.y, v[0].z += w.z, v[0].w += w.w;
        }
    }
    if (!mine) return;
    l = 0.0f;
    for (int w = 0; w < JOIN_SET * SETS / 32; ++w) l += warp_stat[w][jr].y;
    const bool some = l > 0.0f || l != l;
    const float inv = some ? 1.0f / l : 0.0f;
    const int32_t token = (int32_t)a.heads.div((uint32_t)rho), hq = rho - token * a.Hq;
    unsigned char *out = a.out + r * a.out_request + token * a.out_token + hq * a.out_head + e4 * 8;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
        *(uint2 *)(out + i * JOIN_COLS * 8) = make_uint2(narrow2<F16>(v[i].x * inv, v[i].y * inv),
                                                         narrow2<F16>(v[i].z * inv, v[i].w * inv));
    if (e4 == 0 && a.lse != nullptr)
        a.lse[((int64_t)r * a.m + token) * a.Hq + hq] =
            some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// the instance for M query rows
template <bool F16>
auto kernel_of(int64_t M) {
    return M <= 16 ? latent_kernel<F16, 16> : M <= 32 ? latent_kernel<F16, 32> : latent_kernel<F16, 0>;
}

template <bool F16>
constexpr void (*JOINS_OF[5])(LatentArgs) = {latent_join<F16, 1, false>, latent_join<F16, 2, false>,
                                             latent_join<F16, 4, false>, latent_join<F16, 8, false>,
                                             latent_join<F16, 1, true>};

}  // namespace

size_t kvc_latent_partial_bytes(int32_t sm_count) {
    return (size_t)(sm_count / 2) * 2 * SLOT * sizeof(float);
}

// Copy-engine maps of each layer's plane, as [block][token][element] in boxes of `piece` tokens
// and 64 (values) or 32 elements. Where blocks are no multiples of 8 tokens that divide a tile, or a
// map cannot be had, there are none and rows come by cp.async.
static kvr_status make_maps(kvc_cache *c) {
    const int32_t B = c->d.block_size;
    const int32_t piece = std::min(B, KT);
    c->piece = 0;
    c->maps.clear();
    if (piece < 8 || KT % piece != 0 || B % piece != 0) return KVR_OK;
    c->maps.resize(2 * (size_t)c->d.num_layers);
    for (int32_t l = 0; l < c->d.num_layers; ++l)
        for (int k = 0; k < 2; ++k) {
            const uint64_t dims[3] = {KVC_LATENT_DIM, (uint64_t)B, (uint64_t)c->d.num_blocks};
            const int64_t strides[2] = {c->token_stride, c->block_stride};
            const uint32_t box[3] = {k == 0 ? 64u : (uint32_t)REST, (uint32_t)piece, 1};
            if (!kvc_make_map(&c->maps[2 * (size_t)l + k], 2, 3, c->base[l], c->row_bytes, dims, strides,
                              box, k == 0 ? 128 : 64))
                return KVR_OK;
        }
    c->piece = piece;
    return KVR_OK;
}

kvr_status kvc_latent_setup(kvc_cache *c) {
    const int smem = OFF_PREFIX + 4 * (KVC_MAX_REQUESTS + 1);
    static_assert(OFF_PREFIX + 4 * (KVC_MAX_REQUESTS + 1) <= 227 * 1024, "");
    for (auto k : {kernel_of<false>(1), kernel_of<false>(17), kernel_of<false>(33), kernel_of<true>(1),
                   kernel_of<true>(17), kernel_of<true>(33)})
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            cudaGetLastError();
            return KVR_ERR_CUDA;
        }
    cudaFuncAttributes loaded;            // now, and not while a stream is captured
    for (const auto &of_type : {JOINS_OF<false>, JOINS_OF<true>})
        for (int k = 0; k < 5; ++k)
            if (cudaFuncGetAttributes(&loaded, of_type[k]) != cudaSuccess) {
                cudaGetLastError();
                return KVR_ERR_CUDA;
            }
    return make_maps(c);
}

kvr_status kvc_latent_launch(const kvc_cache *c, int32_t layer, const kvc_attend *p, void *stream) {
    LatentArgs a = {};
    a.plane = c->plane(layer, 0);
    a.piece = c->piece;
    if (c->piece > 0) {
        a.values = c->maps[2 * (size_t)layer];
        a.rest = c->maps[2 * (size_t)layer + 1];
    }
    a.split = {c->slots(p->table), p->lengths, c->ws.flags, p->num_requests, p->num_new, p->window};
    a.q = (const unsigned char *)p->q;
    a.out = (unsigned char *)p->out;
    a.lse = p->lse;
    a.q_request = p->q_request_stride, a.q_token = p->q_token_stride, a.q_head = p->q_head_stride;
    a.out_request = p->out_request_stride, a.out_token = p->out_token_stride;
    a.out_head = p->out_head_stride;
    a.partial = c->ws.partial;
    a.prefix = (int32_t *)c->ws.arrived;
    a.ahead = a.prefix + p->num_requests + 1;
    a.m = p->num_new, a.Hq = c->d.query_heads;
    a.heads = kvr_make_div((uint32_t)a.Hq);
    a.scale = p->scale;
    const int64_t M = (int64_t)a.m * a.Hq;
    a.chunks = (int32_t)((M + ROWS - 1) / ROWS);
    const int64_t most = ((int64_t)p->table.width * c->d.block_size + KT - 1) / KT + 1;
    if (most * p->num_requests * a.chunks > INT32_MAX) return KVR_ERR_UNSUPPORTED;
    const int32_t sms = kvc_stream_sms(c, stream);
    a.parts = (int32_t)std::min<int64_t>(std::clamp(sms / 2, 1, PARTS_MOST),
                                         most * p->num_requests * a.chunks);
    a.shape = make_cut_shape(p->num_requests, a.chunks, a.parts, SLACK);
    const bool f16 = c->d.dtype == KVC_DTYPE_F16;
    const size_t smem = OFF_PREFIX + 4 * (size_t)(p->num_requests + 1);
    const kvr_status st =
        kvc_launch(f16 ? kernel_of<true>(M) : kernel_of<false>(M), a, dim3((unsigned)(2 * a.parts)), THREADS, smem, stream, 2);
    if (st != KVR_OK) return st;
    const int64_t groups = (std::min<int64_t>(M, ROWS) + JOIN_ROWS - 1) / JOIN_ROWS;
    const int64_t jobs = (int64_t)p->num_requests * a.chunks, blocks = jobs * groups * JOIN_GRID;
    // parts of a job, on average at most: lengths are known on the device alone
    const int64_t parts = std::min<int64_t>(a.parts, most * jobs / LEAST) / jobs;
    int k = 0;
    while (k < 3 && (4 << k) <= parts && (blocks * JOIN_SET * 2 << k) <= (int64_t)sms * JOIN_RESIDENT) ++k;
    const bool all = parts <= 3 && jobs * groups >= 4 * (int64_t)sms;
    return kvc_launch((f16 ? JOINS_OF<true> : JOINS_OF<false>)[all ? 4 : k], a,
                      dim3((unsigned)(jobs * groups), all ? 1 : JOIN_GRID), JOIN_SET << k, 0, stream);
}
