// cache_attend.cuh -- attention of a request's newest tokens over its paged keys and values.
//
// For each key head h of each request, the M = m G rows (m newest tokens, G query heads of h)
// meet the same keys, so one pass over the cache serves them all. It is bound by HBM: at G = 8
// and 16-bit elements there are 8 flops a byte of cache, 1/30 of what the card can do.
//
// Split. The keys of all (request, head) JOBS, in UNITS of 4 KT keys, form one line that is cut into
// parts, at most one a resident block: equal ones whatever the lengths are, or parts within jobs where
// that makes the longest hardly longer (cache_split.cuh). (Two and three times as many parts: 71 and
// 75 us where one takes 52, as each begins with an empty ring and ends with a share of a join.) Each
// block works the prefix sums of the lengths out by itself, so that the lengths can stay on the device. A part of a job that is not the whole of it leaves (max, sum,
// accumulator) in the workspace, and the last of the job's blocks to arrive copies all of them
// into its ring and joins them, in the order of the keys: results do not depend on who is last.
//
// Inside a block each of 4 warps takes every fourth tile of KT keys and keeps its own ring of
// STAGES tiles filled by 16-byte cp.async: nothing in the loop waits for another warp. (The copy
// engine's boxes took 57 us where these take 53.) A window's first tile begins at its first key. Rows of
// padding (beyond the length, or beyond D) are written as zeros, so that what the pool holds there never
// meets the arithmetic.
//
// Products. S^T = K Q^T and O^T += V^T P^T by mma.sync m16n8k16 with keys (then head elements)
// as the 16 rows and the queries as the 8 columns: with M = 8 nothing is padded, and each warp goes its
// own way with tiles of 16 or 32 keys and its accumulators in registers. tcgen05 products could take
// 128 keys (then head elements) as their rows in the same way; that has not been built. With 8 rows
// nothing could be gained, HBM bounds them; with 32 (a chain of 1.3 us a tile, the tensor pipe at 8 %) and
// over E4M3 (instructions) it might be. K and V^T fragments come by ldmatrix (.trans for V), P^T is
// P's accumulator fragment transposed in registers by movmatrix.
//
// Numbers. S, the running maximum and sum, and O are fp32. P enters its product as two 16-bit
// numbers (the one next below, and the rest), so 15 bits of it count: one rounding of P alone would be as
// large as that of the output. With an E4M3 cache the codes become f16 (exact), Q is scaled per
// row by a power of two to f16 (exact but for elements 2^-14 of the row's largest), P is f16
// alone: 11 bits against the output's rounding and the codes' 4 bits. P is scaled by 2^10 in f16
// so that weights down to 2^-24 of the largest are normal numbers.
//
// Measured, 8 queries a key head of 128: 4 requests of 32768 keys, 4 heads, bf16 (268 MB) 48 us,
// 5.6 TB/s; one of 131072, 8 heads, E4M3 (268 MB) 53 us, 5.1 TB/s; 64 of 8192, 8 heads, bf16 (2.1 GB)
// 322 us, 6.68 TB/s, and with 4 newest tokens, 32 rows, 381 us. What is lost below a plain copy's
// rate is fixed: 5 us from the launch to the first keys (lengths, block ids, keys, each after the one
// before), 6 us from the first block's end to the last's, as not all SMs are as near to all of
// HBM, and 3 to 6 us of joining.
#pragma once

#include <math.h>

#include "cache.h"
#include "cache_split.cuh"

namespace kvc {

struct AttendArgs {
    KvcPlane k_plane, v_plane;
    SplitArgs split;
    const unsigned char *q;
    unsigned char *out;
    float *lse;
    int64_t q_request, q_token, q_head, out_request, out_token, out_head;
    const float *k_scale, *v_scale;
    float *partial;
    uint32_t *arrived;
    int32_t m, H, G, D, f16;
    int32_t chunks;           // passes over a job's keys, RP rows each
    KvrDiv group, by_chunks;  // by G, chunks
    CutShape shape;
    float scale;
};

constexpr int ATTEND_WARPS = 4;
constexpr int ATTEND_THREADS = 32 * ATTEND_WARPS;
// Units that a change of job costs (cache_split.cuh). Parts within jobs took 49.1 where equal ones took
// 52.1 (4 requests of 32768 keys, 4 heads), 27.4 for 33.3 (8 of 16 to 8192, 8 heads), 23.8 for 26.7
// (48 of a window of 1024, 32 rows), and with a group 5 above the equal parts' 48.6 for 51.5 (8 of
// 8192, 8 heads); where nothing was to be gained 0.3 to 0.8 more.
constexpr int SLACK = 8;
constexpr float P_SHIFT = 10.0f;      // log2 of P's scale in f16
// how far (as a power of two) P may exceed its scale before a new maximum is taken: f16 P ends at
// 2^16; bf16 reaches further, but 40 was no faster, and O of values up to 2^110 has to stay finite
template <bool F16>
constexpr float GROWTH_OF = F16 ? 5.0f : 8.0f;

template <int DP, int POOL, int NT>
struct Attend {
    static constexpr int ES = POOL == KVR_DTYPE_FP8_E4M3 ? 1 : 2;
    static constexpr bool F16 = POOL != KVR_DTYPE_BF16;          // type of the products
    static constexpr bool SPLIT = POOL != KVR_DTYPE_FP8_E4M3;    // P as two numbers
    static constexpr int ROW = DP * ES;                          // bytes of a row in the ring
    static constexpr int KT = 2 * 16 * ROW >= 8192 ? 16 : 32;    // keys of a tile
    static constexpr int KS = KT / 16;
    static constexpr int STAGE = 2 * KT * ROW;
    static constexpr int STAGES = STAGE >= 8192 ? 3 : 6;
    static constexpr int RING = ATTEND_WARPS * STAGES * STAGE;
    static constexpr int UNIT = ATTEND_WARPS * KT;               // keys of a unit
    static constexpr int RP = 8 * NT;
    static constexpr int MT = DP / 16;
    static constexpr int PITCH = DP + 4;                         // floats of a row to be joined
    static constexpr int BLOCKS = STAGE > 8192 ? 1 : 2;          // resident on an SM
    static constexpr int Q_BYTES = RP * DP * 2;
    static_assert(ATTEND_WARPS * RP * PITCH * 4 <= RING, "the join reuses the ring");
    // ring, queries, a barrier, then floats: row scales [RP], per-warp statistics [4][RP][2]; 4 ints;
    // then ahead and prefix
    static constexpr int FIXED = RING + Q_BYTES + 16 + 4 * RP + 4 * ATTEND_WARPS * RP * 2 + 16 +
                                 4 * (AHEAD_MOST + 4);
    static constexpr size_t smem(int32_t requests) { return FIXED + 4 * (size_t)(requests + 1); }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4t(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
template <bool F16>
__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
                     "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk `c` of row `r` in an array of rows of ROW bytes, spread so that 8
// consecutive rows' same chunk lies in 8 different 16-byte columns of shared memory.
template <int ROW>
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
    if (ROW >= 128) return r * ROW + ((c ^ (r & 7)) << 4);
    return r * ROW + ((c ^ ((r >> 1) & 3)) << 4);       // 64-byte rows: two share 128 bytes
}

// -- the barrier that a join's copies count at ------------------------------------------

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// Waits for the phase of `parity`, in turns of a microsecond and for about two seconds at most.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
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
    return done != 0;
}
__device__ __forceinline__ void load_bytes(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Two weights (>= 0) as the 16-bit numbers next below them: the rests are positive wherever the
// weights are, so an infinite value times both parts is one infinity, not two that cancel.
template <bool F16>
__device__ __forceinline__ uint32_t below2(float lo, float hi) {
    const uint32_t a = max(__float_as_uint(lo), 1u) - 1u, b = max(__float_as_uint(hi), 1u) - 1u;
    if (!F16) return __byte_perm(a, b, 0x7632);
    uint32_t w;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(__uint_as_float(b)), "f"(__uint_as_float(a)));
    return w;
}

// out (16-bit), four elements of one row, from floats
template <bool F16>
__device__ __forceinline__ uint2 narrow4(float4 v) {
    return make_uint2(narrow2<F16>(v.x, v.y), narrow2<F16>(v.z, v.w));
}

template <int DP, int POOL, int NT>
__global__ void __launch_bounds__(ATTEND_THREADS, (Attend<DP, POOL, NT>::BLOCKS))
attend_kernel(AttendArgs a) {
    using C = Attend<DP, POOL, NT>;
    constexpr float GROWTH = GROWTH_OF<C::F16>;
    constexpr int KT = C::KT, KS = C::KS, RP = C::RP, MT = C::MT, ROW = C::ROW;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t smem0 = (uint32_t)__cvta_generic_to_shared(smem);
    unsigned char *q_smem = smem + C::RING;
    const uint32_t join_bar = smem0 + C::RING + C::Q_BYTES;
    float *row_scale = (float *)(q_smem + C::Q_BYTES + 16);
    float *stat = row_scale + RP;                       // [warp][RP][max, sum]
    int32_t *shared_int = (int32_t *)(stat + ATTEND_WARPS * RP * 2);   // [4]
    int32_t *ahead = shared_int + 4;                    // [AHEAD_MOST + 1]
    int32_t *prefix = ahead + AHEAD_MOST + 4;           // [requests + 1], in units of one job
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t4 = lane % 4;

    if (tid == 0) {
        bar_init(join_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    uint32_t join_phase = 0;
    wait_for_previous();
    let_next_start();

    unit_prefix<C::UNIT>(a.split, 1, prefix, shared_int);
    const int32_t HJ = a.H * a.chunks;
    const int32_t total = prefix[a.split.requests] * HJ;
    const Cut cut(total, a.shape);
    if (cut.group > 0) {
        if (warp == 0) cut.count(prefix, a.split.requests, ahead);
        __syncthreads();
    }
    int32_t x, x_end;
    int32_t known = cut.units_of(blockIdx.x, prefix, ahead, a.shape, &x, &x_end);

    const int32_t M = a.m * a.G;
    const int32_t slot_floats = RP * (a.D + 2);
    const uint32_t ring = smem0 + (uint32_t)(warp * C::STAGES * C::STAGE);
    const float log2e = 1.4426950408889634f;

    while (x < x_end) {
        const Segment seg = segment_at(x, x_end, prefix, a.shape, known);
        known = -1;
        const int32_t r = seg.r, job = seg.job, u0 = seg.u0, u1 = seg.u1, units = seg.units;
        x += u1 - u0;
        const int32_t h = (int32_t)a.by_chunks.div((uint32_t)job), row0 = (job - h * a.chunks) * RP;
        const int32_t rows = min(RP, M - row0);
        uint32_t bad = 0;
        const Span sp = span_of(a.split, r, 1, &bad);   // tiles begin at the first key
        const float ks = POOL == KVR_DTYPE_FP8_E4M3 ? a.k_scale[h] : 1.0f;

        // this warp's tiles; the lane's key of a tile (lane < KT) and its slot
        const int32_t tiles = (sp.n - sp.lo + KT - 1) / KT;
        const int32_t t_begin = u0 * ATTEND_WARPS + warp, t_end = min(u1 * ATTEND_WARPS, tiles);
        const int32_t *table = a.split.slots.ids + (int64_t)r * a.split.slots.stride;
        const int64_t head_off = (int64_t)h * a.k_plane.head_stride;
        // its block, which is looked at a tile later than it is asked for; its byte offset in a plane
        auto block_of = [&](int32_t t) -> int32_t {
            const int32_t j = sp.lo + t * KT + (lane & (KT - 1));
            int32_t id = 0;
            if (t < t_end && j < sp.n) id = __ldg(table + a.split.slots.block.div((uint32_t)j));
            return id;
        };
        auto slot_of = [&](int32_t t, int32_t id) -> int64_t {         // -1: no key
            const int32_t j = sp.lo + t * KT + (lane & (KT - 1));
            const int32_t in = j - (int32_t)(a.split.slots.block.div((uint32_t)j) * a.split.slots.block.d);
            const bool key = t < t_end && j < sp.n, known = id >= 0 && id < a.split.slots.num_blocks;
            if (key && !known) bad = KVC_FLAG_BLOCK;
            return key && known ? id * a.k_plane.block_stride + in * a.k_plane.token_stride + head_off : -1;
        };
        auto issue = [&](int32_t stage, int64_t slot) {
            constexpr int CPR = ROW / 16, RPI = 32 / CPR;   // chunks of a row, rows at a time
            const uint32_t base = ring + (uint32_t)(stage * C::STAGE);
            const int c = lane % CPR;
            const bool in_row = c * 16 < a.D * C::ES;
#pragma unroll
            for (int i = 0; i < KT / RPI; ++i) {
                const int row = i * RPI + lane / CPR;
                const int64_t off = __shfl_sync(~0u, slot, row);
                const bool there = off >= 0 && in_row;
                const int64_t at = there ? off + c * 16 : 0;
                const uint32_t dst = base + swizzled<ROW>(row, c), n = there ? 16 : 0;
                cp_async16(dst, a.k_plane.base + at, n);
                cp_async16(dst + KT * ROW, a.v_plane.base + at, n);
            }
        };
        // the queries, one warp a row, asked for ahead of the keys
        constexpr int QW = RP / ATTEND_WARPS;
        uint4 qw[QW];
#pragma unroll
        for (int n = 0; n < QW; ++n) {
            const int row = n * ATTEND_WARPS + warp;
            const int32_t rho = row0 + row;
            const int32_t i = (int32_t)a.group.div((uint32_t)rho), gq = rho - i * a.G;
            const unsigned char *q = a.q + r * a.q_request + i * a.q_token +
                                     ((int64_t)h * a.G + gq) * a.q_head;
            qw[n] = make_uint4(0, 0, 0, 0);
            if (row < rows && lane * 8 < a.D) qw[n] = __ldg((const uint4 *)q + lane);
        }
        int32_t next_block;
        {
            int32_t ids[C::STAGES];
#pragma unroll
            for (int k = 0; k < C::STAGES; ++k) ids[k] = block_of(t_begin + k * ATTEND_WARPS);
#pragma unroll
            for (int k = 0; k < C::STAGES - 1; ++k) {
                const int32_t t = t_begin + k * ATTEND_WARPS;
                if (t < t_end) issue(k, slot_of(t, ids[k]));
                cp_async_commit();
            }
            next_block = ids[C::STAGES - 1];
        }

        // the queries in the type of the products; rows beyond M are zero
#pragma unroll
        for (int n = 0; n < QW; ++n) {
            const int row = n * ATTEND_WARPS + warp;
            const uint4 w = qw[n];
            float factor = a.scale * log2e * ks;
            if (POOL != KVR_DTYPE_FP8_E4M3) {
                if (lane * 8 < DP)
                    *(uint4 *)(q_smem + swizzled<DP * 2>(row, lane)) = w;
            } else {
                float f[8], top = 0.0f;
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 p = a.f16 ? widen2<true>(ws[k]) : widen2<false>(ws[k]);
                    f[2 * k] = p.x, f[2 * k + 1] = p.y;
                    top = fmaxf(top, fmaxf(fabsf(p.x), fabsf(p.y)));
                }
#pragma unroll
                for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                // down = 2^-e with 2^e <= top < 2^(e+1): exponents kept where both are normal
                uint32_t e = __float_as_uint(top) >> 23;
                e = e < 2 || e > 252 ? 127 : e;
                const float down = __uint_as_float((254 - e) << 23);
                factor *= __uint_as_float(e << 23);
                // element d = 4 t + x of 16 is at 2 t + x (x < 2) or 8 + 2 t + x - 2: where the
                // codes of four neighbours land when two 8-bit elements load as one 16-bit one
                if (lane * 8 < DP) {
                    const int grp = lane / 2, half = lane % 2;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int pos = (k & 1 ? 8 : 0) + 4 * half + (k & 2);
                        *(uint32_t *)(q_smem + swizzled<DP * 2>(row, grp * 2 + pos / 8) +
                                      (pos % 8) * 2) = narrow2<true>(f[2 * k] * down, f[2 * k + 1] * down);
                    }
                }
            }
            if (lane == 0) row_scale[row] = factor;
        }
        __syncthreads();

        float sc[NT][2], top[NT][2], sum[NT][2];
        int32_t end[NT][2];                             // first key that the row does not see
        int32_t seen_all = sp.n;                        // keys below it are seen by every row
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = n * 8 + 2 * t4 + e;
                sc[n][e] = row_scale[row];
                top[n][e] = -INFINITY;
                sum[n][e] = 0.0f;
                const int32_t i = (int32_t)a.group.div((uint32_t)(row0 + min(row, rows - 1)));
                end[n][e] = sp.n - a.m + i + 1;
            }
        seen_all = sp.n - a.m + 1;
        const int32_t seen_from = a.split.window > 0 ? sp.n - a.split.window : 0;   // keys from it on, by all

        float o[MT][NT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;

        int stage = 0;
        for (int32_t t = t_begin; t < t_end; t += ATTEND_WARPS) {
            cp_async_wait<C::STAGES - 2>();
            __syncwarp();
            {
                const int32_t tn = t + (C::STAGES - 1) * ATTEND_WARPS;
                const int into = stage == 0 ? C::STAGES - 1 : stage - 1;
                if (tn < t_end) issue(into, slot_of(tn, next_block));
                cp_async_commit();
                next_block = block_of(tn + ATTEND_WARPS);
            }
            const uint32_t kbase = ring + (uint32_t)(stage * C::STAGE), vbase = kbase + KT * ROW;
            stage = stage == C::STAGES - 1 ? 0 : stage + 1;

            // S^T: keys by rows
            float s[KS][NT][4];
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[k][n][e] = 0.0f;
            const uint32_t q_base = smem0 + C::RING;
#pragma unroll
            for (int d2 = 0; d2 < DP / 32; ++d2) {      // two steps of 16 elements
                uint32_t b[NT][4];                      // [row tile][step][half]
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    ldmatrix4(b[n], q_base + swizzled<DP * 2>(n * 8 + lane % 8, d2 * 4 + lane / 8));
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if (C::ES == 2) {
#pragma unroll
                        for (int st = 0; st < 2; ++st) {
                            uint32_t f[4];
                            ldmatrix4(f, kbase + swizzled<ROW>(k * 16 + lane % 16,
                                                               (d2 * 2 + st) * 2 + lane / 16));
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma<C::F16>(s[k][n], f, b[n][2 * st], b[n][2 * st + 1]);
                        }
                    } else {
                        uint32_t w[4];                  // keys 0-7, 8-15 of the 1st, 2nd 16 elements
                        ldmatrix4(w, kbase + swizzled<ROW>(k * 16 + lane % 16, d2 * 2 + lane / 16));
#pragma unroll
                        for (int st = 0; st < 2; ++st) {
                            uint32_t f[4];
                            f[0] = e4m3_to_f16x2(w[2 * st]);
                            f[1] = e4m3_to_f16x2(w[2 * st + 1]);
                            f[2] = e4m3_to_f16x2(w[2 * st] >> 16);
                            f[3] = e4m3_to_f16x2(w[2 * st + 1] >> 16);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma<C::F16>(s[k][n], f, b[n][2 * st], b[n][2 * st + 1]);
                        }
                    }
                }
            }

            // softmax over the tile's keys, relative to the maximum of those before; a new maximum is
            // looked for only where it is outgrown (each tile anew, softmax took 420 cycles of a tile of
            // 16 keys and 8 rows, and 1580 with 32 rows, instead of 210 and 770)
            const int32_t j0 = sp.lo + t * KT;
            const bool mixed = j0 + KT > seen_all || j0 < seen_from;
            bool outgrown = false;
            float best[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    best[n][e] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float &v = s[k][n][2 * u + e];
                            v *= sc[n][e];
                            if (mixed) {
                                const int32_t j = j0 + k * 16 + u * 8 + g;
                                if (j >= end[n][e] ||
                                    (a.split.window > 0 && j < window_from(end[n][e], a.split.window)))
                                    v = -INFINITY;
                            }
                            best[n][e] = fmaxf(best[n][e], v);
                        }
                    outgrown |= best[n][e] > top[n][e] + GROWTH;
                }
            if (__any_sync(~0u, outgrown)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int w = 4; w < 32; w *= 2)
                            best[n][e] = fmaxf(best[n][e], __shfl_xor_sync(~0u, best[n][e], w));
                        const float next = fmaxf(top[n][e], best[n][e]);
                        const float shrink = next == top[n][e] ? 1.0f : ex2(top[n][e] - next);
                        top[n][e] = next;
                        sum[n][e] *= shrink;
#pragma unroll
                        for (int i = 0; i < MT; ++i) o[i][n][e] *= shrink, o[i][n][2 + e] *= shrink;
                    }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float at = (top[n][e] == -INFINITY ? 0.0f : top[n][e]) - (C::F16 ? P_SHIFT : 0.0f);
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float &v = s[k][n][2 * u + e];
                            v = ex2(v - at);
                            sum[n][e] += v;
                        }
                }

            // O^T += V^T P^T
            uint32_t ph[KS][NT][2], pl[KS][NT][2];
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float p0 = s[k][n][2 * u], p1 = s[k][n][2 * u + 1];
                        if (C::SPLIT) {
                            const uint32_t w = below2<C::F16>(p0, p1);
                            const float2 f = widen2<C::F16>(w);
                            ph[k][n][u] = movmatrix(w);
                            pl[k][n][u] = movmatrix(narrow2<C::F16>(p0 - f.x, p1 - f.y));
                        } else {
                            ph[k][n][u] = movmatrix(narrow2<C::F16>(p0, p1));
                        }
                    }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (C::ES == 2) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t f[4];
                        ldmatrix4t(f, vbase + swizzled<ROW>(k * 16 + lane % 8 + (lane / 16) * 8,
                                                            i * 2 + (lane / 8) % 2));
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma<C::F16>(o[i][n], f, ph[k][n][0], ph[k][n][1]);
                            if (C::SPLIT) mma<C::F16>(o[i][n], f, pl[k][n][0], pl[k][n][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int i2 = 0; i2 < MT / 2; ++i2) {
                        uint32_t w[4];      // keys 0-7, 8-15 of the 1st, 2nd 16 elements, by pairs
                        ldmatrix4t(w, vbase + swizzled<ROW>(k * 16 + lane % 16, i2 * 2 + lane / 16));
#pragma unroll
                        for (int st = 0; st < 2; ++st) {
                            uint32_t f[4];  // even elements, odd elements; keys 0-7, then 8-15
                            f[0] = e4m3_to_f16x2(__byte_perm(w[2 * st], 0, 0x4420));
                            f[1] = e4m3_to_f16x2(__byte_perm(w[2 * st], 0, 0x4431));
                            f[2] = e4m3_to_f16x2(__byte_perm(w[2 * st + 1], 0, 0x4420));
                            f[3] = e4m3_to_f16x2(__byte_perm(w[2 * st + 1], 0, 0x4431));
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma<C::F16>(o[2 * i2 + st][n], f, ph[k][n][0], ph[k][n][1]);
                        }
                    }
                }
            }
        }
        if (bad != 0) atomicOr(a.split.flags, bad);

        // join the four warps: statistics and accumulators through the ring's memory
        cp_async_wait<0>();
        __syncthreads();
        float *acc = (float *)smem;                     // [warp][RP][PITCH]
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = sum[n][e];
#pragma unroll
                for (int w = 4; w < 32; w *= 2) l += __shfl_xor_sync(~0u, l, w);
                const int row = n * 8 + 2 * t4 + e;
                if (g == 0) {
                    stat[(warp * RP + row) * 2] = top[n][e];
                    stat[(warp * RP + row) * 2 + 1] = l;
                }
                float *to = acc + (warp * RP + row) * C::PITCH;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    to[i * 16 + (C::ES == 2 ? g : 2 * g)] = o[i][n][e];
                    to[i * 16 + (C::ES == 2 ? g + 8 : 2 * g + 1)] = o[i][n][2 + e];
                }
            }
        __syncthreads();
        const int32_t job_index = r * HJ + job;
        const bool whole = u0 == 0 && u1 == units;
        const int32_t D4 = a.D / 4;
        float *slot = a.partial + (size_t)(2 * blockIdx.x + (u0 == 0 ? 1 : 0)) * (size_t)slot_floats;
        const float vs = POOL == KVR_DTYPE_FP8_E4M3 ? a.v_scale[h] : 1.0f;
        // a row's maximum and sum are final: its lse, and what its accumulators are multiplied with
        auto settle = [&](int row, float m, float l) -> float {
            const bool some = l > 0.0f || l != l;
            if (a.lse != nullptr) {
                const int32_t rho = row0 + row, i = (int32_t)a.group.div((uint32_t)rho);
                a.lse[((int64_t)r * a.m + i) * ((int64_t)a.H * a.G) + (int64_t)h * a.G + (rho - i * a.G)] =
                    some ? (m - (C::F16 ? P_SHIFT : 0.0f) + log2f(l)) * 0.6931471805599453f : -INFINITY;
            }
            return some ? vs / l : 0.0f;
        };
        auto finish = [&](int row, int d4, float4 v, float inv) {
            const int32_t rho = row0 + row, i = (int32_t)a.group.div((uint32_t)rho);
            v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
            unsigned char *to = a.out + r * a.out_request + i * a.out_token +
                                ((int64_t)h * a.G + (rho - i * a.G)) * a.out_head;
            *(uint2 *)(to + d4 * 8) = a.f16 ? narrow4<true>(v) : narrow4<false>(v);
        };
        // each row's maximum and sum, and the warps' weights in place of their maxima
        if (tid < rows) {
            float m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int w = 0; w < ATTEND_WARPS; ++w) m = fmaxf(m, stat[(w * RP + tid) * 2]);
#pragma unroll
            for (int w = 0; w < ATTEND_WARPS; ++w) {
                const float mw = stat[(w * RP + tid) * 2], lw = stat[(w * RP + tid) * 2 + 1];
                const float f = mw == -INFINITY ? 0.0f : ex2(mw - m);
                // (a warp that saw no key of the row has nothing to add, whatever it multiplied)
                const bool none = mw == -INFINITY && lw == 0.0f;
                l += none ? 0.0f : f * lw;
                stat[(w * RP + tid) * 2] = none ? -1.0f : f;
            }
            if (whole)
                row_scale[tid] = settle(tid, m, l);
            else
                __stcg((float2 *)(slot + RP * a.D) + tid, make_float2(m, l));
        }
        __syncthreads();
#pragma unroll (RP / ATTEND_WARPS < 4 ? RP / ATTEND_WARPS : 4)
        for (int row = warp; row < rows; row += ATTEND_WARPS)
            for (int d4 = lane; d4 < D4; d4 += 32) {
                float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int w = 0; w < ATTEND_WARPS; ++w) {
                    const float f = stat[(w * RP + row) * 2];
                    const float4 p = *(const float4 *)(acc + (w * RP + row) * C::PITCH + d4 * 4);
                    const bool some = !(f < 0.0f);
                    v.x = some ? fmaf(f, p.x, v.x) : v.x, v.y = some ? fmaf(f, p.y, v.y) : v.y;
                    v.z = some ? fmaf(f, p.z, v.z) : v.z, v.w = some ? fmaf(f, p.w, v.w) : v.w;
                }
                if (whole)
                    finish(row, d4, v, row_scale[row]);
                else
                    __stcg((float4 *)(slot + row * a.D) + d4, v);
            }
        if (!whole) {
            // the job's parts: the blocks that hold its first and its last unit, and all between
            int32_t c0, n;
            cut.parts_of(r, job, seg.job_first, units, ahead, a.shape, &c0, &n);
            __syncthreads();
            if (tid == 0) {
                // (fences by one thread cover what the barriers order before and after it)
                __threadfence();
                const uint32_t before = atomicAdd(a.arrived + job_index, 1u);
                shared_int[0] = before == (uint32_t)(n - 1);
                if (before == (uint32_t)(n - 1)) a.arrived[job_index] = 0;
                __threadfence();
            }
            __syncthreads();
            if (shared_int[0]) {
                // the last to come joins them, in the order of the keys: as many parts at a time as
                // the ring holds, each one copy; their weights, then the weighted sums
                constexpr int COLS = DP / 4, ITEMS = RP * COLS / ATTEND_THREADS;
                static_assert(RP * COLS % ATTEND_THREADS == 0 && RP <= ATTEND_THREADS, "");
                const int32_t slot_bytes = slot_floats * 4;
                const int32_t batch = C::RING / slot_bytes;
                float m = -INFINITY, l = 0.0f;          // of row tid / LANES
                float4 v[ITEMS];
#pragma unroll
                for (int e = 0; e < ITEMS; ++e) v[e] = make_float4(0, 0, 0, 0);
                for (int32_t k0 = 0; k0 < n; k0 += batch) {
                    const int32_t here = min(batch, n - k0);
                    // (what is here was read and written by threads, there written by others')
                    asm volatile("fence.proxy.async;" ::: "memory");
                    __syncthreads();
                    if (warp == 0) {
                        if (lane == 0) bar_expect(join_bar, here * slot_bytes);
                        __syncwarp();
                        for (int32_t k = lane; k < here; k += 32) {
                            const int32_t c = k0 + k;
                            load_bytes(smem0 + k * slot_bytes,
                                       a.partial + (size_t)(2 * (c0 + c) + (c == 0 ? 1 : 0)) * (size_t)slot_floats,
                                       slot_bytes, join_bar);
                        }
                    }
                    if (!bar_wait(join_bar, join_phase)) atomicOr(a.split.flags, KVC_FLAG_TIMEOUT);
                    join_phase ^= 1;
                    {
                        // LANES threads a row
                        constexpr int LANES = ATTEND_THREADS / RP;
                        const int row = tid / LANES, at = tid % LANES;
                        float2 *ml = (float2 *)(acc + RP * a.D) + row;
                        float top = m;
                        for (int32_t k = at; k < here; k += LANES)
                            top = fmaxf(top, ml[k * (slot_floats / 2)].x);
#pragma unroll
                        for (int w = 1; w < LANES; w *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
                        const float old = m == -INFINITY ? 0.0f : ex2(m - top);
                        m = top;
                        float add = 0.0f;
                        for (int32_t k = at; k < here; k += LANES) {
                            const float2 q = ml[k * (slot_floats / 2)];
                            const bool none = q.x == -INFINITY && q.y == 0.0f;
                            const float f = q.x == -INFINITY ? 0.0f : ex2(q.x - top);
                            if (!none) add += f * q.y;
                            ml[k * (slot_floats / 2)].x = none ? -1.0f : f;
                        }
#pragma unroll
                        for (int w = 1; w < LANES; w *= 2) add += __shfl_xor_sync(~0u, add, w);
                        l = l * old + add;
                        if (at == 0) {
                            stat[row * 2] = old;
                            if (k0 + batch >= n && row < rows) row_scale[row] = settle(row, m, l);
                        }
                    }
                    __syncthreads();
#pragma unroll
                    for (int e = 0; e < ITEMS; ++e) {
                        const float old = stat[(e * ATTEND_THREADS + tid) / COLS * 2];
                        v[e].x *= old, v[e].y *= old, v[e].z *= old, v[e].w *= old;
                    }
                    // (all of a thread's items of a part at once: one by one, each waits for its loads)
                    const float *part = acc;
#pragma unroll (ITEMS < 8 ? 8 / ITEMS : 1)
                    for (int32_t k = 0; k < here; ++k, part += slot_floats)
#pragma unroll
                        for (int e = 0; e < ITEMS; ++e) {
                            const int item = e * ATTEND_THREADS + tid, row = item / COLS, d4 = item % COLS;
                            const float f = part[RP * a.D + 2 * row];
                            const float4 p = *(const float4 *)(part + row * a.D + 4 * min(d4, D4 - 1));
                            const bool some = !(f < 0.0f);
                            v[e].x = some ? fmaf(f, p.x, v[e].x) : v[e].x;
                            v[e].y = some ? fmaf(f, p.y, v[e].y) : v[e].y;
                            v[e].z = some ? fmaf(f, p.z, v[e].z) : v[e].z;
                            v[e].w = some ? fmaf(f, p.w, v[e].w) : v[e].w;
                        }
                    __syncthreads();
                }
#pragma unroll
                for (int e = 0; e < ITEMS; ++e) {
                    const int item = e * ATTEND_THREADS + tid, row = item / COLS, d4 = item % COLS;
                    if (row < rows && d4 < D4) finish(row, d4, v[e], row_scale[row]);
                }
            }
        }
        __syncthreads();
    }
}

// What the host needs of an instance.
struct AttendPick {
    void (*kernel)(AttendArgs);
    size_t (*smem)(int32_t requests);
    int32_t unit, rp, blocks;
};

template <int DP, int POOL, int NT>
inline AttendPick attend_instance() {
    using C = Attend<DP, POOL, NT>;
    return {attend_kernel<DP, POOL, NT>, &C::smem, C::UNIT, C::RP, C::BLOCKS};
}

// The instance for head dimension D and M rows a job: rows in passes of 8, 16 or 32 (at most 16
// for D > 128, where 32 rows' accumulators would not fit the registers).
template <int POOL>
inline AttendPick attend_pick(int32_t D, int32_t M) {
    const int nt = M <= 8 ? 1 : M <= 16 || D > 128 ? 2 : 4;
    if (D <= 64)
        return nt == 1 ? attend_instance<64, POOL, 1>()
               : nt == 2 ? attend_instance<64, POOL, 2>() : attend_instance<64, POOL, 4>();
    if (D <= 128)
        return nt == 1 ? attend_instance<128, POOL, 1>()
               : nt == 2 ? attend_instance<128, POOL, 2>() : attend_instance<128, POOL, 4>();
    return nt == 1 ? attend_instance<256, POOL, 1>() : attend_instance<256, POOL, 2>();
}

AttendPick attend_pick_bf16(int32_t D, int32_t M);   // one translation unit each
AttendPick attend_pick_f16(int32_t D, int32_t M);
AttendPick attend_pick_e4m3(int32_t D, int32_t M);

}  // namespace kvc
