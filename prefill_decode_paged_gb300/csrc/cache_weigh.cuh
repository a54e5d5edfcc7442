// cache_weigh.cuh -- how much attention the cached keys of a request got from its newest tokens.
//
// w[r][h][j] (+)= sum over the M = m G rows of key head h of exp(x_j - lse), with the scores x and each row's
// log-sum-exp as attention gave them. One pass over the keys alone, half of attention's bytes; with
// lse given nothing has to be joined, each key belongs to one thread, and the order of its sum is fixed.
// (Within attention itself lse is not known yet: the scores would have to be kept, 4 bytes a row and key
// written and read again, as many bytes as the keys of 4 bits themselves at 8 rows.)
//
// Split. The keys of all (request, head) jobs in units of 4 KT keys form one line, cut into equal parts, one a
// resident block (4-bit pools: cut for one head, each part done by a block a head). Inside a block each of 4 warps takes every fourth tile of KT keys through a ring of its own,
// as in attention. S^T = K Q^T by mma.sync m16n8k16, keys by rows; a lane holds 4 keys of 2 rows of every 8,
// and three exchanges give each lane of four one key's sum, so that a warp writes 32 neighbours at once.
// Scores, exponentials and sums are fp32.
//
// Measured: 64 requests of 8192 keys, 8 heads of 128, 8 rows: bf16 166 to 170 us from card to card (6.4 to 6.6 TB/s,
// HBM), E4M3 96 to 102 (5.4 to 5.8), 4 bits 68 (4.7; conversions). 4 requests of up to 32768 E4M3 keys under 64 rows
// 38.7 us: mma.sync at 57 % of its rate. With 32 rows a pass, which takes the keys and their conversion twice, and tiles
// of 16 keys it took 1.4 and 1.04 times as long.
//
// Tiles take the form with a mask, each score compared with its row's end, where scores are capped or biased, rows do not
// fill the instance, or a row sees nothing: 64 requests of 8192 keys capped 173 us in bf16, 119 in E4M3, 93 in 4 bits,
// biased 172, 110 and 79; under 4 of 8 rows 171, 104 and 73. (4 bits in blocks of 16 tokens, each lane looking its own
// key up, 75.)
#pragma once

#include "cache_attend.cuh"

namespace kvc {

struct WeighArgs {
    KvcPlane k_plane;
    SplitArgs split;
    const unsigned char *q;
    const float *lse;
    float *weights;
    int64_t q_request, q_token, q_head, w_request, w_head;
    const float *k_scale;
    const unsigned char *k_block_scales;
    int32_t m, H, G, D, f16, width, add;
    int32_t chunks;           // passes over a job's keys, RP rows each
    int32_t parts;
    KvrDiv group, by_heads;
    CutShape shape;
    float scale;
    Scoring scoring;
};

template <int DP, int POOL, int NT>
struct Weigh {
    static constexpr bool E4 = POOL == KVR_DTYPE_FP8_E4M3, E2 = POOL == KVC_DTYPE_E2M1, CODES = E4 || E2;
    static constexpr int ROW = E2 ? DP / 2 : E4 ? DP : DP * 2;
    static constexpr int SROW = E2 ? DP / 16 : 0;
    static constexpr int KT = ROW > 256 ? 16 : 32;
    static constexpr int KS = KT / 16;
    static constexpr int STAGE = KT * (ROW + SROW);
    static constexpr int BLOCKS = E2 && NT < 4 && DP <= 128 ? 4 : 2;   // resident on an SM
    static constexpr int STAGES =
        STAGE >= 8192 ? (NT * DP >= 1024 ? 2 : 3) : NT * DP >= 1024 ? 4 : BLOCKS == 4 || STAGE > 4096 ? 5 : 6;
    static constexpr int RING = ATTEND_WARPS * STAGES * STAGE;
    static constexpr int UNIT = ATTEND_WARPS * KT;
    // (as in attention: the block scales of a token's heads share a sector)
    static constexpr bool ABREAST = E2;
    // Tiles that lie in one block are addressed from their first row on where instructions count: 4 bits (64 requests
    // of 8192 keys 74 -> 68 us) and 8 bits under many rows (4 prompts, 64 rows 39.9 -> 38.7), not under few (102 -> 104.5)
    static constexpr bool RUNS = E2 || (E4 && NT > 2);
    static constexpr int RP = 8 * NT;
    static constexpr int Q_BYTES = RP * DP * 2;
    // ring, queries, then of each row its factor, its log-sum-exp, its end and its slope; 4 ints; prefix
    static constexpr int FIXED = RING + Q_BYTES + 16 * RP + 16;
    static constexpr size_t smem(int32_t requests) { return FIXED + 4 * (size_t)(requests + 1); }
};

template <int DP, int POOL, int NT>
__global__ void __launch_bounds__(ATTEND_THREADS, (Weigh<DP, POOL, NT>::BLOCKS)) weigh_kernel(WeighArgs a) {
    using C = Weigh<DP, POOL, NT>;
    constexpr int KT = C::KT, KS = C::KS, RP = C::RP, ROW = C::ROW;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t smem0 = (uint32_t)__cvta_generic_to_shared(smem);
    unsigned char *q_smem = smem + C::RING;
    float *row_scale = (float *)(q_smem + C::Q_BYTES);  // factors of the products, log-sum-exps: in powers of two
    float *row_lse = row_scale + RP;
    int32_t *row_end = (int32_t *)(row_lse + RP);       // first key that the row does not see; 0: no row
    float *row_slope = (float *)(row_end + RP);
    int32_t *shared_int = (int32_t *)(row_slope + RP);  // [4]
    int32_t *prefix = shared_int + 4;                   // [requests + 1], in units of one job
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t4 = lane % 4;
    const float log2e = 1.4426950408889634f;

    wait_for_previous();
    let_next_start();
    unit_prefix<C::UNIT>(a.split, 1, prefix, shared_int);
    // (abreast: one block a head goes through the same part of the requests' keys)
    const int32_t parts = C::ABREAST ? a.parts : (int32_t)gridDim.x;
    const int32_t part = C::ABREAST ? (int32_t)a.by_heads.div(blockIdx.x) : (int32_t)blockIdx.x;
    const int32_t total = prefix[a.split.requests] * (C::ABREAST ? 1 : a.H);
    const int32_t each = total / parts, more = total - each * parts;
    int32_t x = part * each + min(part, more);
    const int32_t x_end = x + each + (part < more ? 1 : 0);
    const int32_t M = a.m * a.G;
    const uint32_t ring = smem0 + (uint32_t)(warp * C::STAGES * C::STAGE);

    while (x < x_end) {
        const Segment seg = segment_at(x, x_end, prefix, a.shape);
        const int32_t r = seg.r, h = C::ABREAST ? (int32_t)blockIdx.x - part * a.H : seg.job;
        x += seg.u1 - seg.u0;
        uint32_t bad = 0;
        const Span sp = span_of(a.split, r, 1, &bad);   // tiles begin at the first key
        const float ks = C::CODES ? a.k_scale[h] : 1.0f;
        float *weights = a.weights + r * a.w_request + h * a.w_head;
        const int32_t n = min(sp.n, a.width);           // keys that have a weight
        if (sp.n > a.width) bad |= KVC_FLAG_LENGTH;
        // what lies below the windows gets nothing
        if (seg.u0 == 0 && !a.add)
            for (int32_t j = tid; j < min(sp.lo, n); j += ATTEND_THREADS) weights[j] = 0.0f;

        const int32_t tiles = (sp.n - sp.lo + KT - 1) / KT;
        const int32_t t_begin = seg.u0 * ATTEND_WARPS + warp, t_end = min(seg.u1 * ATTEND_WARPS, tiles);
        const int32_t *table = a.split.slots.ids + (int64_t)r * a.split.slots.stride;
        const int64_t head_off = (int64_t)h * a.k_plane.head_stride;
        // a tile's key of this lane: its block, looked at a tile later than it is asked for; its offset in a plane
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
            if (key && !known) bad |= KVC_FLAG_BLOCK;
            return key && known ? id * a.k_plane.block_stride + in * a.k_plane.token_stride + head_off : -1;
        };
        auto issue = [&](int32_t stage, int64_t slot) {
            constexpr int CPR = ROW / 16, RPI = 32 / CPR;   // chunks of a row, rows at a time
            const uint32_t base = ring + (uint32_t)(stage * C::STAGE);
            const int c = lane % CPR;
            const bool in_row = C::E2 ? c * 32 < a.D : C::E4 ? c * 16 < a.D : c * 8 < a.D;
#pragma unroll
            for (int i = 0; i < KT / RPI; ++i) {
                const int row = i * RPI + lane / CPR;
                const int64_t off = __shfl_sync(~0u, slot, row);
                const bool there = off >= 0 && in_row;
                cp_async16<!C::E2 || ROW >= 128>(base + swizzled<ROW>(row, c), a.k_plane.base + (there ? off + c * 16 : 0),
                           there ? 16 : 0);
            }
            if (C::E2) {                                // each lane its own key's block scales
                constexpr int PIECE = DP == 128 ? 8 : 4;
#pragma unroll
                for (int p = 0; p < C::SROW / PIECE; ++p) {
                    const bool there = slot >= 0 && p * PIECE * 16 < a.D;
                    cp_async_few<PIECE>(base + KT * ROW + lane * C::SROW + p * PIECE,
                                        a.k_block_scales + (there ? slot / 8 + p * PIECE : 0), there ? PIECE : 0);
                }
            }
        };

        // A tile that is whole and in one block: from its first row on
        const bool runs = C::RUNS && a.split.slots.block.d % KT == 0 && sp.lo % KT == 0;
        auto issue_run = [&](int32_t stage, int32_t t, int32_t id) {
            constexpr int CPR = ROW / 16, RPI = 32 / CPR;
            const uint32_t base = ring + (uint32_t)(stage * C::STAGE);
            const int32_t j = sp.lo + t * KT, c = lane % CPR;
            const int32_t in = j - (int32_t)(a.split.slots.block.div((uint32_t)j) * a.split.slots.block.d);
            const int64_t first = id * a.k_plane.block_stride + in * a.k_plane.token_stride + head_off;
            const uint32_t n = (C::E2 ? c * 32 < a.D : c * 16 < a.D) ? 16 : 0;   // (0: nothing is read)
            const unsigned char *k =
                a.k_plane.base + first + (lane / CPR) * a.k_plane.token_stride + (n != 0 ? c * 16 : 0);
            const int64_t step = RPI * a.k_plane.token_stride;
#pragma unroll
            for (int i = 0; i < KT / RPI; ++i, k += step)
                cp_async16<!C::E2 || ROW >= 128>(base + swizzled<ROW>(i * RPI + lane / CPR, c), k, n);
            if (C::E2) {
                constexpr int PIECE = DP == 128 ? 8 : 4;
                const int64_t scale = (first + lane * a.k_plane.token_stride) / 8;
#pragma unroll
                for (int p = 0; p < C::SROW / PIECE; ++p) {
                    const bool there = p * PIECE * 16 < a.D;
                    cp_async_few<PIECE>(base + KT * ROW + lane * C::SROW + p * PIECE,
                                        a.k_block_scales + (there ? scale + p * PIECE : 0), there ? PIECE : 0);
                }
            }
        };
        // (the block's id is the same in all lanes there)
        auto issue_tile = [&](int32_t stage, int32_t t, int32_t id) {
            if constexpr (C::RUNS) {
                if (runs && sp.lo + (t + 1) * KT <= sp.n && id >= 0 && id < a.split.slots.num_blocks) {
                    issue_run(stage, t, id);
                    return;
                }
            }
            issue(stage, slot_of(t, id));
        };

        for (int32_t chunk = 0; chunk < a.chunks; ++chunk) {
            const int32_t row0 = chunk * RP, rows = min(RP, M - row0);
            const bool adding = a.add || chunk > 0;
            // the queries, asked for ahead of the keys
            using Queries = QueryLanes<DP, RP>;
            uint4 qw[Queries::TIMES];
#pragma unroll
            for (int k = 0; k < Queries::TIMES; ++k) {
                const int row = Queries::row(k);
                const int32_t rho = row0 + row;
                const int32_t i = (int32_t)a.group.div((uint32_t)rho), gq = rho - i * a.G;
                const int64_t head = (int64_t)h * a.G + gq;
                const unsigned char *q = a.q + r * a.q_request + i * a.q_token + head * a.q_head;
                qw[k] = make_uint4(0, 0, 0, 0);
                if (row < rows && Queries::lane() * 8 < a.D) qw[k] = __ldg((const uint4 *)q + Queries::lane());
            }
            // (and one thread a row what else there is of it)
            static_assert(RP <= ATTEND_THREADS, "");
            float z_own = 0.0f, slope_own = 0.0f;
            int32_t end_own = 0;                        // (no row: sees no key, and its distances stay within 32 bits)
            if (tid < rows) {
                const int32_t rho = row0 + tid, i = (int32_t)a.group.div((uint32_t)rho);
                const int64_t head = (int64_t)h * a.G + rho - i * a.G;
                z_own = __ldg(a.lse + ((int64_t)r * a.m + i) * ((int64_t)a.H * a.G) + head);
                // (one without a sum has nothing to give, whatever its scores are: it sees no key)
                end_own = z_own == -INFINITY ? 0 : sp.n - a.m + i + 1;
                slope_own = slope_of(a.scoring, (int32_t)head);
            }
            int32_t next_block;
            {
                int32_t ids[C::STAGES];
#pragma unroll
                for (int k = 0; k < C::STAGES; ++k) ids[k] = block_of(t_begin + k * ATTEND_WARPS);
#pragma unroll
                for (int k = 0; k < C::STAGES - 1; ++k) {
                    const int32_t t = t_begin + k * ATTEND_WARPS;
                    if (t < t_end) issue_tile(k, t, ids[k]);
                    cp_async_commit();
                }
                next_block = ids[C::STAGES - 1];
            }
            __syncthreads();                            // the queries before these have been used
#pragma unroll
            for (int k = 0; k < Queries::TIMES; ++k) {
                const int row = Queries::row(k);
                if (row >= RP) continue;
                float factor = a.scale * log2e * ks;
                place_query<DP, POOL>(q_smem, row, qw[k], a.f16, &factor);
                if (Queries::lane() == 0) row_scale[row] = factor;
            }
            if (tid < RP) {
                row_lse[tid] = z_own * log2e;
                row_end[tid] = end_own;
                row_slope[tid] = slope_own;
            }
            __syncthreads();

            float sc[NT][2], z[NT][2];
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sc[k][e] = row_scale[k * 8 + 2 * t4 + e];
                    z[k][e] = row_lse[k * 8 + 2 * t4 + e];
                }
            const bool plain = a.scoring.cap == 0.0f && a.scoring.slopes == nullptr;
            bool none = rows < RP;                                // a row that sees nothing, whatever its place
#pragma unroll
            for (int k = 0; k < NT; ++k) none |= z[k][0] == -INFINITY || z[k][1] == -INFINITY;
            const int32_t seen_all = __any_sync(~0u, none) ? INT32_MIN : sp.n - a.m + 1;   // keys below it are seen by every row
            const int32_t seen_from = a.split.window > 0 ? sp.n - a.split.window : 0;   // keys from it on, by all

            // the lane's own key of a tile, and its weight so far, asked for a tile ahead
            auto key_of = [&](int32_t t) -> int32_t {
                const int32_t j = sp.lo + t * KT + t4 * 8 + g;
                return t < t_end && t4 < 2 * KS && j < n ? j : -1;
            };
            auto old_of = [&](int32_t j) -> float { return adding && j >= 0 ? weights[j] : 0.0f; };
            int32_t own = key_of(t_begin);
            float old = old_of(own);
            int stage = 0;
            for (int32_t t = t_begin; t < t_end; t += ATTEND_WARPS) {
                cp_async_wait<C::STAGES - 2>();
                __syncwarp();
                {
                    const int32_t tn = t + (C::STAGES - 1) * ATTEND_WARPS;
                    const int into = stage == 0 ? C::STAGES - 1 : stage - 1;
                    if (tn < t_end) issue_tile(into, tn, next_block);
                    cp_async_commit();
                    next_block = block_of(tn + ATTEND_WARPS);
                }
                const int32_t next = key_of(t + ATTEND_WARPS);
                const float next_old = old_of(next);
                const uint32_t kbase = ring + (uint32_t)(stage * C::STAGE);
                stage = stage == C::STAGES - 1 ? 0 : stage + 1;

                float s[KS][NT][4];
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[k][c][e] = 0.0f;
                tile_scores<DP, POOL, KT, NT>(s, kbase, smem0 + C::RING, smem + (kbase - smem0) + KT * ROW);

                const int32_t j0 = sp.lo + t * KT;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};            // keys g, g + 8 of each 16
                if (plain && j0 + KT <= seen_all && j0 >= seen_from) {
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int k = 0; k < KS; ++k)
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    sum[2 * k + u] += ex2(fmaf(s[k][c][2 * u + e], sc[c][e], -z[c][e]));
                } else {
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int32_t end = row_end[c * 8 + 2 * t4 + e];
                            const float slope = row_slope[c * 8 + 2 * t4 + e];
#pragma unroll
                            for (int k = 0; k < KS; ++k)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const int32_t j = j0 + k * 16 + u * 8 + g;
                                    const float v = s[k][c][2 * u + e];
                                    const float p =
                                        plain ? ex2(fmaf(v, sc[c][e], -z[c][e]))
                                              : ex2(scored(v * sc[c][e], a.scoring, slope, j - end + 1) - z[c][e]);
                                    const bool seen = j < end && (a.split.window == 0 || j >= window_from(end, a.split.window));
                                    sum[2 * k + u] += seen ? p : 0.0f;
                                }
                        }
                }
                // each lane of four keeps a quarter of the keys
                const bool odd = t4 & 1, high = t4 & 2;
                const float lo = (odd ? sum[1] : sum[0]) + __shfl_xor_sync(~0u, odd ? sum[0] : sum[1], 1);
                const float hi = (odd ? sum[3] : sum[2]) + __shfl_xor_sync(~0u, odd ? sum[2] : sum[3], 1);
                const float all = (high ? hi : lo) + __shfl_xor_sync(~0u, high ? lo : hi, 2);
                if (own >= 0) weights[own] = old + all;
                own = next;
                old = next_old;
            }
            cp_async_wait<0>();
        }
        if (bad != 0) atomicOr(a.split.flags, bad);
        __syncthreads();
    }
}

// What the host needs of an instance.
struct WeighPick {
    void (*kernel)(WeighArgs);
    size_t (*smem)(int32_t requests);
    int32_t unit, rp, blocks;
    bool abreast;
};

template <int DP, int POOL, int NT>
inline WeighPick weigh_instance() {
    using C = Weigh<DP, POOL, NT>;
    static_assert(C::BLOCKS * (C::smem(1) + 1024) <= 228 << 10, "blocks that shared memory holds");
    return {weigh_kernel<DP, POOL, NT>, &C::smem, C::UNIT, C::RP, C::BLOCKS, C::ABREAST};
}

// The instance for head dimension D and M rows a job: rows in passes of 8, 16, 32 or 64.
template <int POOL>
inline WeighPick weigh_pick(int32_t D, int32_t M) {
    const int nt = M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : 8;
    if (D <= 64)
        return nt == 1   ? weigh_instance<64, POOL, 1>()
               : nt == 2 ? weigh_instance<64, POOL, 2>()
               : nt == 4 ? weigh_instance<64, POOL, 4>() : weigh_instance<64, POOL, 8>();
    if (D <= 128)
        return nt == 1   ? weigh_instance<128, POOL, 1>()
               : nt == 2 ? weigh_instance<128, POOL, 2>()
               : nt == 4 ? weigh_instance<128, POOL, 4>() : weigh_instance<128, POOL, 8>();
    return nt == 1   ? weigh_instance<256, POOL, 1>()
           : nt == 2 ? weigh_instance<256, POOL, 2>()
           : nt == 4 ? weigh_instance<256, POOL, 4>() : weigh_instance<256, POOL, 8>();
}

WeighPick weigh_pick_bf16(int32_t D, int32_t M);     // one translation unit each
WeighPick weigh_pick_f16(int32_t D, int32_t M);
WeighPick weigh_pick_e4m3(int32_t D, int32_t M);
WeighPick weigh_pick_e2m1(int32_t D, int32_t M);

}  // namespace kvc
