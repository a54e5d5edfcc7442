// cache_append.cu -- new tokens' keys and values into a paged pool, positions rotated on the way.
//
// Pure data movement with three fp32 operations a rotated element: each input row is read once,
// each pool row and rotated query written once. One block does one token, whose head rows (those
// of the queries, keys and values) are cut into UNITS of 16 elements, two 16-byte pieces each:
//   rotated, halves:      pieces at 8 i and 8 i + R / 2 hold pairs 8 i .. 8 i + 7 as (a | b);
//   rotated, interleaved: pieces at 16 i and 16 i + 8 hold the same pairs side by side;
//   not rotated:          pieces at 16 i and 16 i + 8, passed through (or quantized).
// A thread asks for BATCH units before it looks at the token's position: the slot (position, then
// block id) and the angles are on their way meanwhile. Where the row's units divide the block's
// threads, a thread has the same unit of every row, and loads its angles once. HBM bounds it with
// many tokens: 39834 tokens of 32 + 16 heads of 128, 982 MB, 152 to 159 us from card to card
// (6180 to 6450 GB/s, 91 to 95 % of a plain copy's rate).
#include <algorithm>

#include "cache.h"

namespace {

using namespace kvc;

constexpr int BORDER = 2;     // tokens an SM, above which they are many
// MB of rows (those of E4M3 pools counted as they are read, in 16 bits) above which the stores do not ask
// L2 to keep what they write: half of it. Prompts' 486 MB take 152
// us instead of 161 so; 60 MB would take 22 instead of 24, but what reads them next finds them there.
constexpr int AWAY = 64;
constexpr int MANY_THREADS = 128, FEW_THREADS = 512;
struct Rows {                 // head rows of one input and where they go
    const unsigned char *src;
    int64_t src_token, src_head;
    int32_t heads;
};

struct AppendArgs {
    Rows k, v, q;
    KvcPlane k_plane, v_plane;
    unsigned char *q_out;
    int64_t q_out_token, q_out_head;
    const int32_t *requests, *positions;
    KvcSlots slots;
    const float *rotary;      // [rows][R]
    int32_t rotary_rows, R;
    int32_t dim, q_dim;
    const float *k_scale, *v_scale;
    uint32_t *flags;
    int32_t last;             // the rotated elements are the row's last
    int32_t away;             // what is written need not stay in L2
    KvrDiv units, q_units;    // of a key's and of a query's row
};

struct Unit {
    int32_t e0, e1;           // its two pieces' first elements in the row
    int32_t pair;             // its first pair, -1 if it is not rotated
    bool rotated;
    float cs[8], sn[8];
};

template <bool INTERLEAVED>
__device__ __forceinline__ void place(Unit &u, const AppendArgs &a, int32_t dim, int32_t j) {
    const int32_t R = a.R;
    const int32_t first = a.last ? dim - R : 0;
    const int32_t i = a.last ? j - (dim - R) / 16 : j;      // which rotated unit, if it is one
    u.rotated = R > 0 && i >= 0 && i < R / 16;
    u.e0 = u.rotated ? first + (INTERLEAVED ? 16 * i : 8 * i) : 16 * j;
    u.e1 = u.e0 + (u.rotated && !INTERLEAVED ? R / 2 : 8);
    u.pair = u.rotated ? 8 * i : -1;
}

__device__ __forceinline__ void load_angles(Unit &u, const float *row, int32_t R) {
    const float4 *c = (const float4 *)(row + u.pair), *s = (const float4 *)(row + R / 2 + u.pair);
    const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
    u.cs[0] = c0.x, u.cs[1] = c0.y, u.cs[2] = c0.z, u.cs[3] = c0.w;
    u.cs[4] = c1.x, u.cs[5] = c1.y, u.cs[6] = c1.z, u.cs[7] = c1.w;
    u.sn[0] = s0.x, u.sn[1] = s0.y, u.sn[2] = s0.z, u.sn[3] = s0.w;
    u.sn[4] = s1.x, u.sn[5] = s1.y, u.sn[6] = s1.z, u.sn[7] = s1.w;
}

__device__ __forceinline__ uint4 load16(const unsigned char *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The unit's 16 elements in fp32: x[0..7] piece 0, x[8..15] piece 1; rotated in place.
template <bool F16, bool INTERLEAVED>
__device__ __forceinline__ void turn(const uint4 &p0, const uint4 &p1, const Unit &u, float x[16]) {
    const uint32_t w[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = widen2<F16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    if (!u.rotated) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &a = x[INTERLEAVED ? 2 * i : i], &b = x[INTERLEAVED ? 2 * i + 1 : i + 8];
        const float y = fmaf(a, u.cs[i], -(b * u.sn[i]));
        b = fmaf(b, u.cs[i], a * u.sn[i]);
        a = y;
    }
}

template <typename T>
__device__ __forceinline__ void store(unsigned char *to, T v, bool away) {
    if (away)
        __stcs((T *)to, v);
    else
        *(T *)to = v;
}

template <bool F16>
__device__ __forceinline__ void store_16bit(unsigned char *row, const Unit &u, const float x[16],
                                            bool away) {
    uint4 o0, o1;
    o0.x = narrow2<F16>(x[0], x[1]), o0.y = narrow2<F16>(x[2], x[3]);
    o0.z = narrow2<F16>(x[4], x[5]), o0.w = narrow2<F16>(x[6], x[7]);
    o1.x = narrow2<F16>(x[8], x[9]), o1.y = narrow2<F16>(x[10], x[11]);
    o1.z = narrow2<F16>(x[12], x[13]), o1.w = narrow2<F16>(x[14], x[15]);
    store(row + 2 * u.e0, o0, away);
    store(row + 2 * u.e1, o1, away);
}

// Four E4M3 codes of x * inv, nearest-even, saturated; every code gets its value's sign bit (a
// no-op for all but NaN, whose code is 0x7F otherwise).
__device__ __forceinline__ uint32_t quant4f(const float *x, float inv) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * inv), "f"(x[0] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * inv), "f"(x[2] * inv));
    const uint32_t sign = (__float_as_uint(x[0]) >> 31 << 7) | (__float_as_uint(x[1]) >> 31 << 15) |
                          (__float_as_uint(x[2]) >> 31 << 23) | (__float_as_uint(x[3]) >> 31 << 31);
    return (uint32_t)lo | ((uint32_t)hi << 16) | sign;
}

__device__ __forceinline__ void store_8bit(unsigned char *row, const Unit &u, const float x[16],
                                           float inv, bool away) {
    store(row + u.e0, make_uint2(quant4f(x, inv), quant4f(x + 4, inv)), away);
    store(row + u.e1, make_uint2(quant4f(x + 8, inv), quant4f(x + 12, inv)), away);
}

// Where unit `t` of the token's units is: queries first, then keys, then values.
struct Place {
    int32_t row, j;           // head row of its input, unit of the row
    int32_t kind;             // 0 query, 1 key, 2 value, 3 none
};
__device__ __forceinline__ Place place_of(const AppendArgs &a, int32_t t, int32_t n) {
    Place p;
    const int32_t nq = a.q.heads * (int32_t)a.q_units.d;
    if (t < nq) {
        p.kind = 0;
        p.row = (int32_t)a.q_units.div((uint32_t)t);
        p.j = t - p.row * (int32_t)a.q_units.d;
    } else {
        t -= nq;
        p.row = (int32_t)a.units.div((uint32_t)t);
        p.j = t - p.row * (int32_t)a.units.d;
        p.kind = p.row < a.k.heads ? 1 : 2;
        if (p.kind == 2) p.row -= a.k.heads;
        if (t + nq >= n) p.kind = 3;
    }
    return p;
}

template <bool F16, bool INTERLEAVED, bool E4M3, bool MANY>
__global__ void __launch_bounds__(MANY ? MANY_THREADS : FEW_THREADS, MANY ? 10 : 2)
append_kernel(AppendArgs a) {
    constexpr int BATCH = MANY ? 1 : 2;
    const int32_t THREADS = MANY ? MANY_THREADS : (int32_t)blockDim.x;
    wait_for_previous();
    let_next_start();
    const int64_t token = blockIdx.x;
    const int32_t pos = __ldg(a.positions + token), req = __ldg(a.requests + token);
    const int32_t n = a.q.heads * (int32_t)a.q_units.d + (a.k.heads + a.v.heads) * (int32_t)a.units.d;
    int64_t slot = -1;                       // the token's slot in a plane, in bytes
    const float *angles = nullptr;
    int32_t have = -1;                       // the pair whose angles `u` holds
    Unit u;

    for (int32_t t0 = threadIdx.x; t0 < n; t0 += THREADS * BATCH) {
        uint4 p0[BATCH], p1[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const Place p = place_of(a, t0 + b * THREADS, n);
            if (p.kind < 3) {
                const Rows &in = p.kind == 0 ? a.q : p.kind == 1 ? a.k : a.v;
                Unit w;
                place<INTERLEAVED>(w, a, p.kind == 0 ? a.q_dim : a.dim, p.j);
                const unsigned char *src = in.src + token * in.src_token + p.row * in.src_head;
                p0[b] = load16(src + 2 * w.e0);
                p1[b] = load16(src + 2 * w.e1);
            }
        }
        if (slot < 0) {
            if (pos < 0) return;
            const uint32_t entry = a.slots.block.div((uint32_t)pos);
            uint32_t bad = 0;
            if (req < 0 || req >= a.slots.rows) {
                bad = KVC_FLAG_REQUEST;
            } else if (entry >= (uint32_t)a.slots.width ||
                       (a.rotary != nullptr && pos >= a.rotary_rows)) {
                bad = KVC_FLAG_POSITION;
            } else {
                const int32_t id = __ldg(a.slots.ids + (int64_t)req * a.slots.stride + entry);
                const int32_t off = pos - (int32_t)(entry * a.slots.block.d);
                angles = a.rotary + (int64_t)pos * a.R;
                if (id < 0 || id >= a.slots.num_blocks)
                    bad = KVC_FLAG_BLOCK;
                else
                    slot = id * a.k_plane.block_stride + off * a.k_plane.token_stride;
            }
            if (bad != 0) {
                if (threadIdx.x == 0) atomicOr(a.flags, bad);
                return;
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const Place p = place_of(a, t0 + b * THREADS, n);
            if (p.kind == 3) continue;
            place<INTERLEAVED>(u, a, p.kind == 0 ? a.q_dim : a.dim, p.j);
            if (p.kind == 2) u.rotated = false;
            if (u.rotated && u.pair != have) {
                load_angles(u, angles, a.R);
                have = u.pair;
            }
            float x[16];
            turn<F16, INTERLEAVED>(p0[b], p1[b], u, x);
            if (p.kind == 0) {
                store_16bit<F16>(a.q_out + token * a.q_out_token + p.row * a.q_out_head, u, x,
                                 MANY && a.away);
            } else {
                const KvcPlane &plane = p.kind == 1 ? a.k_plane : a.v_plane;
                unsigned char *dst = plane.base + slot + p.row * plane.head_stride;
                if (E4M3)
                    store_8bit(dst, u, x, 1.0f / __ldg((p.kind == 1 ? a.k_scale : a.v_scale) + p.row),
                               MANY && a.away);
                else
                    store_16bit<F16>(dst, u, x, MANY && a.away);
            }
        }
    }
}

// Many tokens: blocks of 128 threads, one unit a thread at a time and small register sets, as the blocks
// on an SM hide one another's waits. Few: a token is one chain of waits, so each unit has a thread of
// its own, up to 512 and two units a thread. Few and many took (us) 3.0 and 4.0 for 64 tokens of 640
// units, 4.2 and 5.6 for 256; 2.9 and 3.1 for 300 of 384, 4.9 and 3.8 for 600; and with blocks of 192,
// 256 and 384 threads 39834 tokens took 186, 190 and 216 where those of 128 took 162. (The register limits, 48
// for many and 64 for few, make the compiler spill 12 to 64 bytes a thread; looser ones have not been tried.)
template <bool F16, bool E4M3>
kvr_status go(AppendArgs &a, bool interleaved, int32_t tokens, int sms, void *stream) {
    const int64_t n = (int64_t)a.q.heads * a.q_units.d + (int64_t)(a.k.heads + a.v.heads) * a.units.d;
    const bool many = tokens > BORDER * sms;
    const int64_t rounds = (n + FEW_THREADS - 1) / FEW_THREADS;
    const int threads = many ? MANY_THREADS : (int)((n + 32 * rounds - 1) / (32 * rounds)) * 32;
    a.away = tokens * n * 16 * 2 > (int64_t)AWAY << 20;
    const auto kernel =
        many ? (interleaved ? append_kernel<F16, true, E4M3, true> : append_kernel<F16, false, E4M3, true>)
             : (interleaved ? append_kernel<F16, true, E4M3, false> : append_kernel<F16, false, E4M3, false>);
    return kvc_launch(kernel, a, dim3((unsigned)tokens), threads, 0, stream);
}

}  // namespace

kvr_status kvc_append_launch(const kvc_cache *c, int32_t layer, const kvc_append *p, void *stream) {
    AppendArgs a = {};
    const int32_t H = c->d.kv_heads;
    a.k = {(const unsigned char *)p->k, p->k_token_stride, p->k_head_stride, H};
    a.k_plane = c->plane(layer, 0);
    a.k_scale = c->scale_of(layer, 0);
    if (!c->latent()) {
        a.v = {(const unsigned char *)p->v, p->v_token_stride, p->v_head_stride, H};
        a.v_plane = c->plane(layer, 1);
        a.v_scale = c->scale_of(layer, 1);
    }
    a.q = {(const unsigned char *)p->q, p->q_token_stride, p->q_head_stride, p->q_heads};
    a.q_out = (unsigned char *)p->q_out;
    a.q_out_token = p->q_out_token_stride;
    a.q_out_head = p->q_out_head_stride;
    a.requests = p->requests;
    a.positions = p->positions;
    a.slots = c->slots(p->table);
    a.rotary = p->rotary;
    a.rotary_rows = p->rotary_rows;
    a.R = p->rotary == nullptr ? 0 : p->rotary_dim;
    a.dim = c->d.head_dim;
    a.q_dim = p->q_dim;
    a.units = kvr_make_div((uint32_t)a.dim / 16);
    a.q_units = kvr_make_div(std::max(1u, (uint32_t)a.q_dim / 16));
    a.flags = c->ws.flags;
    a.last = (p->flags & KVC_ROTATE_LAST) != 0;
    const bool il = (p->flags & KVC_INTERLEAVED) != 0, f16 = p->dtype == KVC_DTYPE_F16;
    if (c->d.dtype == KVR_DTYPE_FP8_E4M3)
        return f16 ? go<true, true>(a, il, p->num_tokens, c->sm_count, stream)
                   : go<false, true>(a, il, p->num_tokens, c->sm_count, stream);
    return f16 ? go<true, false>(a, il, p->num_tokens, c->sm_count, stream)
               : go<false, false>(a, il, p->num_tokens, c->sm_count, stream);
}
