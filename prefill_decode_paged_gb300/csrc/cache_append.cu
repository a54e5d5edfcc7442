// cache_append.cu -- new tokens' keys and values into a paged pool, positions rotated on the way.
//
// Pure data movement with three fp32 operations a rotated element: each input row is read once,
// each pool row and rotated query written once. One block does one token. A thread owns one
// UNIT of a head row, 16 elements as two 16-byte pieces, and the same unit of every head that
// it comes to, so the cosines and sines of its eight pairs are loaded once a token:
//   rotated, halves:      pieces at 8 i and 8 i + R / 2 hold pairs 8 i .. 8 i + 7 as (a | b);
//   rotated, interleaved: pieces at 16 i and 16 i + 8 hold the same pairs side by side;
//   not rotated:          pieces at 16 i and 16 i + 8, passed through (or quantized).
#include "cache.h"

namespace {

using namespace kvc;

constexpr int THREADS = 128;
constexpr int BATCH = 4;      // rows a thread has in flight

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
};

struct Unit {                 // byte offsets of its two pieces in a row of 16-bit elements
    int32_t e0, e1;           // elements
    bool rotated;
    float cs[8], sn[8];
};

template <bool INTERLEAVED>
__device__ __forceinline__ Unit make_unit(const AppendArgs &a, int32_t dim, int32_t j,
                                          const float *row) {
    Unit u;
    const int32_t R = a.R;
    const int32_t first = a.last ? dim - R : 0;
    const int32_t i = a.last ? j - (dim - R) / 16 : j;      // which rotated unit, if it is one
    u.rotated = R > 0 && i >= 0 && i < R / 16;
    if (u.rotated) {
        u.e0 = first + (INTERLEAVED ? 16 * i : 8 * i);
        u.e1 = u.e0 + (INTERLEAVED ? 8 : R / 2);
        if (row != nullptr) {
            const float4 *c = (const float4 *)(row + 8 * i), *s = (const float4 *)(row + R / 2 + 8 * i);
            const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
            u.cs[0] = c0.x, u.cs[1] = c0.y, u.cs[2] = c0.z, u.cs[3] = c0.w;
            u.cs[4] = c1.x, u.cs[5] = c1.y, u.cs[6] = c1.z, u.cs[7] = c1.w;
            u.sn[0] = s0.x, u.sn[1] = s0.y, u.sn[2] = s0.z, u.sn[3] = s0.w;
            u.sn[4] = s1.x, u.sn[5] = s1.y, u.sn[6] = s1.z, u.sn[7] = s1.w;
        }
    } else {
        u.e0 = 16 * j;
        u.e1 = u.e0 + 8;
    }
    return u;
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

template <bool F16>
__device__ __forceinline__ void store_16bit(unsigned char *row, const Unit &u, const float x[16]) {
    uint4 o0, o1;
    o0.x = narrow2<F16>(x[0], x[1]), o0.y = narrow2<F16>(x[2], x[3]);
    o0.z = narrow2<F16>(x[4], x[5]), o0.w = narrow2<F16>(x[6], x[7]);
    o1.x = narrow2<F16>(x[8], x[9]), o1.y = narrow2<F16>(x[10], x[11]);
    o1.z = narrow2<F16>(x[12], x[13]), o1.w = narrow2<F16>(x[14], x[15]);
    *(uint4 *)(row + 2 * u.e0) = o0;
    *(uint4 *)(row + 2 * u.e1) = o1;
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
                                           float inv) {
    *(uint2 *)(row + u.e0) = make_uint2(quant4f(x, inv), quant4f(x + 4, inv));
    *(uint2 *)(row + u.e1) = make_uint2(quant4f(x + 8, inv), quant4f(x + 12, inv));
}

// Rows [0, count) of this token: the queries (count = q.heads), or keys then values.
template <bool F16, bool INTERLEAVED, bool E4M3>
__global__ void __launch_bounds__(THREADS) append_kernel(AppendArgs a) {
    wait_for_previous();
    let_next_start();
    const int64_t t = blockIdx.x;
    const int32_t pos = __ldg(a.positions + t), req = __ldg(a.requests + t);
    if (pos < 0) return;
    if (a.rotary != nullptr && pos >= a.rotary_rows) {
        if (threadIdx.x == 0) atomicOr(a.flags, KVC_FLAG_POSITION);
        return;
    }
    const float *angles = a.rotary == nullptr ? nullptr : a.rotary + (int64_t)pos * a.R;

    int64_t slot_k = -1, slot_v = -1;        // this token's slot in either plane, in bytes
    const uint32_t entry = a.slots.block.div((uint32_t)pos);
    uint32_t bad = 0;
    if (req < 0 || req >= a.slots.rows) {
        bad = KVC_FLAG_REQUEST;
    } else if (entry >= (uint32_t)a.slots.width) {
        bad = KVC_FLAG_POSITION;
    } else {
        const int32_t id = __ldg(a.slots.ids + (int64_t)req * a.slots.stride + entry);
        const int32_t off = pos - (int32_t)(entry * a.slots.block.d);
        if (id < 0 || id >= a.slots.num_blocks) {
            bad = KVC_FLAG_BLOCK;
        } else {
            slot_k = id * a.k_plane.block_stride + off * a.k_plane.token_stride;
            slot_v = id * a.v_plane.block_stride + off * a.v_plane.token_stride;
        }
    }
    if (bad != 0) {
        if (threadIdx.x == 0) atomicOr(a.flags, bad);
        return;
    }

    // keys and values
    {
        const int32_t units = a.dim / 16, groups = THREADS / units;
        const int32_t j = threadIdx.x % units, g = threadIdx.x / units;
        if (g < groups) {
            const Unit u = make_unit<INTERLEAVED>(a, a.dim, j, angles);
            Unit plain = u;
            plain.rotated = false;
            const int32_t rows = a.k.heads + a.v.heads;
            for (int32_t r0 = g; r0 < rows; r0 += groups * BATCH) {
                uint4 p0[BATCH], p1[BATCH];
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const int32_t r = r0 + b * groups;
                    if (r < rows) {
                        const bool key = r < a.k.heads;
                        const unsigned char *src =
                            key ? a.k.src + t * a.k.src_token + r * a.k.src_head
                                : a.v.src + t * a.v.src_token + (r - a.k.heads) * a.v.src_head;
                        p0[b] = load16(src + 2 * u.e0);
                        p1[b] = load16(src + 2 * u.e1);
                    }
                }
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const int32_t r = r0 + b * groups;
                    if (r < rows) {
                        const bool key = r < a.k.heads;
                        const int32_t h = key ? r : r - a.k.heads;
                        float x[16];
                        turn<F16, INTERLEAVED>(p0[b], p1[b], key ? u : plain, x);
                        unsigned char *dst =
                            key ? a.k_plane.base + slot_k + h * a.k_plane.head_stride
                                : a.v_plane.base + slot_v + h * a.v_plane.head_stride;
                        if (E4M3)
                            store_8bit(dst, u, x, 1.0f / __ldg((key ? a.k_scale : a.v_scale) + h));
                        else
                            store_16bit<F16>(dst, u, x);
                    }
                }
            }
        }
    }
    // queries
    if (a.q.heads > 0) {
        const int32_t units = a.q_dim / 16, groups = THREADS / units;
        const int32_t j = threadIdx.x % units, g = threadIdx.x / units;
        if (g >= groups) return;
        const Unit u = make_unit<INTERLEAVED>(a, a.q_dim, j, angles);
        for (int32_t r0 = g; r0 < a.q.heads; r0 += groups * BATCH) {
            uint4 p0[BATCH], p1[BATCH];
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int32_t r = r0 + b * groups;
                if (r < a.q.heads) {
                    const unsigned char *src = a.q.src + t * a.q.src_token + r * a.q.src_head;
                    p0[b] = load16(src + 2 * u.e0);
                    p1[b] = load16(src + 2 * u.e1);
                }
            }
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                const int32_t r = r0 + b * groups;
                if (r < a.q.heads) {
                    float x[16];
                    turn<F16, INTERLEAVED>(p0[b], p1[b], u, x);
                    store_16bit<F16>(a.q_out + t * a.q_out_token + r * a.q_out_head, u, x);
                }
            }
        }
    }
}

template <bool F16, bool E4M3>
kvr_status go(const AppendArgs &a, bool interleaved, int32_t tokens, void *stream) {
    return kvc_launch(interleaved ? append_kernel<F16, true, E4M3> : append_kernel<F16, false, E4M3>,
                      a, dim3((unsigned)tokens), THREADS, 0, stream);
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
    a.flags = c->ws.flags;
    a.last = (p->flags & KVC_ROTATE_LAST) != 0;
    const bool il = (p->flags & KVC_INTERLEAVED) != 0, f16 = p->dtype == KVC_DTYPE_F16;
    if (c->d.dtype == KVR_DTYPE_FP8_E4M3)
        return f16 ? go<true, true>(a, il, p->num_tokens, stream)
                   : go<false, true>(a, il, p->num_tokens, stream);
    return f16 ? go<true, false>(a, il, p->num_tokens, stream)
               : go<false, false>(a, il, p->num_tokens, stream);
}
