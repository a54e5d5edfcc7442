// cache_append_e2m1.cu -- new tokens' keys and values into a paged pool of 4 bits, positions rotated on the way.
//
// For each group of 16 neighbours y = x / s of a row: b = max(2^-9, E4M3(max |y| / 6)), codes E2M1(y / b), both
// divisions as products with the fp32 reciprocal (the header states each rounding). A thread takes 32 elements,
// two groups, so that it needs no other's maximum:
//   rotated, halves:      those at 16 i and 16 i + R / 2, which hold pairs 16 i .. 16 i + 15 as (a | b);
//   rotated, interleaved: those at 32 i and 32 i + 16, the same pairs side by side;
//   not rotated:          those at 32 i and 32 i + 16.
// One block does one token. Its input rows are asked for before the token's position is known; slot and angles
// are on their way meanwhile. Bound by HBM with many tokens (2 bytes read for 0.56 written), by launch, slot and
// angles, one after another, with few.
#include <algorithm>

#include "cache.h"

namespace {

using namespace kvc;

struct Rows {                 // head rows of one input
    const unsigned char *src;
    int64_t src_token, src_head;
    int32_t heads;
};

struct AppendArgs {
    Rows q, k, v;
    KvcPlane k_plane, v_plane;
    unsigned char *k_block_scales, *v_block_scales;
    unsigned char *q_out;
    int64_t q_out_token, q_out_head;
    const int32_t *requests, *positions, *angles;
    KvcSlots slots;
    const float *rotary;      // [rows][R]
    int32_t rotary_rows, R;
    int32_t dim, q_dim;
    const float *k_scale, *v_scale;
    uint32_t *flags;
    int32_t last;             // the rotated elements are the row's last
    KvrDiv units, q_units;    // of a key's and of a query's row
};

constexpr int MOST_THREADS = 256;

struct Unit {
    int32_t kind;             // 0 query, 1 key, 2 value, 3 none
    int32_t row;              // head row of its input
    int32_t e0, e1;           // its two groups' first elements
    int32_t pair;             // its first pair, -1 if it is not rotated
};

template <bool INTERLEAVED>
__device__ __forceinline__ Unit unit_of(const AppendArgs &a, int32_t t, int32_t n) {
    Unit u;
    const int32_t nq = a.q.heads * (int32_t)a.q_units.d;
    int32_t j, dim;
    if (t < nq) {
        u.kind = 0;
        u.row = (int32_t)a.q_units.div((uint32_t)t);
        j = t - u.row * (int32_t)a.q_units.d;
        dim = a.q_dim;
    } else {
        const int32_t i = t - nq;
        u.row = (int32_t)a.units.div((uint32_t)i);
        j = i - u.row * (int32_t)a.units.d;
        dim = a.dim;
        u.kind = u.row < a.k.heads ? 1 : 2;
        if (u.kind == 2) u.row -= a.k.heads;
        if (t >= n) u.kind = 3;
    }
    const int32_t first = a.last ? dim - a.R : 0, i = j - first / 32;   // which rotated unit, if it is one
    const bool rotated = u.kind != 2 && i >= 0 && i < a.R / 32;
    u.e0 = rotated ? first + (INTERLEAVED ? 32 * i : 16 * i) : 32 * j;
    u.e1 = u.e0 + (rotated && !INTERLEAVED ? a.R / 2 : 16);
    u.pair = rotated ? 16 * i : -1;
    return u;
}

__device__ __forceinline__ uint4 load16(const unsigned char *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Eight codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float *y, float by) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(__fmul_rn(y[0], by)), "f"(__fmul_rn(y[1], by)), "f"(__fmul_rn(y[2], by)),
          "f"(__fmul_rn(y[3], by)), "f"(__fmul_rn(y[4], by)), "f"(__fmul_rn(y[5], by)),
          "f"(__fmul_rn(y[6], by)), "f"(__fmul_rn(y[7], by)));
    return w;
}

// One group of 16: its codes and its block scale.
__device__ __forceinline__ void store_group(unsigned char *codes, unsigned char *scale, const float *x, float inv) {
    float y[16], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        y[i] = __fmul_rn(x[i], inv);
        top = max_nan(top, fabsf(y[i]));
    }
    unsigned short b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.0f), "f"(__fmul_rn(top, 1.0f / 6.0f)));
    b = b == 0 ? 1 : b;                                 // 2^-9
    const float by = 1.0f / widen2<true>(e4m3_to_f16x2(b)).x;
    *(uint2 *)codes = make_uint2(codes8(y, by), codes8(y + 8, by));
    *scale = (unsigned char)b;
}

template <bool F16>
__device__ __forceinline__ void store_16bit(unsigned char *to, const float *x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 o;
        o.x = narrow2<F16>(x[8 * i], x[8 * i + 1]), o.y = narrow2<F16>(x[8 * i + 2], x[8 * i + 3]);
        o.z = narrow2<F16>(x[8 * i + 4], x[8 * i + 5]), o.w = narrow2<F16>(x[8 * i + 6], x[8 * i + 7]);
        *(uint4 *)(to + 16 * i) = o;
    }
}

// x[0..15] the first group, x[16..31] the second, rotated in place.
template <bool F16, bool INTERLEAVED>
__device__ __forceinline__ void turn(const uint4 p[4], const Unit &u, const float *angles, int32_t R,
                                     float x[32]) {
    const uint32_t *w = (const uint32_t *)p;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float2 f = widen2<F16>(w[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
    if (u.pair < 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 c = __ldg((const float4 *)(angles + u.pair) + i);
        const float4 s = __ldg((const float4 *)(angles + R / 2 + u.pair) + i);
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = 4 * i + k;
            float &a = x[INTERLEAVED ? 2 * e : e], &b = x[INTERLEAVED ? 2 * e + 1 : e + 16];
            // (one rounding each, so that a value next to a border goes the same way everywhere)
            const float y = __fsub_rn(__fmul_rn(a, cs[k]), __fmul_rn(b, sn[k]));
            b = __fadd_rn(__fmul_rn(b, cs[k]), __fmul_rn(a, sn[k]));
            a = y;
        }
    }
}

template <bool F16, bool INTERLEAVED>
__global__ void __launch_bounds__(MOST_THREADS, 4) append_e2m1_kernel(AppendArgs a) {
    wait_for_previous();
    let_next_start();
    const int64_t token = blockIdx.x;
    const int32_t pos = __ldg(a.positions + token), req = __ldg(a.requests + token);
    const int32_t turned = a.angles != nullptr ? __ldg(a.angles + token) : pos;
    const int32_t n = a.q.heads * (int32_t)a.q_units.d + (a.k.heads + a.v.heads) * (int32_t)a.units.d;
    int64_t slot = -1;                       // the token's slot in a plane, in bytes of codes
    for (int32_t t = threadIdx.x; t < n; t += blockDim.x) {
        const Unit u = unit_of<INTERLEAVED>(a, t, n);
        const Rows &in = u.kind == 0 ? a.q : u.kind == 1 ? a.k : a.v;
        const unsigned char *src = in.src + token * in.src_token + u.row * in.src_head;
        const uint4 p[4] = {load16(src + 2 * u.e0), load16(src + 2 * u.e0 + 16), load16(src + 2 * u.e1),
                            load16(src + 2 * u.e1 + 16)};
        if (slot < 0) {
            if (pos < 0) return;
            const uint32_t entry = a.slots.block.div((uint32_t)pos);
            uint32_t bad = 0;
            if (req < 0 || req >= a.slots.rows) {
                bad = KVC_FLAG_REQUEST;
            } else if (entry >= (uint32_t)a.slots.width ||
                       (a.rotary != nullptr && (turned < 0 || turned >= a.rotary_rows))) {
                bad = KVC_FLAG_POSITION;
            } else {
                const int32_t id = __ldg(a.slots.ids + (int64_t)req * a.slots.stride + entry);
                const int32_t off = pos - (int32_t)(entry * a.slots.block.d);
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
        float x[32];
        turn<F16, INTERLEAVED>(p, u, a.rotary + (int64_t)turned * a.R, a.R, x);
        if (u.kind == 0) {
            unsigned char *to = a.q_out + token * a.q_out_token + u.row * a.q_out_head;
            store_16bit<F16>(to + 2 * u.e0, x);
            store_16bit<F16>(to + 2 * u.e1, x + 16);
        } else {
            const int64_t at = slot + u.row * a.k_plane.head_stride;
            unsigned char *codes = (u.kind == 1 ? a.k_plane : a.v_plane).base + at;
            unsigned char *scales = (u.kind == 1 ? a.k_block_scales : a.v_block_scales) + at / 8;
            const float inv = 1.0f / __ldg((u.kind == 1 ? a.k_scale : a.v_scale) + u.row);
            store_group(codes + u.e0 / 2, scales + u.e0 / 16, x, inv);
            store_group(codes + u.e1 / 2, scales + u.e1 / 16, x + 16, inv);
        }
    }
}

}  // namespace

kvr_status kvc_append_e2m1_launch(const kvc_cache *c, int32_t layer, const kvc_append *p, const int32_t *angles,
                                  void *stream) {
    AppendArgs a = {};
    const int32_t H = c->d.kv_heads;
    a.k = {(const unsigned char *)p->k, p->k_token_stride, p->k_head_stride, H};
    a.v = {(const unsigned char *)p->v, p->v_token_stride, p->v_head_stride, H};
    a.q = {(const unsigned char *)p->q, p->q_token_stride, p->q_head_stride, p->q_heads};
    a.k_plane = c->plane(layer, 0);
    a.v_plane = c->plane(layer, 1);
    a.k_block_scales = c->block_scales(layer, 0);
    a.v_block_scales = c->block_scales(layer, 1);
    a.k_scale = c->scale_of(layer, 0);
    a.v_scale = c->scale_of(layer, 1);
    a.q_out = (unsigned char *)p->q_out;
    a.q_out_token = p->q_out_token_stride;
    a.q_out_head = p->q_out_head_stride;
    a.requests = p->requests;
    a.positions = p->positions;
    a.angles = angles;
    a.slots = c->slots(p->table);
    a.rotary = p->rotary;
    a.rotary_rows = p->rotary_rows;
    a.R = p->rotary == nullptr ? 0 : p->rotary_dim;
    a.dim = c->d.head_dim;
    a.q_dim = p->q_dim;
    a.units = kvr_make_div((uint32_t)a.dim / 32);
    a.q_units = kvr_make_div(std::max(1u, (uint32_t)a.q_dim / 32));
    a.flags = c->ws.flags;
    a.last = (p->flags & KVC_ROTATE_LAST) != 0;
    const bool il = (p->flags & KVC_INTERLEAVED) != 0, f16 = p->dtype == KVC_DTYPE_F16;
    const int64_t n = (int64_t)p->q_heads * a.q_units.d + 2 * (int64_t)H * a.units.d;
    const int64_t rounds = (n + MOST_THREADS - 1) / MOST_THREADS;
    const int threads = (int)((n + 32 * rounds - 1) / (32 * rounds)) * 32;
    const auto kernel = f16 ? (il ? append_e2m1_kernel<true, true> : append_e2m1_kernel<true, false>)
                            : (il ? append_e2m1_kernel<false, true> : append_e2m1_kernel<false, false>);
    return kvc_launch(kernel, a, dim3((unsigned)p->num_tokens), threads, 0, stream);
}
