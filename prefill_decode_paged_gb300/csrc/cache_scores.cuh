// cache_scores.cuh -- scores that are more than a scaled product: capped by a tanh, biased by the distance.
//
// All in powers of two, as the softmax takes them: y = scale log2(e) q.k becomes c tanh(y / c) with c = cap
// log2(e), and slope log2(e) (j - p) is added. tanh costs a polynomial, an exponential and a reciprocal a score; over 16
// and 8 bits attention hides them.
#pragma once

#include "cache.h"

namespace kvc {

struct Scoring {
    float cap, per_cap;       // cap log2(e) and its reciprocal; cap 0: none
    const float *slopes;      // [query heads]; NULL: none
};

inline Scoring make_scoring(const kvc_scoring *s) {
    const float log2e = 1.4426950408889634f;
    if (s == nullptr) return {0.0f, 0.0f, nullptr};
    const float c = s->cap * log2e;
    return {c, s->cap > 0.0f ? 1.0f / c : 0.0f, s->slopes};
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c tanh(v / c), within 2^-19 of itself. Below 0.3 the series of tanh up to u^9 (what is left out is 2^-24 of u there);
// above, 1 - 2 / (1 + e^2u), which would lose the small ones: the exponential's error, 2^-22 and 2^-23 for each unit of 2u, counts
// 2 e^2u / (1 + e^2u)^2 times, the reciprocal's, 2^-23, up to 1.3 times, and tanh is at least 0.29: in all 4.6 parts in 2^22, and
// one more for the constants' rounding. Infinities give +-c, NaN stays.
__device__ __forceinline__ float capped(float v, float c, float per_c) {
    const float u = v * per_c, w = u * u;
    float t = fmaf(w, 62.0f / 2835.0f, -17.0f / 315.0f);
    t = fmaf(w, t, 2.0f / 15.0f);
    t = fmaf(w, t, -1.0f / 3.0f);
    const float near = fmaf(u * w, t, u);
    const float far = fmaf(-2.0f, reciprocal(1.0f + ex2(u * 2.8853900817779268f)), 1.0f);
    return c * (fabsf(u) < 0.3f ? near : far);
}

// A query head's slope, in powers of two.
__device__ __forceinline__ float slope_of(const Scoring &s, int32_t head) {
    return s.slopes == nullptr ? 0.0f : __ldg(s.slopes + head) * 1.4426950408889634f;
}

// The score of a key `away` tokens from the query (0: the query's own, before it negative).
__device__ __forceinline__ float scored(float v, const Scoring &s, float slope, int32_t away) {
    if (s.cap > 0.0f) v = capped(v, s.cap, s.per_cap);
    if (s.slopes != nullptr) v = fmaf(slope, (float)away, v);
    return v;
}

}  // namespace kvc
