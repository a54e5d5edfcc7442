// cache_split.cuh -- how the attention kernels divide the keys of all requests among their parts.
//
// The units (a fixed number of keys) of all jobs form one line: request by request, job by job of
// a request (key heads, or passes of query rows), units of a job in the order of its keys. It is
// cut into parts, one a block or cluster: equal ones, which may end within a job and go on in the
// next; or, where that makes the longest part hardly longer, parts within jobs.
#pragma once

#include "cache.h"

namespace kvc {

// A request's keys that some of its newest tokens see: [first, n). What lies below is not read, and
// its block may be gone from the table. Tiles begin at `lo`, which may be a little before `first`.
struct Span {
    int32_t n, lo, first;
};

struct SplitArgs {
    KvcSlots slots;
    const int32_t *lengths;
    uint32_t *flags;
    int32_t requests, m, window;
};

// The first key that a query which sees the keys below `end` sees. (A window may be any positive
// int32 and `end` negative, for a token before a short request's first: their difference may not
// be taken as it is.)
__host__ __device__ __forceinline__ int32_t window_from(int32_t end, int32_t window) {
    return max(end, 0) - window;
}

// The keys of a request of n tokens, of which the newest m attend; `lo` is the multiple of `align`
// next below (1: the first key itself).
__host__ __device__ __forceinline__ Span span_of(int32_t n, int32_t m, int32_t window, int32_t align) {
    const int32_t first = window > 0 ? max(0, window_from(n - m + 1, window)) : 0;
    return {n, first / align * align, first};
}

// Request r's. A length out of range counts as the nearest in range.
__device__ __forceinline__ Span span_of(const SplitArgs &a, int32_t r, int32_t align,
                                        uint32_t *bad) {
    int32_t n = __ldg(a.lengths + r);
    const int32_t most = a.slots.width * (int32_t)a.slots.block.d;
    if (n < 0 || n > most) {
        *bad = KVC_FLAG_LENGTH;
        n = n < 0 ? 0 : most;
    }
    return span_of(n, a.m, a.window, align);
}

// prefix[r] = units of one job of each of the requests before r (at least one a request, so that
// a request without keys still has its outputs written). All threads of the block, a multiple of
// 32 of them; `scratch` holds one int a warp; ends with a barrier.
template <int UNIT>
__device__ __forceinline__ void unit_prefix(const SplitArgs &a, int32_t align, int32_t *prefix,
                                            int32_t *scratch) {
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    uint32_t bad = 0;
    const int32_t per = (a.requests + (int)blockDim.x - 1) / (int)blockDim.x;
    const int32_t r0 = min(a.requests, tid * per), r1 = min(a.requests, r0 + per);
    int32_t sum = 0;
    for (int32_t r = r0; r < r1; ++r) {
        const Span s = span_of(a, r, align, &bad);
        sum += max(1, (s.n - s.lo + UNIT - 1) / UNIT);
        prefix[r + 1] = sum;
    }
    if (bad != 0 && blockIdx.x == 0) atomicOr(a.flags, bad);
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int32_t y = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int32_t before = incl - sum;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    for (int32_t r = r0; r < r1; ++r) prefix[r + 1] += before;
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
}

// The line's cut into parts. A part has LEAST units at least, but in jobs that have fewer, as
// each costs its job a share of the join.
//
// Equal parts (group 0): the first `more` have one unit more than the others. Parts within jobs:
// a job of u units is cut into ceil(u / group) equal ones, with the smallest group that at most
// `most` parts come of whatever the lengths are: sum ceil(u / group) <= (total + jobs (group - 1)) /
// group <= most. (With room for more, the fewer that have LEAST units.) A change of job within a
// part costs the part a new start, as long as `slack` units take.
//
// (What the host knows of the divisors comes as multipliers: all this lies before a block's first
// load, and a division takes a hundred cycles.)
//
// LEAST of 1, 2, 4 and 8 (us, inputs not in L2): keys and values of 8 heads with 8 queries each, one request
// of 4096 keys 15.0, 14.8, 12.5, 13.9; its 4 newest tokens 30.8, 30.4, 24.7, 26.4; 16 requests of 512 keys 14.3,
// 14.4, 14.4, 11.8; one of 1024 9.6, 9.2, 9.8, 11.9; one request of 4096 latents with 16 heads 18.1, 17.1,
// 15.8, 16.6.
constexpr int32_t LEAST = 4;
constexpr int32_t AHEAD_MOST = 128;       // requests up to which parts may be within jobs

struct CutShape {
    int32_t requests, of_request, most, slack;   // of_request: jobs of a request
    KvrDiv by_jobs, by_most, by_rest;            // by of_request, most, and most - jobs
};
inline CutShape make_cut_shape(int32_t requests, int32_t of_request, int32_t most, int32_t slack) {
    const int64_t jobs = (int64_t)requests * of_request;
    return {requests, of_request, most, slack, kvr_make_div((uint32_t)of_request),
            kvr_make_div((uint32_t)most), kvr_make_div(jobs < most ? (uint32_t)(most - jobs) : 1u)};
}

struct Cut {
    int32_t total, parts, each, more, group;

    // The parts are counted later where group > 0.
    __host__ __device__ __forceinline__ Cut(int32_t total_, const CutShape &s) : total(total_) {
        const int32_t jobs = s.requests * s.of_request;
        parts = min(s.most, max(total / LEAST, jobs));
        each = parts == s.most ? (int32_t)s.by_most.div((uint32_t)total)
                               : (int32_t)((uint32_t)total / (uint32_t)parts);
        more = total - each * parts;
        group = 0;
        if (jobs > 1 && jobs < s.most && s.requests <= AHEAD_MOST && total > jobs * LEAST) {
            const int32_t g =
                max(LEAST, (int32_t)s.by_rest.div((uint32_t)(total - jobs + s.most - jobs - 1)));
            if (g <= each + s.slack) group = g;
        }
    }
    // parts that a job of so many units has
    __host__ __device__ __forceinline__ int32_t of_job(int32_t units) const {
        return group == LEAST ? max(1, units / LEAST)
                              : (int32_t)((uint32_t)(units + group - 1) / (uint32_t)group);
    }
    // equal parts: where part c begins, and the part that holds unit x
    __host__ __device__ __forceinline__ int32_t start(int32_t c) const { return c * each + min(c, more); }
    __host__ __device__ __forceinline__ int32_t part_of(int32_t x) const {
        const int32_t edge = more * (each + 1);
        return x < edge ? (int32_t)((uint32_t)x / (uint32_t)(each + 1))
                        : more + (int32_t)((uint32_t)(x - edge) / (uint32_t)max(each, 1));
    }
    // ahead[r]: parts of one job of each of the requests before r. By one warp; needs a barrier.
    __device__ __forceinline__ void count(const int32_t *prefix, int32_t requests, int32_t *ahead) const {
        const int lane = threadIdx.x % 32;
        constexpr int PER = AHEAD_MOST / 32;
        int32_t own[PER], sum = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int32_t r = lane * PER + k;
            own[k] = r < requests ? of_job(prefix[r + 1] - prefix[r]) : 0;
            sum += own[k];
        }
        int32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int32_t y = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += y;
        }
        int32_t before = incl - sum;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int32_t r = lane * PER + k;
            if (r <= requests) ahead[r] = before;
            before += own[k];
        }
        if (lane == 31 && requests == AHEAD_MOST) ahead[requests] = before;
    }
    // units [x, x_end) of part c, none if there is no such part; the request of x, or -1: unknown
    __host__ __device__ __forceinline__ int32_t units_of(int32_t c, const int32_t *prefix,
                                                         const int32_t *ahead, const CutShape &s,
                                                         int32_t *x, int32_t *x_end) const {
        *x = *x_end = 0;
        if (group == 0) {
            if (c < parts) *x = start(c), *x_end = start(c + 1);
            return -1;
        }
        if (c >= ahead[s.requests] * s.of_request) return -1;
        int32_t lo = 0, hi = s.requests - 1;
        const int32_t cj = (int32_t)s.by_jobs.div((uint32_t)c);
        while (lo < hi) {
            const int32_t mid = (lo + hi + 1) / 2;
            if (ahead[mid] <= cj) lo = mid; else hi = mid - 1;
        }
        const int32_t units = prefix[lo + 1] - prefix[lo], n = ahead[lo + 1] - ahead[lo];
        const int32_t at = c - ahead[lo] * s.of_request;
        const int32_t job = (int32_t)((uint32_t)at / (uint32_t)n), k = at - job * n;
        const int32_t size = (int32_t)((uint32_t)units / (uint32_t)n), rest = units - size * n;
        *x = prefix[lo] * s.of_request + job * units + k * size + min(k, rest);
        *x_end = *x + size + (k < rest ? 1 : 0);
        return lo;
    }
    // job `job` of request r, whose first unit and number of units are these: its first part, and
    // how many it has
    __host__ __device__ __forceinline__ void parts_of(int32_t r, int32_t job, int32_t first, int32_t units,
                                             const int32_t *ahead, const CutShape &s, int32_t *c0,
                                             int32_t *n) const {
        if (group == 0) {
            *c0 = part_of(first);
            *n = part_of(first + units - 1) - *c0 + 1;
        } else {
            *n = of_job(units);
            *c0 = ahead[r] * s.of_request + job * *n;
        }
    }
};

// What of the line a part does next: units [u0, u1) of job `job` (of `units`) of request r.
struct Segment {
    int32_t r, job, u0, u1, units;
    int32_t job_first;        // the job's first unit in the line
};
// `known`: the request of x, or -1.
__host__ __device__ __forceinline__ Segment segment_at(int32_t x, int32_t x_end, const int32_t *prefix,
                                                       const CutShape &shape, int32_t known = -1) {
    Segment s;
    int32_t lo = known < 0 ? 0 : known, hi = known < 0 ? shape.requests - 1 : known;
    const int32_t jobs = shape.of_request, xj = (int32_t)shape.by_jobs.div((uint32_t)x);
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) / 2;
        if (prefix[mid] <= xj) lo = mid; else hi = mid - 1;
    }
    s.r = lo;
    const int32_t first = prefix[lo];
    s.units = prefix[lo + 1] - first;
    const int32_t start = first * jobs;
    s.job = (int32_t)((uint32_t)(x - start) / (uint32_t)s.units);
    s.job_first = start + s.job * s.units;
    s.u0 = x - s.job_first;
    s.u1 = min(s.units, s.u0 + (x_end - x));
    return s;
}

}  // namespace kvc
