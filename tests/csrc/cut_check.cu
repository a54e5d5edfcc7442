// cut_check.cu -- test harness: how the attention kernels divide the keys, walked on the CPU.
//
// Includes the kernels' own header and walks every part of a launch as a block does, for random
// lengths: each unit of each job belongs to one part, parts are no more than the launch has blocks,
// and a job's parts are those that its join asks for.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "cache_split.cuh"

using namespace kvc;

#define REQUIRE(x)                                                              \
    do {                                                                        \
        if (!(x)) {                                                             \
            printf("%s: %d requests, %d jobs, %d blocks, slack %d\n", #x, requests, \
                   jobs, most, slack);                                          \
            return 1;                                                           \
        }                                                                       \
    } while (0)

int main() {
    std::mt19937 rng(5);
    auto pick = [&](std::vector<int> of) { return of[rng() % of.size()]; };
    int within = 0, across = 0;
    for (int trial = 0; trial < 4000; ++trial) {
        const int requests = trial % 5 == 0 ? pick({1, 127, 128, 129}) : 1 + (int)(rng() % 140);
        const int jobs = pick({1, 2, 3, 8}), most = pick({1, 2, 76, 152, 304});
        const int slack = pick({0, 8, 50}), longest = pick({1, 3, 20, 200, 3000});
        std::vector<int32_t> prefix(requests + 1, 0), ahead(requests + 1, 0);
        for (int r = 0; r < requests; ++r) prefix[r + 1] = prefix[r] + 1 + (int)(rng() % longest);
        const int32_t total = prefix[requests] * jobs;
        const CutShape shape = make_cut_shape(requests, jobs, most, slack);
        const Cut cut(total, shape);
        (cut.group > 0 ? within : across) += 1;
        if (cut.group > 0)
            for (int r = 0; r < requests; ++r) ahead[r + 1] = ahead[r] + cut.of_job(prefix[r + 1] - prefix[r]);
        REQUIRE(cut.group == 0 || ahead[requests] * jobs <= most);

        // the parts of every unit's job, as the blocks walk them
        std::vector<std::vector<int32_t>> parts((size_t)requests * jobs);
        int32_t at = 0;
        for (int32_t c = 0; c < most; ++c) {
            int32_t x, x_end;
            int32_t known = cut.units_of(c, prefix.data(), ahead.data(), shape, &x, &x_end);
            REQUIRE(x == at || x == x_end);
            int segments = 0;
            while (x < x_end) {
                const Segment s = segment_at(x, x_end, prefix.data(), shape, known);
                known = -1;
                REQUIRE(s.r >= 0 && s.r < requests && s.job >= 0 && s.job < jobs);
                REQUIRE(s.units == prefix[s.r + 1] - prefix[s.r]);
                REQUIRE(s.job_first == prefix[s.r] * jobs + s.job * s.units && s.job_first + s.u0 == x);
                REQUIRE(0 <= s.u0 && s.u0 < s.u1 && s.u1 <= s.units);
                REQUIRE(segments == 0 || s.u0 == 0);
                parts[(size_t)s.r * jobs + s.job].push_back(c);
                x += s.u1 - s.u0;
                at = x;
                ++segments;
            }
            REQUIRE(cut.group == 0 || segments <= 1);
        }
        REQUIRE(at == total);
        for (int r = 0; r < requests; ++r)
            for (int j = 0; j < jobs; ++j) {
                const int32_t units = prefix[r + 1] - prefix[r];
                int32_t c0, n;
                cut.parts_of(r, j, prefix[r] * jobs + j * units, units, ahead.data(), shape, &c0, &n);
                const std::vector<int32_t> &p = parts[(size_t)r * jobs + j];
                REQUIRE((int32_t)p.size() == n);
                for (int k = 0; k < n; ++k) REQUIRE(p[k] == c0 + k);
            }
    }
    printf("%d within, %d across\n", within, across);
    return within > 200 && across > 200 ? 0 : 1;
}
