// span_check.cu -- test harness: the keys that a request's newest tokens see, on the CPU.
//
// Includes the kernels' own header and compares with 64 bits, for lengths, numbers of newest tokens
// and windows up to the largest that the calls accept.
#include <stdio.h>

#include <algorithm>
#include <random>
#include <vector>

#include "cache_split.cuh"

using namespace kvc;

int main() {
    std::mt19937 rng(7);
    const int64_t longest = (int64_t)INT32_MAX - KVC_MAX_REQUESTS;
    std::vector<int64_t> lengths = {0, 1, 2, 3, 4, 5, 100, longest - 1, longest}, news = {1, 2, 4, 9, 4096},
                         windows = {1, 2, 1024, longest, INT32_MAX - 4096, INT32_MAX - 1, INT32_MAX};
    for (int k = 0; k < 60; ++k) {
        lengths.push_back(rng() % (longest + 1) >> rng() % 31);
        windows.push_back(1 + (rng() % INT32_MAX >> rng() % 31));
    }
    int checked = 0;
    for (int64_t n : lengths)
        for (int64_t m : news)
            for (int64_t w : windows)
                for (int64_t align : {1, 16, 32}) {
                    const int64_t first = std::max<int64_t>(0, n - m + 1 - w);
                    const Span s = span_of((int32_t)n, (int32_t)m, (int32_t)w, (int32_t)align);
                    bool good = s.n == n && s.first == first && s.lo == first / align * align;
                    // a query that sees a key: where its window begins
                    for (int64_t i = 0; i < m; i += m > 9 ? 511 : 1) {
                        const int64_t end = n - m + i + 1;
                        const int64_t from = window_from((int32_t)end, (int32_t)w);
                        good = good && (end <= 0 || from == end - w);
                    }
                    if (!good) {
                        printf("n %lld m %lld window %lld align %lld: lo %d\n", (long long)n, (long long)m,
                               (long long)w, (long long)align, s.lo);
                        return 1;
                    }
                    ++checked;
                }
    for (int64_t n : lengths) {
        const Span s = span_of((int32_t)n, 4, 0, 32);
        if (s.n != n || s.lo != 0 || s.first != 0) return 1;
    }
    printf("%d\n", checked);
    return 0;
}
