// share_check.cu -- test harness: which entries the threads of an eviction take, on the CPU.
//
// Includes the kernels' own header and compares with 64 bits, up to the largest numbers of entries and threads that
// the calls accept.
#include <stdio.h>

#include <algorithm>

#include "cache.h"

using namespace kvc;

int main() {
    const int64_t most = (int64_t)INT32_MAX - KVC_MAX_REQUESTS;
    // (blocks of a cluster; blocks that go into other blocks)
    const int64_t all[] = {256, 2048, 512, 4096, 128, 128 * 1024, 128 << 20, 1 << 30};
    int checked = 0;
    for (int64_t end : {(int64_t)0, (int64_t)1, (int64_t)5000, most / 3, most - 4096, most - 1, most})
        for (int64_t from : {(int64_t)0, end / 2, std::max<int64_t>(0, end - 5000), std::max<int64_t>(0, end - 1), end})
            for (int64_t threads : all)
                for (int64_t t : {(int64_t)0, (int64_t)1, threads / 2, most % threads, threads - 128, threads - 1}) {
                    int64_t want = from + t, got = 0;
                    Share s((int32_t)from, (int32_t)end, (int32_t)t, (int32_t)threads);
                    bool good = s.more() == (want < end);
                    // the first, and from a later one on the last few
                    if (s.more()) {
                        good = good && s.at() == want;
                        const int64_t skip = std::max<int64_t>(0, (end - 1 - want) / threads - 3);
                        want += skip * threads;
                        Share late((int32_t)(want - t), (int32_t)end, (int32_t)t, (int32_t)threads);
                        for (; late.more() && got < 10; late.next(), want += threads, ++got)
                            good = good && late.at() == want && want < end;
                        good = good && !late.more() && want >= end && got > 0;
                    }
                    if (!good) {
                        printf("from %lld end %lld thread %lld of %lld\n", (long long)from, (long long)end, (long long)t,
                               (long long)threads);
                        return 1;
                    }
                    ++checked;
                }
    printf("%d\n", checked);
    return 0;
}
