// cache_attend_scored_e2m1.cu -- the attention kernel's instances with capped or biased scores for one element type.
#include "cache_attend.cuh"

kvc::AttendPick kvc::attend_pick_scored_e2m1(int32_t D, int32_t M) {
    return attend_pick<KVC_DTYPE_E2M1, true>(D, M);
}
