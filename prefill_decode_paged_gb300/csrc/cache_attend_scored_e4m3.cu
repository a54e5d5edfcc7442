// cache_attend_scored_e4m3.cu -- the attention kernel's instances with capped or biased scores for one element type.
#include "cache_attend.cuh"

kvc::AttendPick kvc::attend_pick_scored_e4m3(int32_t D, int32_t M) {
    return attend_pick<KVR_DTYPE_FP8_E4M3, true>(D, M);
}
