// cache_attend_scored_bf16.cu -- the attention kernel's instances with capped or biased scores for one element type.
#include "cache_attend.cuh"

kvc::AttendPick kvc::attend_pick_scored_bf16(int32_t D, int32_t M) {
    return attend_pick<KVR_DTYPE_BF16, true>(D, M);
}
