// cache_attend_bf16.cu -- the attention kernel's instances for one element type of the pool.
#include "cache_attend.cuh"

kvc::AttendPick kvc::attend_pick_bf16(int32_t D, int32_t M) {
    return attend_pick<KVR_DTYPE_BF16, false>(D, M);
}
