// cache_attend_e4m3.cu -- the attention kernel's instances for one element type of the pool.
#include "cache_attend.cuh"

kvc::AttendPick kvc::attend_pick_e4m3(int32_t D, int32_t M) {
    return attend_pick<KVR_DTYPE_FP8_E4M3, false>(D, M);
}
