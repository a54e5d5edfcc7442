// cache_attend_f16.cu -- the attention kernel's instances for one element type of the pool.
#include "cache_attend.cuh"

kvc::AttendPick kvc::attend_pick_f16(int32_t D, int32_t M) {
    return attend_pick<KVC_DTYPE_F16>(D, M);
}
