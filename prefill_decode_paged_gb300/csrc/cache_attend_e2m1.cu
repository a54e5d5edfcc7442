// cache_attend_e2m1.cu -- the attention kernel's instances for one element type of the pool.
#include "cache_attend.cuh"

kvc::AttendPick kvc::attend_pick_e2m1(int32_t D, int32_t M) {
    return attend_pick<KVC_DTYPE_E2M1, false>(D, M);
}
