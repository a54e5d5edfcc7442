// cache_weigh_f16.cu -- the instances of the kernel of weights for one element type of the pool.
#include "cache_weigh.cuh"

kvc::WeighPick kvc::weigh_pick_f16(int32_t D, int32_t M) { return weigh_pick<KVC_DTYPE_F16>(D, M); }
