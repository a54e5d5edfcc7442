// cache_weigh_e4m3.cu -- the instances of the kernel of weights for one element type of the pool.
#include "cache_weigh.cuh"

kvc::WeighPick kvc::weigh_pick_e4m3(int32_t D, int32_t M) { return weigh_pick<KVR_DTYPE_FP8_E4M3>(D, M); }
