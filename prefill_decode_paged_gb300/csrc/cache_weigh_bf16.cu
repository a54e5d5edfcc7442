// cache_weigh_bf16.cu -- the instances of the kernel of weights for one element type of the pool.
#include "cache_weigh.cuh"

kvc::WeighPick kvc::weigh_pick_bf16(int32_t D, int32_t M) { return weigh_pick<KVR_DTYPE_BF16>(D, M); }
