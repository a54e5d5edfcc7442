// cache_latent.h -- the launches of cache_latent.cu.
#pragma once

#include "cache.h"

kvr_status kvc_latent_launch(const kvc_cache *c, int32_t layer, const kvc_attend *a, void *stream);
kvr_status kvc_latent_setup(kvc_cache *c);
size_t kvc_latent_partial_bytes(int32_t sm_count);
