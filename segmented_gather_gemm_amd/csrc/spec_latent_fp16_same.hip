// The latent attention's instances of fp16 queries and a cache of the same type.
#include "spec_latent_tile.h"

namespace sgg {

hipError_t launch_latent_fp16_same(const LatentParams& p, const LatentShape& s,
                            hipStream_t stream) {
  return launch_latent<true, false>(p, s, stream);
}

}  // namespace sgg
