// The latent attention's instances of bf16 queries and an 8-bit cache.
#include "spec_latent_tile.h"

namespace sgg {

hipError_t launch_latent_bf16_e4m3(const LatentParams& p, const LatentShape& s,
                            hipStream_t stream) {
  return launch_latent<false, true>(p, s, stream);
}

}  // namespace sgg
