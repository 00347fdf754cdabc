// The latent attention's instances of fp16 queries and an 8-bit cache.
#include "spec_latent_tile.h"

namespace sgg {

hipError_t launch_latent_fp16_e4m3(const LatentParams& p, const LatentShape& s,
                            hipStream_t stream) {
  return launch_latent<true, true>(p, s, stream);
}

}  // namespace sgg
