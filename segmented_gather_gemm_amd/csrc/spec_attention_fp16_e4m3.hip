// The attention kernels for fp16 queries and an 8-bit cache.
#include "spec_attention_tile.h"

namespace sgg {

hipError_t launch_attention_fp16_e4m3(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
  return launch_attention<true, true>(p, s, stream);
}

}  // namespace sgg
