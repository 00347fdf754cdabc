// The attention kernels for fp16 queries and a cache of the same type.
#include "spec_attention_tile.h"

namespace sgg {

hipError_t launch_attention_fp16_same(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
  return launch_attention<true, false>(p, s, stream);
}

}  // namespace sgg
