// The attention kernels for bf16 queries and a cache of the same type.
#include "spec_attention_tile.h"

namespace sgg {

hipError_t launch_attention_bf16_same(const AttnParams& p, const AttnShape& s, hipStream_t stream) {
  return launch_attention<false, false>(p, s, stream);
}

}  // namespace sgg
