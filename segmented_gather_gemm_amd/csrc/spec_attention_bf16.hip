// The attention kernels for bf16 queries.
#include "spec_attention_tile.h"

namespace sgg {

hipError_t launch_attention_bf16(const AttnParams& p, const AttnShape& s, bool e4m3,
                                 hipStream_t stream) {
  return e4m3 ? launch_attention<false, true>(p, s, stream)
              : launch_attention<false, false>(p, s, stream);
}

}  // namespace sgg
