// The attention kernels for fp16 queries.
#include "spec_attention_tile.h"

namespace sgg {

hipError_t launch_attention_fp16(const AttnParams& p, const AttnShape& s, bool e4m3,
                                 hipStream_t stream) {
  return e4m3 ? launch_attention<true, true>(p, s, stream)
              : launch_attention<true, false>(p, s, stream);
}

}  // namespace sgg
