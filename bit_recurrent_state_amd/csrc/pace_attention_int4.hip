// The attention kernels over an int4 cache (pace_attention.h).
#include "pace_attention.h"

namespace pace {

hipError_t launch_attention_int4(const AttnParams& p, const AttnPlan& plan, int d, int group, int io_bf16,
                                 hipStream_t stream) {
  return launch_attention_kind<PACE_CACHE_INT4>(p, plan, d, group, io_bf16, stream);
}

}  // namespace pace
