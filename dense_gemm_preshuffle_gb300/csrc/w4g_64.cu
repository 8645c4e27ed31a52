// 4-bit weights in groups of 64.
#include "w4g.h"
#include "w4g_run.cuh"

namespace gp {

int w4g_launch_64(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream) {
  return fp16 ? w4g_launch_type<true, 64>(p, gated, num_sms, stream)
              : w4g_launch_type<false, 64>(p, gated, num_sms, stream);
}

}  // namespace gp
