// 4-bit weights in groups of 32.
#include "w4g.h"
#include "w4g_run.cuh"

namespace gp {

int w4g_launch_32(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream) {
  return fp16 ? w4g_launch_type<true, 32>(p, gated, num_sms, stream)
              : w4g_launch_type<false, 32>(p, gated, num_sms, stream);
}

}  // namespace gp
