// Interface of the 4-bit products' translation units.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace gp {

struct StreamParams;

int w4g_launch_32(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_64(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_128(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);

}  // namespace gp
