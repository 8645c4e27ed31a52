// Interface of the 4-bit products' translation units.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace gp {

struct StreamParams;

// Two row tiles of 16 a warp step, from the width on at which every
// resident block still gets several of them; else one.
inline bool w4g_two_tiles(int64_t row_tiles, int num_sms) { return row_tiles >= 8 * (int64_t)num_sms; }

int w4g_launch_32(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_64(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_128(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);

}  // namespace gp
