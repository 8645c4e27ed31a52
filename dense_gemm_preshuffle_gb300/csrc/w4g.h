// Interface of the 4-bit products' translation units.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace gp {

struct StreamParams;

// Row tiles of 16 of a step (1, 2 or 4, at most `most`): what leaves the
// fewest row tiles to the block with most of them, where `slots` blocks are
// resident, and of equals the largest, whose steps share A's loads and sums.
inline int w4g_tiles_a_step(int row_tiles, int slots, int most) {
  int best = 1, fewest = 0x7fffffff;
  for (int r = 1; r <= most; r *= 2) {
    const int groups = (row_tiles + r - 1) / r;
    const int load = (groups + slots - 1) / slots * r;
    if (load <= fewest) best = r, fewest = load;
  }
  return best;
}

int w4g_launch_32(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_64(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_128(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);

}  // namespace gp
