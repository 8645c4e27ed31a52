// The tile kernel of 4-bit weights in groups of 32.
#include "w4g_tile.cuh"

namespace gp {

int w4g_tile_32(const W4gTileMaps& maps, const W4gTileParams& p, int rows, bool fp16, int num_sms, cudaStream_t stream) {
  return tile_launch_group<32>(maps, p, rows, fp16, num_sms, stream);
}

}  // namespace gp
