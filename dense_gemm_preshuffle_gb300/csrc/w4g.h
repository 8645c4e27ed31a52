// Interface of the 4-bit products' translation units.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace gp {

struct StreamParams;

// The tile kernel (w4g_tile.cuh): units of 128 rows of weights, or 64 of each
// of two matrices, with a number of rows of A.
struct W4gTileParams {
  uint16_t* C;
  int64_t ldc;
  int block_bytes, kblocks;  // of the packed matrices
  int M, N;
  int tiles, units;  // units: tiles * chunks of rows of A
  int cluster;       // CTAs that share a unit
  int gated, act, has_zeros, scale_fp16, b_constant;
  uint32_t* status;
  uint64_t wait_limit_ns;
  int debug_skip_load;
};

int w4g_launch_32(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_64(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);
int w4g_launch_128(const StreamParams& p, bool fp16, bool gated, int num_sms, cudaStream_t stream);

struct W4gTileMaps {
  CUtensorMap a;     // A: boxes of 64 values x `rows` rows (32 or 64) in the 128-byte swizzle
  CUtensorMap w, u;  // packed blocks as [row tile][block of K][block_bytes / 8] words of 8 bytes, four row tiles a box
};
int w4g_tile_32(const W4gTileMaps& maps, const W4gTileParams& p, int rows, bool fp16, int num_sms, cudaStream_t stream);
int w4g_tile_64(const W4gTileMaps& maps, const W4gTileParams& p, int rows, bool fp16, int num_sms, cudaStream_t stream);
int w4g_tile_128(const W4gTileMaps& maps, const W4gTileParams& p, int rows, bool fp16, int num_sms, cudaStream_t stream);

}  // namespace gp
