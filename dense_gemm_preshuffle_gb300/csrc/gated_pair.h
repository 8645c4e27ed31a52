// Interface of the gated block's tensor-core kernels (gated_pair.cu).
#pragma once
#include "kernels.h"

namespace gp {

enum GatedMode : int { GATED_FORWARD = 0, GATED_SLOPES = 1, GATED_INPUT = 2, GATED_WEIGHTS = 3 };

// Tensor maps of one launch; 128-byte swizzle throughout.  K-major operands
// have boxes of 64 x 128 rows, MN-major ones 64 x 64, 16-bit outputs (and dH)
// 64 x 32, fp32 parts 32 x 32 x 1.
struct GatedMaps {
  CUtensorMap a[2];     // INPUT: dg, du; WEIGHTS: dg, du (by output); else the activation
  CUtensorMap b[2];     // gate, up; WEIGHTS: the activation
  CUtensorMap c[2];     // the outputs
  CUtensorMap dh;       // SLOPES
  CUtensorMap partial;  // INPUT, WEIGHTS with parts > 1: [outputs * parts][rows][pitch] fp32
};

struct GatedPairParams {
  uint32_t* status;
  uint64_t wait_limit_ns;
  int rows, cols;        // of one output
  uint16_t* out[2];      // the outputs again, for the columns past the last multiple of 8:
  int64_t ld[2];         // a TMA store writes whole 16-byte units
  int tail;              // first of those columns, or cols where there are none
  int tiles_m, tiles_n;  // 256 rows x 128 (FORWARD, SLOPES) or 256 columns
  int num_tiles;         // outputs * parts * tiles_m * tiles_n
  int ksteps;            // reduction steps of 64
  int ksteps_half;       // INPUT: the steps of dg G, before those of du U
  int parts;             // parts of the reduction, each a tile of its own
  int raster_g;
  int act;
  int fp16;
  int b_constant;
  int debug_skip_load;
};

int gated_pair_launch(int mode, const GatedMaps& maps, const GatedPairParams& p, int num_sms, cudaStream_t stream);
// out = the sum of `parts` fp32 parts, for one or two outputs.
int gated_add_parts_launch(const float* partial, int parts, int outputs, int64_t rows, int64_t cols, int64_t pitch,
                           void* out0, int64_t ld0, void* out1, int64_t ld1, bool fp16, int num_sms,
                           cudaStream_t stream);
// FORWARD and SLOPES for few tokens or little work (gated_stream.cu): whether
// it takes them, and the launch, into out0 (and out1 for SLOPES) of pitch ld.
bool gated_stream_choice(int64_t M, int64_t N, int64_t K, int num_sms);
int gated_stream_launch(const GatedArgs& a, void* out0, void* out1, int64_t ld, const HostContext& ctx,
                        cudaStream_t stream);

}  // namespace gp
