// The 4-bit products of one group size (one translation unit each).
#pragma once
#include "stream.cuh"
#include "w4g.h"

namespace gp {

namespace {

template <bool FP16, int GROUP, int NT>
int w4g_launch_nt(const StreamParams& p, bool gated, int num_sms, cudaStream_t stream) {
  using P = Packed4<FP16, GROUP>;
  // Two blocks an SM; 32 rows of A need more registers than that leaves for
  // two row tiles, and take one block with a deeper ring.
  constexpr int BLOCKS = NT == 4 ? 1 : 2, STAGES = NT == 4 ? 8 : 4;
  if (gated) return launch_stream<P, 2, 1, NT, STAGES, 8, BLOCKS>(p, num_sms, stream);
  if (w4g_two_tiles(p.row_tiles, num_sms)) return launch_stream<P, 1, 2, NT, STAGES, 8, BLOCKS>(p, num_sms, stream);
  return launch_stream<P, 1, 1, NT, STAGES, 8, BLOCKS>(p, num_sms, stream);
}

template <bool FP16, int GROUP>
int w4g_launch_type(const StreamParams& p, bool gated, int num_sms, cudaStream_t stream) {
  if (p.M <= 8) return w4g_launch_nt<FP16, GROUP, 1>(p, gated, num_sms, stream);
  if (p.M <= 16) return w4g_launch_nt<FP16, GROUP, 2>(p, gated, num_sms, stream);
  return w4g_launch_nt<FP16, GROUP, 4>(p, gated, num_sms, stream);
}

}  // namespace

}  // namespace gp
