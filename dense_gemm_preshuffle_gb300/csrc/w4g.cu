// Products with 4-bit group-scaled weights: a packed buffer as the streaming
// kernel's operand.
#include "stream.cuh"
#include "w4g.h"

namespace gp {

int w4g_run_launch(const W4gArgs& a, const HostContext& ctx, cudaStream_t stream) {
  const W4gLayout l = w4g_layout(a.N, a.K, a.group, a.has_zeros);
  StreamParams p{};
  p.A = static_cast<const uint16_t*>(a.A);
  p.lda = a.lda;
  p.W[0] = a.W;
  p.W[1] = a.U;
  p.C = static_cast<uint16_t*>(a.C);
  p.ldc = a.ldc;
  p.block_bytes = (int)l.block_bytes;
  p.has_zeros = a.has_zeros ? 1 : 0;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.K = (int)a.K;
  p.steps = (int)l.kblocks;
  p.row_tiles = (int)((a.N + 15) / 16);
  p.act = a.act;
  p.scale_fp16 = a.scale_fp16 ? 1 : 0;
  p.b_constant = a.b_constant ? 1 : 0;
  const bool gated = a.U != nullptr;
  switch (a.group) {
    case 32: return w4g_launch_32(p, a.fp16, gated, ctx.num_sms, stream);
    case 64: return w4g_launch_64(p, a.fp16, gated, ctx.num_sms, stream);
    default: return w4g_launch_128(p, a.fp16, gated, ctx.num_sms, stream);
  }
}

}  // namespace gp
