// The gated products for a few tokens: the streaming kernel over the rows of
// G and U as they are.
#include "gated_pair.h"
#include "stream.cuh"

namespace gp {

namespace {

template <bool FP16, int NT>
int launch_nt(const StreamParams& p, int num_sms, cudaStream_t stream) {
  return launch_stream<Rows16<FP16, 2, 1, 8>, 2, 1, NT, 3, 8, 2>(p, num_sms, stream);
}

template <bool FP16>
int launch_type(const StreamParams& p, int num_sms, cudaStream_t stream) {
  if (p.M <= 8) return launch_nt<FP16, 1>(p, num_sms, stream);
  if (p.M <= 16) return launch_nt<FP16, 2>(p, num_sms, stream);
  return launch_nt<FP16, 4>(p, num_sms, stream);
}

}  // namespace

int gated_stream_launch(const GatedArgs& a, const HostContext& ctx, cudaStream_t stream) {
  StreamParams p{};
  p.A = static_cast<const uint16_t*>(a.A);
  p.lda = a.lda;
  p.W[0] = static_cast<const uint8_t*>(a.G);
  p.W[1] = static_cast<const uint8_t*>(a.U);
  p.ldw[0] = a.ldg;
  p.ldw[1] = a.ldu;
  p.C = static_cast<uint16_t*>(a.H);
  p.ldc = a.ldh;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.K = (int)a.K;
  constexpr int kStepK = Rows16<false, 2, 1, 8>::kStepK;
  p.steps = (int)((a.K + kStepK - 1) / kStepK);
  p.row_tiles = (int)((a.N + 15) / 16);
  p.act = a.act;
  p.b_constant = a.b_constant ? 1 : 0;
  return a.fp16 ? launch_type<true>(p, ctx.num_sms, stream) : launch_type<false>(p, ctx.num_sms, stream);
}

}  // namespace gp
