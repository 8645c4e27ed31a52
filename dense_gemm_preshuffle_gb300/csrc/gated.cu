// Gated feed-forward products H = act(A G^T) * (A U^T) and their gradients:
// tiles of 32 x 32 outputs, fp32 sums, operands staged in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gated_math.cuh"
#include "kernels.h"

namespace gp {

namespace {

__device__ __forceinline__ float load16(const uint16_t* p, bool fp16) {
  return fp16 ? __half2float(__ushort_as_half(*p)) : __bfloat162float(__ushort_as_bfloat16(*p));
}
__device__ __forceinline__ uint16_t round16(float v, bool fp16) {
  return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ ActSlope act_of(float v, int act) {
  switch (act) {
    case GP_ACT_RELU: return act_slope<GP_ACT_RELU>(v);
    case GP_ACT_SILU: return act_slope<GP_ACT_SILU>(v);
    default: return act_slope<GP_ACT_GELU>(v);
  }
}

// A matrix read as element (row, k) at p[row * rs + k * ks].
struct View {
  const uint16_t* p;
  int64_t rs, ks;
};

// acc += sum_k P(r, k) Q(c, k) for this thread's (r, c) of a 32 x 32 tile.
__device__ float tile_sum(const View& P, const View& Q, int64_t r0, int64_t c0, int64_t rows, int64_t cols, int64_t K,
                          bool fp16, float acc) {
  __shared__ float sp[32][33], sq[32][33];
  const int tx = threadIdx.x, ty = threadIdx.y;
  for (int64_t k0 = 0; k0 < K; k0 += 32) {
    const int64_t k = k0 + tx;
    sp[ty][tx] = (r0 + ty < rows && k < K) ? load16(P.p + (r0 + ty) * P.rs + k * P.ks, fp16) : 0.0f;
    sq[ty][tx] = (c0 + ty < cols && k < K) ? load16(Q.p + (c0 + ty) * Q.rs + k * Q.ks, fp16) : 0.0f;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; ++i) acc = fmaf(sp[ty][i], sq[tx][i], acc);
    __syncthreads();
  }
  return acc;
}

// H, or (with dH) dg and du.
__global__ void gated_kernel(View A, View G, View U, const uint16_t* dH, int64_t lddh, uint16_t* H, uint16_t* H2,
                             int64_t ldh, int64_t M, int64_t N, int64_t K, int act, bool fp16) {
  const int64_t m0 = (int64_t)blockIdx.y * 32, n0 = (int64_t)blockIdx.x * 32;
  const float g = tile_sum(A, G, m0, n0, M, N, K, fp16, 0.0f);
  const float u = tile_sum(A, U, m0, n0, M, N, K, fp16, 0.0f);
  const int64_t m = m0 + threadIdx.y, n = n0 + threadIdx.x;
  if (m >= M || n >= N) return;
  const ActSlope s = act_of(g, act);
  if (dH == nullptr) {
    H[m * ldh + n] = round16(s.value * u, fp16);
  } else {
    const float d = load16(dH + m * lddh + n, fp16);
    H[m * ldh + n] = round16(d * u * s.slope, fp16);
    H2[m * ldh + n] = round16(d * s.value, fp16);
  }
}

// C[r, c] = sum_k P(r, k) Q(c, k) + sum_k P2(r, k) Q2(c, k)
__global__ void product_kernel(View P, View Q, View P2, View Q2, int64_t rows, int64_t cols, int64_t K, uint16_t* C,
                               int64_t ldc, bool fp16) {
  const int64_t r0 = (int64_t)blockIdx.y * 32, c0 = (int64_t)blockIdx.x * 32;
  float acc = tile_sum(P, Q, r0, c0, rows, cols, K, fp16, 0.0f);
  if (P2.p != nullptr) acc = tile_sum(P2, Q2, r0, c0, rows, cols, K, fp16, acc);
  const int64_t r = r0 + threadIdx.y, c = c0 + threadIdx.x;
  if (r < rows && c < cols) C[r * ldc + c] = round16(acc, fp16);
}

View view(const void* p, int64_t rs, int64_t ks) { return {static_cast<const uint16_t*>(p), rs, ks}; }

dim3 grid_of(int64_t rows, int64_t cols) { return dim3((unsigned)((cols + 31) / 32), (unsigned)((rows + 31) / 32)); }

int last_error() { return cudaGetLastError() == cudaSuccess ? GP_OK : GP_ERR_CUDA; }

int64_t pitch(int64_t n) { return (n + 7) / 8 * 8; }

}  // namespace

size_t gated_workspace_bytes(int64_t M, int64_t N, int64_t K) { return (size_t)(4 * M * pitch(N)); }

int gated_run_launch(const GatedArgs& a, const HostContext&, cudaStream_t stream) {
  gated_kernel<<<grid_of(a.M, a.N), dim3(32, 32), 0, stream>>>(
      view(a.A, a.lda, 1), view(a.G, a.ldg, 1), view(a.U, a.ldu, 1), nullptr, 0, static_cast<uint16_t*>(a.H), nullptr,
      a.ldh, a.M, a.N, a.K, a.act, a.fp16);
  return last_error();
}

int gated_backward_launch(const GatedArgs& a, const HostContext&, cudaStream_t stream) {
  const int64_t ldw = pitch(a.N);
  uint16_t* dg = static_cast<uint16_t*>(a.workspace);
  uint16_t* du = dg + a.M * ldw;
  gated_kernel<<<grid_of(a.M, a.N), dim3(32, 32), 0, stream>>>(
      view(a.A, a.lda, 1), view(a.G, a.ldg, 1), view(a.U, a.ldu, 1), static_cast<const uint16_t*>(a.dH), a.lddh, dg,
      du, ldw, a.M, a.N, a.K, a.act, a.fp16);
  if (a.dA != nullptr)
    product_kernel<<<grid_of(a.M, a.K), dim3(32, 32), 0, stream>>>(
        view(dg, ldw, 1), view(a.G, 1, a.ldg), view(du, ldw, 1), view(a.U, 1, a.ldu), a.M, a.K, a.N,
        static_cast<uint16_t*>(a.dA), a.ldda, a.fp16);
  if (a.dG != nullptr) {
    product_kernel<<<grid_of(a.N, a.K), dim3(32, 32), 0, stream>>>(view(dg, 1, ldw), view(a.A, 1, a.lda), View{},
                                                                    View{}, a.N, a.K, a.M,
                                                                    static_cast<uint16_t*>(a.dG), a.lddg, a.fp16);
    product_kernel<<<grid_of(a.N, a.K), dim3(32, 32), 0, stream>>>(view(du, 1, ldw), view(a.A, 1, a.lda), View{},
                                                                    View{}, a.N, a.K, a.M,
                                                                    static_cast<uint16_t*>(a.dU), a.lddu, a.fp16);
  }
  return last_error();
}

}  // namespace gp
