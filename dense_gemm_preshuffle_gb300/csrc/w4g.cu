// Products with 4-bit group-scaled weights: one warp per output column, each
// lane over its share of the packed words, fp32 sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gated_math.cuh"
#include "kernels.h"

namespace gp {

namespace {

__device__ __forceinline__ float load16(const uint16_t* p, bool fp16) {
  return fp16 ? __half2float(__ushort_as_half(*p)) : __bfloat162float(__ushort_as_bfloat16(*p));
}

__device__ float dot(const uint16_t* A, bool fp16, const uint8_t* packed, const W4gLayout& l, int64_t n, int64_t K,
                     int group, bool scale_fp16, bool has_zeros) {
  const int lane = threadIdx.x & 31;
  const int gpb = 128 / group;
  const int h = (int)(n >> 3) & 1, g = (int)n & 7;
  float sum = 0.0f;
  for (int64_t w = lane; w < K / 8; w += 32) {
    const int64_t block = (n >> 4) * l.kblocks + w / 16;
    const int b = (int)(w % 16);
    const uint32_t v = reinterpret_cast<const uint32_t*>(packed)[block * 256 + (h * 32 + 4 * g + b % 4) * 4 + b / 4];
    const int64_t at = (block * gpb + (b * 8) / group) * 16 + 2 * g + h;
    const float s = load16(reinterpret_cast<const uint16_t*>(packed + l.scales) + at, scale_fp16);
    const float z = has_zeros ? (float)packed[l.zeros + at] : 8.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int bit = 4 * (k / 2) + 16 * (k & 1);
      sum = fmaf(load16(A + w * 8 + k, fp16), ((float)((v >> bit) & 15u) - z) * s, sum);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

__global__ void w4g_kernel(W4gArgs a, W4gLayout l) {
  const int64_t n = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  if (n >= a.N) return;
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    const uint16_t* A = static_cast<const uint16_t*>(a.A) + m * a.lda;
    float v = dot(A, a.fp16, a.W, l, n, a.K, a.group, a.scale_fp16, a.has_zeros);
    if (a.U != nullptr) {
      const float u = dot(A, a.fp16, a.U, l, n, a.K, a.group, a.scale_fp16, a.has_zeros);
      v = u * (a.act == GP_ACT_RELU   ? act_value<GP_ACT_RELU>(v)
               : a.act == GP_ACT_SILU ? act_value<GP_ACT_SILU>(v)
                                      : act_value<GP_ACT_GELU>(v));
    }
    if (threadIdx.x % 32 == 0)
      static_cast<uint16_t*>(a.C)[m * a.ldc + n] =
          a.fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

}  // namespace

int w4g_run_launch(const W4gArgs& a, const HostContext&, cudaStream_t stream) {
  const W4gLayout l = w4g_layout(a.N, a.K, a.group, a.has_zeros);
  const dim3 grid((unsigned)((a.N + 7) / 8), (unsigned)(a.M < 65535 ? a.M : 65535));
  w4g_kernel<<<grid, 256, 0, stream>>>(a, l);
  return cudaGetLastError() == cudaSuccess ? GP_OK : GP_ERR_CUDA;
}

}  // namespace gp
