// The offline preshuffle of 4-bit group-scaled weights and its inverse.  The
// layout, blocks of 16 rows x 128 K values in the order in which the kernel's
// lanes read them, is documented at gemm_preshuffle_w4g.
#include "kernels.h"

namespace gp {

W4gLayout w4g_layout(int64_t N, int64_t K, int group, bool has_zeros) {
  W4gLayout l{};
  l.row_tiles = (N + 63) / 64 * 4;
  l.kblocks = (K + 127) / 128;
  l.block_bytes = 1024 + (has_zeros ? 48 : 32) * (128 / group);
  l.bytes = l.row_tiles * l.kblocks * l.block_bytes;
  return l;
}

namespace {

__device__ __forceinline__ int64_t block_at(int64_t n, int64_t c, const W4gLayout& l) {
  return ((n >> 4) * l.kblocks + c) * l.block_bytes;
}

// Where the 32-bit word `w` of row n (its values 8w .. 8w + 7) sits, in bytes.
__device__ __forceinline__ int64_t word_at(int64_t n, int64_t w, const W4gLayout& l) {
  const int h = (int)(n >> 3) & 1, g = (int)n & 7, i = (int)(w >> 2) & 3, t = (int)w & 3;
  return block_at(n, w >> 4, l) + (h * 32 + 4 * g + t) * 16 + 4 * i;
}

// Which of a block's scales (and zero points) row n's group j has.
__device__ __forceinline__ int scale_in_block(int64_t n, int64_t j, int gpb) {
  const int h = (int)(n >> 3) & 1, g = (int)n & 7;
  return (g * gpb + (int)(j % gpb)) * 2 + h;
}

// Eight codes k0..k7 in the low-nibble-first order of a row -> the packed
// word's order, bits 0, 16, 4, 20, 8, 24, 12, 28: (word >> 4j) & 0x000F000F
// is then the pair (k2j, k2j+1), one in each half.
__device__ __forceinline__ uint32_t spread(uint32_t w) {
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    out |= ((w >> (8 * j)) & 0xFu) << (4 * j);
    out |= ((w >> (8 * j + 4)) & 0xFu) << (16 + 4 * j);
  }
  return out;
}

__device__ __forceinline__ uint32_t unspread(uint32_t w) {
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    out |= ((w >> (4 * j)) & 0xFu) << (8 * j);
    out |= ((w >> (16 + 4 * j)) & 0xFu) << (8 * j + 4);
  }
  return out;
}

// One thread per 8 codes of the padded matrix, then one per scale.
__global__ void w4g_pack_kernel(const uint32_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                                int64_t K, int group, W4gLayout l, uint8_t* packed) {
  const int64_t words = l.row_tiles * 16 * l.kblocks * 16;
  const int gpb = 128 / group;
  const int64_t groups = (K + group - 1) / group, pgroups = l.kblocks * gpb;
  const int64_t nscales = l.row_tiles * 16 * pgroups;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x < words + nscales; x += step) {
    if (x < words) {
      const int64_t n = x / (l.kblocks * 16), w = x % (l.kblocks * 16);
      const bool in = n < N && w * 8 < K;
      const uint32_t v = in ? spread(codes[n * (K / 8) + w]) : 0u;
      *reinterpret_cast<uint32_t*>(packed + word_at(n, w, l)) = v;
    } else {
      const int64_t y = x - words, n = y / pgroups, j = y % pgroups;
      const bool in = n < N && j < groups;
      uint8_t* block = packed + block_at(n, j / gpb, l) + 1024;
      const int i = scale_in_block(n, j, gpb);
      reinterpret_cast<uint16_t*>(block)[i] = in ? scales[n * groups + j] : (uint16_t)0;
      if (zeros != nullptr) block[32 * gpb + i] = in ? zeros[n * groups + j] : (uint8_t)0;
    }
  }
}

__global__ void w4g_unpack_kernel(const uint8_t* packed, int64_t N, int64_t K, int group, W4gLayout l,
                                  uint32_t* codes, uint16_t* scales, uint8_t* zeros) {
  const int64_t words = N * (K / 8);
  const int gpb = 128 / group;
  const int64_t groups = (K + group - 1) / group;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; x < words + N * groups; x += step) {
    if (x < words) {
      const int64_t n = x / (K / 8), w = x % (K / 8);
      codes[x] = unspread(*reinterpret_cast<const uint32_t*>(packed + word_at(n, w, l)));
    } else {
      const int64_t y = x - words, n = y / groups, j = y % groups;
      const uint8_t* block = packed + block_at(n, j / gpb, l) + 1024;
      const int i = scale_in_block(n, j, gpb);
      scales[y] = reinterpret_cast<const uint16_t*>(block)[i];
      if (zeros != nullptr) zeros[y] = block[32 * gpb + i];
    }
  }
}

int blocks_for(int64_t items) {
  const int64_t b = (items + 255) / 256;
  return (int)(b < 65536 ? b : 65536);
}

}  // namespace

int w4g_pack_launch(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t N, int64_t K,
                    int group, uint8_t* packed, cudaStream_t stream) {
  const W4gLayout l = w4g_layout(N, K, group, zeros != nullptr);
  const int64_t items = l.row_tiles * 16 * l.kblocks * (16 + 128 / group);
  w4g_pack_kernel<<<blocks_for(items), 256, 0, stream>>>(reinterpret_cast<const uint32_t*>(codes), scales, zeros, N, K,
                                                         group, l, packed);
  return cudaGetLastError() == cudaSuccess ? GP_OK : GP_ERR_CUDA;
}

int w4g_unpack_launch(const uint8_t* packed, int64_t N, int64_t K, int group, bool has_zeros, uint8_t* codes,
                      uint16_t* scales, uint8_t* zeros, cudaStream_t stream) {
  const W4gLayout l = w4g_layout(N, K, group, has_zeros);
  const int64_t items = N * (K / 8) + N * ((K + group - 1) / group);
  w4g_unpack_kernel<<<blocks_for(items), 256, 0, stream>>>(packed, N, K, group, l, reinterpret_cast<uint32_t*>(codes),
                                                           scales, zeros);
  return cudaGetLastError() == cudaSuccess ? GP_OK : GP_ERR_CUDA;
}

}  // namespace gp
