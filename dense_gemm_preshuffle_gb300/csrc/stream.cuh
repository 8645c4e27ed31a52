// Products of a few rows of A with weights that are streamed once:
//
//   C[m, n] = sum_k A[m, k] W[n, k],   or   act(A W^T) * (A U^T)
//
// for M up to a few dozen, where the time is that of reading the weights.
// The weights never pass through shared memory as tiles that warps share:
//   - A step is one warp's work on R tiles of 16 weight rows (of W, and with
//     MATS = 2 of U): every lane fetches, with 16-byte cp.async, exactly the
//     bytes that its own mma.sync fragments need, into a ring of its own in
//     shared memory, and reads only those back.  There are no barriers and
//     no producer: cp.async.wait_group orders a lane with itself, and STAGES
//     steps of every warp are in flight.
//   - The weights are the MMA's 16-row operand and A's rows its 8 columns
//     (NT such groups), so that M = 1..8 costs one MMA.  K is permuted alike
//     for both: lane t of a row's four takes 8 consecutive values, which are
//     the values 2t, 2t+1, 2t+8, 2t+9 of two MMAs.  The sum does not change.
//   - The warps of a block take a row tile's steps in turn; their sums meet in
//     shared memory in a fixed order.  Blocks are persistent over the tiles,
//     and the loads of the next tile are in flight while one is summed.
//   - A is read through L1, which keeps it from tile to tile.
// mma.sync, not tcgen05: at M <= 32 the arithmetic is a few percent of
// either's rate, and register fragments spare the weights two trips through
// shared memory.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gated_math.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace gp {

struct StreamParams {
  const uint16_t* A;
  int64_t lda;
  const uint8_t* W[2];       // packed 4-bit weights, or 16-bit rows
  int64_t ldw[2];            // 16-bit rows: elements
  uint16_t* C;
  int64_t ldc;
  int64_t scales, zeros;     // 4 bits: byte offsets of these regions; zeros 0: 8 throughout
  int M, N, K;
  int steps;                 // steps of a row tile
  int row_tiles;             // ceil(N / 16)
  int groups;                // ceil(row_tiles / R): a block's unit of rows
  int items;                 // groups * chunks of 8 * NT rows of A
  int act;
  int scale_fp16;
  int b_constant;
};

namespace {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  // bytes < 16: the rest is zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// d += a (16 rows x 16) . b (16 x 8), fp32 sums.
template <bool FP16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (FP16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight values of row m of A from k on, as four pairs; zeros past M or K.
template <bool CHECK_K>
__device__ __forceinline__ uint4 load_a8(const uint16_t* row, bool in, int k, int K) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (!in) return v;
  if (!CHECK_K || k + 8 <= K) {
    v = __ldg(reinterpret_cast<const uint4*>(row + k));
  } else if (k < K) {  // a row's last, short run of values
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < K) w[e / 2] |= (uint32_t)__ldg(row + k + e) << (16 * (e & 1));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

__device__ __forceinline__ float act_of(float v, int act) {
  switch (act) {
    case GP_ACT_RELU: return act_value<GP_ACT_RELU>(v);
    case GP_ACT_SILU: return act_value<GP_ACT_SILU>(v);
    default: return act_value<GP_ACT_GELU>(v);
  }
}

// ---------------------------------------------------------------- weights
// A policy fetches a lane's bytes of a step and multiplies them:
//   kStepK     K values of a step
//   kBytes     ring bytes of a step and row tile
//   Extra      what a step needs besides the ring, loaded one step ahead
//   fetch / extra / multiply

// 16-bit rows as the caller has them: row g and row g + 8 of a tile, 16
// bytes a lane and half step of 32 values.
template <bool FP16_>
struct Rows16 {
  static constexpr bool FP16 = FP16_;
  static constexpr int kHalves = 2;
  static constexpr int kStepK = 32 * kHalves;
  static constexpr int kBytes = 1024 * kHalves;
  static constexpr bool kCheckK = true;
  struct Extra {};

  static __device__ __forceinline__ void fetch(const StreamParams& p, int mat, int tile, int step, uint32_t dst,
                                               int lane) {
    const int64_t n = (int64_t)tile * 16 + (lane >> 2);
#pragma unroll
    for (int i = 0; i < kHalves; ++i) {
      const int k = step * kStepK + i * 32 + (lane & 3) * 8;
      const int left = min(max(p.K - k, 0), 8) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t row = n + 8 * h;
        const bool in = row < p.N && left > 0;
        const uint8_t* src = p.W[mat] + (in ? (row * p.ldw[mat] + k) * 2 : 0);
        cp_async16(dst + (uint32_t)(((i * 2 + h) * 32 + lane) * 16), src, in ? left : 0);
      }
    }
  }
  static __device__ __forceinline__ Extra extra(const StreamParams&, int, int, int, int) { return {}; }

  template <int TILES, int NT>
  static __device__ __forceinline__ void multiply(const StreamParams& p, const uint16_t* const (&row)[NT],
                                                  const bool (&in)[NT], int step, uint32_t src, int lane,
                                                  const Extra (&)[TILES], float (&sum)[TILES][NT][4]) {
#pragma unroll
    for (int i = 0; i < kHalves; ++i) {
      uint4 x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[t] = load_a8<true>(row[t], in[t], step * kStepK + i * 32 + (lane & 3) * 8, p.K);
#pragma unroll
      for (int r = 0; r < TILES; ++r) {
        const uint32_t at = src + (uint32_t)(r * kBytes + (i * 64 + lane) * 16);
        const uint4 w0 = lds128(at), w1 = lds128(at + 512);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816<FP16>(sum[r][t], w0.x, w1.x, w0.y, w1.y, x[t].x, x[t].y);
          mma16816<FP16>(sum[r][t], w0.z, w1.z, w0.w, w1.w, x[t].z, x[t].w);
        }
      }
    }
  }
};

// 4-bit weights in blocks of 16 rows x 128 values, as packed.  A code becomes
// a 16-bit float without arithmetic:
//   fp16: the subnormal q 2^-24, so the sums are scaled by 2^24;
//   bf16: 128 + q, the low bits of 128's fraction.
// W = (q - z) s, so a group's sum is s (sum q a - z sum a), with 128 added
// to z for bf16.  The sums of a come from one more MMA, by a matrix of ones,
// and serve every row tile of the step.
template <bool FP16_, int GROUP>
struct Packed4 {
  static constexpr bool FP16 = FP16_;
  static constexpr int kStepK = 128;
  static constexpr int kBytes = 1024;
  static constexpr int kGroups = 128 / GROUP;  // groups of a block
  struct Extra {
    uint32_t scale[kGroups];  // rows g (low) and g + 8
    uint32_t zero[(kGroups + 1) / 2];  // two bytes a group
  };

  static __device__ __forceinline__ void fetch(const StreamParams& p, int mat, int tile, int step, uint32_t dst,
                                               int lane) {
    const bool in = tile < p.row_tiles;
    const uint8_t* src = p.W[mat] + (in ? ((int64_t)tile * p.steps + step) * 1024 + lane * 16 : 0);
    cp_async16(dst + (uint32_t)(lane * 16), src, in ? 16 : 0);
    cp_async16(dst + (uint32_t)(512 + lane * 16), src + (in ? 512 : 0), in ? 16 : 0);
  }

  static __device__ __forceinline__ Extra extra(const StreamParams& p, int mat, int tile, int step, int lane) {
    Extra e{};
    if (tile >= p.row_tiles) return e;
    const int64_t at = (((int64_t)tile * p.steps + step) * 8 + (lane >> 2)) * kGroups * 2;  // first of the rows' scales
    const uint8_t* s = p.W[mat] + p.scales + at * 2;
    if constexpr (kGroups == 1) {
      e.scale[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
    } else if constexpr (kGroups == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
      e.scale[0] = v.x, e.scale[1] = v.y;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
      e.scale[0] = v.x, e.scale[1] = v.y, e.scale[2] = v.z, e.scale[3] = v.w;
    }
    if (p.zeros != 0) {
      const uint8_t* z = p.W[mat] + p.zeros + at;
      if constexpr (kGroups == 1) {
        e.zero[0] = __ldg(reinterpret_cast<const uint16_t*>(z));
      } else if constexpr (kGroups == 2) {
        e.zero[0] = __ldg(reinterpret_cast<const uint32_t*>(z));
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(z));
        e.zero[0] = v.x, e.zero[1] = v.y;
      }
    }
    return e;
  }

  template <int SHIFT>
  static __device__ __forceinline__ uint32_t pair(uint32_t w) {
    constexpr uint32_t magic = FP16 ? 0u : 0x43004300u;
    return ((w >> SHIFT) & 0x000F000Fu) | magic;
  }

  static __device__ __forceinline__ float2 scales_of(uint32_t w, int scale_fp16) {
    if (scale_fp16) return __half22float2(*reinterpret_cast<__half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }

  template <int TILES, int NT>
  static __device__ __forceinline__ void multiply(const StreamParams& p, const uint16_t* const (&row)[NT],
                                                  const bool (&in)[NT], int step, uint32_t src, int lane,
                                                  const Extra (&extra)[TILES], float (&sum)[TILES][NT][4]) {
    constexpr uint32_t one = FP16 ? 0x3C003C00u : 0x3F803F80u;
    uint4 x[4][NT];
    auto load_x = [&](int i) {
#pragma unroll
      for (int t = 0; t < NT; ++t)  // K % 32 == 0: eight values are all inside or all outside
        x[i][t] = load_a8<false>(row[t], in[t] && step * 128 + i * 32 < p.K, step * 128 + i * 32 + (lane & 3) * 8, p.K);
    };
    constexpr int kAhead = NT <= 2 ? 4 : 1;  // all of the step's A at once, or one quarter ahead (registers)
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_x(i);
    uint32_t q[TILES][2][4];
#pragma unroll
    for (int r = 0; r < TILES; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 v = lds128(src + (uint32_t)(r * kBytes + h * 512 + lane * 16));
        q[r][h][0] = v.x, q[r][h][1] = v.y, q[r][h][2] = v.z, q[r][h][3] = v.w;
      }
    float acc[TILES][NT][4], sa[NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i + kAhead < 4) load_x(i + kAhead);
      if (i % (GROUP / 32) == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sa[t][e] = 0.0f;
#pragma unroll
            for (int r = 0; r < TILES; ++r) acc[r][t][e] = 0.0f;
          }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma16816<FP16>(sa[t], one, one, one, one, x[i][t].x, x[i][t].y);
        mma16816<FP16>(sa[t], one, one, one, one, x[i][t].z, x[i][t].w);
      }
#pragma unroll
      for (int r = 0; r < TILES; ++r) {
        const uint32_t w0 = q[r][0][i], w1 = q[r][1][i];
        const uint32_t a0 = pair<0>(w0), a1 = pair<0>(w1), a2 = pair<4>(w0), a3 = pair<4>(w1);
        const uint32_t b0 = pair<8>(w0), b1 = pair<8>(w1), b2 = pair<12>(w0), b3 = pair<12>(w1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          mma16816<FP16>(acc[r][t], a0, a1, a2, a3, x[i][t].x, x[i][t].y);
          mma16816<FP16>(acc[r][t], b0, b1, b2, b3, x[i][t].z, x[i][t].w);
        }
      }
      if ((i + 1) % (GROUP / 32) == 0) {
        const int j = i / (GROUP / 32);
#pragma unroll
        for (int r = 0; r < TILES; ++r) {
          const float2 s = scales_of(extra[r].scale[j], p.scale_fp16);
          float z0 = 8.0f, z1 = 8.0f;
          if (p.zeros != 0) {
            const uint32_t z = extra[r].zero[j / 2] >> (16 * (j & 1));
            z0 = (float)(z & 0xFFu);
            z1 = (float)((z >> 8) & 0xFFu);
          }
          if (!FP16) z0 += 128.0f, z1 += 128.0f;
          constexpr float unit = FP16 ? 16777216.0f : 1.0f;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float zz = e < 2 ? z0 : z1, ss = e < 2 ? s.x : s.y;
              const float v = FP16 ? fmaf(acc[r][t][e], unit, -zz * sa[t][e & 1]) : fmaf(-zz, sa[t][e & 1], acc[r][t][e]);
              sum[r][t][e] = fmaf(ss, v, sum[r][t][e]);
            }
        }
      }
    }
  }
};

// ---------------------------------------------------------------- kernel

template <class P, int MATS, int R, int NT, int STAGES>
struct StreamCfg {
  static constexpr int kTiles = MATS * R;
  static constexpr int kRowPitch = kTiles * 16 + 4;  // +4: a warp's fragment stores hit distinct banks
  static constexpr int kStepBytes = kTiles * P::kBytes;
  static constexpr int smem(int warps) {
    return warps * STAGES * kStepBytes + warps * 8 * NT * kRowPitch * 4;
  }
};

// BLOCKS: blocks that share an SM.
template <class P, int MATS, int R, int NT, int STAGES, int WARPS, int BLOCKS>
__global__ void __launch_bounds__(32 * WARPS, BLOCKS) stream_kernel(StreamParams p) {
  using C = StreamCfg<P, MATS, R, NT, STAGES>;
  constexpr int TILES = C::kTiles;
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem + WARPS * STAGES * C::kStepBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * STAGES * C::kStepBytes);

  // The load cursor runs STAGES - 1 steps ahead of the compute cursor, across items.
  int l_item = (int)blockIdx.x, l_tile = l_item % p.groups * R;
  int l_step = warp, l_slot = 0;
  const bool works = warp < p.steps;
  auto fetch_next = [&]() {
    if (works && l_item < p.items) {
#pragma unroll
      for (int a = 0; a < MATS; ++a)
#pragma unroll
        for (int r = 0; r < R; ++r)
          P::fetch(p, a, l_tile + r, l_step, ring + (uint32_t)(l_slot * C::kStepBytes + (a * R + r) * P::kBytes), lane);
      l_step += WARPS;
      if (l_step >= p.steps) {
        l_step = warp;
        l_item += (int)gridDim.x;
        l_tile = l_item % p.groups * R;
      }
      if (++l_slot == STAGES) l_slot = 0;
    }
    cp_async_commit();
  };
  auto extras = [&](int tile, int step, typename P::Extra (&e)[TILES]) {
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int r = 0; r < R; ++r) e[a * R + r] = P::extra(p, a, tile + r, step, lane);
  };

  if (!p.b_constant) {
    pdl_launch_dependents();
    pdl_wait();
  }
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch_next();
  typename P::Extra ahead[TILES];
  const int l_first = (int)blockIdx.x % p.groups * R;
  if (works && (int)blockIdx.x < p.items) extras(l_first, warp, ahead);
  if (p.b_constant) {  // the weights are on their way; A may be the previous kernel's output
    pdl_launch_dependents();
    pdl_wait();
  }

  int slot = 0;
  for (int item = (int)blockIdx.x; item < p.items; item += (int)gridDim.x) {
    const int group = item % p.groups;
    const int m0 = item / p.groups * (8 * NT);
    const int next_item = item + (int)gridDim.x;
    const int next_tile = next_item < p.items ? next_item % p.groups * R : -1;
    const uint16_t* row[NT];
    bool in[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int m = m0 + t * 8 + (lane >> 2);
      in[t] = m < p.M;
      row[t] = p.A + (int64_t)(in[t] ? m : 0) * p.lda;
    }
    float sum[TILES][NT][4];
#pragma unroll
    for (int r = 0; r < TILES; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[r][t][e] = 0.0f;

    for (int step = warp; step < p.steps; step += WARPS) {
      typename P::Extra now[TILES];
#pragma unroll
      for (int r = 0; r < TILES; ++r) now[r] = ahead[r];
      const bool last = step + WARPS >= p.steps;
      const int tile = last ? next_tile : group * R;
      if (tile >= 0) extras(tile, last ? warp : step + WARPS, ahead);
      cp_async_wait<STAGES - 2>();
      P::template multiply<TILES, NT>(p, row, in, step, ring + (uint32_t)(slot * C::kStepBytes), lane, now, sum);
      fetch_next();  // into the slot that the step before this one read
      if (++slot == STAGES) slot = 0;
    }

    // The warps' sums, [warp][row of A][weight row], added in warp order.
    float* mine = red + warp * 8 * NT * C::kRowPitch;
#pragma unroll
    for (int r = 0; r < TILES; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(t * 8 + 2 * (lane & 3) + (e & 1)) * C::kRowPitch + r * 16 + (lane >> 2) + 8 * (e >> 1)] = sum[r][t][e];
    __syncthreads();
    const int live = min(8 * NT, p.M - m0);
    const int used = min(WARPS, p.steps);  // warps past that hold zeros
    for (int x = threadIdx.x; x < live * R * 16; x += 32 * WARPS) {
      const int m = x / (R * 16), n = x % (R * 16);
      float v[MATS];
#pragma unroll
      for (int a = 0; a < MATS; ++a) {
        v[a] = 0.0f;
        for (int w = 0; w < used; ++w) v[a] += red[(w * 8 * NT + m) * C::kRowPitch + a * R * 16 + n];
      }
      const float out = MATS == 2 ? act_of(v[0], p.act) * v[MATS - 1] : v[0];
      const int64_t col = (int64_t)group * (R * 16) + n;
      if (col < p.N)
        p.C[(int64_t)(m0 + m) * p.ldc + col] = P::FP16 ? __half_as_ushort(__float2half_rn(out))
                                                       : __bfloat16_as_ushort(__float2bfloat16_rn(out));
    }
    __syncthreads();  // before the next item's sums replace these
  }
  cp_async_wait<0>();
}

template <class P, int MATS, int R, int NT, int STAGES, int WARPS, int BLOCKS>
int launch_stream(StreamParams p, int num_sms, cudaStream_t stream) {
  using C = StreamCfg<P, MATS, R, NT, STAGES>;
  auto kern = stream_kernel<P, MATS, R, NT, STAGES, WARPS, BLOCKS>;
  static std::atomic<bool> attr_set[64];
  if (const int rc = smem_attr_once(attr_set, kern, C::smem(WARPS)); rc != GP_OK) return rc;
  p.groups = (p.row_tiles + R - 1) / R;
  const int64_t items = p.groups * (((int64_t)p.M + 8 * NT - 1) / (8 * NT));
  if (items > 0x40000000) return GP_ERR_SHAPE;  // more outputs than the memory holds
  p.items = (int)items;
  const int slots = BLOCKS * num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.items < slots ? p.items : slots));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = C::smem(WARPS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return GP_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? GP_OK : GP_ERR_CUDA;
}

}  // namespace

}  // namespace gp
