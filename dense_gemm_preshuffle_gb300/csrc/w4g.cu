// Products with 4-bit group-scaled weights: the choice of kernel, and a packed
// buffer as the streaming kernel's operand or the tile kernel's.
#include <cstdlib>

#include "stream.cuh"
#include "w4g.h"

namespace gp {

namespace {

// The tile kernel's units, and CTAs to each: a cluster where units are few and
// every CTA keeps 8 blocks of K or more.
struct Tiles {
  int rows, cluster;
  int64_t across, units;
};
Tiles tiles_of(const W4gArgs& a, int64_t kblocks, int num_sms) {
  Tiles t{};
  t.rows = a.M <= 32 ? 32 : 64;
  const int64_t width = a.U != nullptr ? 64 : 128;
  t.across = (a.N + width - 1) / width;
  t.units = t.across * ((a.M + t.rows - 1) / t.rows);
  t.cluster = 1;
  for (int c = 2; c <= kMaxCluster; ++c)
    if (t.units <= clusters_at_once(c, num_sms) && kblocks >= 8 * c) t.cluster = c;
  return t;
}

// Whether the tile kernel takes a call: never up to 16 rows of A (16 x 16384 x
// 8192, groups of 128: 26.4 us against the streaming kernel's 24.1); above, by
// a model of both.  Streaming: 3 us and the codes' bytes at the rate of one
// pass of 16 rows.  Tiles: 5 us, 1.5 us a unit and the time of 256 values of K
// by group size.  Measured, streaming and tiles: 32 x 16384 x 8192 42.8 and
// 30.5 us, 32 x 4096 x 4096 8.7 and 9.5, 64 x 7168 x 4096 24.5 and 15.3; a
// gated pair in groups of 64, 32 x 12000 x 10176, 96.3 and 85.4.
bool tile_choice(const W4gArgs& a, const W4gLayout& l, int num_sms) {
  static const int forced = [] {
    const char* e = std::getenv("GP_W4G_TILE");
    return (e == nullptr || *e == '\0') ? -1 : std::atoi(e);
  }();
  if (forced >= 0) return forced != 0;
  if (a.M <= 16) return false;
  const int g = a.group == 128 ? 0 : a.group == 64 ? 1 : 2;
  constexpr double kRate[3] = {2.6e6, 2.4e6, 1.8e6};                     // bytes / us
  constexpr double kStep[2][3] = {{0.8, 0.95, 1.6}, {1.03, 1.28, 2.5}};  // us
  const Tiles t = tiles_of(a, l.kblocks, num_sms);
  const double bytes = (a.U != nullptr ? 1.0 : 0.5) * (double)a.N * (double)a.K;
  const double stream_us = 3.0 + (double)((a.M + 15) / 16) * bytes / kRate[g];
  const double rounds = (double)((t.units * t.cluster + num_sms - 1) / num_sms);
  const double steps = (double)((l.kblocks + 1) / 2 + t.cluster - 1) / (double)t.cluster;
  return 5.0 + rounds * (1.5 + steps * kStep[t.rows == 64][g]) < stream_us;
}

int tile_launch(const W4gArgs& a, const W4gLayout& l, const HostContext& ctx, cudaStream_t stream) {
  W4gTileParams p{};
  p.C = static_cast<uint16_t*>(a.C);
  p.ldc = a.ldc;
  p.block_bytes = (int)l.block_bytes;
  p.kblocks = (int)l.kblocks;
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.gated = a.U != nullptr ? 1 : 0;
  const Tiles t = tiles_of(a, l.kblocks, ctx.num_sms);
  // more outputs than the memory holds; and steps are counted in 32 bits
  if (t.units > 0x10000000 || (t.units / ctx.num_sms + 1) * l.kblocks * 4 > 0x7FFFFFFF) return GP_ERR_SHAPE;
  p.tiles = (int)t.across;
  p.units = (int)t.units;
  p.cluster = t.cluster;
  p.act = a.act;
  p.has_zeros = a.has_zeros ? 1 : 0;
  p.scale_fp16 = a.scale_fp16 ? 1 : 0;
  p.b_constant = a.b_constant ? 1 : 0;
  p.status = ctx.status;
  p.wait_limit_ns = ctx.wait_limit_ns;
  p.debug_skip_load = take_debug_skip_load();
  W4gTileMaps maps;
  int rc = encode_map_2d(&maps.a, a.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.A,
                         (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.lda * 2, 64, (uint32_t)t.rows,
                         CU_TENSOR_MAP_SWIZZLE_128B);
  auto blocks = [&](CUtensorMap* map, const uint8_t* packed) {
    return encode_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_INT64, packed, (uint64_t)l.block_bytes / 8, (uint64_t)l.kblocks,
                         (uint64_t)l.row_tiles, (uint64_t)l.block_bytes, (uint64_t)(l.kblocks * l.block_bytes),
                         (uint32_t)l.block_bytes / 8, 2, 4, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  if (rc == GP_OK) rc = blocks(&maps.w, a.W);
  if (rc == GP_OK && p.gated) rc = blocks(&maps.u, a.U);
  if (rc != GP_OK) return rc;
  switch (a.group) {
    case 32: return w4g_tile_32(maps, p, t.rows, a.fp16, ctx.num_sms, stream);
    case 64: return w4g_tile_64(maps, p, t.rows, a.fp16, ctx.num_sms, stream);
    default: return w4g_tile_128(maps, p, t.rows, a.fp16, ctx.num_sms, stream);
  }
}

}  // namespace

int w4g_run_launch(const W4gArgs& a, const HostContext& ctx, cudaStream_t stream) {
  const W4gLayout l = w4g_layout(a.N, a.K, a.group, a.has_zeros);
  if (tile_choice(a, l, ctx.num_sms)) return tile_launch(a, l, ctx, stream);
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
