// Gated feed-forward products H = act(A G^T) * (A U^T) and their gradients:
// the choice of kernels, their tensor maps and the workspace.
#include "gated_pair.h"

namespace gp {

namespace {

// The sizes that decide how the work is split are taken for this many SM
// pairs (a GB300 has 152 SMs), so that the workspace's size is known on the
// host without a device.
constexpr int kPairs = 76;

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t cdiv(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Parts of a reduction of `ksteps` steps for a product of `tiles` 256 x 256
// tiles (`outputs` matrices of rows x cols): the fewest microseconds by a
// simple model.  A step of a tile takes 0.28 us when the tensor cores are
// busy, a tile about 8 steps to fill and drain, and summing the parts writes
// and reads them at about 5 TB/s behind one more launch.
int parts_of(int64_t tiles, int64_t ksteps, int64_t outputs, int64_t rows, int64_t cols) {
  int best = 1;
  double best_us = 0;
  for (int s = 1; s <= 16 && s * 4 <= ksteps; ++s) {
    const double waves = (double)cdiv(tiles * s, kPairs);
    double us = waves * 0.28 * (double)(cdiv(ksteps, s) + 8);
    if (s > 1) us += 3.0 + (double)s * (double)(outputs * rows * cols) * 8.0 / 5.0e6;
    if (s == 1 || us < best_us) {
      best = s;
      best_us = us;
    }
  }
  return best;
}

int input_parts(int64_t M, int64_t N, int64_t K) {
  return parts_of(cdiv(M, 256) * cdiv(K, 256), 2 * cdiv(N, 64), 1, M, K);
}
int weight_parts(int64_t M, int64_t N, int64_t K) {
  return parts_of(2 * cdiv(N, 256) * cdiv(K, 256), cdiv(M, 64), 2, N, K);
}

// dg | du | fp32 parts
struct Workspace {
  int64_t pitch;         // of dg and du, in elements
  int64_t part_pitch;    // of the fp32 parts
  int64_t du, partial, bytes;
};
Workspace workspace_of(int64_t M, int64_t N, int64_t K) {
  Workspace w{};
  w.pitch = round_up(N, 8);
  w.part_pitch = round_up(K, 4);
  w.du = M * w.pitch * 2;
  w.partial = 2 * w.du;
  const int64_t ip = input_parts(M, N, K), wp = weight_parts(M, N, K);
  const int64_t in = ip > 1 ? ip * M : 0, wt = wp > 1 ? 2 * wp * N : 0;
  w.bytes = w.partial + (in > wt ? in : wt) * w.part_pitch * 4;
  return w;
}

struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
};

int map16(CUtensorMap* map, const Matrix& m, bool fp16, uint32_t box_rows) {
  return encode_map_2d(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, m.p,
                       (uint64_t)m.cols, (uint64_t)m.rows, (uint64_t)m.ld * 2, 64, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// One of the caller's outputs: the map ends at the last multiple of 8
// columns, the rest is the kernel's own stores (see gated_pair.cu).
int map_output(GatedMaps& maps, GatedPairParams& p, int i, const Matrix& m, bool fp16) {
  const int64_t whole = m.cols / 8 * 8;
  p.out[i] = static_cast<uint16_t*>(const_cast<void*>(m.p));
  p.ld[i] = m.ld;
  p.tail = (int)whole;
  return map16(&maps.c[i], {m.p, m.rows, whole > 0 ? whole : 8, m.ld}, fp16, 32);
}

// M tiles per group of the tile order: all of them while the group's rows of
// the left operand stay within a third of L2, else 16 (as for gemm_run).
int raster(int64_t tiles_m, int64_t row_bytes, int64_t l2_bytes) {
  if (tiles_m > kRasterG && tiles_m * 256 * row_bytes <= l2_bytes / 3) return (int)tiles_m;
  return kRasterG;
}

GatedPairParams params_of(const GatedArgs& a, const HostContext& ctx) {
  GatedPairParams p{};
  p.status = ctx.status;
  p.wait_limit_ns = ctx.wait_limit_ns;
  p.act = a.act;
  p.fp16 = a.fp16 ? 1 : 0;
  p.parts = 1;
  p.debug_skip_load = take_debug_skip_load();
  return p;
}

int set_tiles(GatedPairParams& p, int64_t outputs, int64_t rows, int64_t cols, int64_t tile_cols, int64_t ksteps) {
  const int64_t tm = cdiv(rows, 256), tn = cdiv(cols, tile_cols);
  const int64_t total = tm * tn * outputs * p.parts;
  if (total >= (int64_t(1) << 31)) return GP_ERR_SHAPE;
  p.rows = (int)rows;
  p.cols = (int)cols;
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.num_tiles = (int)total;
  p.ksteps = (int)ksteps;
  return GP_OK;
}

// FORWARD, or SLOPES where dH is given.
int products_launch(const GatedArgs& a, const HostContext& ctx, const Matrix& out0, const Matrix& out1,
                    cudaStream_t stream) {
  const int mode = a.dH != nullptr ? GATED_SLOPES : GATED_FORWARD;
  GatedMaps maps{};
  GatedPairParams p = params_of(a, ctx);
  p.b_constant = a.b_constant ? 1 : 0;
  int rc = set_tiles(p, 1, a.M, a.N, 128, cdiv(a.K, 64));
  if (rc != GP_OK) return rc;
  p.raster_g = raster(p.tiles_m, a.K * 2, ctx.l2_bytes);
  if ((rc = map16(&maps.a[0], {a.A, a.M, a.K, a.lda}, a.fp16, 128)) != GP_OK) return rc;
  if ((rc = map16(&maps.b[0], {a.G, a.N, a.K, a.ldg}, a.fp16, 128)) != GP_OK) return rc;
  if ((rc = map16(&maps.b[1], {a.U, a.N, a.K, a.ldu}, a.fp16, 128)) != GP_OK) return rc;
  if (mode == GATED_FORWARD) {
    if ((rc = map_output(maps, p, 0, out0, a.fp16)) != GP_OK) return rc;
  } else {  // into the workspace, whose rows are padded
    if ((rc = map16(&maps.c[0], out0, a.fp16, 32)) != GP_OK) return rc;
    if ((rc = map16(&maps.c[1], out1, a.fp16, 32)) != GP_OK) return rc;
    if ((rc = map16(&maps.dh, {a.dH, a.M, a.N, a.lddh}, a.fp16, 32)) != GP_OK) return rc;
  }
  return gated_pair_launch(mode, maps, p, ctx.num_sms, stream);
}

int map_parts(CUtensorMap* map, float* partial, int64_t slices, int64_t rows, int64_t cols, int64_t pitch) {
  return encode_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, partial, (uint64_t)cols, (uint64_t)rows,
                       (uint64_t)slices, (uint64_t)pitch * 4, (uint64_t)pitch * 4 * (uint64_t)rows, 32, 32, 1,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

size_t gated_workspace_bytes(int64_t M, int64_t N, int64_t K) { return (size_t)workspace_of(M, N, K).bytes; }

int gated_run_launch(const GatedArgs& a, const HostContext& ctx, cudaStream_t stream) {
  if (gated_stream_choice(a.M, a.N, a.K, ctx.num_sms)) return gated_stream_launch(a, a.H, nullptr, a.ldh, ctx, stream);
  return products_launch(a, ctx, {a.H, a.M, a.N, a.ldh}, {}, stream);
}

int gated_backward_launch(const GatedArgs& a, const HostContext& ctx, cudaStream_t stream) {
  const Workspace w = workspace_of(a.M, a.N, a.K);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const Matrix dg{ws, a.M, a.N, w.pitch}, du{ws + w.du, a.M, a.N, w.pitch};
  float* partial = reinterpret_cast<float*>(ws + w.partial);
  int rc = gated_stream_choice(a.M, a.N, a.K, ctx.num_sms)
               ? gated_stream_launch(a, ws, ws + w.du, w.pitch, ctx, stream)
               : products_launch(a, ctx, dg, du, stream);
  if (rc != GP_OK) return rc;
  if (a.dA != nullptr) {
    GatedMaps maps{};
    GatedPairParams p = params_of(a, ctx);
    p.parts = input_parts(a.M, a.N, a.K);
    p.ksteps_half = (int)cdiv(a.N, 64);
    if ((rc = set_tiles(p, 1, a.M, a.K, 256, 2 * cdiv(a.N, 64))) != GP_OK) return rc;
    p.raster_g = raster(p.tiles_m, a.N * 4, ctx.l2_bytes);
    if ((rc = map16(&maps.a[0], dg, a.fp16, 128)) != GP_OK) return rc;
    if ((rc = map16(&maps.a[1], du, a.fp16, 128)) != GP_OK) return rc;
    if ((rc = map16(&maps.b[0], {a.G, a.N, a.K, a.ldg}, a.fp16, 64)) != GP_OK) return rc;
    if ((rc = map16(&maps.b[1], {a.U, a.N, a.K, a.ldu}, a.fp16, 64)) != GP_OK) return rc;
    if ((rc = map_output(maps, p, 0, {a.dA, a.M, a.K, a.ldda}, a.fp16)) != GP_OK) return rc;
    if (p.parts > 1 && (rc = map_parts(&maps.partial, partial, p.parts, a.M, a.K, w.part_pitch)) != GP_OK) return rc;
    if ((rc = gated_pair_launch(GATED_INPUT, maps, p, ctx.num_sms, stream)) != GP_OK) return rc;
    if (p.parts > 1 && (rc = gated_add_parts_launch(partial, p.parts, 1, a.M, a.K, w.part_pitch, a.dA, a.ldda,
                                                    nullptr, 0, a.fp16, ctx.num_sms, stream)) != GP_OK)
      return rc;
  }
  if (a.dG != nullptr) {
    GatedMaps maps{};
    GatedPairParams p = params_of(a, ctx);
    p.parts = weight_parts(a.M, a.N, a.K);
    if ((rc = set_tiles(p, 2, a.N, a.K, 256, cdiv(a.M, 64))) != GP_OK) return rc;
    p.raster_g = raster(p.tiles_m, a.M * 2, ctx.l2_bytes);
    if ((rc = map16(&maps.a[0], dg, a.fp16, 64)) != GP_OK) return rc;
    if ((rc = map16(&maps.a[1], du, a.fp16, 64)) != GP_OK) return rc;
    if ((rc = map16(&maps.b[0], {a.A, a.M, a.K, a.lda}, a.fp16, 64)) != GP_OK) return rc;
    if ((rc = map_output(maps, p, 0, {a.dG, a.N, a.K, a.lddg}, a.fp16)) != GP_OK) return rc;
    if ((rc = map_output(maps, p, 1, {a.dU, a.N, a.K, a.lddu}, a.fp16)) != GP_OK) return rc;
    if (p.parts > 1 && (rc = map_parts(&maps.partial, partial, 2 * p.parts, a.N, a.K, w.part_pitch)) != GP_OK)
      return rc;
    if ((rc = gated_pair_launch(GATED_WEIGHTS, maps, p, ctx.num_sms, stream)) != GP_OK) return rc;
    if (p.parts > 1 && (rc = gated_add_parts_launch(partial, p.parts, 2, a.N, a.K, w.part_pitch, a.dG, a.lddg, a.dU,
                                                    a.lddu, a.fp16, ctx.num_sms, stream)) != GP_OK)
      return rc;
  }
  return GP_OK;
}

}  // namespace gp
