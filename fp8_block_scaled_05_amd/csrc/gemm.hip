// Launchers of the block-scaled FP8 GEMM (kernel template in gemm_kernel.hpp).
//
// Tile shapes by problem shape (measured on MI355X with the dense, grouped and
// few-row workloads):
// - large M: 256x256 tiles, 8 waves of 128x64, two LDS stages (128 KB); the
//   large tile halves the L2->LDS traffic per flop compared with 128x256,
//   which matters more than the deeper pipeline a smaller tile would allow;
//   the same shape serves the grouped path.  When the dense raster would end
//   in a partial round of workgroups, its last tiles run as pairs of
//   128x256 tiles (a half-length last round); a group whose last tile-row
//   holds at most 128 rows runs that row as 128x256 tiles;
// - few rows (decode-like, weight-bandwidth bound): short tiles so that the
//   weight matrix is spread over many workgroups and every weight byte is
//   read once; 1 wave along M; four LDS stages (three K groups in flight).
//   E4M3 output (quantized per 128 output columns) needs tiles of whole
//   128-column groups, so it takes the 64x128 tile for every M <= 64.
// - M > 64 with too few 256x256 tiles to fill the compute units: 128x256 or
//   64x128 tiles when they finish in fewer rounds of workgroups by the
//   estimate below (bitwise the same results: every tile shape sums each
//   output's K groups in the same order).
// The weight-gradient GEMM (B scaled per row and K group) uses the same tiles.

#include "gemm_kernel.hpp"

namespace fp8bs {

namespace {
using gemm::LargeCfg;
using gemm::LargeTail;
using gemm::Rows32Cfg;
using gemm::Rows64Cfg;
using gemm::Tiles;
using gemm::pick_tiles;
}  // namespace

hipError_t launch_block_gemm(const GemmArgs& args, OutKind out, hipStream_t stream) {
  // E4M3 output quantizes whole 128-column tiles inside a workgroup: the
  // 32-column few-row tile cannot, so E4M3 output uses the 64x128 tile
  if (args.M <= 32 && out != kOutE4M3) return gemm::launch<Rows32Cfg, gemm::kDense>(args, out, stream);
  if (args.M <= 64) return gemm::launch<Rows64Cfg, gemm::kDense>(args, out, stream);
  switch (pick_tiles(args)) {
    case Tiles::kSmall: return gemm::launch<Rows64Cfg, gemm::kDense>(args, out, stream);
    case Tiles::kHalf: return gemm::launch<LargeTail, gemm::kDense>(args, out, stream);
    default: return gemm::launch<LargeCfg, gemm::kDense, LargeTail>(args, out, stream);
  }
}

hipError_t launch_block_gemm_rowscaled(const GemmArgs& args, OutKind out, hipStream_t stream) {
  using gemm::RowScaledB;
  if (args.M <= 32) return gemm::launch<RowScaledB<Rows32Cfg>, gemm::kDense>(args, out, stream);
  if (args.M <= 64) return gemm::launch<RowScaledB<Rows64Cfg>, gemm::kDense>(args, out, stream);
  switch (pick_tiles(args)) {
    case Tiles::kSmall:
      return gemm::launch<RowScaledB<Rows64Cfg>, gemm::kDense>(args, out, stream);
    case Tiles::kHalf:
      return gemm::launch<RowScaledB<LargeTail>, gemm::kDense>(args, out, stream);
    default:
      return gemm::launch<RowScaledB<LargeCfg>, gemm::kDense, RowScaledB<LargeTail>>(args, out,
                                                                                     stream);
  }
}

hipError_t launch_kgrouped_gemm_rowscaled(const GemmArgs& args, OutKind out,
                                          hipStream_t stream) {
  using gemm::RowScaledB;
  return gemm::launch<RowScaledB<LargeCfg>, gemm::kGroupK, RowScaledB<LargeTail>>(args, out,
                                                                                   stream);
}

hipError_t launch_grouped_gemm(const GemmArgs& args, OutKind out, hipStream_t stream) {
  return gemm::launch<LargeCfg, gemm::kGroupRows, LargeTail>(args, out, stream);
}

}  // namespace fp8bs
