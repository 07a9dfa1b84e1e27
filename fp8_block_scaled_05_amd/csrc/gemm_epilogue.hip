// The dense block-scaled FP8 GEMM with a linear layer's epilogue:
//   z = A . B^T + bias,  y = act(z) + residual,
// y in bf16 or E4M3, z kept in bf16 on request (the backward pass needs it).
// The product is the template of gemm_kernel.hpp; its FP32 sums are finished
// in registers, so z and y are rounded once each and act sees the unrounded
// z.  Tile shapes are the plain product's (the same estimate).

#include "epilogue.hpp"
#include "gemm_kernel.hpp"

namespace fp8bs {

namespace {

struct LinearEpilogue {
  Epilogue e;

  // Lane (g, l) holds rows 16 i + 4 g + r and FN consecutive columns (see
  // gemm::store_tile).
  template <class C>
  __device__ __forceinline__ void apply(const GemmArgs& p, const gemm::TileCoords& t,
                                        v4f (&acc)[C::FM][C::FN], int wm, int wn,
                                        int lane) const {
    const int g4 = lane >> 4, l16 = lane & 15;
    const int64_t col = t.col0 + wn * C::TN + C::FN * l16;
    const int64_t wrow0 = t.row0 + wm * C::TM;
    if (e.bias) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const float b = col + j < p.N ? e.bias[col + j] : 0.0f;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] += b;
      }
    }
    if (e.z) {
      GemmArgs pz = p;
      pz.ldc = e.ldz;
      gemm::TileCoords tz = t;
      tz.c = e.z;
      gemm::store_tile<C, kOutBF16>(pz, tz, acc, wm, wn, lane);
    }
    with_activation(e.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = activate<decltype(act)::value>(acc[i][j][r]);
    });
    if (e.residual) {
      using VT = typename gemm::Vec<uint16_t, C::FN>::type;
      const bool vec = reinterpret_cast<uintptr_t>(e.residual) % (C::FN * 2) == 0 &&
                       e.ldr % C::FN == 0 && col + C::FN <= p.N;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t row = wrow0 + 16 * i + 4 * g4 + r;
          if (row >= t.row_end) continue;
          const uint16_t* src = e.residual + row * e.ldr + col;
          if (vec) {
            VT v;
            if constexpr (C::FN == 1) {
              v[0] = *src;
            } else {
              v = *reinterpret_cast<const VT*>(src);
            }
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
              acc[i][j][r] += __uint_as_float((uint32_t)v[j] << 16);
          } else {
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
              if (col + j < p.N) acc[i][j][r] += __uint_as_float((uint32_t)src[j] << 16);
          }
        }
    }
  }
};

template <class C, class TAIL = C>
hipError_t launch_tiles(const GemmArgs& a, const LinearEpilogue& ep, OutKind out,
                        hipStream_t stream) {
  int64_t full = 0;
  const int64_t blocks = gemm::grid_size<C, gemm::kDense, TAIL>(a, full);
  if (blocks == 0) return hipSuccess;
  if (blocks < 0) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(C::THREADS);
  if (out == kOutBF16)
    return launch_kernel(gemm::block_gemm_epilogue_kernel<C, TAIL, kOutBF16, LinearEpilogue>, grid,
                         block, stream, a, full, ep);
  return launch_kernel(gemm::block_gemm_epilogue_kernel<C, TAIL, kOutE4M3, LinearEpilogue>, grid,
                       block, stream, a, full, ep);
}

}  // namespace

hipError_t launch_block_gemm_epilogue(const GemmArgs& args, const Epilogue& e, OutKind out,
                                      hipStream_t stream) {
  const LinearEpilogue ep{e};
  if (args.M <= 64) return launch_tiles<gemm::Rows64Cfg>(args, ep, out, stream);
  switch (gemm::pick_tiles(args)) {
    case gemm::Tiles::kSmall: return launch_tiles<gemm::Rows64Cfg>(args, ep, out, stream);
    case gemm::Tiles::kHalf: return launch_tiles<gemm::LargeTail>(args, ep, out, stream);
    default: return launch_tiles<gemm::LargeCfg, gemm::LargeTail>(args, ep, out, stream);
  }
}

}  // namespace fp8bs
