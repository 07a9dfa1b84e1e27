// The dense block-scaled FP8 GEMM with a linear layer's epilogue:
//   z = A . B^T + bias,  y = act(z) + residual,
// y in bf16 or E4M3, z kept in bf16 on request (the backward pass needs it).
// The product is the template of gemm_kernel.hpp; its FP32 sums are finished
// in registers, so z and y are rounded once each and act sees the unrounded
// z.  Tile shapes are the plain product's (the same estimate).
//
// MFMA-bound at large M.  4096 x 18432 x 7168 with bias, gelu and z: 460 us,
// beside 437 for the plain product (z alone +12: 151 MB of stores at the tiles'
// ends); 4096 x 7168 x 18432 with bias and residual: 480 beside 434.  Settled
// clock, which board power sets; a few calls after idling take 510 and 493.

#include "epilogue.hpp"
#include "gemm_kernel.hpp"

namespace fp8bs {

namespace {

struct LinearEpilogue {
  static constexpr bool kStream = true;
  Epilogue e;

  // Bias and residual of a lane's outputs, rows 16 i + 4 g + r and FN
  // consecutive columns (see gemm::store_tile).  Tiles with registers to spare
  // (kEarly) load them before the K loop, which hides their latency: 333 x 2050 x
  // 2048 with all parts, by 64x128 tiles, 17.8 against 15.5 us.  Larger tiles load
  // them after it.
  template <class C>
  struct Early {
    static constexpr bool kEarly = C::FM * C::FN <= 8;
    float bias[kEarly ? C::FN : 1];
    uint16_t res[kEarly ? C::FM : 1][kEarly ? 4 : 1][kEarly ? C::FN : 1];
  };

  template <class C>
  __device__ __forceinline__ void load_bias(const GemmArgs& p, int64_t col, float* bias) const {
#pragma unroll
    for (int j = 0; j < C::FN; ++j) bias[j] = e.bias[col + j < p.N ? col + j : p.N - 1];
  }

  template <class C>
  __device__ __forceinline__ void load(const GemmArgs& p, const gemm::TileCoords& t, int wm,
                                       int wn, int lane, Early<C>& early) const {
    if constexpr (Early<C>::kEarly) {
      const int64_t col = t.col0 + wn * C::TN + C::FN * (lane & 15);
      const int64_t row0 = t.row0 + wm * C::TM + 4 * (lane >> 4);
      if (e.bias) load_bias<C>(p, col, early.bias);
      if (e.residual) {
        // rows and columns past the end repeat the last: loaded, never stored
        const int64_t last = t.row_end - 1;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t row = row0 + 16 * i + r;
            const uint16_t* src = e.residual + (row < last ? row : last) * e.ldr;
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
              early.res[i][r][j] = src[col + j < p.N ? col + j : p.N - 1];
          }
      }
    }
  }

  template <class C>
  __device__ __forceinline__ void apply(const GemmArgs& p, const gemm::TileCoords& t,
                                        v4f (&acc)[C::FM][C::FN], int wm, int wn, int lane,
                                        const Early<C>& early) const {
    constexpr bool EARLY = Early<C>::kEarly;
    const int64_t col = t.col0 + wn * C::TN + C::FN * (lane & 15);
    const int64_t row0 = t.row0 + wm * C::TM + 4 * (lane >> 4);
    if (e.bias) {
      float late[C::FN];
      if constexpr (!EARLY) load_bias<C>(p, col, late);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const float b = EARLY ? early.bias[EARLY ? j : 0] : late[j];
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
      gemm::store_tile<C, kOutBF16, true>(pz, tz, acc, wm, wn, lane);
    }
    with_activation(e.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = activate<decltype(act)::value>(acc[i][j][r]);
        __builtin_amdgcn_sched_barrier(0);  // few temporaries beside the sums
      }
    });
    if (e.residual) {
      if constexpr (EARLY) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
              acc[i][j][r] += __uint_as_float((uint32_t)early.res[i][r][j] << 16);
      } else {
        add_residual<C>(p, t, acc, row0, col, t.row0 + (wm + 1) * C::TM <= t.row_end);
      }
    }
  }

  // acc += residual, loaded here.  row0, col: the lane's first; inside: every
  // row of the wave exists.
  template <class C>
  __device__ __forceinline__ void add_residual(const GemmArgs& p, const gemm::TileCoords& t,
                                               v4f (&acc)[C::FM][C::FN], int64_t row0, int64_t col,
                                               bool inside) const {
    using VT = typename gemm::Vec<uint16_t, C::FN>::type;
    const bool vec = reinterpret_cast<uintptr_t>(e.residual) % (C::FN * 2) == 0 &&
                     e.ldr % C::FN == 0 && col + C::FN <= p.N;
    const uint16_t* const src = e.residual + row0 * e.ldr + col;
    if (inside && __all(vec)) {
      // the whole wave: the loads of HB MFMA rows in flight together
      constexpr int HB = C::FM < 4 ? C::FM : 4;
#pragma unroll
      for (int i0 = 0; i0 < C::FM; i0 += HB) {
        VT v[HB][4];
#pragma unroll
        for (int i = 0; i < HB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[i][r] = *reinterpret_cast<const VT*>(src + (16 * (i0 + i) + r) * e.ldr);
#pragma unroll
        for (int i = 0; i < HB; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
              acc[i0 + i][j][r] += __uint_as_float((uint32_t)v[i][r][j] << 16);
        __builtin_amdgcn_sched_barrier(0);  // few loads beside the sums
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (row0 + 16 * i + r >= t.row_end) continue;
        const uint16_t* at = src + (16 * i + r) * e.ldr;
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
          if (col + j < p.N) acc[i][j][r] += __uint_as_float((uint32_t)at[j] << 16);
      }
  }
};

// Tiles of a bf16 output whose 64x64 tiles are at most three per compute unit
// (an E4M3 output needs whole 128-column tiles): the K loop of such a launch is
// latency, and smaller tiles in more workgroups have more loads in flight.  us,
// with bias, silu, residual and z:
//                        128x256  64x128  64x64  32x64
//    200 x 1000 x 512              10.6    7.4    5.9
//    128 x 4096 x 7168             27.0   19.5   21.3   (128 tiles of 64x64)
//    333 x 2050 x 2048             15.6   11.5   10.9
//    300 x 2048 x 4096             19.8   14.4   17.2   (160)
//    700 x 4096 x 2048     30.4           21.9          (704)
//   1000 x 4096 x 7168     63.2           72.6          (1024)
// The rule goes by the tiles alone.  K moves the ends of it: at 128 tiles and a
// K of 7168 it takes 32x64 where 64x64 is 8% faster, at 198 tiles and a K of 2048
// (333 x 2050) 64x64 where 32x64 is 5% faster.
using SmallCfg = gemm::Cfg<64, 64, 2, 2, 4, 1>;
using TinyCfg = gemm::Cfg<32, 64, 2, 2, 4, 1>;

template <class C, class TAIL = C>
hipError_t launch_tiles(const GemmArgs& a, const LinearEpilogue& ep, OutKind out,
                        hipStream_t stream) {
  int64_t full = 0;
  const int64_t blocks = gemm::grid_size<C, gemm::kDense, TAIL>(a, full);
  if (blocks == 0) return hipSuccess;
  if (blocks < 0) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(C::THREADS);
  if constexpr (C::BN % 128 == 0) {
    if (out == kOutE4M3)
      return launch_kernel(gemm::block_gemm_epilogue_kernel<C, TAIL, kOutE4M3, LinearEpilogue>,
                           grid, block, stream, a, full, ep);
  }
  if constexpr (C::BN != gemm::Rows64Cfg::BN) {
    if (out == kOutBF16)
      return launch_kernel(gemm::block_gemm_epilogue_kernel<C, TAIL, kOutBF16, LinearEpilogue>,
                           grid, block, stream, a, full, ep);
  }
  return hipErrorInvalidConfiguration;
}

}  // namespace

hipError_t launch_block_gemm_epilogue(const GemmArgs& args, const Epilogue& e, OutKind out,
                                      hipStream_t stream) {
  const LinearEpilogue ep{e};
  if (out == kOutBF16) {
    const int64_t cus = gemm::device_cus() > 0 ? gemm::device_cus() : 256;
    const int64_t tiles = ((args.M + 63) / 64) * ((args.N + 63) / 64);
    if (2 * tiles <= cus) return launch_tiles<TinyCfg>(args, ep, out, stream);
    if (tiles <= 3 * cus) return launch_tiles<SmallCfg>(args, ep, out, stream);
  }
  if (args.M <= 64 && out == kOutE4M3)
    return launch_tiles<gemm::Rows64Cfg>(args, ep, out, stream);
  switch (gemm::pick_tiles(args)) {
    // one round of 64x128 tiles at most: E4M3 outputs, the others are taken above
    case gemm::Tiles::kSmall: return launch_tiles<gemm::Rows64Cfg>(args, ep, out, stream);
    case gemm::Tiles::kHalf: return launch_tiles<gemm::LargeTail>(args, ep, out, stream);
    default: return launch_tiles<gemm::LargeCfg, gemm::LargeTail>(args, ep, out, stream);
  }
}

}  // namespace fp8bs
