// The gated block-scaled FP8 product of a feed-forward block, dense and grouped
// (MoE):
//   gate = A . Wg^T, up = A . Wu^T,  y = act(gate) up,
// y in bf16 or E4M3 (the down projection's operand), gate and up kept in bf16 on
// request (the backward pass needs them).  W holds Wg's rows, then Wu's.
//
// The product is the template of gemm_kernel.hpp with its GatedB tiles: half of
// the waves along N hold gate sums, the other half up sums of the same columns,
// so its K loop is the plain product's.  At the end the two waves of a pair swap
// through LDS, each giving away two of the four rows of every MFMA tile, and
// every wave finishes the half of the rows that it keeps.  y is formed from the
// FP32 sums and rounded once.
//
// What bounds it, at 4096 x 18432 x 7168 (2.16e12 operations).  A bf16 output: the
// FP8 matrix cores, as the plain product of the same W, whose 913 us it takes 930
// of, 984 with z.  An E4M3 output: exact products (gemm::Exact) at half the FP8
// rate with the codes' widening between them, bound by instruction issue and board
// power, 1.75 to 1.90 ms with z by the clock that a card holds, 0.03 less without (a
// plain FP16 product of these sizes by the installed BLAS 1.76).  32 groups of 512
// rows x 2048 x 7168: 492 and 883 us.  The 256x256 kernels keep a few registers in
// scratch (10 dense, 24 grouped), outside their K loop.

#include "epilogue.hpp"
#include "gemm_kernel.hpp"

namespace fp8bs {

namespace {

typedef float v2f __attribute__((ext_vector_type(2)));

struct GateEpilogue {
  Gate e;

  template <class C>
  struct Early {};
  template <class C>
  __device__ __forceinline__ void load(const GemmArgs&, const gemm::TileCoords&, int, int, int,
                                       Early<C>&) const {}

  // Wave (wm, wn): half wn / (WN/2), columns (wn mod WN/2) TN .. of the tile.  Its
  // lane (g, l) holds rows 16 i + 4 g + r and FN consecutive columns from FN l;
  // it keeps rows r = 2 half and 2 half + 1.
  template <class C, int OUT>
  __device__ __forceinline__ void finish(const GemmArgs& p, const gemm::TileCoords& t,
                                         v4f (&acc)[C::FM][C::FN], int wm, int wn, int lane,
                                         uint8_t* st0, uint8_t* st1, float* red,
                                         float* rcp) const {
    constexpr int HW = C::WN / 2;
    constexpr int CHUNK = C::FM * C::FN * 512;     // bytes a wave gives away
    // chunks that use a stage; a pair's are in one
    constexpr int FIT = C::STAGE_BYTES / CHUNK / C::WN * C::WN;
    static_assert(C::FN % 2 == 0, "two columns per LDS access");
    static_assert(2 * FIT >= C::NWAVES, "the chunks fit two stages");
    const int wave = wm * C::WN + wn;
    const int half = wn / HW, wc = wn % HW;
    const int l16 = lane & 15;
    if (e.z) {
      GemmArgs pz = p;
      pz.ldc = e.ldz;
      gemm::TileCoords tz = t;
      tz.c = e.z + half * p.N;
      gemm::store_tile<C, kOutBF16, true>(pz, tz, acc, wm, wc, lane);
    }
    // f(the stage that holds the chunks of this wave and of its pair, its index there)
    auto chunks = [&](auto&& f) {
      if constexpr (FIT >= C::NWAVES) {
        f(st0, wave);
      } else {
        if (wave < FIT) {
          f(st0, wave);
        } else {
          f(st1, wave - FIT);
        }
      }
    };
    __syncthreads();  // every wave has read its last operands
    chunks([&](uint8_t* st, int w) {
      v4f* const out = reinterpret_cast<v4f*>(st + w * CHUNK) + lane;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; j += 2) {
          const v4f a = acc[i][j], b = acc[i][j + 1];
          out[(i * (C::FN / 2) + j / 2) * 64] =
              half ? v4f{a[0], a[1], b[0], b[1]} : v4f{a[2], a[3], b[2], b[3]};
        }
    });
    __syncthreads();
    v2f y[C::FM][C::FN];  // first the gate, then act(gate) up
    v2f up[C::FM][C::FN];
    chunks([&](uint8_t* st, int w) {
      const v4f* const in = reinterpret_cast<const v4f*>(st + (w ^ HW) * CHUNK) + lane;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; j += 2) {
          const v4f o = in[(i * (C::FN / 2) + j / 2) * 64];
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const v4f a = acc[i][j + d];
            const v2f mine = half ? v2f{a[2], a[3]} : v2f{a[0], a[1]};
            const v2f theirs = v2f{o[2 * d], o[2 * d + 1]};
            y[i][j + d] = half ? theirs : mine;
            up[i][j + d] = half ? mine : theirs;
          }
        }
    });
    with_activation(e.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) y[i][j][r] = activate<decltype(act)::value>(y[i][j][r]);
    });
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) y[i][j][r] *= up[i][j][r];

    // the lane's first row in the tile and first column of y
    const int row0 = wm * C::TM + 4 * (lane >> 4) + 2 * half;
    const int64_t col = t.col0 + wc * C::TN + C::FN * l16;
    if constexpr (OUT == kOutE4M3) {
      store_codes<C>(p, t, y, row0, wc, col, l16, red, rcp);
    } else {
      store_bf16<C>(p, t, y, row0, col);
    }
  }

  template <class C>
  static __device__ __forceinline__ void store_bf16(const GemmArgs& p, const gemm::TileCoords& t,
                                                    const v2f (&y)[C::FM][C::FN], int row0,
                                                    int64_t col) {
    using VT = typename gemm::Vec<uint32_t, C::FN / 2>::type;
    uint16_t* const out = static_cast<uint16_t*>(t.c);
    const bool vec = reinterpret_cast<uintptr_t>(out) % (C::FN * 2) == 0 && p.ldc % C::FN == 0;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = t.row0 + row0 + 16 * i + r;
        if (row >= t.row_end) continue;
        uint16_t* const dst = out + row * p.ldc + col;
        VT w;
#pragma unroll
        for (int q = 0; q < C::FN / 2; ++q) w[q] = bf16x2_rne(y[i][2 * q][r], y[i][2 * q + 1][r]);
        if (vec) {
          *reinterpret_cast<VT*>(dst) = w;
        } else {
#pragma unroll
          for (int q = 0; q < C::FN / 2; ++q) {
            dst[2 * q] = (uint16_t)w[q];
            dst[2 * q + 1] = (uint16_t)(w[q] >> 16);
          }
        }
      }
  }

  // As gemm::store_tile_e4m3 for the rows that the wave keeps: a row's 128
  // columns are those of HW waves; a NaN keeps the code of NaN.
  template <class C>
  static __device__ __forceinline__ void store_codes(const GemmArgs& p, const gemm::TileCoords& t,
                                                     const v2f (&y)[C::FM][C::FN], int row0, int wc,
                                                     int64_t col, int l16, float* red,
                                                     float* rcp) {
    static_assert(C::BNO == 128 && C::FN == 4, "a tile holds one 128-column block of y");
    constexpr int HW = C::WN / 2;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) m = fmaxf(m, fabsf(y[i][j][r]));
        m = max_row16(m);
        if (l16 == 0) red[wc * C::BM + row0 + 16 * i + r] = m;
      }
    __syncthreads();
    for (int rt = threadIdx.x; rt < C::BM; rt += C::THREADS) {
      float amax = 0.0f;
#pragma unroll
      for (int w = 0; w < HW; ++w) amax = fmaxf(amax, red[w * C::BM + rt]);
      float s, rr;
      group_scale(amax, s, rr);
      rcp[rt] = rr;
      const int64_t row = t.row0 + rt;
      if (row < t.row_end) p.sc[t.col0 / 128 * p.ldsc + row] = s;
    }
    __syncthreads();
    uint8_t* const out = static_cast<uint8_t*>(t.c);
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t row = t.row0 + row0 + 16 * i + r;
        if (row >= t.row_end) continue;
        const float f = rcp[row0 + 16 * i + r];
        const uint32_t lo = codes2<false>(y[i][0][r] * f, y[i][1][r] * f, 0u);
        *reinterpret_cast<uint32_t*>(out + row * p.ldc + col) =
            codes2<true>(y[i][2][r] * f, y[i][3][r] * f, lo);
      }
  }
};

template <class C, class TAIL, int SCHED, int OUT>
__global__ __launch_bounds__(C::THREADS) void gated_kernel(GemmArgs p, int64_t full,
                                                           GateEpilogue ep) {
  gemm::block_gemm_tile<C, TAIL, SCHED, OUT>(p, full, ep);
}

// OUT: bf16 from the FP8 instruction's sums, whose error lies far below bf16's
// rounding, or E4M3 from exact products, whose FP32 scales show it (see
// gemm::Exact).
template <class C0, int SCHED, int OUT, class TAIL0 = C0>
hipError_t launch_tiles(const GemmArgs& a, const GateEpilogue& ep, hipStream_t stream) {
  using CG = gemm::GatedB<C0>;
  using TG = gemm::GatedB<TAIL0>;
  using C = typename std::conditional<OUT == kOutE4M3, gemm::Exact<CG>, CG>::type;
  using TAIL = typename std::conditional<OUT == kOutE4M3, gemm::Exact<TG>, TG>::type;
  int64_t full = 0;
  const int64_t blocks = gemm::grid_size<C, SCHED, TAIL>(a, full);
  if (blocks == 0) return hipSuccess;
  if (blocks < 0) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(C::THREADS);
  return launch_kernel(gated_kernel<C, TAIL, SCHED, OUT>, grid, block, stream, a, full, ep);
}

// An E4M3 output needs 128 columns of y, 256 rows of W, per tile.
using Exact128 = gemm::Cfg<128, 256, 2, 4, 3, 4>;
using Exact128Tail = gemm::Cfg<64, 256, 2, 4, 3, 4>;
using Exact64 = gemm::Cfg<64, 256, 1, 4, 3, 8>;
using Exact32 = gemm::Cfg<32, 256, 1, 4, 3, 8>;
// bf16 outputs of few tiles, as the epilogue's.  Eight tile-rows of a dense product
// to a run share an XCD's weights in its L2: 333 x 2048 x 2048 11.0 us, with one
// 13.1; 1000 x 2048 x 7168 in E4M3 60.5 and 65.8.  Groups' tile-rows have weights
// of their own, and runs only keep them apart: 4 groups of 200 x 2048 x 2048 11.5
// with one, 14.6 with eight, 32 of 256 x 2048 x 7168 157.9 and 161.4.
using SmallCfg = gemm::Cfg<64, 64, 2, 2, 4, 8>;
using TinyCfg = gemm::Cfg<32, 64, 2, 2, 4, 8>;
using GroupSmallCfg = gemm::Cfg<64, 64, 2, 2, 4, 1>;
using GroupTinyCfg = gemm::Cfg<32, 64, 2, 2, 4, 1>;

// fp32 [M][N] -> codes and scales, 16 lanes per 1x128 tile.
__global__ __launch_bounds__(256) void quant_f32_kernel(const float* x, int64_t M, int64_t N,
                                                        uint8_t* q, int64_t ldq, float* s,
                                                        int64_t lds) {
  const int64_t tile = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t NB = N / 128;
  if (tile >= M * NB) return;  // 16 lanes together
  const int64_t row = tile / NB, nb = tile % NB, col = nb * 128 + (threadIdx.x & 15) * 8;
  const float4 a = *reinterpret_cast<const float4*>(x + row * N + col);
  const float4 b = *reinterpret_cast<const float4*>(x + row * N + col + 4);
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  float sc, r;
  group_scale(max_row16(m), sc, r);
  *reinterpret_cast<u32x2*>(q + row * ldq + col) = codes8(v, r);
  if ((threadIdx.x & 15) == 0) s[nb * lds + row] = sc;
}

}  // namespace

hipError_t launch_quant_f32(const float* x, int64_t M, int64_t N, uint8_t* q, int64_t ldq,
                            float* s, int64_t lds, hipStream_t stream) {
  const int64_t blocks = (M * (N / 128) + 15) / 16;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  return launch_kernel(quant_f32_kernel, dim3((unsigned)blocks), dim3(256), stream, x, M, N, q,
                       ldq, s, lds);
}

// Tiles by their number, as the epilogue's.  us, each call after one with other
// weights, rows of 32 / 64 / 128 for E4M3 and 32x64 / 64x64 / 128x256 / 256x256 for
// bf16:
//    100 x  2048 x 2048     17.0   21.6   29.6      7.8    8.6   19.7   26.7
//    333 x  2048 x 2048     17.8   22.0   29.6     12.2   11.5   19.7   27.8
//    512 x  2048 x 2048     18.0   22.1   29.6     15.9   11.8   19.7   27.6
//    576 x  2048 x 2048     32.0   21.9   29.5     17.6   16.9   19.9   27.6
//    250 x  2048 x 7168     44.1   58.2   84.2     21.9   18.8   53.7   74.7
//   1000 x  2048 x 7168     90.5   60.4   84.1     66.7   51.3   54.3   77.8
//   1100 x  2048 x 7168    125.7  114.3   84.8     76.1   63.3   55.5   78.1
//   1500 x  2048 x 7168    128.7  120.1   86.2     98.5   76.8   68.4   86.4
//     70 x 18432 x 7168    100.4  116.7   86.4     86.1   75.8   87.0   96.0
//    128 x 18432 x 7168    145.8  119.5   89.9    108.8   90.4   90.9   98.3
//    200 x 18432 x 7168    188.1  174.9  149.8    165.3  125.4  158.7  101.3
// The bf16 rule loses where 64x64 tiles pass four to a compute unit over a long K
// (1100 rows).
hipError_t launch_block_gemm_gated(const GemmArgs& args, const Gate& gate, OutKind out,
                                   hipStream_t stream) {
  const GateEpilogue ep{gate};
  const int64_t cus = gemm::device_cus() > 0 ? gemm::device_cus() : 256;
  if (out == kOutE4M3) {
    const int64_t tiles = (args.M + 63) / 64 * (args.N / 128);
    if (2 * tiles <= cus) return launch_tiles<Exact32, gemm::kDense, kOutE4M3>(args, ep, stream);
    if (tiles <= cus) return launch_tiles<Exact64, gemm::kDense, kOutE4M3>(args, ep, stream);
    return launch_tiles<Exact128, gemm::kDense, kOutE4M3, Exact128Tail>(args, ep, stream);
  }
  const int64_t tiles = (args.M + 63) / 64 * (args.N / 32);
  if (2 * tiles <= cus) return launch_tiles<TinyCfg, gemm::kDense, kOutBF16>(args, ep, stream);
  if (tiles <= 5 * cus) return launch_tiles<SmallCfg, gemm::kDense, kOutBF16>(args, ep, stream);
  GemmArgs whole = args;  // the estimate counts W's rows
  whole.N = 2 * args.N;
  if (gemm::pick_tiles(whole) == gemm::Tiles::kLarge)
    return launch_tiles<gemm::LargeCfg, gemm::kDense, kOutBF16, gemm::LargeTail>(args, ep, stream);
  return launch_tiles<gemm::LargeTail, gemm::kDense, kOutBF16>(args, ep, stream);
}

// The groups' rows are known on the device alone: the rules go by the most
// tile-rows that M rows of G groups can fill.  us, 32x64 / 64x64 / 128x256 /
// 256x256 for bf16 and rows of 32 / 64 / 128 for E4M3:
//   G 8  M  333 N  512 K 2048    8.8   10.0   20.7   20.8     18.0   22.7   30.8
//   G 4  M  200 N 2048 K 2048   12.1   13.4   25.0   25.2     19.4   23.4   31.5
//   G 16 M 2000 N  512 K 2048   21.2   20.5   27.2   32.6     39.1   24.5   31.5
//   G 32 M  256 N 2048 K 7168  162.3  158.6  185.4  185.5    207.1  166.2  165.7
//   G 32 M 1000 N 2048 K 7168  189.3  178.0  258.2  203.2    196.8  205.9  216.2
//   G 32 M 2048 N 2048 K 7168  265.4  223.8  261.8  268.6    324.7  227.9  235.8
//   G 8  M 3000 N 1024 K 4096   76.5   64.8   51.9   60.3    122.1   80.5   59.2
// Few rows to a group (the weights' stream) take 64x64 tiles whatever their number,
// in bf16 up to 32 rows to a group.  The rules lose at 64 rows to a group (bf16 269
// us where 224 could be) and, in E4M3, at 32 to 64 (216 where 197, 236 where 228).
hipError_t launch_grouped_gemm_gated(const GemmArgs& args, const Gate& gate, OutKind out,
                                     hipStream_t stream) {
  const GateEpilogue ep{gate};
  const int64_t cus = gemm::device_cus() > 0 ? gemm::device_cus() : 256;
  const int64_t groups = args.G < args.M ? args.G : args.M;
  const int64_t rows = args.M / 64 + groups;  // tile-rows of 64
  if (out == kOutE4M3) {
    const int64_t tiles = rows * (args.N / 128);
    if (2 * tiles <= cus) return launch_tiles<Exact32, gemm::kGroupRows, kOutE4M3>(args, ep, stream);
    if (tiles <= cus) return launch_tiles<Exact64, gemm::kGroupRows, kOutE4M3>(args, ep, stream);
    return launch_tiles<Exact128, gemm::kGroupRows, kOutE4M3, Exact128Tail>(args, ep, stream);
  }
  const int64_t tiles = rows * (args.N / 32);
  if (tiles <= 2 * cus)
    return launch_tiles<GroupTinyCfg, gemm::kGroupRows, kOutBF16>(args, ep, stream);
  if (tiles <= 3 * cus || args.M <= 32 * args.G)
    return launch_tiles<GroupSmallCfg, gemm::kGroupRows, kOutBF16>(args, ep, stream);
  if ((args.M / 256 + groups) * (args.N / 128) <= cus)
    return launch_tiles<gemm::LargeTail, gemm::kGroupRows, kOutBF16>(args, ep, stream);
  return launch_tiles<gemm::LargeCfg, gemm::kGroupRows, kOutBF16, gemm::LargeTail>(args, ep,
                                                                                   stream);
}

}  // namespace fp8bs
