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
  // columns are those of HW waves.
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
        const uint32_t lo = cvt2_e4m3<false>(y[i][0][r] * f, y[i][1][r] * f, 0u);
        *reinterpret_cast<uint32_t*>(out + row * p.ldc + col) =
            cvt2_e4m3<true>(y[i][2][r] * f, y[i][3][r] * f, lo);
      }
  }
};

template <class C, class TAIL, int SCHED, int OUT>
__global__ __launch_bounds__(C::THREADS) void gated_kernel(GemmArgs p, int64_t full,
                                                           GateEpilogue ep) {
  gemm::block_gemm_tile<C, TAIL, SCHED, OUT>(p, full, ep);
}

template <class C0, int SCHED, class TAIL0 = C0>
hipError_t launch_tiles(const GemmArgs& a, const GateEpilogue& ep, OutKind out,
                        hipStream_t stream) {
  using C = gemm::GatedB<C0>;
  using TAIL = gemm::GatedB<TAIL0>;
  int64_t full = 0;
  const int64_t blocks = gemm::grid_size<C, SCHED, TAIL>(a, full);
  if (blocks == 0) return hipSuccess;
  if (blocks < 0) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(C::THREADS);
  if constexpr (C::BNO == 128) {
    if (out == kOutE4M3)
      return launch_kernel(gated_kernel<C, TAIL, SCHED, kOutE4M3>, grid, block, stream, a, full,
                           ep);
  }
  if (out == kOutBF16)
    return launch_kernel(gated_kernel<C, TAIL, SCHED, kOutBF16>, grid, block, stream, a, full, ep);
  return hipErrorInvalidConfiguration;
}

// An E4M3 output needs 128 columns of y, 256 rows of W, per tile: 64 rows of A
// where the card is not filled otherwise, in three LDS stages.
using Rows64Wide = gemm::Cfg<64, 256, 1, 4, 3, 1>;

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
  uint32_t lo = cvt2_e4m3<false>(v[0] * r, v[1] * r, 0u);
  lo = cvt2_e4m3<true>(v[2] * r, v[3] * r, lo);
  uint32_t hi = cvt2_e4m3<false>(v[4] * r, v[5] * r, 0u);
  hi = cvt2_e4m3<true>(v[6] * r, v[7] * r, hi);
  *reinterpret_cast<u32x2*>(q + row * ldq + col) = u32x2{lo, hi};
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

hipError_t launch_block_gemm_gated(const GemmArgs& args, const Gate& gate, OutKind out,
                                   hipStream_t stream) {
  const GateEpilogue ep{gate};
  GemmArgs whole = args;  // the tiles' estimate counts W's rows
  whole.N = 2 * args.N;
  switch (gemm::pick_tiles(whole)) {
    case gemm::Tiles::kSmall: return launch_tiles<Rows64Wide, gemm::kDense>(args, ep, out, stream);
    case gemm::Tiles::kHalf:
      return launch_tiles<gemm::LargeTail, gemm::kDense>(args, ep, out, stream);
    default:
      return launch_tiles<gemm::LargeCfg, gemm::kDense, gemm::LargeTail>(args, ep, out, stream);
  }
}

hipError_t launch_grouped_gemm_gated(const GemmArgs& args, const Gate& gate, OutKind out,
                                     hipStream_t stream) {
  return launch_tiles<gemm::LargeCfg, gemm::kGroupRows, gemm::LargeTail>(args, GateEpilogue{gate},
                                                                         out, stream);
}

}  // namespace fp8bs
