// Backward of the gated product y = act(gate) up for gfx950, up to the operands
// of its three backward GEMMs:
//   dgate = dy up act'(gate),  dup = dy act(gate)
// in FP32, quantized by the online E4M3 rule per 1x128 tile (the data gradient's
// operand, contraction over gate and up columns) and per 128 rows of a column,
// transposed (the weight gradient's); y = act(gate) up is formed again from the
// kept values and quantized per 128 rows for the down projection's weight
// gradient.
//
// HBM-bound: 6 bytes in and 5 codes out per element of y.  One workgroup per
// 128x128 block of y holds both gradients and y in registers, so everything is
// read once and nothing but codes and scales is written.  A thread holds 8
// values of each of 4 rows (16 lanes span a row): row maxima are a 16-lane
// reduction, column maxima go over the thread's rows, its wave's row groups and
// the waves.  The codes are transposed through LDS, all three blocks between the
// same barriers.  4096 x 18432, silu: 166 us, 5.0 TB/s beside a plain copy's 5.2
// (842 MB, each input read once; 184 with the blocks dealt round-robin over the
// XCDs, 170 with the column codes left to the caches).  333 x 2048: 11 us, launch
// and latency.

#include "epilogue.hpp"
#include "transpose.hpp"

namespace fp8bs {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 4;     // rows per thread, 32 apart
constexpr int kPitch = 132;  // LDS row pitch of the staged codes (bytes)

// One 128x128 block on its way to codes per column, transposed.
struct Columns {
  float cmax[kWaves][128];
  float rcp[128];
  uint8_t tile[128 * kPitch];
};

// Column maxima of the block v (kRows rows of 8 columns per thread) by waves.
__device__ __forceinline__ void column_maxima(const float (&v)[kRows][8], Columns& L) {
  const int lane = threadIdx.x & 15;
  float cm[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    cm[c] = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) cm[c] = fmaxf(cm[c], fabsf(v[i][c]));
    cm[c] = fmaxf(cm[c], __shfl_xor(cm[c], 16, 64));
    cm[c] = fmaxf(cm[c], __shfl_xor(cm[c], 32, 64));
  }
  if ((threadIdx.x & 63) < 16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) L.cmax[threadIdx.x >> 6][lane * 8 + c] = cm[c];
  }
}

// Scale and reciprocal of column c.
__device__ __forceinline__ void column_scale(int c, Columns& L, float* st) {
  float m = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, L.cmax[w][c]);
  float s, r;
  group_scale(m, s, r);
  L.rcp[c] = r;
  st[c] = s;
}

__device__ __forceinline__ void stage_codes(const float (&v)[kRows][8], Columns& L) {
  const int lane = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  float r[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) r[c] = L.rcp[lane * 8 + c];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const u32x2 w = codes8(v[i], r);
    uint32_t* const dst = reinterpret_cast<uint32_t*>(L.tile + (r0 + 32 * i) * kPitch + lane * 8);
    dst[0] = w.x;
    dst[1] = w.y;
  }
}

// The staged codes to qt[c][0 .. 127]: 16 consecutive threads cover the 128 rows
// of one output row (whole lines).
__device__ __forceinline__ void store_columns(const Columns& L, uint8_t* qt, int64_t ldqt) {
  const int m0 = (threadIdx.x & 15) * 8, c0 = (threadIdx.x >> 4) * 4;
  uint32_t in[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    in[i] = *reinterpret_cast<const uint32_t*>(L.tile + (m0 + i) * kPitch + c0);
  u32x2 out[4];
  transpose8x4(in, out);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    __builtin_nontemporal_store(out[c],
                                reinterpret_cast<u32x2*>(qt + (int64_t)(c0 + c) * ldqt + m0));
  }
}

// The block's rows as codes per 1x128 tile (rows past M are not stored).
__device__ __forceinline__ void store_rows(const float (&v)[kRows][8], int64_t row0, int64_t M,
                                           uint8_t* q, int64_t ldq, float* s) {
  const int lane = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(v[i][c]));
    float sc, r;
    group_scale(max_row16(m), sc, r);
    const int64_t row = row0 + 32 * i;
    const u32x2 w = codes8(v[i], r);
    if (row < M) {
      __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(q + row * ldq + lane * 8));
      if (lane == 0) s[row] = sc;
    }
  }
}

template <int ACT>
__global__ __launch_bounds__(kThreads) void gated_backward_kernel(GatedGradArgs a) {
  __shared__ __attribute__((aligned(16))) Columns L[3];  // dgate, dup, y
  const int64_t NB = a.N / 128;
  // each XCD a contiguous run of blocks (workgroup b runs on XCD b mod 8), so that
  // neighbouring stretches of a row of dy and z come through one L2
  const int64_t x = blockIdx.x % 8, n = gridDim.x / 8, r8 = gridDim.x % 8;
  const int64_t block = x * n + (x < r8 ? x : r8) + blockIdx.x / 8;
  const int64_t nb = block % NB, mb = block / NB;
  const int lane = threadIdx.x & 15;
  const int64_t row0 = mb * 128 + (threadIdx.x >> 4), col = nb * 128 + lane * 8;
  float dg[kRows][8], du[kRows][8], y[kRows][8];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = row0 + 32 * i;
    const int64_t rc = row < a.M ? row : a.M - 1;
    const u32x4 vd = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(a.dy + rc * a.lddy + col));
    const u32x4 vg =
        __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.z + rc * a.ldz + col));
    const u32x4 vu =
        __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.z + rc * a.ldz + a.N + col));
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float d = c & 1 ? bf16_hi(vd[c / 2]) : bf16_lo(vd[c / 2]);
      const float g = c & 1 ? bf16_hi(vg[c / 2]) : bf16_lo(vg[c / 2]);
      const float u = c & 1 ? bf16_hi(vu[c / 2]) : bf16_lo(vu[c / 2]);
      const float ag = activate<ACT>(g);
      dg[i][c] = d * u * activate_grad<ACT>(g);
      du[i][c] = d * ag;
      y[i][c] = ag * u;
    }
    if (row >= a.M) {  // padding: in no maximum, codes 0
#pragma unroll
      for (int c = 0; c < 8; ++c) dg[i][c] = du[i][c] = y[i][c] = 0.0f;
    }
  }
  store_rows(dg, row0, a.M, a.q + nb * 128, a.ldq, a.s + nb * a.lds);
  store_rows(du, row0, a.M, a.q + a.N + nb * 128, a.ldq, a.s + (NB + nb) * a.lds);
  column_maxima(dg, L[0]);
  column_maxima(du, L[1]);
  if (a.yt) column_maxima(y, L[2]);
  __syncthreads();
  const int64_t n0 = nb * 128, m0 = mb * 128;
  const int c = threadIdx.x & 127;
  if (threadIdx.x < 128) {
    column_scale(c, L[0], a.st + mb * a.ldst + n0);
  } else if (threadIdx.x < 256) {
    column_scale(c, L[1], a.st + mb * a.ldst + a.N + n0);
  } else if (threadIdx.x < 384 && a.yt) {
    column_scale(c, L[2], a.syt + mb * a.ldsyt + n0);
  }
  __syncthreads();
  stage_codes(dg, L[0]);
  stage_codes(du, L[1]);
  if (a.yt) stage_codes(y, L[2]);
  __syncthreads();
  store_columns(L[0], a.qt + n0 * a.ldqt + m0, a.ldqt);
  store_columns(L[1], a.qt + (a.N + n0) * a.ldqt + m0, a.ldqt);
  if (a.yt) store_columns(L[2], a.yt + n0 * a.ldyt + m0, a.ldyt);
}

}  // namespace

hipError_t launch_gated_backward(const GatedGradArgs& a, int act, hipStream_t stream) {
  const int64_t blocks = (a.M + 127) / 128 * (a.N / 128);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(kThreads);
  switch (act) {
    case kActRelu: return launch_kernel(gated_backward_kernel<kActRelu>, grid, block, stream, a);
    case kActSilu: return launch_kernel(gated_backward_kernel<kActSilu>, grid, block, stream, a);
    case kActGelu: return launch_kernel(gated_backward_kernel<kActGelu>, grid, block, stream, a);
    default: return launch_kernel(gated_backward_kernel<kActNone>, grid, block, stream, a);
  }
}

}  // namespace fp8bs
