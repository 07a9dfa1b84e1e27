// Backward of the linear layer's epilogue, up to the operands of its two
// backward GEMMs, for gfx950: dz = dy act'(z) in FP32, quantized by the online
// E4M3 rule both per 1x128 tile (the data gradient's operand) and per 128 rows
// of a column, transposed (the weight gradient's), and dbias = sum of dz over
// the rows.
//
// HBM-bound: 4 bytes in, 2 codes and two 1/128 scales out per element.  One
// workgroup per 128x128 block holds its dz in registers, so dy and z are read
// once and dz never reaches memory.  A thread holds 8 values of each of 8 rows
// (16 lanes span a row): the row maxima are a 16-lane reduction, the column
// maxima and sums go over the thread's rows, its wave's row groups and the
// waves.  The column sums of the blocks are left in the workspace and added
// up, in order, by a second launch.  4096 x 18432, gelu: 95 us, 4.8 TB/s, the rate
// of a plain copy (453 MB moved, each input read once).  At 333 x 2048 the two
// launches are latency: 9 + 3 us.

#include "epilogue.hpp"
#include "transpose.hpp"

namespace fp8bs {

namespace {

struct BackwardArgs {
  const uint16_t* dy;
  int64_t lddy;
  const uint16_t* z;
  int64_t ldz;
  int64_t M, NB;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;
  uint8_t* qt;
  int64_t ldqt;
  float* st;
  int64_t ldst;
  float* part;  // [ceil(M/128)][N] column sums
};

// v of lane i (compile time) of the 16 lanes of this one's row.
template <int I>
__device__ __forceinline__ float of_row_lane(float v) {
  return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), (I << 5) | 0x10));
}

template <int ACT>
__global__ __launch_bounds__(256) void epilogue_backward_kernel(BackwardArgs a) {
  constexpr int kPitch = 136;  // LDS row pitch of the staged codes (bytes)
  __shared__ float colmax[4][128], colsum[4][128];
  __shared__ __attribute__((aligned(16))) float rcp[128];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kPitch];
  const int64_t nb = blockIdx.x % a.NB, mb = blockIdx.x / a.NB;
  const int lane = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int64_t col = nb * 128 + lane * 8;

  float d[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = mb * 128 + r0 + 16 * i;
    const int64_t rc = row < a.M ? row : a.M - 1;
    const u32x4 y = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4*>(a.dy + rc * a.lddy + col));
    u32x4 z = {0u, 0u, 0u, 0u};
    if constexpr (ACT != kActNone)
      z = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.z + rc * a.ldz + col));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d[i][2 * e] = bf16_lo(y[e]) * activate_grad<ACT>(bf16_lo(z[e]));
      d[i][2 * e + 1] = bf16_hi(y[e]) * activate_grad<ACT>(bf16_hi(z[e]));
    }
    if (row >= a.M) {  // padding: in no maximum, no sum, codes 0
#pragma unroll
      for (int c = 0; c < 8; ++c) d[i][c] = 0.0f;
    }
  }
  float cm[8], cs[8], rm[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) cm[c] = cs[c] = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m = fmaxf(m, fabsf(d[i][c]));
      cm[c] = fmaxf(cm[c], fabsf(d[i][c]));
      cs[c] += d[i][c];
    }
    rm[i] = max_row16(m);
  }
  // lane i (mod 8) forms the scale of row i, for all 16 lanes of the row: the
  // IEEE divisions would otherwise be a tenth of the kernel's instructions
  float mine = rm[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mine = (lane & 7) == i ? rm[i] : mine;
  float scale, rcp_mine;
  group_scale(mine, scale, rcp_mine);
  {
    const int64_t row = mb * 128 + r0 + 16 * lane;
    if (lane < 8 && row < a.M) a.s[nb * a.lds + row] = scale;
  }
  static_for<0, 8>([&](auto i_) {
    constexpr int i = decltype(i_)::value;
    const float r = of_row_lane<i>(rcp_mine);
    uint32_t lo = codes2<false>(d[i][0] * r, d[i][1] * r, 0u);
    lo = codes2<true>(d[i][2] * r, d[i][3] * r, lo);
    uint32_t hi = codes2<false>(d[i][4] * r, d[i][5] * r, 0u);
    hi = codes2<true>(d[i][6] * r, d[i][7] * r, hi);
    const int64_t row = mb * 128 + r0 + 16 * i;
    if (row < a.M)
      __builtin_nontemporal_store(u32x2{lo, hi}, reinterpret_cast<u32x2*>(a.q + row * a.ldq + col));
  });
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    cm[c] = fmaxf(cm[c], __shfl_xor(cm[c], 16, 64));
    cm[c] = fmaxf(cm[c], __shfl_xor(cm[c], 32, 64));
    cs[c] += __shfl_xor(cs[c], 16, 64);
    cs[c] += __shfl_xor(cs[c], 32, 64);
  }
  if ((threadIdx.x & 63) < 16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      colmax[threadIdx.x >> 6][lane * 8 + c] = cm[c];
      colsum[threadIdx.x >> 6][lane * 8 + c] = cs[c];
    }
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    const int c = threadIdx.x;
    float sc, r;
    group_scale(fmaxf(fmaxf(colmax[0][c], colmax[1][c]), fmaxf(colmax[2][c], colmax[3][c])), sc, r);
    rcp[c] = r;
    a.st[mb * a.ldst + nb * 128 + c] = sc;
    a.part[mb * (a.NB * 128) + nb * 128 + c] =
        (colsum[0][c] + colsum[1][c]) + (colsum[2][c] + colsum[3][c]);
  }
  __syncthreads();
  const float4 ra = *reinterpret_cast<const float4*>(rcp + lane * 8);
  const float4 rb = *reinterpret_cast<const float4*>(rcp + lane * 8 + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t lo = codes2<false>(d[i][0] * ra.x, d[i][1] * ra.y, 0u);
    lo = codes2<true>(d[i][2] * ra.z, d[i][3] * ra.w, lo);
    uint32_t hi = codes2<false>(d[i][4] * rb.x, d[i][5] * rb.y, 0u);
    hi = codes2<true>(d[i][6] * rb.z, d[i][7] * rb.w, hi);
    *reinterpret_cast<u32x2*>(tile + (r0 + 16 * i) * kPitch + lane * 8) = u32x2{lo, hi};
  }
  __syncthreads();
  // 16 consecutive threads cover the 128 rows of one output row (whole
  // 128-byte lines per store)
  const int m0 = (threadIdx.x & 15) * 8, c0 = (threadIdx.x >> 4) * 8;
  uint32_t lo[8], hi[8], olo[8], ohi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(tile + (m0 + i) * kPitch + c0);
    lo[i] = v.x;
    hi[i] = v.y;
  }
  transpose8x8(lo, hi, olo, ohi);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int64_t n = nb * 128 + c0 + c;
    *reinterpret_cast<u32x2*>(a.qt + n * a.ldqt + mb * 128 + m0) = u32x2{olo[c], ohi[c]};
  }
}

// dbias from the blocks' column sums: 64 columns per workgroup, its four waves
// taking every fourth block (a fixed order).
__global__ __launch_bounds__(256) void epilogue_bias_kernel(const float* part, int64_t MB,
                                                            int64_t N, float* dbias) {
  __shared__ float sum[4][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;  // N is a multiple of 128
  float s = 0.0f;
#pragma unroll 8
  for (int64_t b = wave; b < MB; b += 4) s += part[b * N + n];
  sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0) dbias[n] = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
}

}  // namespace

size_t epilogue_backward_workspace(int64_t M, int64_t N) {
  return size_t((M + 127) / 128) * size_t(N) * 4;
}

hipError_t launch_epilogue_backward(const uint16_t* dy, int64_t lddy, const uint16_t* z,
                                    int64_t ldz, int act, int64_t M, int64_t N, uint8_t* q,
                                    int64_t ldq, float* s, int64_t lds, uint8_t* qt, int64_t ldqt,
                                    float* st, int64_t ldst, float* dbias, void* workspace,
                                    hipStream_t stream) {
  const int64_t MB = (M + 127) / 128, blocks = MB * (N / 128);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  // one block of rows: its sums are dbias
  float* part = MB == 1 ? dbias : static_cast<float*>(workspace);
  const BackwardArgs a{dy, lddy, z, ldz, M, N / 128, q, ldq, s, lds, qt, ldqt, st, ldst, part};
  const dim3 grid((unsigned)blocks), block(256);
  hipError_t e;
  switch (act) {
    case kActRelu:
      e = launch_kernel(epilogue_backward_kernel<kActRelu>, grid, block, stream, a);
      break;
    case kActSilu:
      e = launch_kernel(epilogue_backward_kernel<kActSilu>, grid, block, stream, a);
      break;
    case kActGelu:
      e = launch_kernel(epilogue_backward_kernel<kActGelu>, grid, block, stream, a);
      break;
    default:
      e = launch_kernel(epilogue_backward_kernel<kActNone>, grid, block, stream, a);
  }
  if (e != hipSuccess || MB == 1) return e;
  return launch_kernel(epilogue_bias_kernel, dim3((unsigned)(N / 64)), dim3(256), stream,
                       static_cast<const float*>(part), MB, N, dbias);
}

}  // namespace fp8bs
