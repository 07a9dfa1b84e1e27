// Root-mean-square norm of a transformer block for gfx950, with the residual's
// addition in front and the online E4M3 quantization per 1x128 tile behind it,
// and its backward pass.
//
//   h = RN_bf16(x + residual), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd g
//   n = h rstd, u = g dy, c = mean(u n)
//   dx = rstd (u - n c) + dh,  dg = sum over the rows of dy n
//
// HBM-bound: forward 7 to 9 bytes per element, backward 8.  A row lies in the
// registers of the threads that share it (8 consecutive values per thread and
// load, 16 lanes to a 128-wide tile), so every input is read once.  The threads
// of a row are one wave, whose sums need no barrier, or up to sixteen.

#include "device.hpp"
#include "internal.hpp"

namespace fp8bs {

namespace {

// Sum over a wave64; every lane receives it.
__device__ __forceinline__ float sum_wave64(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  v += dpp_f32<0x140>(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// Sum over the threads of a row (blockDim.x, whole waves); every thread
// receives it, always in the same order.  `red`: 16 floats that no wave of the
// row still reads from an earlier call.
__device__ __forceinline__ float sum_row(float v, float* red) {
  v = sum_wave64(v);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += red[w];
  return s;
}

__device__ __forceinline__ void unpack8(const u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = bf16_lo(v[e]);
    f[2 * e + 1] = bf16_hi(v[e]);
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
               bf16x2_rne(f[6], f[7])};
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// Squares of finite values past 2^64 leave FP32: such a row is summed again at
// this scale, whose square takes no bit from a sum that large.
constexpr float kTiny = 0x1p-80f;

template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.M) return;  // rows of one wave only: nobody waits
  const int T = (int)blockDim.x;
  const int K = (int)a.K;
  u32x4 h[V];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
    h[i] = u32x4{0u, 0u, 0u, 0u};
    if (col >= K) continue;
    h[i] = *reinterpret_cast<const u32x4*>(a.x + row * a.ldx + col);
    if (a.residual) {
      const u32x4 r = *reinterpret_cast<const u32x4*>(a.residual + row * a.ldr + col);
      float f[8], fr[8];
      unpack8(h[i], f);
      unpack8(r, fr);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += fr[e];
      h[i] = pack8(f);
    }
    if (a.h) *reinterpret_cast<u32x4*>(a.h + row * a.ldh + col) = h[i];
    float f[8];
    unpack8(h[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(f[e], f[e], sum);
  }
  sum = sum_row(sum, red[0]);
  float rstd = 1.0f / sqrtf(sum / (float)K + a.eps);
  if (sum == __builtin_inff()) {  // the same for every thread of the row
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack8(h[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(f[e] * kTiny, f[e] * kTiny, sum);
    }
    sum = sum_row(sum, red[1]);
    rstd = kTiny / sqrtf(sum / (float)K);
  }
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
    if (col >= K) continue;
    float f[8], g[8];
    unpack8(h[i], f);
    load8(a.weight + col, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * g[e];
    if (a.y) *reinterpret_cast<u32x4*>(a.y + row * a.ldy + col) = pack8(f);
    if (a.q) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
      float s, r;
      group_scale(max_row16(m), s, r);
      uint32_t lo = cvt2_e4m3<false>(f[0] * r, f[1] * r, 0u);
      lo = cvt2_e4m3<true>(f[2] * r, f[3] * r, lo);
      uint32_t hi = cvt2_e4m3<false>(f[4] * r, f[5] * r, 0u);
      hi = cvt2_e4m3<true>(f[6] * r, f[7] * r, hi);
      *reinterpret_cast<u32x2*>(a.q + row * a.ldq + col) = u32x2{lo, hi};
      if ((threadIdx.x & 15) == 0) a.s[(int64_t)(col / 128) * a.lds + row] = s;
    }
  }
}

// Rows b, b + blocks, ... of one workgroup; its sums for dg go to part[b].
template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_backward_kernel(NormGradArgs a) {
  __shared__ float red[2][16];
  __shared__ float fold[64 * 8 * 4];  // rows of one wave: the other rows' sums
  const int T = (int)blockDim.x, K = (int)a.K, R = (int)blockDim.y;
  float g[V][8], dg[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = g[i][e] = 0.0f;
    if (col < K) load8(a.weight + col, g[i]);
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.y; row < a.M;
       row += (int64_t)gridDim.x * R, turn ^= 1) {
    u32x4 y[V], h[V], d[V];
    const float rstd = a.rstd[row];
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * T + (int)threadIdx.x) * 8;
      y[i] = h[i] = d[i] = u32x4{0u, 0u, 0u, 0u};
      if (col >= K) continue;
      y[i] = *reinterpret_cast<const u32x4*>(a.dy + row * a.lddy + col);
      h[i] = *reinterpret_cast<const u32x4*>(a.h + row * a.ldh + col);
      if (a.dh) d[i] = *reinterpret_cast<const u32x4*>(a.dh + row * a.lddh + col);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float fy[8], fh[8];
      unpack8(y[i], fy);
      unpack8(h[i], fh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = fh[e] * rstd;
        c = __builtin_fmaf(fy[e] * g[i][e], n, c);
        dg[i][e] = __builtin_fmaf(fy[e], n, dg[i][e]);
      }
    }
    c = sum_row(c, red[turn]) / (float)K;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * T + (int)threadIdx.x) * 8;
      if (col >= K) continue;
      float fy[8], fh[8], fd[8];
      unpack8(y[i], fy);
      unpack8(h[i], fh);
      unpack8(d[i], fd);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        fd[e] = __builtin_fmaf(rstd, fy[e] * g[i][e] - fh[e] * rstd * c, fd[e]);
      *reinterpret_cast<u32x4*>(a.dx + row * a.lddx + col) = pack8(fd);
    }
  }
  float* const out = a.part + (int64_t)blockIdx.x * K;
  if (R > 1) {  // V == 1, T == 64: added up in row order
#pragma unroll
    for (int e = 0; e < 8; ++e) fold[(threadIdx.y * 8 + e) * 64 + threadIdx.x] = dg[0][e];
    __syncthreads();
    if (threadIdx.y != 0) return;
    for (int r = 1; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e) dg[0][e] += fold[(r * 8 + e) * 64 + threadIdx.x];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
    if (col >= K) continue;
    *reinterpret_cast<float4*>(out + col) = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
    *reinterpret_cast<float4*>(out + col + 4) =
        make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
  }
}

// dg from the workgroups' sums: 64 columns per workgroup, its four waves taking
// every fourth sum (a fixed order).
__global__ __launch_bounds__(256) void rmsnorm_weight_kernel(const float* part, int parts,
                                                             int64_t K, float* dg) {
  __shared__ float sum[4][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t k = (int64_t)blockIdx.x * 64 + lane;  // K is a multiple of 128
  float s = 0.0f;
#pragma unroll 8
  for (int b = wave; b < parts; b += 4) s += part[b * K + k];
  sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0) dg[k] = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
}

// Threads of a row and loads of 8 values per thread.
struct RowPlan {
  int vecs, threads, rows;  // rows: rows per workgroup (of one wave each)
};

RowPlan row_plan(int64_t K) {
  const int lanes = (int)(K / 8);
  RowPlan p;
  p.vecs = lanes <= 512 ? 1 : lanes <= 2048 ? 2 : 4;
  p.threads = ((lanes + p.vecs - 1) / p.vecs + 63) / 64 * 64;
  p.rows = p.threads == 64 ? 4 : 1;
  return p;
}

// Workgroups of the backward pass, each with its own sums for dg.
constexpr int64_t kNormParts = 256;
int64_t norm_parts(int64_t M, int64_t K) {
  const int64_t rows = row_plan(K).rows, blocks = (M + rows - 1) / rows;
  return blocks < kNormParts ? blocks : kNormParts;
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t stream) {
  const RowPlan p = row_plan(a.K);
  const int64_t blocks = (a.M + p.rows - 1) / p.rows;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block((unsigned)p.threads, (unsigned)p.rows);
  switch (p.vecs) {
    case 1: return launch_kernel(rmsnorm_kernel<1>, grid, block, stream, a);
    case 2: return launch_kernel(rmsnorm_kernel<2>, grid, block, stream, a);
    default: return launch_kernel(rmsnorm_kernel<4>, grid, block, stream, a);
  }
}

size_t rmsnorm_backward_workspace(int64_t M, int64_t K) {
  return size_t(norm_parts(M, K)) * size_t(K) * 4;
}

hipError_t launch_rmsnorm_backward(NormGradArgs a, float* dg, void* workspace,
                                   hipStream_t stream) {
  const RowPlan p = row_plan(a.K);
  const int64_t parts = norm_parts(a.M, a.K);
  // one workgroup: its sums are dg
  a.part = parts == 1 ? dg : static_cast<float*>(workspace);
  const dim3 block((unsigned)p.threads, (unsigned)p.rows);
  hipError_t e = hipSuccess;
  if (parts > 0) {
    const dim3 grid((unsigned)parts);
    switch (p.vecs) {
      case 1: e = launch_kernel(rmsnorm_backward_kernel<1>, grid, block, stream, a); break;
      case 2: e = launch_kernel(rmsnorm_backward_kernel<2>, grid, block, stream, a); break;
      default: e = launch_kernel(rmsnorm_backward_kernel<4>, grid, block, stream, a);
    }
  }
  if (e != hipSuccess || parts == 1) return e;
  // no rows: dg is zero
  return launch_kernel(rmsnorm_weight_kernel, dim3((unsigned)(a.K / 64)), dim3(256), stream,
                       static_cast<const float*>(workspace), (int)parts, a.K, dg);
}

}  // namespace fp8bs
