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
//
// At 4096 x 7168: forward 36 us, 42 with y and rstd (6.2 TB/s of 265 MB; a large
// copy reaches 5.2), bf16 output alone 19 (its operands lie in the last-level
// cache), backward 49 (4.8 TB/s of 235 MB).  One row 4 us: a load, a sum over the
// row's waves and a store in turn.  Rows past 16384 (four loads per thread): forward
// 5.2 to 5.8 TB/s, backward 3.1 to 3.7, one workgroup to a compute unit with 44 of
// its registers in scratch (2048 x 32768 167 us; 4096 x 16384 98, 5.5 TB/s).

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
// receives it, always in the same order.  `red`: 16 floats, shared by the
// workgroup's rows, that no wave still reads from an earlier call.
__device__ __forceinline__ float sum_row(float v, float* red) {
  v = sum_wave64(v);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;  // rows of one wave: nobody waits
  red += (int)threadIdx.y * waves;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += red[w];
  return s;
}

// 16 or 8 bytes to p; STREAM: past the caches' retention.
template <bool STREAM, class T>
__device__ __forceinline__ void store_vec(T v, void* p) {
  if constexpr (STREAM) {
    __builtin_nontemporal_store(v, static_cast<T*>(p));
  } else {
    *static_cast<T*>(p) = v;
  }
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

// Squares of finite values past 2^64 leave FP32, and so may their mean with an eps
// near FP32's largest value: such a row is summed again at this scale, whose square
// takes no bit from a sum that large.
constexpr float kTiny = 0x1p-80f;

template <int V, bool STREAM>
__global__ __launch_bounds__(1024) void rmsnorm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= a.M) return;  // rows of one wave only: nobody waits
  const int T = (int)blockDim.x;
  const int K = (int)a.K;
  u32x4 h[V];
  // the weight is on its way during the sum, where registers allow
  constexpr bool EARLY = V <= 2;
  float g[EARLY ? V : 1][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
    h[i] = u32x4{0u, 0u, 0u, 0u};
    if (col >= K) continue;
    if constexpr (EARLY) load8(a.weight + col, g[i]);
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
    if (a.h) store_vec<STREAM>(h[i], a.h + row * a.ldh + col);
    float f[8];
    unpack8(h[i], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(f[e], f[e], sum);
  }
  sum = sum_row(sum, red[0]);
  const float var = sum / (float)K + a.eps;
  float rstd = 1.0f / sqrtf(var);
  if (var == __builtin_inff()) {  // the same for every thread of the row
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack8(h[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(f[e] * kTiny, f[e] * kTiny, sum);
    }
    sum = sum_row(sum, red[1]);
    rstd = kTiny / sqrtf(__builtin_fmaf(a.eps * kTiny, kTiny, sum / (float)K));
  }
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
    if (col >= K) continue;
    float f[8];
    unpack8(h[i], f);
    if constexpr (!EARLY) load8(a.weight + col, g[0]);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * g[EARLY ? i : 0][e];
    if (a.y) store_vec<STREAM>(pack8(f), a.y + row * a.ldy + col);
    if (a.q) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
      float s, r;
      group_scale(max_row16(m), s, r);
      store_vec<STREAM>(codes8(f, r), a.q + row * a.ldq + col);
      if ((threadIdx.x & 15) == 0) a.s[(int64_t)(col / 128) * a.lds + row] = s;
    }
  }
}

// R rows at a time (blockDim.y), workgroup b the groups b, b + blocks, ... of
// them; its sums for dg go to part[b].
template <int V, bool STREAM>
__global__ __launch_bounds__(1024) void rmsnorm_backward_kernel(NormGradArgs a) {
  __shared__ float red[2][16];
  __shared__ __attribute__((aligned(16))) float fold[V > 2 ? 4 : 512 * 8 * V];
  const int T = (int)blockDim.x, K = (int)a.K, R = (int)blockDim.y;
  // the weight stays in registers where they allow it
  constexpr bool KEEP = V <= 2;
  float g[KEEP ? V : 1][8], dg[V][8];
  auto weight = [&](int i) -> const float (&)[8] {
    if constexpr (!KEEP) load8(a.weight + (i * T + (int)threadIdx.x) * 8, g[0]);
    return g[KEEP ? i : 0];
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[i][e] = g[KEEP ? i : 0][e] = 0.0f;
    if constexpr (KEEP) {
      if (col < K) load8(a.weight + col, g[i]);
    }
  }
  auto load = [&](const uint16_t* p) {
    const u32x4* v = reinterpret_cast<const u32x4*>(p);
    return STREAM ? __builtin_nontemporal_load(v) : *v;
  };
  int turn = 0;
  // all rows of a group go through the same number of turns: they may meet
  for (int64_t first = (int64_t)blockIdx.x * R; first < a.M;
       first += (int64_t)gridDim.x * R, turn ^= 1) {
    const int64_t row = first + threadIdx.y;
    const bool live = row < a.M;
    u32x4 y[V], h[V], d[V];
    const float rstd = live ? a.rstd[row] : 0.0f;
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * T + (int)threadIdx.x) * 8;
      y[i] = h[i] = d[i] = u32x4{0u, 0u, 0u, 0u};
      if (col >= K || !live) continue;
      y[i] = load(a.dy + row * a.lddy + col);
      h[i] = load(a.h + row * a.ldh + col);
      if (a.dh) d[i] = load(a.dh + row * a.lddh + col);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if ((i * T + (int)threadIdx.x) * 8 >= K) continue;
      float fy[8], fh[8];
      unpack8(y[i], fy);
      unpack8(h[i], fh);
      const float (&w)[8] = weight(i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = fh[e] * rstd;
        c = __builtin_fmaf(fy[e] * w[e], n, c);
        dg[i][e] = __builtin_fmaf(fy[e], n, dg[i][e]);
      }
    }
    c = sum_row(c, red[turn]) / (float)K;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (i * T + (int)threadIdx.x) * 8;
      if (col >= K || !live) continue;
      float fy[8], fh[8], fd[8];
      unpack8(y[i], fy);
      unpack8(h[i], fh);
      unpack8(d[i], fd);
      const float (&w)[8] = weight(i);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        fd[e] = __builtin_fmaf(rstd, fy[e] * w[e] - fh[e] * rstd * c, fd[e]);
      *reinterpret_cast<u32x4*>(a.dx + row * a.lddx + col) = pack8(fd);
    }
  }
  // the rows' sums, halves onto halves
  if constexpr (V <= 2) {
    for (int half = R / 2; half > 0; half /= 2) {
      const int y = (int)threadIdx.y;
      __syncthreads();
      if (y >= half && y < 2 * half) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            fold[((i * 8 + e) * half + y - half) * T + threadIdx.x] = dg[i][e];
      }
      __syncthreads();
      if (y < half) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) dg[i][e] += fold[((i * 8 + e) * half + y) * T + threadIdx.x];
      }
    }
  }
  if (threadIdx.y != 0) return;
  float* const out = a.part + (int64_t)blockIdx.x * K;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (i * T + (int)threadIdx.x) * 8;
    if (col >= K) continue;
    *reinterpret_cast<float4*>(out + col) = make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]);
    *reinterpret_cast<float4*>(out + col + 4) =
        make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]);
  }
}

// dg from the workgroups' sums: 64 columns per workgroup, its sixteen waves taking
// every sixteenth sum, all their loads at once (a fixed order).
__global__ __launch_bounds__(1024) void rmsnorm_weight_kernel(const float* part, int parts,
                                                              int64_t K, float* dg) {
  __shared__ float sum[16][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t k = (int64_t)blockIdx.x * 64 + lane;  // K is a multiple of 128
  float s = 0.0f;
#pragma unroll 16
  for (int b = wave; b < parts; b += 16) s += part[b * K + k];
  sum[wave][lane] = s;
  __syncthreads();
  if (wave != 0) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 16; ++w) s += sum[w][lane];
  dg[k] = s;
}

// Threads of a row and loads of 8 values per thread.
struct RowPlan {
  int vecs, threads;
};

RowPlan row_plan(int64_t K) {
  const int lanes = (int)(K / 8);
  RowPlan p;
  p.vecs = lanes <= 512 ? 1 : lanes <= 2048 ? 2 : 4;
  p.threads = ((lanes + p.vecs - 1) / p.vecs + 63) / 64 * 64;
  return p;
}

// Workgroups of the backward pass, each with its own sums for dg, at most one per
// compute unit, and rows that one takes at a time, up to 1024 threads: 16384 x 1024
// by two waves to a compute unit 79 us, by sixteen 31 (two workgroups each, with
// twice the sums, 34).  Below 64 workgroups one row at a time; above, few
// workgroups pay, their sums are read again (333 x 2048 by 167 of them 9.8 us, by
// 84 8.6; 1531 x 512 by 192 10.1, by 96 8.8).
constexpr int64_t kNormParts = 256;
int rows_at_once(int64_t M, int threads) {
  int r = 1;
  while (2 * r * threads <= 1024 && r * 64 < M) r *= 2;
  return r;
}
int64_t norm_parts(int64_t M, int64_t K) {
  const int64_t rows = rows_at_once(M, row_plan(K).threads), blocks = (M + rows - 1) / rows;
  return blocks < kNormParts ? blocks : kNormParts;
}

// Elements from which on outputs are stored, and the backward pass's inputs read,
// past the caches' retention: 4096 x 7168 forward 46 -> 34 us, backward 51 -> 49.
constexpr int64_t kStreamFrom = int64_t(1) << 21;

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& all, hipStream_t stream) {
  const RowPlan p = row_plan(all.K);
  const int64_t rows = p.threads == 64 ? 4 : 1;  // per workgroup
  const dim3 block((unsigned)p.threads, (unsigned)rows);
  const bool stream_out = all.M * all.K >= kStreamFrom;
  // a grid has fewer than 2^32 threads: rows past that go in further launches
  const int64_t most = (int64_t(1) << 31) / p.threads * rows;
  for (int64_t first = 0; first < all.M; first += most) {
    NormArgs a = all;
    a.M = all.M - first < most ? all.M - first : most;
    a.x += first * a.ldx;
    if (a.residual) a.residual += first * a.ldr;
    if (a.h) a.h += first * a.ldh;
    if (a.y) a.y += first * a.ldy;
    if (a.rstd) a.rstd += first;
    if (a.q) {
      a.q += first * a.ldq;
      a.s += first;
    }
    const dim3 grid((unsigned)((a.M + rows - 1) / rows));
    auto go = [&](auto V) {
      constexpr int v = decltype(V)::value;
      return stream_out ? launch_kernel(rmsnorm_kernel<v, true>, grid, block, stream, a)
                        : launch_kernel(rmsnorm_kernel<v, false>, grid, block, stream, a);
    };
    hipError_t e;
    switch (p.vecs) {
      case 1: e = go(std::integral_constant<int, 1>{}); break;
      case 2: e = go(std::integral_constant<int, 2>{}); break;
      default: e = go(std::integral_constant<int, 4>{});
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
  const dim3 block((unsigned)p.threads, (unsigned)rows_at_once(a.M, p.threads));
  hipError_t e = hipSuccess;
  if (parts > 0) {
    const dim3 grid((unsigned)parts);
    auto go = [&](auto V) {
      constexpr int v = decltype(V)::value;
      return a.M * a.K >= kStreamFrom
                 ? launch_kernel(rmsnorm_backward_kernel<v, true>, grid, block, stream, a)
                 : launch_kernel(rmsnorm_backward_kernel<v, false>, grid, block, stream, a);
    };
    switch (p.vecs) {
      case 1: e = go(std::integral_constant<int, 1>{}); break;
      case 2: e = go(std::integral_constant<int, 2>{}); break;
      default: e = go(std::integral_constant<int, 4>{});
    }
  }
  if (e != hipSuccess || parts == 1) return e;
  // no rows: dg is zero
  return launch_kernel(rmsnorm_weight_kernel, dim3((unsigned)(a.K / 64)), dim3(1024), stream,
                       static_cast<const float*>(workspace), (int)parts, a.K, dg);
}

}  // namespace fp8bs
