// Softmax cross entropy of the head's logits, with its gradients, for gfx950.
//
// With logits l(m, v) = x(m) . w(v) (bf16 operands, FP32 sums), the loss of row
// m with target t is lse(m) - l(m, t), lse(m) = log sum_v exp l(m, v).  The
// logits never reach memory:
// - forward: the tiles of the product reduce their logits in registers to one
//   (maximum, sum of exp(l - maximum)) pair per row and wave of columns, and
//   one wave (few rows: one workgroup) per row joins the pairs.
// - backward: with P = exp(l - lse) and G = P - onehot(t), the gradients are
//   dx(m) = dloss(m) sum_v G(m, v) w(v) and dw(v) = sum_m G(m, v) dloss(m) x(m).
//   The vocabulary is taken in pieces: a piece's logits are rebuilt and left
//   as G in bf16 in the workspace, then one launch forms the piece's dw and
//   its part of dx (FP32, added up over the pieces in the workspace).
//
// Roundings.  G is rounded to bf16 (it feeds MFMAs) and carries no dloss, so
// the target's entry, which dominates both gradients, keeps its value near
// -1.  dx takes dloss in FP32 at the end.  dw takes it through x: with
// c = max |dloss| its operand is bf16(x dloss / c), which is x itself where
// dloss is one value for all rows (a mean or a sum), and c in FP32 at the end.
//
// Rows whose target is ignore_index (or outside [0, V)) carry no loss: they
// are left out of all products (the rows that remain are packed together), so
// they cost nothing and whatever they hold, NaN and infinities too, reaches
// no output.

#include "epilogue.hpp"
#include "gemm_bf16.hpp"

namespace fp8bs {

namespace {

using gemm16::kCol;
using gemm16::kRow;
using gemm16::kStep;
using gemm16::Operand;

// Logits: q are the rows of x, p the vocabulary.  Large tiles, their half for a
// last tile of at most 128 rows, and the small tile of few rows or small heads
// (deep stream).
using LogitsCfg = gemm16::Cfg<256, 256, 2, 4, 2, kRow, kRow>;
using LogitsHalf = gemm16::Cfg<256, 128, 4, 2, 2, kRow, kRow>;
using LogitsQuarter = gemm16::Cfg<128, 128, 2, 4, 2, kRow, kRow>;  // see logits_tiles
using LogitsSmall = gemm16::Cfg<128, 64, 4, 1, 4, kRow, kRow>;
// Up to 16 rows, two workgroups per compute unit: copies no rows of x that do not
// exist, and so has more of w in flight (1 x 129280 x 7168, w through the caches:
// 326 us small, 304 so; past them, as launch_few takes it, 265).
using LogitsToken = gemm16::Cfg<128, 16, 2, 1, 3, kRow, kRow>;
// Both at half the width, for heads whose 64x64 tiles fit one round of workgroups:
// a step of fewer copies is shorter (55 x 1615 x 4736: 29 us small, 20 so; 20 x
// 7889 x 4352: 33 and 25; with 395 such tiles, 300 x 5000 x 4096: 41 and 48).
using LogitsNarrow = gemm16::Cfg<64, 64, 2, 2, 4, kRow, kRow>;
using LogitsTokenNarrow = gemm16::Cfg<64, 16, 2, 1, 4, kRow, kRow>;
static_assert(LogitsNarrow::TP == LogitsSmall::TP, "pairs");
// dx: q rows, p hidden, k vocabulary.  dw: q vocabulary, p hidden, k rows.
// Large, and small (two workgroups per compute unit).
using DxCfg = gemm16::Cfg<256, 256, 2, 4, 2, kCol, kRow>;
using DwCfg = gemm16::Cfg<256, 256, 2, 4, 2, kCol, kCol>;
using DxSmall = gemm16::Cfg<128, 128, 2, 2, 2, kCol, kRow>;
using DwSmall = gemm16::Cfg<128, 128, 2, 2, 2, kCol, kCol>;

constexpr int64_t kTile = 256;
constexpr int64_t kMaxTiles = INT32_MAX;  // of one launch: tile numbers are 32 bits
constexpr int64_t kPad = 2 * kStep;  // k-steps come in pairs
// One tile of rows is not packed: 17 x 32003 x 2048 26 us, packed 29; 64 x 129280 x
// 7168 370 and 378.
constexpr int64_t kFewXentRows = LogitsSmall::BQ;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of V columns: whole kPad columns, since dx's k-steps read G up to there.
template <class C>
__host__ __device__ constexpr int64_t tiles_of(int64_t V) {
  return C::BP < kPad ? (V + kPad - 1) / kPad * (kPad / C::BP) : (V + C::BP - 1) / C::BP;
}

int64_t compute_units() { return gemm::device_cus() > 0 ? gemm::device_cus() : 256; }

// Workgroups for `tiles` tiles, `per_cu` of them resident on a compute unit,
// every one taking its share.
dim3 tile_grid(int64_t tiles, int64_t per_cu = 1) {
  const int64_t most = compute_units() * per_cu;
  return dim3((unsigned)(tiles < most ? tiles : most));
}

// What the row pass leaves for the others.
struct Header {
  int32_t rows;     // rows with a loss
  int32_t uniform;  // dloss is one positive, finite value over those rows (backward)
  float c;          // max |dloss| (1 where that is 0 or not finite)
};

struct Rows {
  Header* h;
  int32_t* index;  // packed row -> row
  int32_t* place;  // row -> packed row, or -1
  int32_t* target; // of the packed rows
  float* lse;      // of the packed rows (backward)
  float* dloss;    // of the packed rows (backward)
};

struct RowArgs {
  const int64_t* target;
  int64_t M, V, ignore;
  Rows r;
  const float *lse, *dloss;      // backward
  float *loss_out, *lse_out;     // forward: zeroed for the rows without a loss
  const uint16_t* x;
  int64_t ldx, K;
  uint16_t *xc, *xs;             // see pack_row; xs: backward
};

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;

// One workgroup: numbers the rows with a loss, in order.  write: leaves it all in
// a.r (and the zeros); index: optional, receives the rows of the packed rows
// first .. first + kRowWaves - 1.  Returns the header, to every thread.
__device__ __forceinline__ Header number_rows(const RowArgs& a, bool write, int32_t* index,
                                              int32_t first) {
  __shared__ int32_t count[16];
  __shared__ float red[2][16];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  Header h{0, 0, 1.0f};
  float top = 0.0f, low = INFINITY, high = -INFINITY;
  bool nan = false;
  for (int64_t m0 = 0; m0 < a.M; m0 += kRowThreads) {
    const int64_t m = m0 + threadIdx.x;
    const int64_t t = m < a.M ? a.target[m] : a.ignore;
    const float d = m < a.M && a.dloss ? a.dloss[m] : 0.0f;
    const float l = m < a.M && a.dloss && write ? a.lse[m] : 0.0f;
    const bool valid = m < a.M && t != a.ignore && t >= 0 && t < a.V;
    const unsigned long long mask = __ballot(valid);
    __syncthreads();
    if (lane == 0) count[wave] = __popcll(mask);
    __syncthreads();
    int32_t at = h.rows, all = 0;
    for (int w = 0; w < 16; ++w) {
      at += w < wave ? count[w] : 0;
      all += count[w];
    }
    h.rows += all;
    at += __popcll(mask & ((1ull << lane) - 1ull));
    if (valid && index && at >= first && at < first + kRowWaves) index[at - first] = (int32_t)m;
    if (valid && a.dloss) {
      top = fmaxf(top, fabsf(d));
      low = fminf(low, d);
      high = fmaxf(high, d);
      nan = nan || d != d;
    }
    if (!write || m >= a.M) continue;
    if (valid) {
      a.r.index[at] = (int32_t)m;
      a.r.target[at] = (int32_t)t;
      if (a.dloss) {
        a.r.lse[at] = l;
        a.r.dloss[at] = d;
      }
    } else if (a.loss_out) {
      a.loss_out[m] = a.lse_out[m] = 0.0f;
    }
    a.r.place[m] = valid ? at : -1;
  }
  if (a.dloss) {
    top = max_wave64(top);
    high = max_wave64(high);
    low = -max_wave64(-low);
    nan = __any(nan);
    if (lane == 0) {
      red[0][wave] = top;
      red[1][wave] = !nan && (low == high || low > high) ? low : NAN;  // low > high: no rows
    }
    __syncthreads();
    bool same = true;
    float v = INFINITY;
    top = 0.0f;
    for (int w = 0; w < 16; ++w) {
      top = fmaxf(top, red[0][w]);
      const float x = red[1][w];
      if (x == INFINITY) continue;  // a wave without rows, or of infinite dloss (top)
      same = same && x == x && (v == INFINITY || v == x);
      v = x;
    }
    h.c = top > 0.0f && top < INFINITY ? top : 1.0f;
    // an infinite dloss is not taken as one value for all: it has to reach dw,
    // which takes it through x (c is 1 then)
    h.uniform = same && v == top && v > 0.0f && v < INFINITY ? 1 : 0;
  }
  if (write && threadIdx.x == 0) *a.r.h = h;
  return h;
}

__global__ __launch_bounds__(kRowThreads) void xent_rows_kernel(RowArgs a) {
  number_rows(a, true, nullptr, 0);
}

// Packed row q of x, by one wave; zeros for rows past the last up to a multiple
// of kPad (the last k-steps of dw's product); xs (backward, dloss not uniform):
// the row times dloss / c.  Nothing is packed where x is used in place: all
// rows count and, in the backward pass, end at such a multiple.
__device__ __forceinline__ void pack_row(const RowArgs& a, const Header& h, int64_t q,
                                         int64_t row) {
  const int lane = threadIdx.x & 63;
  const int64_t rows = h.rows, upto = (rows + kPad - 1) / kPad * kPad;
  const bool scaled = a.xs != nullptr && !h.uniform;
  if (q >= upto || (rows == a.M && (a.xs == nullptr || (rows == upto && !scaled)))) return;
  const bool real = q < rows;
  const uint16_t* src = a.x + (real ? row : 0) * a.ldx;
  const float f = scaled && real ? a.dloss[row] / h.c : 1.0f;
  for (int64_t k = lane * 8; k < a.K; k += 512) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (real) v = *reinterpret_cast<const u32x4*>(src + k);
    *reinterpret_cast<u32x4*>(a.xc + q * a.K + k) = v;
    if (scaled) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = bf16x2_rne(bf16_lo(v[e]) * f, bf16_hi(v[e]) * f);
      *reinterpret_cast<u32x4*>(a.xs + q * a.K + k) = w;
    }
  }
}

__global__ __launch_bounds__(256) void xent_pack_kernel(RowArgs a) {
  const int64_t q = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const Header h = *a.r.h;
  pack_row(a, h, q, q < h.rows ? a.r.index[q] : 0);
}

// Both in one launch: every workgroup numbers the rows for itself, the first one
// writes the numbers down.  Up to kFusedRows rows: every workgroup reads all
// targets (loss of 4096 x 1003 x 512 25.9 us fused, 27.6 not; of 6144 x 1003 x
// 2048 63.7 and 59.5).
constexpr int64_t kFusedRows = 4096;
__global__ __launch_bounds__(kRowThreads) void xent_rows_pack_kernel(RowArgs a) {
  __shared__ int32_t index[kRowWaves];
  const int first = (int)blockIdx.x * kRowWaves, wave = threadIdx.x >> 6;
  const Header h = number_rows(a, blockIdx.x == 0, index, first);
  __syncthreads();
  pack_row(a, h, first + wave, first + wave < h.rows ? index[wave] : 0);
}

hipError_t launch_rows(const RowArgs& a, hipStream_t stream) {
  const int64_t padded = cdiv(a.M, kPad) * kPad;
  if (a.M <= kFusedRows && a.M > 0)
    return launch_kernel(xent_rows_pack_kernel, dim3((unsigned)(padded / kRowWaves)),
                         dim3(kRowThreads), stream, a);
  const hipError_t e = launch_kernel(xent_rows_kernel, dim3(1), dim3(kRowThreads), stream, a);
  if (e != hipSuccess || a.M == 0) return e;
  return launch_kernel(xent_pack_kernel, dim3((unsigned)(padded / 4)), dim3(256), stream, a);
}

// Tile number `i` of a raster of PT x QT tiles: 8 p-tiles x all q-tiles, in
// blocks of 8 x 4, before the next 8 p-tiles.
struct TileAt {
  uint32_t p, q;
};
__device__ __forceinline__ TileAt raster(uint32_t i, uint32_t PT, uint32_t QT) {
  constexpr uint32_t GP = 8, GQ = 4;
  const uint32_t p0 = i / (GP * QT) * GP, r = i % (GP * QT);
  const uint32_t gp = PT - p0 < GP ? PT - p0 : GP;
  const uint32_t q0 = r / (GQ * gp) * GQ, rr = r % (GQ * gp);
  const uint32_t gq = QT - q0 < GQ ? QT - q0 : GQ;
  return {p0 + rr / gq, q0 + rr % gq};
}

// Tile number in the raster of the number `i` of T in order of work:
// workgroups go round-robin to the 8 XCDs, 32 compute units each.  Every full
// round of 256 tiles gives each XCD 32 consecutive tiles of the raster (an
// 8 x 4 block sharing its L2) and the XCDs neighbouring blocks, so that a
// panel of the large operand, which several XCDs need, is wanted by all of
// them at one time and comes from HBM once.  The rest of the tiles is dealt
// evenly.  A bijection of [0, T).
__device__ __forceinline__ uint32_t in_rounds(uint32_t i, uint32_t T) {
  const uint32_t full = T / 256 * 256;
  if (i >= full) return full + (uint32_t)gemm::xcd_remap(i - full, T - full);
  const uint32_t x = i % 8, j = i / 8;
  return j / 32 * 256 + x * 32 + j % 32;
}

// Tiles number w, w + G, ... of T for workgroup w of G.
__device__ __forceinline__ int share(uint32_t T, uint32_t w, uint32_t G) {
  return w < T ? (int)((T - w - 1) / G + 1) : 0;
}

__device__ __forceinline__ uint32_t ld2(int64_t ld) { return (uint32_t)(2 * ld); }

struct LossArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* xc;  // packed rows, row stride K (null: few rows, not packed)
  const uint16_t* w;
  int64_t ldw;
  int64_t M, V, K;
  Rows r;
  const int64_t* target;  // few rows: of the rows themselves
  float2* part;           // [rows][blocks]: maximum, sum of a wave's TP columns
  int64_t blocks;         // room for the pairs of a row
  float* at;              // logit of each row's target
};

// Magnitude past which a finite logit times log2 e may leave FP32's range.
constexpr float kFar = 0x1p126f;

// A tile's logits -> its rows' pairs over each wave's TP columns, and the
// targets' logits.
template <class C, bool FEW>
__device__ __forceinline__ void reduce_logits(const LossArgs& a, int64_t rows, int64_t p0,
                                              int64_t q0, gemm16::Acc<C>& acc) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wp = wave / C::WQ, wq = wave % C::WQ;
  const int64_t pw = p0 + wp * C::TP;  // the wave's first column
  if (pw >= a.V) return;
  const int64_t left = a.V - pw;
  const int n = left < C::TP ? (int)left : C::TP;  // its valid columns
  const int pl = gemm16::p_lane<C>(g);
  if (n < C::TP) {  // the vocabulary ends here
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool past = gemm16::p_tile<C>(i) + r >= n - pl;
#pragma unroll
        for (int j = 0; j < C::FQ; ++j) acc[i][j][r] = past ? -INFINITY : acc[i][j][r];
      }
  }
#pragma unroll
  for (int j = 0; j < C::FQ; ++j) {
    const int64_t q = q0 + wq * C::TQ + 16 * j + l16;
    const bool real = q < rows;
    float m = acc[0][j][0];
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) m = fmaxf(m, acc[i][j][r]);
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    // the target's logit, on the one lane that holds it
    int64_t t = -1;
    if (real) t = FEW ? a.target[q] : (int64_t)a.r.target[q];
    const int64_t tp = t - pw;
    if (__any(tp >= 0 && tp < n)) {
      const int d = tp >= 0 && tp < n ? (int)tp - pl : -1;
      float at = 0.0f;
      bool here = false;
#pragma unroll
      for (int i = 0; i < C::FP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool hit = d == gemm16::p_tile<C>(i) + r;
          at = hit ? acc[i][j][r] : at;
          here = here || hit;
        }
      if (here) a.at[q] = at;
    }
    // l - m with log2 e folded in is one FMA.  A block of -inf logits alone has no
    // sum; beside a maximum past kFar the fold would overflow, and of two infinities
    // the difference has no value, so there the sums become the differences first
    const bool far = fabsf(m) > kFar && m != -INFINITY;
    if (__any(far)) {
#pragma unroll
      for (int i = 0; i < C::FP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float l = acc[i][j][r];
          acc[i][j][r] = !far ? l : l == m ? 0.0f : l - m;
        }
    }
    const float b = far || m == -INFINITY ? 0.0f : -m * kLog2e;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        s += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], kLog2e, b));
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (real && g == 0) a.part[q * a.blocks + pw / C::TP] = make_float2(m, s);
    __builtin_amdgcn_sched_barrier(0);  // one j at a time: few registers beside the sums
  }
}

// Rows of a last q-tile of at most 128 rows that runs as half tiles; 0: there
// is none.  Half tiles go over w a second time, so they are taken only where w
// stays in the last-level cache between (kCachedBytes), and only where the
// rounds of workgroups come out shorter, a round of half tiles taking 3/4 of one
// of large tiles (they do not halve a k-step's latency).  Measured: 613 x
// 32003 x 2048, 2 rounds against 1.75: 106 and 95 us; 300 x 129280 x 7168,
// read twice from HBM: 755 and 841 us.
constexpr int64_t kCachedBytes = int64_t(192) << 20;
__device__ __forceinline__ uint32_t half_rows(int64_t rows, int64_t V, int64_t K, uint32_t G) {
  const uint32_t rem = (uint32_t)(rows % LogitsCfg::BQ);
  if (rem == 0 || rem > LogitsHalf::BQ || 2 * V * K > kCachedBytes) return 0;
  const uint32_t PT = (uint32_t)((V + LogitsCfg::BP - 1) / LogitsCfg::BP);
  const uint32_t full = PT * (uint32_t)(rows / LogitsCfg::BQ), idle = full % G ? G - full % G : 0;
  const uint32_t plain = 4 * ((full + PT + G - 1) / G);
  const uint32_t over = PT > idle ? PT - idle : 0;
  const uint32_t halved = full ? 4 * ((full + G - 1) / G) + 3 * ((over + G - 1) / G)
                               : 3 * ((PT + G - 1) / G);
  return halved < plain ? rem : 0;
}

// The product of logits behind both directions: done(C{}, p0, q0, acc) takes the
// tiles that hold rows [0, rows).  Small tiles: one per workgroup.  Large
// tiles: every workgroup takes its share, then its share of the half tiles, the
// workgroups left out of the last round of large ones first.
template <class C, class F>
__device__ __forceinline__ void logits_tiles(const uint16_t* x, int64_t ldx, int64_t rows,
                                             const uint16_t* w, int64_t ldw, int64_t V, int64_t K,
                                             uint32_t QT, uint8_t* const (&stages)[4], F&& done) {
  const uint32_t PT = (uint32_t)tiles_of<C>(V);
  auto job = [&](auto c, int64_t p0, int64_t q0) {
    using T = decltype(c);
    return gemm16::Job{{w + p0 * ldw, ld2(ldw), (int)(V - p0 < T::BP ? V - p0 : T::BP), 0},
                       {x + q0 * ldx, ld2(ldx), (int)(rows - q0 < T::BQ ? rows - q0 : T::BQ), 0},
                       (int)(K / kStep)};
  };
  if constexpr (C::STAGES > 2) {
    if (blockIdx.x >= PT * QT) return;  // whole workgroup
    const TileAt t = raster(in_rounds(blockIdx.x, PT * QT), PT, QT);
    const int64_t p0 = (int64_t)t.p * C::BP, q0 = (int64_t)t.q * C::BQ;
    gemm16::Acc<C> acc;
    gemm16::clear<C>(acc);
    if (q0 < rows && p0 < V) {  // otherwise padding: zeros in any case
      const gemm16::Job j = job(C{}, p0, q0);
      gemm16::product_deep<C>(j.p, j.q, j.steps, stages, acc);
    }
    done(C{}, p0, q0, acc);
  } else {
    const uint32_t w0 = blockIdx.x, G = gridDim.x;
    auto run = [&](auto c, uint32_t id, uint32_t qt, int64_t first_q) {
      using T = decltype(c);
      const uint32_t pt = (uint32_t)((V + T::BP - 1) / T::BP), n = pt * qt;
      auto at = [&](int i) { return raster(in_rounds(id + (uint32_t)i * G, n), pt, qt); };
      gemm16::run_tiles<T>(
          share(n, id, G), stages,
          [&](int i) {
            const TileAt t = at(i);
            return job(c, (int64_t)t.p * T::BP, first_q + (int64_t)t.q * T::BQ);
          },
          [&](int i, gemm16::Acc<T>& acc) {
            const TileAt t = at(i);
            done(c, (int64_t)t.p * T::BP, first_q + (int64_t)t.q * T::BQ, acc);
          });
    };
    const uint32_t half = half_rows(rows, V, K, G), full = half ? QT - 1 : QT;
    run(C{}, w0, full, 0);
    if (half) {
      const uint32_t taken = PT * full % G;
      const uint32_t id = w0 >= taken ? w0 - taken : w0 + G - taken;
      // at most half a round of them is cut once more (613 x 32003 x 2048: 90 us
      // with halves, 85 so); both have pairs of 64 columns
      static_assert(LogitsQuarter::TP == LogitsHalf::TP, "pairs");
      if (2 * PT <= G)
        run(LogitsQuarter{}, id, 1, rows - half);
      else
        run(LogitsHalf{}, id, 1, rows - half);
    }
  }
}

// Forward.  FEW: the rows as they are, in one tile of q.
//
// Many rows: MFMA-bound, in fact by the clock that the board's power allows.
// 4096 x 129280 x 7168: 5.3 ms, 1.43 PFLOP/s, MFMA pipe busy 0.77 of the cycles
// (the library's product alone, which stores the logits: 5.28 ms).  613 x 32003
// x 2048: 79 us, 1.02 PFLOP/s, one round of large tiles and one of quarters.  One
// row: the stream of w, 265 us for 1.85 GB, 7.0 TB/s, read once.
template <class C, bool FEW>
__global__ __launch_bounds__(C::THREADS) void xent_loss_kernel(LossArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  FP8BS_GEMM16_STAGES(C);
  const int64_t rows = FEW ? a.M : a.r.h->rows;
  const bool direct = FEW || rows == a.M;
  logits_tiles<C>(direct ? a.x : a.xc, direct ? a.ldx : a.K, rows, a.w, a.ldw, a.V, a.K,
                  (uint32_t)((rows + C::BQ - 1) / C::BQ), stages,
                  [&](auto c, int64_t p0, int64_t q0, gemm16::Acc<decltype(c)>& acc) {
                    reduce_logits<decltype(c), FEW>(a, rows, p0, q0, acc);
                  });
#endif
}

// The sum s of a pair with maximum m, taken to the larger maximum `top`.  Equal
// maxima are not subtracted: of two infinities the difference has no value.  A NaN
// sum stays NaN, also beside a maximum of -inf (a block of NaN and -inf logits, to
// which the columns past the vocabulary belong).
__device__ __forceinline__ float rescaled(float m, float s, float top) {
  return m == top ? s : s * __builtin_amdgcn_exp2f((m - top) * kLog2e);
}

// (m, s) += (m2, s2)
__device__ __forceinline__ void join_pair(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  s = rescaled(m, s, top) + rescaled(m2, s2, top);
  m = top;
}

// Joins the pairs of a (packed) row: a wave per row, or with FEW, where the
// rows are too few to fill the chip, a workgroup per row.  G: workgroups of the
// product; tp, tp_half: columns per pair, of its large (or small) tiles and of
// its half tiles.
template <bool FEW>
__global__ __launch_bounds__(256) void xent_join_kernel(LossArgs a, uint32_t G, int tp,
                                                        int tp_half, int64_t ignore, float* loss,
                                                        float* lse) {
  __shared__ float2 part[4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t q = FEW ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  const int64_t rows = FEW ? a.M : a.r.h->rows;
  if (q >= rows) return;
  int w = tp;
  if (tp != tp_half && q >= rows - (int64_t)half_rows(rows, a.V, a.K, G)) w = tp_half;
  const int64_t blocks = (a.V + w - 1) / w;
  const float2* p = a.part + q * a.blocks;
  // loaded ahead, and U pairs in flight per lane: with a row's 4040 pairs (FEW, V
  // = 129280) taken one by one 9.7 us, so 4.6 us
  const int64_t row = FEW ? q : (int64_t)a.r.index[q], t = FEW ? a.target[q] : 0;
  const float at = a.at[q];
  constexpr int U = FEW ? 16 : 8, STEP = FEW ? 256 : 64;
  float m = -INFINITY, s = 0.0f;
  for (int64_t b0 = FEW ? threadIdx.x : lane; b0 < blocks; b0 += U * STEP) {
    float2 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = p[b0 + u * STEP < blocks ? b0 + u * STEP : blocks - 1];
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b0 + u * STEP >= blocks) v[u] = make_float2(-INFINITY, 0.0f);
      top = fmaxf(top, v[u].x);
    }
    s = rescaled(m, s, top);
#pragma unroll
    for (int u = 0; u < U; ++u) s += rescaled(v[u].x, v[u].y, top);
    m = top;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) join_pair(m, s, __shfl_xor(m, d, 64), __shfl_xor(s, d, 64));
  if constexpr (FEW) {
    if (lane == 0) part[wave] = make_float2(m, s);
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int k = 1; k < 4; ++k) join_pair(m, s, part[k].x, part[k].y);
    if (t == ignore || t < 0 || t >= a.V) {
      loss[q] = lse[q] = 0.0f;
      return;
    }
  }
  if (lane != 0) return;
  const float l = m + logf(s);
  lse[row] = l;
  loss[row] = l - at;
}

struct GradArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t *xc, *xs;  // packed rows, and those times dloss / c
  const uint16_t* w;
  int64_t ldw;
  int64_t M, V, K;
  Rows r;
  uint16_t* g;      // [rows, whole tiles][ldg] of the piece
  int64_t ldg;      // columns of a piece, a multiple of 256
  int64_t v0, nv;   // the piece's vocabulary [v0, v0 + nv)
  float* dxp;       // FP32 parts of dx, [splits][rows][K], at most dx_rows rows in all
  int64_t dx_rows;
  uint16_t* dw;
  int64_t lddw;
};

// A tile's logits -> G.  Rows past the last and columns past the vocabulary
// are zeros up to whole tiles.
template <class C>
__device__ __forceinline__ void store_g(const GradArgs& a, int64_t rows, int64_t p0, int64_t q0,
                                        gemm16::Acc<C>& acc) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int wp = wave / C::WQ, wq = wave % C::WQ;
  const int64_t pw = p0 + wp * C::TP;
  const int64_t left = a.nv - pw;  // columns from pw on (<= 0: none)
  const int pl = gemm16::p_lane<C>(g);
  const int n = (left < C::TP ? (int)left : C::TP) - pl;  // the lane's first column past them
  static_assert(C::NI % 2 == 0, "runs of 8 or 16 columns per lane");
#pragma unroll
  for (int j = 0; j < C::FQ; ++j) {
    const int64_t q = q0 + wq * C::TQ + 16 * j + l16;
    const bool real = q < rows;
    const float lse = real ? a.r.lse[q] : 0.0f;
    const bool far = fabsf(lse) > kFar;  // see reduce_logits
    if (__any(far)) {
#pragma unroll
      for (int i = 0; i < C::FP; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] -= far ? lse : 0.0f;
    }
    const float b = far ? 0.0f : -lse * kLog2e;
    const int64_t tp = real ? (int64_t)a.r.target[q] - (a.v0 + pw) : -1;
    const int t = tp >= 0 && tp < C::TP ? (int)tp - pl : -1;
    const int last = real ? n : -C::TP;  // a row past the last: zeros
    uint16_t* dst = a.g + q * a.ldg + pw + pl;
#pragma unroll
    for (int i0 = 0; i0 < C::FP; i0 += 2) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int i = i0 + e / 2, r = 2 * (e & 1) + z;
          const int p = gemm16::p_tile<C>(i) + r;
          float v = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][r], kLog2e, b));
          v = t == p ? v - 1.0f : v;
          f[z] = p < last ? v : 0.0f;
        }
        o[e] = bf16x2_rne(f[0], f[1]);
      }
      *reinterpret_cast<u32x4*>(dst + gemm16::p_tile<C>(i0)) = u32x4{o[0], o[1], o[2], o[3]};
    }
    __builtin_amdgcn_sched_barrier(0);  // one j at a time: few registers beside the sums
  }
}

// Backward, first launch of a piece: logits rebuilt, G stored, with zeros in
// rows up to a multiple of kPad (dw's last k-steps).  MFMA-bound as the forward:
// 4096 x 129280 x 7168 5.4 ms, 1.40 PFLOP/s, MFMA pipe busy 0.73.
template <class C>
__global__ __launch_bounds__(C::THREADS) void xent_grad_logits_kernel(GradArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  FP8BS_GEMM16_STAGES(C);
  const int64_t rows = a.r.h->rows;
  static_assert(kPad % C::BQ == 0 || C::BQ % kPad == 0, "whole tiles of padded rows");
  static_assert(LogitsHalf::BQ % kPad == 0, "whole tiles of padded rows");
  const int64_t padded = (rows + kPad - 1) / kPad * kPad;
  logits_tiles<C>(rows == a.M ? a.x : a.xc, rows == a.M ? a.ldx : a.K, rows, a.w + a.v0 * a.ldw,
                  a.ldw, a.nv, a.K, (uint32_t)((padded + C::BQ - 1) / C::BQ), stages,
                  [&](auto c, int64_t p0, int64_t q0, gemm16::Acc<decltype(c)>& acc) {
                    store_g<decltype(c)>(a, rows, p0, q0, acc);
                  });
#endif
}

// A tile of a piece's part of dx, added to the earlier pieces'.
template <class C>
__device__ __forceinline__ void add_dx(const GradArgs& a, int64_t rows, bool first, int64_t split,
                                       int64_t p0, int64_t q0, const gemm16::Acc<C>& acc) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int64_t pw = p0 + wave / C::WQ * C::TP;
  float* out = a.dxp + split * rows * a.K;
  if (pw >= a.K) return;  // K is a multiple of 128: a wave's columns exist or do not
#pragma unroll
  for (int j = 0; j < C::FQ; ++j) {
    const int64_t q = q0 + wave % C::WQ * C::TQ + 16 * j + l16;
    if (q >= rows) continue;
#pragma unroll
    for (int i = 0; i < C::FP; ++i) {
      v4f* d = reinterpret_cast<v4f*>(out + q * a.K + pw + gemm16::p_lane<C>(g) +
                                      gemm16::p_tile<C>(i));
      *d = first ? acc[i][j] : *d + acc[i][j];
    }
  }
}

// v[t] of lane row g (16 lanes each) <-> v[g] of lane row t.
__device__ __forceinline__ void transpose_lane_rows(uint32_t (&v)[4]) {
  typedef uint32_t pair __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int t = 0; t < 4; t += 2) {  // bit 0 of t and of g
    const pair r = __builtin_amdgcn_permlane16_swap(v[t], v[t + 1], false, false);
    v[t] = r.x;
    v[t + 1] = r.y;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {  // bit 1
    const pair r = __builtin_amdgcn_permlane32_swap(v[t], v[t + 2], false, false);
    v[t] = r.x;
    v[t + 2] = r.y;
  }
}

// A tile of a piece's dw.  Lane row g holds columns 4 g .. + 3 of every MFMA
// tile; transposed over four tiles it holds the 16 columns of tile g, and a row
// of dw is stored in whole 128-byte lines, past the caches (613 x 32003 x 2048: 273
// us through them, 254 past them).
template <class C>
__device__ __forceinline__ void store_dw(const GradArgs& a, int64_t p0, int64_t q0,
                                         const gemm16::Acc<C>& acc) {
  static_assert(C::FP % 4 == 0 && C::NI == 1, "groups of four MFMA tiles");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  const int64_t pw = p0 + wave / C::WQ * C::TP;
  const float c = a.r.h->c;
  if (pw >= a.K) return;  // wave-uniform: a wave's columns exist or do not
#pragma unroll
  for (int j = 0; j < C::FQ; ++j) {
    const int64_t q = q0 + wave % C::WQ * C::TQ + 16 * j + l16;
    uint16_t* const row = a.dw + (a.v0 + q) * a.lddw + pw + 16 * g;
#pragma unroll
    for (int i0 = 0; i0 < C::FP; i0 += 4) {
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const v4f v = acc[i0 + t][j] * c;
        lo[t] = bf16x2_rne(v[0], v[1]);
        hi[t] = bf16x2_rne(v[2], v[3]);
      }
      transpose_lane_rows(lo);
      transpose_lane_rows(hi);
      if (q < a.nv) {
        u32x4* d = reinterpret_cast<u32x4*>(row + 16 * i0);
        __builtin_nontemporal_store(u32x4{lo[0], hi[0], lo[1], hi[1]}, d);
        __builtin_nontemporal_store(u32x4{lo[2], hi[2], lo[3], hi[3]}, d + 1);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // one j at a time: few registers beside the sums
  }
}

// Parts that the contraction of dx over a whole piece is cut into: the number
// whose launch (see xent_grad_kernel) ends first by an estimate in k-steps of a
// workgroup, the parts' own cost included: they are written and added up again,
// PART_COST / 4 steps for every 2^20 numbers.  Lane i estimates i + 1 parts;
// whole numbers, so that every wave of every kernel comes to the same.
// kTileSteps: a tile's start and end in steps.
constexpr uint32_t kTileSteps = 3, kMostParts = 32;
template <uint32_t PART_COST>
__device__ __forceinline__ uint32_t dx_splits(const GradArgs& a, int64_t rows, uint32_t tiles_x,
                                              uint32_t tiles_w, uint32_t G) {
  const uint32_t s = threadIdx.x % kMostParts + 1;
  const uint32_t dx = ((uint32_t)(a.ldg / kStep) + s - 1) / s + kTileSteps;
  const uint32_t dw = (uint32_t)((rows + kStep - 1) / kStep) + kTileSteps;
  const uint32_t NX = tiles_x * s, last = NX % G, behind = last ? G - last : 0;
  uint32_t t = NX / G * dx;
  if (last) {
    uint32_t ahead = dx / dw;
    if (ahead * behind > tiles_w) ahead = tiles_w / behind;
    const uint32_t rem = tiles_w - ahead * behind;
    const uint32_t more = rem > behind ? (rem - behind + G - 1) / G : 0;
    const uint32_t all = (rem + G - 1) / G;
    t += ahead ? dx + all * dw : (dx + more * dw > all * dw ? dx + more * dw : all * dw);
  } else {
    t += (tiles_w + G - 1) / G * dw;
  }
  t += (uint32_t)((uint64_t)s * (uint64_t)rows * (uint64_t)a.K * PART_COST >> 22);
  // every part has work in the first piece, which sets them all
  const uint32_t pads = (uint32_t)(((a.V < a.ldg ? a.V : a.ldg) + kPad - 1) / kPad);
  const bool fits = s == 1 || (s <= pads && s * rows <= a.dx_rows);
  uint32_t best = fits ? (t < 0x3ffffff ? t : 0x3ffffff) << 6 | s : ~0u;
#pragma unroll
  for (int d = 1; d < (int)kMostParts; d <<= 1) {
    const uint32_t o = __shfl_xor(best, d, 64);
    best = o < best ? o : best;
  }
  return __builtin_amdgcn_readfirstlane(best) & 63;
}

// A small tile's step takes about half as long.
template <class CX>
constexpr uint32_t part_cost() {
  return CX::BP == 256 ? 3 : 6;
}

// Backward, second launch of a piece: tiles of its part of dx, then of its
// dw.  The dx tiles, long, go round the workgroups; those left out of the last
// round of them take dw tiles worth a dx tile's steps meanwhile; the other dw
// tiles go round all workgroups.
//
// MFMA-bound; both products in one launch, so that neither's last partial round
// leaves compute units idle.  4096 x 129280 x 7168: 11.1 ms, 1.37 PFLOP/s, MFMA
// pipe busy 0.72.  613 x 32003 x 2048: 172 us, 0.93 PFLOP/s; dw's tiles have ten
// steps there and end in stores of 131 MB.
template <class CX, class CW>
__global__ __launch_bounds__(CX::THREADS, 2) void xent_grad_kernel(GradArgs a, int first) {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(CX::STAGE_BYTES == CW::STAGE_BYTES && CX::STAGES == CW::STAGES &&
                    CX::THREADS == CW::THREADS, "one workgroup shape");
  FP8BS_GEMM16_STAGES(CX);
  const int64_t rows = a.r.h->rows;
  const uint32_t w = blockIdx.x, G = gridDim.x;
  const uint32_t PT = (uint32_t)((a.K + CX::BP - 1) / CX::BP);
  const uint32_t QX = (uint32_t)((rows + CX::BQ - 1) / CX::BQ);
  // k-steps in pairs; G is zero past the vocabulary, up to whole tiles
  const uint32_t pairs = (uint32_t)((a.nv + 2 * kStep - 1) / (2 * kStep));
  // by the full piece, the same for all: a shorter last piece may use fewer
  const uint32_t whole =
      dx_splits<part_cost<CX>()>(a, rows, PT * QX, PT * (uint32_t)(a.ldg / CW::BQ), G);
  const uint32_t splits = whole < pairs ? whole : pairs;
  const uint32_t NX = PT * QX * splits;
  {
    using C = CX;
    auto at = [&](int i, uint32_t& split) {
      const uint32_t n = in_rounds(w + (uint32_t)i * G, NX);
      split = n / (PT * QX);
      return raster(n % (PT * QX), PT, QX);
    };
    gemm16::run_tiles<C>(
        share(NX, w, G), stages,
        [&](int i) {
          uint32_t split;
          const TileAt t = at(i, split);
          const int64_t p0 = (int64_t)t.p * C::BP, q0 = (int64_t)t.q * C::BQ;
          const int64_t s0 = (int64_t)pairs * split / splits * 2;
          const int64_t s1 = (int64_t)pairs * (split + 1) / splits * 2, k0 = s0 * kStep;
          return gemm16::Job{{a.w + (a.v0 + k0) * a.ldw + p0, ld2(a.ldw),
                              (int)(a.K - p0 < C::BP ? a.K - p0 : C::BP), (int)(a.nv - k0)},
                             // G: whole tiles of rows
                             {a.g + q0 * a.ldg + k0, ld2(a.ldg), C::BQ, 0},
                             (int)(s1 - s0)};
        },
        [&](int i, const gemm16::Acc<C>& acc) {
          uint32_t split;
          const TileAt t = at(i, split);
          add_dx<C>(a, rows, first, split, (int64_t)t.p * C::BP, (int64_t)t.q * C::BQ, acc);
        });
  }
  {
    using C = CW;
    const uint32_t QW = (uint32_t)((a.nv + C::BQ - 1) / C::BQ), NW = PT * QW;
    const uint32_t steps = (uint32_t)((rows + 2 * kStep - 1) / (2 * kStep) * 2);
    // early tiles: `ahead` for each of the workgroups behind the last round
    const uint32_t last = NX % G, behind = last ? G - last : 0;
    uint32_t ahead = last ? (2 * pairs / splits + kTileSteps) / (steps + kTileSteps) : 0;
    if (ahead * behind > NW) ahead = NW / behind;
    const uint32_t early = ahead * behind, mine = behind && w >= last ? ahead : 0;
    // too few dw tiles for that: the workgroups without a dx tile come first
    const uint32_t id = early ? w : (w >= last ? w - last : w + G - last);
    auto at = [&](int i) {
      const uint32_t n = (uint32_t)i < mine ? w - last + (uint32_t)i * behind
                                            : early + id + ((uint32_t)i - mine) * G;
      return raster(n < early ? n : early + in_rounds(n - early, NW - early), PT, QW);
    };
    const int n = (int)mine + share(NW - early, id, G);
    auto finish = [&](int i, const gemm16::Acc<C>& acc) {
      const TileAt t = at(i);
      store_dw<C>(a, (int64_t)t.p * C::BP, (int64_t)t.q * C::BQ, acc);
    };
    if (steps == 0) {  // no row has a loss
      gemm16::Acc<C> zero;
      gemm16::clear<C>(zero);
      for (int i = 0; i < n; ++i) finish(i, zero);
      return;
    }
    const bool direct = a.r.h->uniform && rows == a.M && rows % kPad == 0;
    const uint16_t* x = direct ? a.x : a.r.h->uniform ? a.xc : a.xs;
    const int64_t ldx = direct ? a.ldx : a.K;
    gemm16::run_tiles<C>(
        n, stages,
        [&](int i) {
          const TileAt t = at(i);
          const int64_t p0 = (int64_t)t.p * C::BP, q0 = (int64_t)t.q * C::BQ;
          return gemm16::Job{{x + p0, ld2(ldx), (int)(a.K - p0 < C::BP ? a.K - p0 : C::BP),
                              (int)steps * kStep},
                             {a.g + q0, ld2(a.ldg), C::BQ, (int)steps * kStep},
                             (int)steps};
        },
        finish);
  }
#endif
}

// dx: adds up its parts (zeros for a row without a loss), 4 columns per thread.
// HBM-bound (43 us at 4096 x 7168).
template <class CX, class CW>
__global__ __launch_bounds__(256) void xent_dx_kernel(GradArgs a, uint32_t G, uint32_t chunks,
                                                      uint16_t* dx, int64_t lddx) {
  const int64_t m = blockIdx.x / chunks;
  const int64_t k = (int64_t)(blockIdx.x % chunks) * 1024 + threadIdx.x * 4;
  const int64_t q = a.r.place[m], rows = a.r.h->rows;
  const uint32_t PT = (uint32_t)((a.K + CX::BP - 1) / CX::BP);
  const uint32_t QX = (uint32_t)((rows + CX::BQ - 1) / CX::BQ);
  const uint32_t splits =
      dx_splits<part_cost<CX>()>(a, rows, PT * QX, PT * (uint32_t)(a.ldg / CW::BQ), G);
  if (k >= a.K) return;
  u32x2 o = {0u, 0u};
  if (q >= 0) {
    v4f s = *reinterpret_cast<const v4f*>(a.dxp + q * a.K + k);
#pragma unroll 4
    for (uint32_t z = 1; z < splits; ++z)
      s += *reinterpret_cast<const v4f*>(a.dxp + (z * rows + q) * a.K + k);
    s = s * a.r.dloss[q];
    o = u32x2{bf16x2_rne(s[0], s[1]), bf16x2_rne(s[2], s[3])};
  }
  *reinterpret_cast<u32x2*>(dx + m * lddx + k) = o;
}

// Workspace, in order; every part starts at a multiple of 256 bytes.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  template <class T>
  T* take(size_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += (n * sizeof(T) + 255) & ~size_t(255);
    return p;
  }
};

Rows take_rows(Carver& c, int64_t M, bool grad) {
  Rows r{};
  r.h = c.take<Header>(1);
  r.index = c.take<int32_t>(M);
  r.place = c.take<int32_t>(M);
  r.target = c.take<int32_t>(M);
  if (grad) {
    r.lse = c.take<float>(M);
    r.dloss = c.take<float>(M);
  }
  return r;
}

// Whether a head's logits take the small tiles: by the estimated rounds of
// workgroups, a round of 256x256 tiles taking 100, of their halves (see half_rows)
// 75, of 128x64 tiles 38 and the first 10 more (loss of 100 x 10000 x 2048: 37 us
// large, 24 small; 100 x 32003 x 2048: 40 and 51; 256 x 32003 x 2048: 53 and 81).
bool small_logits(int64_t M, int64_t V, int64_t K) {
  const int64_t cus = compute_units();
  const bool half = M <= LogitsHalf::BQ && 2 * V * K <= kCachedBytes;
  return 10 + 38 * cdiv(cdiv(M, LogitsSmall::BQ) * cdiv(V, LogitsSmall::BP), cus) <
         (half ? 75 : 100) * cdiv(cdiv(M, LogitsCfg::BQ) * cdiv(V, LogitsCfg::BP), cus);
}

// Whether its small tiles are the narrow ones.
bool narrow_logits(int64_t M, int64_t V) {
  return cdiv(M, LogitsNarrow::BQ) * cdiv(V, LogitsNarrow::BP) <= compute_units();
}

struct LossPlan {
  Rows r;
  uint16_t* xc;
  float2* part;
  int64_t blocks;
  float* at;
  bool small;
  size_t bytes;
};

LossPlan loss_plan(void* ws, int64_t M, int64_t V, int64_t K) {
  Carver c{static_cast<uint8_t*>(ws)};
  LossPlan p{};
  const bool few = M <= kFewXentRows;
  p.small = few || small_logits(M, V, K);
  // half tiles have narrower waves than large ones
  p.blocks = p.small ? cdiv(V, LogitsSmall::TP) : cdiv(V, LogitsHalf::TP);
  p.part = c.take<float2>(M * p.blocks);
  p.at = c.take<float>(M);
  if (!few) {
    p.r = take_rows(c, M, false);
    p.xc = c.take<uint16_t>(cdiv(M, kPad) * kPad * K);
  }
  p.bytes = c.used;
  return p;
}

// The vocabulary is cut into equal pieces, whole tiles each, whose G takes at
// most kPieceBytes.  Fewer pieces waste fewer partial rounds of tiles, which is
// worth more than reading G back from the 256-MB last-level cache: 4096 x 129280
// x 7168 in pieces of 256 MB 16.76 ms, of 1 GB 16.50; 16384 x 50257 x 4096 15.93
// and 15.41.
constexpr int64_t kPieceBytes = int64_t(1) << 30;

// The parts of dx take at most this (or one part).  2000 x 129280 x 512: four parts
// 1218 us, as many as are estimated best 837.
constexpr int64_t kDxBytes = int64_t(256) << 20;

struct GradPlan {
  Rows r;
  uint16_t *xc, *xs, *g;
  int64_t ldg, pieces;
  float* dxp;
  int64_t dx_rows;
  bool small_logits, small;
  size_t bytes;
};

GradPlan grad_plan(void* ws, int64_t M, int64_t V, int64_t K) {
  Carver c{static_cast<uint8_t*>(ws)};
  GradPlan p{};
  const int64_t Mt = cdiv(M > 0 ? M : 1, kTile) * kTile;
  int64_t most = kPieceBytes / (2 * Mt) / kTile * kTile;
  most = most < kTile ? kTile : most;
  p.pieces = cdiv(V, most);
  p.ldg = cdiv(cdiv(V, p.pieces), kTile) * kTile;
  p.pieces = cdiv(V, p.ldg);
  p.small_logits = small_logits(M, p.ldg, K);
  // Small tiles where dw has too few large ones to go round (1000 x 4096 x 1024, 64
  // of them: 67 us large, 57 small; 1000 x 6144 x 1024, 96: 75 and 79) or dx so
  // few that its parts cannot either (130 x 129280 x 512, 2: 184 and 152; 400 x
  // 129280 x 512, 4: 245 and 271).
  const int64_t KT = cdiv(K, kTile);
  p.small = p.ldg / kTile * KT < 96 || Mt / kTile * KT < 4;
  // room for the parts of dx (see dx_splits)
  const int64_t room = kDxBytes / (4 * K);
  const int64_t parts = kMostParts * M < room ? kMostParts * M : room;
  p.dx_rows = M > parts ? M : parts;
  p.r = take_rows(c, M, true);
  p.xc = c.take<uint16_t>(cdiv(M, kPad) * kPad * K);
  p.xs = c.take<uint16_t>(cdiv(M, kPad) * kPad * K);
  p.g = c.take<uint16_t>(Mt * p.ldg);
  p.dxp = c.take<float>(p.dx_rows * K);
  p.bytes = c.used;
  return p;
}

// The forward call of few rows, one tile of q.  A w that cannot stay in the
// last-level cache until it is read again is read past it (1 x 129280 x 7168: 304
// us through the caches, 268 past them; 1 x 20000 x 4096, which stays: 31 and 48).
constexpr int64_t kStreamBytes = int64_t(256) << 20;
template <class C>
hipError_t launch_few(const LossArgs& a, int64_t ignore, float* loss, float* lse,
                      hipStream_t stream) {
  const int64_t tiles = tiles_of<C>(a.V);
  if (tiles > kMaxTiles) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)tiles), block(C::THREADS);
  const hipError_t e =
      2 * a.V * a.K > kStreamBytes
          ? launch_kernel(xent_loss_kernel<gemm16::Streamed<C>, true>, grid, block, stream, a)
          : launch_kernel(xent_loss_kernel<C, true>, grid, block, stream, a);
  if (e != hipSuccess) return e;
  return launch_kernel(xent_join_kernel<true>, dim3((unsigned)a.M), dim3(256), stream, a, 0u,
                       C::TP, C::TP, ignore, loss, lse);
}

}  // namespace

size_t xent_workspace(int64_t M, int64_t V, int64_t K) { return loss_plan(nullptr, M, V, K).bytes; }
size_t xent_grad_workspace(int64_t M, int64_t V, int64_t K) {
  return grad_plan(nullptr, M, V, K).bytes;
}

hipError_t launch_xent(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
                       const int64_t* target, int64_t ignore, float* loss, float* lse, int64_t M,
                       int64_t V, int64_t K, void* workspace, hipStream_t stream) {
  const LossPlan p = loss_plan(workspace, M, V, K);
  const LossArgs a{x, ldx, p.xc, w, ldw, M, V, K, p.r, target, p.part, p.blocks, p.at};
  const dim3 block(LogitsSmall::THREADS), large(LogitsCfg::THREADS);
  const bool narrow = narrow_logits(M, V);
  if (M <= LogitsToken::BQ)
    return narrow ? launch_few<LogitsTokenNarrow>(a, ignore, loss, lse, stream)
                  : launch_few<LogitsToken>(a, ignore, loss, lse, stream);
  if (M <= kFewXentRows)
    return narrow ? launch_few<LogitsNarrow>(a, ignore, loss, lse, stream)
                  : launch_few<LogitsSmall>(a, ignore, loss, lse, stream);
  const int64_t tiles = !p.small ? cdiv(V, LogitsCfg::BP) * cdiv(M, LogitsCfg::BQ)
                        : narrow ? tiles_of<LogitsNarrow>(V) * cdiv(M, LogitsNarrow::BQ)
                                 : cdiv(V, LogitsSmall::BP) * cdiv(M, LogitsSmall::BQ);
  if (tiles > kMaxTiles) return hipErrorInvalidConfiguration;
  hipError_t e = launch_rows({target, M, V, ignore, p.r, nullptr, nullptr, loss, lse, x, ldx, K,
                              p.xc, nullptr}, stream);
  if (e != hipSuccess) return e;
  e = !p.small ? launch_kernel(xent_loss_kernel<LogitsCfg, false>, tile_grid(tiles), large, stream,
                               a)
      : narrow ? launch_kernel(xent_loss_kernel<LogitsNarrow, false>, dim3((unsigned)tiles), block,
                               stream, a)
               : launch_kernel(xent_loss_kernel<LogitsSmall, false>, dim3((unsigned)tiles), block,
                               stream, a);
  if (e != hipSuccess) return e;
  return launch_kernel(xent_join_kernel<false>, dim3((unsigned)cdiv(M, 4)), dim3(256), stream, a,
                       tile_grid(tiles).x, p.small ? LogitsSmall::TP : LogitsCfg::TP,
                       p.small ? LogitsSmall::TP : LogitsHalf::TP, ignore, loss, lse);
}

namespace {

template <class CX, class CW>
hipError_t launch_pieces(const GradPlan& p, GradArgs a, int per_cu, uint16_t* dx, int64_t lddx,
                         hipStream_t stream) {
  using CL = LogitsCfg;
  using CS = LogitsSmall;
  using CN = LogitsNarrow;
  static_assert(CS::BQ == CN::BQ && CS::THREADS == CN::THREADS, "rows and waves alike");
  const bool narrow = narrow_logits(a.M, p.ldg);
  const int64_t QL = cdiv(a.M, CL::BQ), QS = cdiv(a.M, kPad) * (kPad / CS::BQ);
  const int64_t tl = p.small_logits ? QS * (p.ldg / (narrow ? CN::BP : CS::BP))
                                    : QL * (p.ldg / CL::BP);
  const int64_t KT = cdiv(a.K, CX::BP), chunks = cdiv(a.K, 1024);
  const int64_t most = KT * (cdiv(a.M, CX::BQ) * kMostParts + p.ldg / CW::BQ);
  if (tl > kMaxTiles || most > kMaxTiles || a.M * chunks > kMaxTiles)
    return hipErrorInvalidConfiguration;
  const dim3 grid = tile_grid(most, per_cu);
  for (int64_t i = 0; i < p.pieces; ++i) {
    const int64_t left = a.V - i * p.ldg;
    a.v0 = i * p.ldg;
    a.nv = left < p.ldg ? left : p.ldg;
    hipError_t e = hipSuccess;
    if (a.M > 0)
      e = !p.small_logits ? launch_kernel(xent_grad_logits_kernel<CL>, tile_grid(tl),
                                          dim3(CL::THREADS), stream, a)
          : narrow        ? launch_kernel(xent_grad_logits_kernel<CN>, dim3((unsigned)tl),
                                          dim3(CN::THREADS), stream, a)
                          : launch_kernel(xent_grad_logits_kernel<CS>, dim3((unsigned)tl),
                                          dim3(CS::THREADS), stream, a);
    if (e != hipSuccess) return e;
    e = launch_kernel(xent_grad_kernel<CX, CW>, grid, dim3(CX::THREADS), stream, a,
                      i == 0 ? 1 : 0);
    if (e != hipSuccess) return e;
  }
  if (a.M == 0) return hipSuccess;
  return launch_kernel(xent_dx_kernel<CX, CW>, dim3((unsigned)(a.M * chunks)), dim3(256), stream, a,
                       grid.x, (uint32_t)chunks, dx, lddx);
}

}  // namespace

hipError_t launch_xent_backward(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw,
                                const int64_t* target, int64_t ignore, const float* lse,
                                const float* dloss, uint16_t* dx, int64_t lddx, uint16_t* dw,
                                int64_t lddw, int64_t M, int64_t V, int64_t K, void* workspace,
                                hipStream_t stream) {
  const GradPlan p = grad_plan(workspace, M, V, K);
  const GradArgs a{x,   ldx, p.xc, p.xs,  w, ldw, M,     V,         K,
                   p.r, p.g, p.ldg, 0,    0, p.dxp, p.dx_rows, dw, lddw};
  const hipError_t e = launch_rows({target, M, V, ignore, p.r, lse, dloss, nullptr, nullptr, x, ldx,
                                    K, p.xc, p.xs}, stream);
  if (e != hipSuccess) return e;
  return p.small ? launch_pieces<DxSmall, DwSmall>(p, a, 2, dx, lddx, stream)
                 : launch_pieces<DxCfg, DwCfg>(p, a, 1, dx, lddx, stream);
}

}  // namespace fp8bs
