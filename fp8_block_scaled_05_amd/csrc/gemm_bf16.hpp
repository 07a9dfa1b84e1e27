// bf16 matrix product template for gfx950, the engine of the head's cross
// entropy (xent.hip).
//
// D[q][p] = sum_k P(p, k) Q(q, k), FP32 accumulation in
// V_MFMA_F32_16X16X32_BF16.  Either operand is stored with k contiguous (kRow:
// [rows][ld]) or with its rows contiguous (kCol: [k][ld], a transposed view
// read without being transposed in memory).  P is the MFMA's first operand, so
// a lane's four accumulators of a 16x16 tile are four consecutive p of one q:
// p is the output's contiguous dimension.
//
// Structure: WP x WQ waves per BP x BQ output tile; k advances in steps of 64
// (128 bytes per row), copied HBM->LDS by direct buffer loads into one of
// STAGES buffers, STAGES - 1 steps ahead of the step that feeds the MFMAs.
// - kRow stage: rows of 128 bytes, the eight 16-byte chunks XOR-swizzled
//   (lds_swizzle), read as 16-byte fragments.
// - kCol stage: 64 k-rows of 2 BP (or BQ) bytes, the 16-byte chunk c of k-row
//   k in slot c ^ 2 f(k), f(k) = (k & 3) | ((k >> 4) & 1) << 2, so that the
//   eight k-rows that half a wave reads at once lie in different banks; read
//   with the transposing 8-byte LDS load (DS_READ_B64_TR_B16: of 16 lanes
//   that read 4 k-rows x 16 rows, lane l receives row l's four k).
// MFMA half h (of the step's two) takes for lane group g the k values
// 16 g + 8 h .. + 7 of the step, the same for both layouts, so products pair
// matching k.
#pragma once

#include "gemm_kernel.hpp"

namespace fp8bs {
namespace gemm16 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

using gemm::lds_swizzle;

enum Layout { kRow = 0, kCol = 1 };

constexpr int kStep = 64;  // k per LDS stage
constexpr int kNonTemporal = 2;  // cache policy bit of a buffer load

template <int BP_, int BQ_, int WP_, int WQ_, int STAGES_, int LP_, int LQ_>
struct Cfg {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, STAGES = STAGES_;
  static constexpr int LP = LP_, LQ = LQ_;
  static constexpr int NWAVES = WP * WQ, THREADS = 64 * NWAVES;
  static constexpr int TP = BP / WP, TQ = BQ / WQ;
  static constexpr int FP = TP / 16, FQ = TQ / 16;
  // kRow P: the rows are staged permuted within a wave's TP rows so that a
  // lane's accumulators are runs of 4 NI consecutive p
  static constexpr int NI = LP == kCol ? 1 : (FP % 4 == 0 ? 4 : FP % 2 == 0 ? 2 : 1);
  static constexpr int Q_OFF = BP * 128;
  static constexpr int STAGE_BYTES = (BP + BQ) * 128;
  // 1-KB copies per wave and stage, of P then of Q: copy c of wave w is block
  // c NWAVES + w of its operand
  static constexpr int CP = BP / 8 / NWAVES, CQ = BQ / 8 / NWAVES, COPIES = CP + CQ;
  static_assert(BP / 8 % NWAVES == 0 && BQ / 8 % NWAVES == 0, "copies must split evenly");
  static_assert(TP % 16 == 0 && TQ % 16 == 0, "whole MFMA tiles");
  static_assert(LP == kRow || BP >= 128, "swizzle of the k-major stage");
  static_assert(LQ == kRow || BQ >= 128, "swizzle of the k-major stage");
  static_assert(STAGES * STAGE_BYTES <= 160 * 1024, "LDS budget");
  static constexpr bool STREAM_P = false;
};

// The same with P read past the caches: for a P that is read once and would not
// stay in them.
template <class C>
struct Streamed : C {
  static constexpr bool STREAM_P = true;
};

// One operand of a tile.  base: the tile's first row (kRow) or its first
// column of k-row 0 (kCol), at the product's first k.  rows: valid rows, >= 1
// (further rows repeat the last; kCol: a multiple of 8).  k_rows (kCol): valid
// k-rows, >= 1; further ones repeat the last, so the other operand has to
// hold zeros there.
struct Operand {
  const uint16_t* base;
  uint32_t ld;  // bytes
  int rows;
  int k_rows;
};

// Tile row held by LDS row r of a permuted kRow P stage (see NI).
template <class C>
__device__ __forceinline__ int p_row(int r) {
  const int w = r / C::TP, x = r % C::TP, i = x / 16, rr = x % 16;
  return w * C::TP + 16 * C::NI * (i / C::NI) + 4 * C::NI * (rr / 4) + 4 * (i % C::NI) + rr % 4;
}

// First p, within the wave's TP, of the four that lane group g holds in MFMA
// tile i: p_tile(i) + p_lane(g).  (Split so that what depends on i is a
// constant of the unrolled code.)
template <class C>
__device__ __forceinline__ constexpr int p_tile(int i) {
  return 16 * C::NI * (i / C::NI) + 4 * (i % C::NI);
}
template <class C>
__device__ __forceinline__ constexpr int p_lane(int g) {
  return 4 * C::NI * g;
}

__device__ __forceinline__ int col_swizzle(int k) { return 2 * ((k & 3) | (((k >> 4) & 1) << 2)); }

// Per-lane LDS byte offsets of a wave's fragments inside a stage, opaque to
// the optimizer (see gemm::FragOffs).  kRow: o[h] is the 16-byte read of half
// h, tile i at + 2048 i.  kCol: o[0] is tile 0's transposing read, tile i at
// ^ 32 i (the swizzle leaves those bits to be XORed), half h and its k quad e at
// + (8 h + 4 e) k-rows.
struct FragOffs {
  int o[2];
};

template <class C, bool IS_P>
__device__ __forceinline__ FragOffs frag_offsets(int w, int lane) {
  constexpr int T = IS_P ? C::TP : C::TQ, B = IS_P ? C::BP : C::BQ;
  constexpr int OFF = IS_P ? 0 : C::Q_OFF;
  const int g = lane >> 4, l16 = lane & 15;
  FragOffs f;
  if constexpr ((IS_P ? C::LP : C::LQ) == kRow) {
    const int slot = (2 * g) ^ lds_swizzle(l16);
    f.o[0] = OFF + (w * T + l16) * 128 + slot * 16;
    f.o[1] = OFF + (w * T + l16) * 128 + (slot ^ 1) * 16;
  } else {
    static_assert(OFF % 256 == 0 && 2 * B % 256 == 0 && T % 64 == 0, "bits 5 to 7 are the tile's");
    const int k = 16 * g + (l16 >> 2);
    const int chunk = w * T / 8 + ((l16 & 3) >> 1);
    f.o[0] = OFF + k * (2 * B) + (chunk ^ col_swizzle(k)) * 16 + (l16 & 1) * 8;
    f.o[1] = 0;
  }
  asm volatile("" : "+v"(f.o[0]), "+v"(f.o[1]));
  return f;
}

// MFMA operand of tile i and half h.
template <class C, bool IS_P>
__device__ __forceinline__ bf16x8 load_frag(uint8_t* st, const FragOffs& f, int i, int h) {
  constexpr int L = IS_P ? C::LP : C::LQ;
  constexpr int B = IS_P ? C::BP : C::BQ;
  if constexpr (L == kRow) {
    return *reinterpret_cast<const bf16x8*>(st + f.o[h] + 2048 * i);
  } else {
    uint8_t* at = st + (f.o[0] ^ (32 * i)) + 8 * h * 2 * B;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * 2 * B));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

template <class C>
using Acc = v4f[C::FP][C::FQ];

template <class C>
__device__ __forceinline__ void clear(Acc<C>& acc) {
#pragma unroll
  for (int i = 0; i < C::FP; ++i)
#pragma unroll
    for (int j = 0; j < C::FQ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
}

// One operand's share of a wave's copies HBM->LDS: N 1-KB copies per k-step,
// copy c of wave w being block c NWAVES + w.  Byte offsets are relative to the
// operand's base at the step's first k.
template <class C, bool IS_P>
struct Copier {
  static constexpr int B = IS_P ? C::BP : C::BQ, N = IS_P ? C::CP : C::CQ;
  static constexpr bool COL = (IS_P ? C::LP : C::LQ) == kCol;
  static constexpr int CH = B / 8;  // kCol: 16-byte chunks of a k-row
  // kCol: copy c takes k-row k0 + c DK; its chunk goes by c mod 2
  static constexpr int DK = 64 / CH * C::NWAVES;
  static_assert(!COL || DK % 16 == 0, "swizzle by the copy's parity");

  const uint8_t* base;
  uint32_t ld;  // bytes
  int k_rows;
  uint32_t at[COL ? 3 : N];  // kRow: the copies' offsets; kCol: k0 and the two chunks' offsets
  int lds;                 // of copy 0

  __device__ __forceinline__ Copier(const Operand& o, int wave, int lane)
      : base(reinterpret_cast<const uint8_t*>(o.base)), ld(o.ld), k_rows(o.k_rows),
        lds((IS_P ? 0 : C::Q_OFF) + wave * 1024) {
    if constexpr (COL) {
      const int k0 = wave * (64 / CH) + lane / CH, last = (o.rows - 1) / 8;
      at[0] = (uint32_t)k0;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int chunk = (lane % CH) ^ col_swizzle(k0 + z * DK);
        at[1 + z] = (uint32_t)((chunk < last ? chunk : last) * 16);
      }
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const int r = (c * C::NWAVES + wave) * 8 + (lane >> 3);
        int row = IS_P ? p_row<C>(r) : r;
        row = row < o.rows ? row : o.rows - 1;
        at[c] = (uint32_t)row * ld + (uint32_t)(((lane & 7) ^ lds_swizzle(r)) * 16);
      }
    }
  }

  // copy c of k-step s into stage st
  __device__ __forceinline__ void issue(int s, uint8_t* st, int c) const {
#if defined(__HIP_DEVICE_COMPILE__)
    uint32_t v;
    int first = s * kStep;
    if constexpr (COL) {
      // k-rows past the last repeat it
      first = first < k_rows ? first : k_rows - 1;
      const uint32_t left = (uint32_t)(k_rows - 1 - first);
      const uint32_t lim = left < kStep - 1 ? left : kStep - 1;
      const uint32_t k = at[0] + (uint32_t)(c * DK);
      v = (k < lim ? k : lim) * ld + at[1 + (c & 1)];
    } else {
      v = at[c];
    }
    const __amdgpu_buffer_rsrc_t rs =
        gemm::make_rsrc(base + (uint64_t)(uint32_t)first * (COL ? ld : 2u));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (gemm::lds_void*)(st + lds + c * C::NWAVES * 1024), 16, v, 0, 0,
        IS_P && C::STREAM_P ? kNonTemporal : 0);
#endif
  }
};

// Both operands' copies; copy c < CP is P's.
template <class C>
struct Copiers {
  Copier<C, true> p;
  Copier<C, false> q;
  __device__ __forceinline__ Copiers(const Operand& op, const Operand& oq, int wave, int lane)
      : p(op, wave, lane), q(oq, wave, lane) {}
  __device__ __forceinline__ void issue(int s, uint8_t* st, int c) const {
    if (c < C::CP) {
      p.issue(s, st, c);
    } else {
      q.issue(s, st, c - C::CP);
    }
  }
  __device__ __forceinline__ void issue_all(int s, uint8_t* st) const {
#pragma unroll
    for (int c = 0; c < C::COPIES; ++c) issue(s, st, c);
  }
};

// acc += the product over `steps` k-steps (steps >= 0), few MFMAs per step:
// the stream of the operands bounds it, so STAGES - 1 steps are in flight.
template <class C>
__device__ __forceinline__ void product_deep(const Operand& op, const Operand& oq, int steps,
                                             uint8_t* const (&stages)[4], Acc<C>& acc) {
  if (steps <= 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const auto fp = frag_offsets<C, true>(wave / C::WQ, lane);
  const auto fq = frag_offsets<C, false>(wave % C::WQ, lane);
  const Copiers<C> cp(op, oq, wave, lane);
  // step s lives in stage s % STAGES; past the last step its copies are
  // issued again, never read, so that the wait counts stay constants
  // Rows 4 KB apart share their memory channels: workgroups that walk k in step
  // would all ask the same few, so each starts elsewhere in k (72569 x 4096, one
  // row: 158 and 140 us; at other strides the start costs 1%)
  const int start = (int)((blockIdx.x * (op.ld % 4096 == 0 ? 5u : 0u)) % (uint32_t)steps);
  auto last = [&](int s) {
    const int t = s < steps ? s : steps - 1;
    return t + start < steps ? t + start : t + start - steps;
  };
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) cp.issue_all(last(s), stages[s]);
  for (int s = 0; s < steps; s += C::STAGES) {
#pragma unroll
    for (int u = 0; u < C::STAGES; ++u) {
      if (s + u < steps) {
        gemm::barrier_after_vmcnt<(C::STAGES - 2) * C::COPIES>();
        cp.issue_all(last(s + u + C::STAGES - 1), stages[(u + C::STAGES - 1) % C::STAGES]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bf16x8 q[C::FQ];
#pragma unroll
          for (int j = 0; j < C::FQ; ++j) q[j] = load_frag<C, false>(stages[u], fq, j, h);
#pragma unroll
          for (int i = 0; i < C::FP; ++i) {
            const bf16x8 p = load_frag<C, true>(stages[u], fp, i, h);
#pragma unroll
            for (int j = 0; j < C::FQ; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q[j], acc[i][j], 0, 0, 0);
          }
        }
      }
    }
  }
  // every copy has landed and every wave has left the stages
  gemm::barrier_after_vmcnt<0>();
}

// A tile of a product: its operands and its k-steps (even, >= 2).
struct Job {
  Operand p, q;
  int steps;
};

// The tiles number 0 .. n - 1 of one workgroup, MFMA-bound: job(i) describes
// tile i, done(i, acc) takes its finished sums (it may not touch the stages).
//
// Two stages.  A step is 2 FP rows of FQ MFMAs (half h = row / FP, tile i =
// row mod FP).  Row r's P fragment is read from LDS at row r - D, so that the
// read is D FQ MFMAs old when it is used; the Q fragments of the second half
// are read over the first rows.  The step's one barrier stands D rows before
// its end, when the last fragment of the stage has been read: behind it the
// next stage has landed, so the last D rows read the first fragments of the
// next step, and the copies of the step after it refill the stage just left,
// one per row (a burst would fill the copy queue and hold up the wave).  The
// matrix cores so have work through the barrier and the step's change.
//
// The stream of steps runs on over the tiles: the last steps of a tile copy
// the first two of the next, whose first fragments are in registers when the
// tile's sums are handed on, so a tile pays for no empty pipeline.  Past the
// last tile its own first steps are copied again, unused.  The loop over a
// tile's steps is one body without a peeled end: with one, the compiler moves
// the accumulators between the copies of the step, and spills.
//
// Steps taken (rebuilt logits, 4096 x 32512 x 7168): fragments read at the row
// that uses them and a barrier between steps 1.85 ms; read D rows ahead 1.46;
// copies one per row and tiles in rounds 1.39; the stream over the tiles 1.35.
// Four stages of half the k measured slower (twice the L2 requests: loss of 4096
// x 129280 x 7168 5.7 ms against 5.3).
template <class C, class JobF, class DoneF>
__device__ __forceinline__ void run_tiles(int n, uint8_t* const (&stages)[4], JobF&& job_of,
                                          DoneF&& done) {
  static_assert(C::STAGES == 2, "two stages");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const auto fp = frag_offsets<C, true>(wave / C::WQ, lane);
  const auto fq = frag_offsets<C, false>(wave % C::WQ, lane);
  constexpr int D = 3, R = 2 * C::FP, RING = D + 1;
  static_assert(R % RING == 0 && C::FP > D, "ring of P fragments");
  static_assert(C::COPIES - D <= R - D, "copies fit a step's rows");
  // the copies of a step go on into the next step's rows up to this one
  constexpr int LAST_ROW = C::COPIES - D;
  bf16x8 p[RING], q[2][C::FQ];

  if (n <= 0) return;
  Job job = job_of(0);
  Copiers<C> cp(job.p, job.q, wave, lane);
  int off = 0;  // steps of the stream before cp's first
  // the XCDs start at different eighths of k, so that they do not all ask the
  // same memory channels for the same stretch of their operands at one time
  // (4096 x 65536 x 3968 loss 1514 and 1487 us); with k-major operands, whose k
  // runs over rows, it gains nothing and costs registers
  constexpr bool APART = C::LP == kRow && C::LQ == kRow;
  const int xcd = (int)(blockIdx.x % 8);
  int len = job.steps, from = len * xcd / 8;
  auto at = [&](int s) { return !APART ? s : s + from < len ? s + from : s + from - len; };
  auto step = [&](int s, uint8_t* st, uint8_t* next, Acc<C>& acc, const Job& then, bool turn) {
    static_for<0, R>([&](auto r_) {
      constexpr int r = decltype(r_)::value, h = r / C::FP, i = r % C::FP;
      if constexpr (r == R - D) {
        gemm::barrier_after_vmcnt<0>();
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (r == LAST_ROW) {
        if (turn) {  // what is copied from here on is the next tile's
          cp = Copiers<C>(then.p, then.q, wave, lane);
          off = s + 2;
          len = then.steps;
          from = len * xcd / 8;
        }
      }
      if constexpr (r + D < R) {
        p[(r + D) % RING] = load_frag<C, true>(st, fp, (r + D) % C::FP, (r + D) / C::FP);
      } else {
        p[(r + D) % RING] = load_frag<C, true>(next, fp, r + D - R, 0);
      }
      static_for<0, C::FQ>([&](auto j_) {
        constexpr int j = decltype(j_)::value;
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[r % RING], q[h][j], acc[i][j], 0, 0, 0);
        // Q fragments: the second half's over the first FQ rows, the next
        // step's over the last D rows
        if constexpr (j == 0 && r < C::FQ) q[1][r] = load_frag<C, false>(st, fq, r, 1);
        if constexpr (r >= R - D) {
          constexpr int m = (r - (R - D)) * C::FQ + j;  // of D FQ
          if constexpr (m < C::FQ) q[0][m] = load_frag<C, false>(next, fq, m, 0);
        }
        constexpr int c = (r + D) % R;
        if constexpr (j == 0 && c < C::COPIES) {
          if constexpr (r >= R - D) cp.issue(at(s + 2 - off), st, c);
          else cp.issue(at(s + 1 - off), next, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  };

  cp.issue_all(at(0), stages[0]);
#pragma unroll
  for (int c = 0; c < D && c < C::COPIES; ++c) cp.issue(at(1), stages[1], c);
  gemm::barrier_after_vmcnt<(D < C::COPIES ? D : C::COPIES)>();
#pragma unroll
  for (int j = 0; j < C::FQ; ++j) q[0][j] = load_frag<C, false>(stages[0], fq, j, 0);
#pragma unroll
  for (int r = 0; r < D; ++r) p[r] = load_frag<C, true>(stages[0], fp, r, 0);

  for (int i = 0;;) {
    const bool more = i + 1 < n;
    const Job then = job_of(more ? i + 1 : i);
    Acc<C> acc;
    clear<C>(acc);
    for (int s = 0; s < job.steps; s += 2) {
      step(s, stages[0], stages[1], acc, then, s + 2 == job.steps);
      step(s + 1, stages[1], stages[0], acc, then, false);
    }
    off = 0;
    done(i, acc);
    if (!more) break;
    job = then;
    ++i;
  }
  // the copies past the last step have landed, and every wave has left the
  // stages
  gemm::barrier_after_vmcnt<0>();
}

// The stage buffers: separate objects, so that the compiler can tell reads of
// one stage from copies in flight to another.
#define FP8BS_GEMM16_STAGES(C)                                                       \
  __shared__ __attribute__((aligned(16))) uint8_t st0_[C::STAGE_BYTES];              \
  __shared__ __attribute__((aligned(16))) uint8_t st1_[C::STAGE_BYTES];              \
  __shared__ __attribute__((aligned(16))) uint8_t st2_[C::STAGES > 2 ? C::STAGE_BYTES : 16]; \
  __shared__ __attribute__((aligned(16))) uint8_t st3_[C::STAGES > 3 ? C::STAGE_BYTES : 16]; \
  uint8_t* const stages[4] = {st0_, st1_, st2_, st3_}

}  // namespace gemm16
}  // namespace fp8bs
