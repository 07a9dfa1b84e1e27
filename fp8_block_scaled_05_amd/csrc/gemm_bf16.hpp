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
};

// One operand of a tile.  base: the tile's first row (kRow) or its first
// column of k-row 0 (kCol), at the product's first k.  rows: valid rows, >= 1
// (further rows repeat the last; kCol: a multiple of 8).  k_rows (kCol): valid
// k-rows, >= 1; further ones repeat the last, so the other operand has to
// hold zeros there.
struct Operand {
  const uint16_t* base;
  int64_t ld;
  int rows;
  int64_t k_rows;
};

// Tile row held by LDS row r of a permuted kRow P stage (see NI).
template <class C>
__device__ __forceinline__ int p_row(int r) {
  const int w = r / C::TP, x = r % C::TP, i = x / 16, rr = x % 16;
  return w * C::TP + 16 * C::NI * (i / C::NI) + 4 * C::NI * (rr / 4) + 4 * (i % C::NI) + rr % 4;
}

// First p, within the wave's TP, of the four that lane group g holds in MFMA
// tile i.
template <class C>
__device__ __forceinline__ constexpr int p_of(int i, int g) {
  return 16 * C::NI * (i / C::NI) + 4 * C::NI * g + 4 * (i % C::NI);
}

__device__ __forceinline__ int col_swizzle(int k) { return 2 * ((k & 3) | (((k >> 4) & 1) << 2)); }

// Byte offset, from the operand's base at the step's first k, of the 16 bytes
// that lane `lane` of 1-KB copy `c` moves.  k_lim: last valid k-row of the
// step (kCol).
template <class C, bool IS_P>
__device__ __forceinline__ uint32_t copy_offset(const Operand& o, int c, int lane, int k_lim) {
  constexpr int B = IS_P ? C::BP : C::BQ;
  if constexpr ((IS_P ? C::LP : C::LQ) == kRow) {
    const int r = c * 8 + (lane >> 3);
    int row = IS_P ? p_row<C>(r) : r;
    row = row < o.rows ? row : o.rows - 1;
    return (uint32_t)row * (uint32_t)(o.ld * 2) + (uint32_t)(((lane & 7) ^ lds_swizzle(r)) * 16);
  } else {
    constexpr int CH = B / 8;          // 16-byte chunks of a k-row
    constexpr int RPC = 64 / CH;       // k-rows per copy
    const int k = c * RPC + lane / CH;
    int chunk = (lane % CH) ^ col_swizzle(k);
    const int last = (o.rows - 1) / 8;
    chunk = chunk < last ? chunk : last;
    const int kk = k < k_lim ? k : k_lim;
    return (uint32_t)kk * (uint32_t)(o.ld * 2) + (uint32_t)(chunk * 16);
  }
}

// Per-lane LDS byte offsets of a wave's fragments inside a stage, opaque to
// the optimizer (see gemm::FragOffs).  kRow: [0], [1] are the 16-byte reads of
// halves 0 and 1, tile i at + 2048 i.  kCol: [i] is tile i's transposing read,
// half h and its k quad e at + (8 h + 4 e) k-rows.
template <int L, int F>
struct FragOffs {
  int o[L == kRow ? 2 : F];
};

template <class C, bool IS_P>
__device__ __forceinline__ FragOffs<IS_P ? C::LP : C::LQ, IS_P ? C::FP : C::FQ> frag_offsets(
    int w, int lane) {
  constexpr int L = IS_P ? C::LP : C::LQ, F = IS_P ? C::FP : C::FQ;
  constexpr int T = IS_P ? C::TP : C::TQ, B = IS_P ? C::BP : C::BQ;
  constexpr int OFF = IS_P ? 0 : C::Q_OFF;
  const int g = lane >> 4, l16 = lane & 15;
  FragOffs<L, F> f;
  if constexpr (L == kRow) {
    const int slot = (2 * g) ^ lds_swizzle(l16);
    f.o[0] = OFF + (w * T + l16) * 128 + slot * 16;
    f.o[1] = OFF + (w * T + l16) * 128 + (slot ^ 1) * 16;
    asm volatile("" : "+v"(f.o[0]), "+v"(f.o[1]));
  } else {
    const int k = 16 * g + (l16 >> 2);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int chunk = (w * T + 16 * i) / 8 + ((l16 & 3) >> 1);
      f.o[i] = OFF + k * (2 * B) + (chunk ^ col_swizzle(k)) * 16 + (l16 & 1) * 8;
      asm volatile("" : "+v"(f.o[i]));
    }
  }
  return f;
}

// MFMA operand of tile i and half h.
template <class C, bool IS_P, class FO>
__device__ __forceinline__ bf16x8 load_frag(uint8_t* st, const FO& f, int i, int h) {
  constexpr int L = IS_P ? C::LP : C::LQ;
  constexpr int B = IS_P ? C::BP : C::BQ;
  if constexpr (L == kRow) {
    return *reinterpret_cast<const bf16x8*>(st + f.o[h] + 2048 * i);
  } else {
    const s16x4 a =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(st + f.o[i] + (8 * h) * 2 * B));
    const s16x4 b =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(st + f.o[i] + (8 * h + 4) * 2 * B));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
}

template <class C>
using Acc = v4f[C::FP][C::FQ];

// acc += the product over `steps` k-steps (steps >= 0).
template <class C>
__device__ __forceinline__ void product(const Operand& op, const Operand& oq, int64_t steps,
                                        uint8_t* const (&stages)[4], Acc<C>& acc) {
  if (steps <= 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int wp = wave / C::WQ, wq = wave % C::WQ;
  const auto fp = frag_offsets<C, true>(wp, lane);
  const auto fq = frag_offsets<C, false>(wq, lane);

  const int64_t step_p = C::LP == kCol ? op.ld * (2 * kStep) : 2 * kStep;
  const int64_t step_q = C::LQ == kCol ? oq.ld * (2 * kStep) : 2 * kStep;
  uint32_t off[C::COPIES];
#pragma unroll
  for (int c = 0; c < C::COPIES; ++c)
    off[c] = c < C::CP
                 ? copy_offset<C, true>(op, c * C::NWAVES + wave, lane, kStep - 1)
                 : copy_offset<C, false>(oq, (c - C::CP) * C::NWAVES + wave, lane, kStep - 1);

  // copies of k-step s (past the last step: the last again, never read)
  auto issue = [&](int64_t s, uint8_t* st) {
    const int64_t sc = s < steps ? s : steps - 1;
    const __amdgpu_buffer_rsrc_t rp =
        gemm::make_rsrc(reinterpret_cast<const uint8_t*>(op.base) + sc * step_p);
    const __amdgpu_buffer_rsrc_t rq =
        gemm::make_rsrc(reinterpret_cast<const uint8_t*>(oq.base) + sc * step_q);
    // k-rows that end inside this step: further ones repeat the last
    const int64_t lp = op.k_rows - 1 - sc * kStep, lq = oq.k_rows - 1 - sc * kStep;
    const bool cut_p = C::LP == kCol && lp < kStep - 1, cut_q = C::LQ == kCol && lq < kStep - 1;
#pragma unroll
    for (int c = 0; c < C::CP; ++c) {
      const int b = c * C::NWAVES + wave;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rp, (gemm::lds_void*)(st + b * 1024), 16,
          cut_p ? copy_offset<C, true>(op, b, lane, (int)lp) : off[c], 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < C::CQ; ++c) {
      const int b = c * C::NWAVES + wave;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rq, (gemm::lds_void*)(st + C::Q_OFF + b * 1024), 16,
          cut_q ? copy_offset<C, false>(oq, b, lane, (int)lq) : off[C::CP + c], 0, 0, 0);
    }
  };
  auto compute = [&](uint8_t* st) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 q[C::FQ];
#pragma unroll
      for (int j = 0; j < C::FQ; ++j) q[j] = load_frag<C, false>(st, fq, j, h);
#pragma unroll
      for (int i = 0; i < C::FP; ++i) {
        const bf16x8 p = load_frag<C, true>(st, fp, i, h);
#pragma unroll
        for (int j = 0; j < C::FQ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q[j], acc[i][j], 0, 0, 0);
      }
    }
  };

  // step s lives in stage s % STAGES; STAGES - 1 steps are in flight ahead
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) issue(s, stages[s]);
  for (int64_t s = 0; s < steps; s += C::STAGES) {
#pragma unroll
    for (int u = 0; u < C::STAGES; ++u) {
      if (s + u < steps) {
        gemm::barrier_after_vmcnt<(C::STAGES - 2) * C::COPIES>();
        issue(s + u + C::STAGES - 1, stages[(u + C::STAGES - 1) % C::STAGES]);
        compute(stages[u]);
      }
    }
  }
  // every copy has landed and every wave has left the stages
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
