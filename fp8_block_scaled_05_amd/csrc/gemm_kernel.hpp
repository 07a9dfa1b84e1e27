// Block-scaled FP8 GEMM kernel template for gfx950 (dense and grouped/MoE).
//
// C = A . B^T with E4M3 operands.  For every 128-wide K group kb the kernel
// forms the FP8 x FP8 partial product of that group in FP32 (one
// V_MFMA_F32_16X16X128_F8F6F4 covers a 16x16 output tile's whole group) and
// promotes it into the FP32 running sum with one multiply-add by
// S_A(m,kb) * S_W(n/128,kb).  Pages: "Advantages of using FP8 for GEMM
// operations in DeepSeek-V3", items 1, 5 and 8 (FP8 GEMM for dense and MoE
// layers; partial results promoted to FP32 registers at fixed intervals of
// the accumulation); "How the unified E4M3 format adds to DeepSeek-V3's
// efficiency", section "Enhanced numerical stability".  The promotion
// interval is the 128-K group, where the scales change.
//
// Structure: WM x WN waves per BM x BN output tile; each wave owns a
// (BM/WM) x (BN/WN) sub-tile made of 16x16 MFMA tiles.  Every K group of A
// and B is copied HBM->LDS by direct buffer_load ... lds (no register
// staging) into one of STAGES LDS buffers; the group's scales go through
// registers into a separate LDS array (with block-scaled B as the finished
// promotion factors S_A(row) * S_W(block), so that the MFMA loop does no
// arithmetic for them).  STAGES-1 groups are in flight while
// one feeds the MFMAs, and the copies of the next group are spread between
// the MFMA rows.  LDS rows are 128 bytes; the eight 16-byte chunks of a row
// are stored XOR-swizzled (lds_swizzle) so that the fragment reads are free
// of bank conflicts.  The lane K order inside an MFMA operand (32 bytes =
// chunks 2g, 2g+1 for lane group g) is the same for A and B, so products
// pair matching K.  Each MFMA's FP32 promotion is issued a few MFMAs later
// (a ring of partial products), so the VALU multiply-adds overlap the matrix
// cores.  B rows are staged permuted within each wave's columns so that a
// lane's MFMA columns are consecutive output columns (vector stores).
//
// Variants: fp32, bf16 or E4M3 output (the last quantized per 1x128 tile
// along N in the epilogue, the next GEMM's input); B scaled per 128x128
// block or, with RowScaledB, per row and K group (weight gradients); dense
// or grouped (MoE) tile schedules.
#pragma once

#include <atomic>

#include "device.hpp"
#include "internal.hpp"

namespace fp8bs {
namespace gemm {

typedef __attribute__((address_space(3))) void lds_void;

// LDS placement of the eight 16-byte K chunks of a 128-byte tile row: chunk c
// of row r is stored in slot c ^ lds_swizzle(r).  The function depends on
// r mod 16 only, so the MFMA reads (16 consecutive rows per fragment) can
// compute it from the lane index; with it the ds_read_b128 fragment reads of
// a wave are free of LDS bank conflicts on gfx950 (measured with
// SQ_LDS_BANK_CONFLICT; plain r & 7 or (r >> 1) & 7 leave 2-way conflicts).
__device__ __forceinline__ int lds_swizzle(int r) { return (r ^ ((r >> 3) & 1)) & 7; }

template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int GROUP_M_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int STAGES = STAGES_, GROUP_M = GROUP_M_;
  static constexpr int NWAVES = WM * WN, THREADS = 64 * NWAVES;
  static constexpr int TM = BM / WM, TN = BN / WN;  // wave sub-tile
  static constexpr int FM = TM / 16, FN = TN / 16;  // 16x16 MFMA tiles per wave
  // weight-block scales of the tile: one per 128 columns
  static constexpr int SB_COUNT = (BN + 127) / 128;
  // B scales per 128x128 block (false) or per row and K group (RowScaledB)
  static constexpr bool ROWB = false;
  // columns of C per tile (half of the tile's B rows with GatedB)
  static constexpr bool GATED = false;
  static constexpr int BNO = BN;
  // matrix products on f16 (see Exact)
  static constexpr bool EXACT = false;
  // block-scaled B: the staged scales are the promotion factors
  // S_A(row) * S_W(block) for each of the tile's SB_COUNT weight blocks
  static constexpr bool PREMUL = true;
  // LDS stage: A rows | B rows; the scales of a stage live in a separate
  // array (activation scales, then weight-block scales) so that the compiler
  // can tell their register->LDS writes from the in-flight tile copies
  static constexpr int A_OFF = 0;
  static constexpr int B_OFF = BM * 128;
  static constexpr int STAGE_BYTES = B_OFF + BN * 128;
  // 1 KB (8 rows) per wave-wide direct load
  static constexpr int TILE_LOADS = (BM + BN) / 8 / NWAVES;
  // the scales go through registers and are written to LDS after the
  // compute, SREG items per thread per stage.  Block-scaled B: item
  // nb * BM + row is the factor S_A(row) * S_W(nb) of tile row `row` and the
  // tile's weight block nb, loaded as its two scales and multiplied before
  // the LDS write (spare items repeat the last block's factors)
  static constexpr int SCALE_ITEMS = SB_COUNT * BM;
  static constexpr int SREG = (SCALE_ITEMS + THREADS - 1) / THREADS;
  // every thread writes its SREG slots (no branch, so no merged wait counts)
  static constexpr int SCALE_FLOATS = SREG * THREADS;
  // vector-memory ops per wave per stage (two scale loads per item)
  static constexpr int LOADS = TILE_LOADS + 2 * SREG;
  static_assert((BM + BN) / 8 % NWAVES == 0, "tile loads must split evenly over waves");
  static_assert(TM % 16 == 0 && TN % 16 == 0, "wave sub-tile must be whole MFMA tiles");
  static_assert(TN <= 128 && 128 % TN == 0, "a wave's columns must share one weight block");
  static_assert(STAGES >= 2 && STAGES <= 4, "2 to 4 LDS stages");
  static_assert(STAGES * STAGE_BYTES <= 160 * 1024, "LDS budget");
  static_assert(LOADS <= 63, "vmcnt range");
};

// The same tile configuration with B scaled per row and 128-K group (one
// scale per column of C per group, like the activation tiles of A) instead of
// per 128x128 block: the weight-gradient GEMM dW = dY^T . X, whose operands
// are both token-grouped activations.
template <class C>
struct RowScaledB : C {
  // items: the BM activation scales, then the BN row scales of B (the
  // factors differ per output element, so they are formed in the MFMA loop)
  static constexpr bool ROWB = true, PREMUL = false;
  static constexpr int SCALE_ITEMS = C::BM + C::BN;
  static constexpr int SREG = (SCALE_ITEMS + C::THREADS - 1) / C::THREADS;
  static constexpr int SCALE_FLOATS = SREG * C::THREADS;
  static constexpr int LOADS = C::TILE_LOADS + SREG;
  static_assert(LOADS <= 63, "vmcnt range");
};

// The same tile configuration for the gated product, whose B holds 2N rows:
// the gate's, then the up projection's.  A tile's first BN/2 B rows are BN/2
// columns' gate rows, the others the same columns' up rows, so that one half of
// the waves along N forms the gate and the other half the up projection, each
// with one weight block, as in the plain product.  N is a multiple of 128.
template <class C>
struct GatedB : C {
  static constexpr bool GATED = true;
  static constexpr int BNO = C::BN / 2;
  // factor items: the gate's weight block, then the up projection's
  static constexpr int SB_COUNT = 2;
  static constexpr int SCALE_ITEMS = 2 * C::BM;
  static constexpr int SREG = (SCALE_ITEMS + C::THREADS - 1) / C::THREADS;
  static constexpr int SCALE_FLOATS = SREG * C::THREADS;
  static constexpr int LOADS = C::TILE_LOADS + 2 * SREG;
  static_assert(C::WN % 2 == 0 && BNO <= 128, "a half's columns share one weight block");
  static_assert(LOADS <= 63, "vmcnt range");
};

// The same tile configuration with exact products: the FP8 matrix instruction
// aligns every 8 products of a lane to their largest and drops what lies 2^-13
// below it (measured), which leaves 1.5e-5 of the sums' size; here the codes are
// widened to f16 (exact) in registers and take four f16 instructions of 32 K each,
// which round like FP32 sums but run at half the rate.
template <class C>
struct Exact : C {
  static constexpr bool EXACT = true;
};

// s_waitcnt vmcnt(N) with the other counters left alone (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// Workgroup barrier after this wave's LDS writes (lgkmcnt) and all but its
// last N vector-memory ops have completed.  __syncthreads() would also wait
// for every direct-to-LDS copy still in flight (its release fence covers
// them), which would drain the copy pipeline at every K group; the memory
// clobber keeps the compiler from moving LDS accesses across the barrier.
template <int N>
__device__ __forceinline__ void barrier_after_vmcnt() {
  wait_vmcnt<N>();
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct TileCoords {
  int64_t row0, row_end, col0;
  const uint8_t* b;
  const float* sb;
  int64_t kb0, KB;  // the tile's K groups: kb0 .. kb0 + KB - 1 (KB >= 1)
  void* c;          // output matrix of the tile (row0, col0 relative to it)
};

// Tile schedules of one launch.
enum Sched {
  kDense = 0,     // one GEMM
  kGroupRows = 1, // row ranges of A per group, one B per group (MoE forward)
  kGroupK = 2     // K ranges per group, one C per group (MoE weight gradient)
};

// Workgroups are dealt round-robin to the 8 XCDs (workgroup b runs on XCD
// b mod 8): give each XCD a contiguous run of the raster of T tiles (the
// first T mod 8 XCDs one tile more than the others), so that concurrently
// resident tiles of one XCD share A and B in its L2.  A bijection of [0, T).
// Used where all tiles cost the same (dense); the grouped schedules, whose
// tiles differ in cost, keep the round-robin order instead.
__device__ __forceinline__ int64_t xcd_remap(int64_t bid, int64_t T) {
  const int64_t x = bid % 8, q = T / 8, r = T % 8;
  return x * q + (x < r ? x : r) + bid / 8;
}

// Coordinates of tile number `i` of a raster with MT tile-rows, which walks
// GROUP_M tile-rows before moving along N: tile-row tm, first column col0.
template <class C>
__device__ __forceinline__ void raster(const GemmArgs& p, int64_t i, int64_t MT, int64_t& tm,
                                       int64_t& col0) {
  const int64_t NT = (p.N + C::BNO - 1) / C::BNO;
  const int64_t per_group = (int64_t)C::GROUP_M * NT;
  const int64_t first_m = (i / per_group) * C::GROUP_M;
  const int64_t gsz = (MT - first_m) < C::GROUP_M ? (MT - first_m) : C::GROUP_M;
  const int64_t in_grp = i % per_group;
  tm = first_m + in_grp % gsz;
  col0 = (in_grp / gsz) * C::BNO;
}

template <class C>
__device__ __forceinline__ void dense_tile(const GemmArgs& p, int64_t i, TileCoords& t) {
  int64_t tm;
  raster<C>(p, i, (p.M + C::BM - 1) / C::BM, tm, t.col0);
  t.b = p.b;
  t.sb = p.sb;
  t.row0 = tm * C::BM;
  t.row_end = p.M;
  t.kb0 = 0;
  t.KB = p.K / 128;
  t.c = p.c;
}

// Range [lo, hi) of group g from the device offsets, clamped to [0, limit]
// and to hi >= lo: offsets that break the documented contract then give
// unspecified results but no access outside the operands.
__device__ __forceinline__ void group_range(const GemmArgs& p, int64_t g, int64_t limit,
                                            int64_t& lo, int64_t& hi) {
  lo = p.group_offsets[g];
  hi = p.group_offsets[g + 1];
  lo = lo < 0 ? 0 : (lo > limit ? limit : lo);
  hi = hi < lo ? lo : (hi > limit ? limit : hi);
}

// Grouped along K: group g owns the K range [off[g], off[g+1]) (multiples of
// 128) and its own output C_g = c + g * c_group_stride; every group has the
// same MT x NT tiles, walked group after group.  KB == 0 for an empty group.
template <class C>
__device__ __forceinline__ void kgrouped_tile(const GemmArgs& p, int64_t i, TileCoords& t,
                                              int out_bytes) {
  const int64_t MT = (p.M + C::BM - 1) / C::BM;
  const int64_t per = MT * ((p.N + C::BN - 1) / C::BN);
  const int64_t g = i / per;
  int64_t tm;
  raster<C>(p, i % per, MT, tm, t.col0);
  t.b = p.b;
  t.sb = p.sb;
  t.row0 = tm * C::BM;
  t.row_end = p.M;
  int64_t o0, o1;
  group_range(p, g, p.K / 128 * 128, o0, o1);
  t.kb0 = o0 / 128;
  t.KB = o1 / 128 - t.kb0;
  t.c = static_cast<char*>(p.c) + g * p.c_group_stride * out_bytes;
}

// Inclusive prefix sum over the 64 lanes of a wave.
__device__ __forceinline__ int wave_incl_sum(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, (unsigned)d, 64);
    v += lane >= d ? u : 0;
  }
  return v;
}

// Grouped raster: group g owns ceil(M_g / BM) tile-rows, in group order.
// The offsets are scanned 64 groups at a time by the whole wave (every wave
// of the workgroup computes the same, uniform, result).
template <class C>
__device__ __forceinline__ int group_row_tiles(const GemmArgs& p, int64_t g) {
  if (g >= p.G) return 0;
  int64_t lo, hi;
  group_range(p, g, p.M, lo, hi);
  return (int)((hi - lo + C::BM - 1) / C::BM);
}

// Total tile-rows over all groups.
template <class C>
__device__ __forceinline__ int64_t grouped_row_tiles(const GemmArgs& p) {
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  for (int64_t base = 0; base < p.G; base += 64)
    total += __builtin_amdgcn_readlane(wave_incl_sum(group_row_tiles<C>(p, base + lane)), 63);
  return total;
}

// Tile `i` of the grouped raster with MT (the total) tile-rows.
template <class C>
__device__ __forceinline__ void grouped_tile(const GemmArgs& p, int64_t i, int64_t MT,
                                             TileCoords& t) {
  const int64_t NB = (p.N + 127) / 128 * (C::GATED ? 2 : 1);
  const int lane = threadIdx.x & 63;
  int64_t tm;
  raster<C>(p, i, MT, tm, t.col0);
  // find the group holding tile-row tm (< MT, so the loop always finds it)
  int64_t seen = 0, g = 0, local = 0;
  for (int64_t base = 0; base < p.G; base += 64) {
    const int cnt = group_row_tiles<C>(p, base + lane);
    const int incl = wave_incl_sum(cnt);
    const int64_t chunk = __builtin_amdgcn_readlane(incl, 63);
    if (tm < seen + chunk) {
      const unsigned long long m = __ballot(seen + incl > tm);
      const int first = __builtin_ctzll(m);
      g = base + first;
      local = tm - seen - __builtin_amdgcn_readlane(incl - cnt, first);
      break;
    }
    seen += chunk;
  }
  int64_t lo, hi;
  group_range(p, g, p.M, lo, hi);
  t.row0 = lo + local * C::BM;
  t.row_end = hi;
  t.b = p.b + g * p.b_group_stride;
  t.sb = p.sb + g * NB * p.sb_ld;
  t.kb0 = 0;
  t.KB = p.K / 128;
  t.c = p.c;
}

// Loop-invariant per-lane byte offsets of one stage's direct copies,
// relative to wave-uniform bases (so each copy needs one 32-bit VGPR).
template <class C>
struct LoadPlan {
  uint32_t tile[C::TILE_LOADS];
  int32_t scale[C::SREG];  // element offset from the tile's S_A (or S_W) column base
  int32_t scaleb[C::SREG]; // factor items: element offset of the S_W block scale
};

// One stage's scales in registers: the S_A (or row-scaled S_W) value of each
// item, and with block-scaled B the item's S_W block scale.
template <class C>
struct ScaleRegs {
  float a[C::SREG];
  float b[C::PREMUL ? C::SREG : 1];
};

template <class C>
__device__ __forceinline__ void make_plan(const GemmArgs& p, const TileCoords& t, int wave,
                                          int lane, LoadPlan<C>& lp) {
  const int64_t NB = (p.N + 127) / 128;
  (void)wave;
  const int rows_a = (int)(t.row_end - t.row0);       // >= 1
  const int rows_b = (int)(p.N - t.col0);             // >= 1
#pragma unroll
  for (int j = 0; j < C::TILE_LOADS; ++j) {
    const int rbase = (wave * C::TILE_LOADS + j) * 8;  // first of 8 rows, A then B
    const int r = rbase + (lane >> 3);
    const int chunk = (lane & 7) ^ lds_swizzle(r);
    if (rbase < C::BM) {
      const int rr = r < rows_a ? r : rows_a - 1;
      lp.tile[j] = (uint32_t)rr * (uint32_t)p.lda + chunk * 16;
    } else {
      // B rows are staged permuted within each wave's TN columns: LDS row
      // 16 f + l of a wave's block holds tile column FN l + f, so the lane
      // that produces MFMA column l of fragment f holds, over f, FN
      // consecutive output columns (one vector store per output row)
      const int rb = r - C::BM, rw = rb % C::TN;
      const int wb = rb / C::TN % (C::GATED ? C::WN / 2 : C::WN);
      const int col = wb * C::TN + C::FN * (rw % 16) + rw / 16;
      uint32_t rr = col < rows_b ? col : rows_b - 1;
      // the up rows, N further (all of W lies within 32-bit offsets)
      if (C::GATED && rb >= C::BN / 2) rr += (uint32_t)p.N;
      lp.tile[j] = rr * (uint32_t)p.ldb + chunk * 16;
    }
  }
#pragma unroll
  for (int s = 0; s < C::SREG; ++s) {
    const int item = (int)threadIdx.x + s * C::THREADS;
    if constexpr (C::PREMUL) {
      // item = nb * BM + row: factor of tile row `row` and weight block nb
      // (blocks past the end of N, and spare items, repeat the last)
      const int row = item % C::BM;
      const int64_t nbl = NB - 1 - t.col0 / 128;
      int nb = item / C::BM;
      nb = nb < C::SB_COUNT ? nb : C::SB_COUNT - 1;
      lp.scale[s] = row < rows_a ? row : rows_a - 1;
      lp.scaleb[s] = (int)((C::GATED ? nb * NB : nb < nbl ? nb : nbl) * p.sb_ld);
    } else if (item < C::BM) {
      lp.scale[s] = item < rows_a ? item : rows_a - 1;
    } else {
      // row-scaled B: row scale of tile column j (columns past N repeat the last)
      const int j = item - C::BM;
      lp.scale[s] = j < rows_b ? j : rows_b - 1;
    }
  }
}

// Buffer resources (base + byte range in SGPRs) of the tile's A rows, B rows,
// activation scales and weight-block scales.  Offsets never leave the range:
// rows past the edge are clamped to the last valid row.
struct Rsrc {
  __amdgpu_buffer_rsrc_t a, b;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base) {
  // raw (stride 0) buffer over [base, base + 4 GiB); 0x00020000 is the
  // gfx9 word-3 setting for untyped dword access
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, 0xFFFFFFFF,
                                           0x00020000);
}

template <class C>
__device__ __forceinline__ Rsrc make_rsrc_set(const GemmArgs& p, const TileCoords& t) {
  Rsrc r;
  r.a = make_rsrc(p.a + t.row0 * p.lda + t.kb0 * 128);
  r.b = make_rsrc(t.b + t.col0 * p.ldb + t.kb0 * 128);
  return r;
}

// Issue tile copy number `idx` (0 <= idx < TILE_LOADS) of K group kb into one
// stage: a 1 KB block (8 rows x 128 B) of A, then of B.
template <class C>
__device__ __forceinline__ void issue_copy(const GemmArgs& p, const Rsrc& rs,
                                           const LoadPlan<C>& lp, int64_t kb, uint8_t* st,
                                           int wave, int idx) {
  (void)p;
  const int rbase = (wave * C::TILE_LOADS + idx) * 8;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rbase < C::BM ? rs.a : rs.b,
                                           (lds_void*)(st + rbase * 128), 16, lp.tile[idx],
                                           (int)(kb * 128), 0, 0);
}

// The scales of K group kb, one fp32 per item, into registers.  Issued before
// the group's tile copies, so that waiting for them (before they are written
// to LDS) leaves the tile copies in flight.
template <class C>
__device__ __forceinline__ void load_scales(const GemmArgs& p, const TileCoords& t,
                                            const LoadPlan<C>& lp, int64_t kb,
                                            ScaleRegs<C>& v) {
  const float* sa = p.sa + (t.kb0 + kb) * p.ldsa + t.row0;
  const float* sb = C::ROWB ? t.sb + (t.kb0 + kb) * p.sb_ld + t.col0
                            : t.sb + (t.col0 / 128) * p.sb_ld + t.kb0 + kb;
#pragma unroll
  for (int s = 0; s < C::SREG; ++s) {
    const int item = (int)threadIdx.x + s * C::THREADS;
    // one load instruction per item slot on every wave (uniform vmcnt counts)
    if constexpr (C::PREMUL) {
      (void)item;
      v.a[s] = sa[lp.scale[s]];
      v.b[s] = sb[lp.scaleb[s]];
    } else {
      const float* src = item < C::BM ? sa : sb;
      v.a[s] = src[lp.scale[s]];
    }
  }
}

template <class C>
__device__ __forceinline__ void store_scales(float* sc, const ScaleRegs<C>& v) {
#pragma unroll
  for (int s = 0; s < C::SREG; ++s)
    sc[(int)threadIdx.x + s * C::THREADS] = C::PREMUL ? v.a[s] * v.b[s] : v.a[s];
}

template <class C>
__device__ __forceinline__ void issue_stage(const GemmArgs& p, const Rsrc& rs,
                                            const LoadPlan<C>& lp, int64_t kb, uint8_t* st,
                                            int wave) {
#pragma unroll
  for (int idx = 0; idx < C::TILE_LOADS; ++idx) issue_copy<C>(p, rs, lp, kb, st, wave, idx);
}

typedef int v4i __attribute__((ext_vector_type(4)));

// Per-lane LDS byte offsets of a wave's MFMA operands inside a stage (the
// same for every stage).  They are made opaque to the optimizer once, so that
// each fragment address is the stage base plus one register plus a constant:
// the LDS lowering then tags every read with the stage's alias scope, and the
// wait-count pass can tell reads of a landed stage from copies still in
// flight to the other stages (an untagged read waits for every copy).
struct FragOffs {
  int a_lo, a_hi, b_lo, b_hi;  // K chunks 2g and 2g+1 of lane group g
  int sa;                      // float index of the lane's first row factor (block-scaled B:
                               // in its wave's weight block) or activation scale (row-scaled B)
  int sbc;                     // row-scaled B: float index of the lane's first column scale
};

template <class C>
__device__ __forceinline__ FragOffs frag_offsets(int wm, int wn, int lane) {
  const int l16 = lane & 15;
  // rows r (r mod 16 == l16) and the K chunk pair 2g, 2g+1 of lane group
  // g = lane / 16; chunk c of row r sits in slot c ^ lds_swizzle(r)
  const int slot0 = (2 * (lane >> 4)) ^ lds_swizzle(l16);
  FragOffs f;
  f.a_lo = C::A_OFF + (wm * C::TM + l16) * 128 + slot0 * 16;
  f.a_hi = C::A_OFF + (wm * C::TM + l16) * 128 + (slot0 ^ 1) * 16;
  f.b_lo = C::B_OFF + (wn * C::TN + l16) * 128 + slot0 * 16;
  f.b_hi = C::B_OFF + (wn * C::TN + l16) * 128 + (slot0 ^ 1) * 16;
  const int block = C::GATED ? wn / (C::WN / 2) : wn * C::TN / 128;
  f.sa = wm * C::TM + 4 * (lane >> 4) + (C::PREMUL ? block * C::BM : 0);
  // the lane's FN output columns are consecutive (permuted B staging)
  f.sbc = C::BM + wn * C::TN + C::FN * l16;
  asm volatile("" : "+v"(f.a_lo), "+v"(f.a_hi), "+v"(f.b_lo), "+v"(f.b_hi), "+v"(f.sa));
  return f;
}

// Two 16-byte LDS reads -> one 32-byte MFMA operand (K chunks 2g, 2g+1).
__device__ __forceinline__ v8i load_frag(const uint8_t* st, int lo, int hi, int row_bytes) {
  const v4i a = *reinterpret_cast<const v4i*>(st + lo + row_bytes);
  const v4i b = *reinterpret_cast<const v4i*>(st + hi + row_bytes);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// One K group from one LDS stage.  The wave's FM x FN MFMAs are issued in
// row-major order; the FP32 promotion of the MFMA issued RING steps earlier
// (long finished) follows each issue, so the VALU multiply-adds overlap the
// matrix cores.  The next stage's copies are spread between the MFMA rows (a
// burst of them would stall the wave at issue while the load pipe drains).
template <class C, bool REFILL, class Refill>
__device__ __forceinline__ void compute_stage(const uint8_t* st, const float* sc,
                                              const FragOffs& fo, v4f (&acc)[C::FM][C::FN],
                                              Refill&& issue_copy_n) {
  constexpr int NM = C::FM * C::FN;
  constexpr int RING = 4;
  // the promotion factors of row i are read until step i*FN + FN - 1 + RING
  // and their slot is refilled at step (i + WS)*FN
  constexpr int WS = 2 + (RING - 1) / C::FN;
  // With two stages the copies of the next group must land before this
  // step ends: issue them over the first half of the rows.  With more stages
  // they have a whole step of slack and are spread over all rows.
  constexpr int ISSUE_ROWS = C::STAGES == 2 ? (C::FM + 1) / 2 : C::FM;
  constexpr int PER_ROW = (C::TILE_LOADS + ISSUE_ROWS - 1) / ISSUE_ROWS;
  // block-scaled B: the stage holds the row factors of the wave's weight
  // block (fo.sa points into them); row-scaled B: the lane's FN column
  // scales, applied per MFMA tile
  static_assert(C::PREMUL != C::ROWB, "block-scaled B stages finished factors");
  float sbj[C::FN];
  if constexpr (C::ROWB) {
    if constexpr (C::FN % 4 == 0) {
#pragma unroll
      for (int q = 0; q < C::FN / 4; ++q) {
        const float4 v = *reinterpret_cast<const float4*>(sc + fo.sbc + 4 * q);
        sbj[4 * q] = v.x;
        sbj[4 * q + 1] = v.y;
        sbj[4 * q + 2] = v.z;
        sbj[4 * q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < C::FN; ++q) sbj[q] = sc[fo.sbc + q];
    }
  }
  // a lane's 4 rows of MFMA row i: one 16-byte LDS read (rows 16 i + 4 g .. + 3)
  const float* w4 = sc + fo.sa;
  v8i bf[C::FN];
#pragma unroll
  for (int j = 0; j < C::FN; ++j) bf[j] = load_frag(st, fo.b_lo, fo.b_hi, 16 * j * 128);
  v8i af[2];
  float4 s4[2];
  float w[WS][4];
  af[0] = load_frag(st, fo.a_lo, fo.a_hi, 0);
  s4[0] = *reinterpret_cast<const float4*>(w4);
  v4f ring[RING];
#pragma unroll
  for (int t = 0; t < NM + RING; ++t) {
    if (t >= RING) {
      const int u = t - RING, i = u / C::FN, j = u % C::FN;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float f = C::ROWB ? w[i % WS][r] * sbj[j] : w[i % WS][r];
        acc[i][j][r] = __builtin_fmaf(ring[u % RING][r], f, acc[i][j][r]);
      }
    }
    if (t < NM) {
      const int i = t / C::FN, j = t % C::FN;
      if (j == 0) {
        // this row's factors (S_A(row) * S_W, or S_A(row) with row-scaled B);
        // prefetch the next row
        w[i % WS][0] = s4[i & 1].x;
        w[i % WS][1] = s4[i & 1].y;
        w[i % WS][2] = s4[i & 1].z;
        w[i % WS][3] = s4[i & 1].w;
        if (i + 1 < C::FM) {
          af[(i + 1) & 1] = load_frag(st, fo.a_lo, fo.a_hi, 16 * (i + 1) * 128);
          s4[(i + 1) & 1] = *reinterpret_cast<const float4*>(w4 + 16 * (i + 1));
        }
      }
      ring[t % RING] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          af[i & 1], bf[j], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
      if (j == C::FN - 1 && REFILL) {
#pragma unroll
        for (int c = i * PER_ROW; c < (i + 1) * PER_ROW && c < C::TILE_LOADS; ++c) issue_copy_n(c);
      }
    }
    // One scheduling region per MFMA.  The partial products are separate
    // values, so without a fence the scheduler places each promotion right
    // after the MFMA that produces it (register pressure is lower there),
    // which stalls the wave on the MFMA latency (hazard NOPs); fenced, the
    // promotion stays RING MFMAs behind its producer.
    __builtin_amdgcn_sched_barrier(0);
  }
  // Keep this group's promotion inside this step: without a use here the
  // compiler sinks the multiply-adds past the next barrier, which piles two
  // groups' VALU work into one step.
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) asm volatile("" : "+v"(acc[i][j]));
}

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Eight E4M3 codes (two dwords) as f16, exact.
__device__ __forceinline__ f16x8 widen8(int lo, int hi) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// What a step of the exact product hands to the next one: the widened operands of
// its first row of tiles, the last pair of tiles, still to be promoted, and its
// row's factors.
template <class C>
struct ExactState {
  f16x8 a[4], b[C::FN][4];
  v8i raw_b[2];    // of the last two B operands, still to be widened
  v4f part[2];
  float4 w, wn;    // factors of the row before and of the first row
};

// One K group with exact products (block-scaled B).  Quarter q of a lane's 32 K
// bytes is the operand of instruction q, on both sides.  The wave's B operands
// stay widened for the step; a row's A operands are widened while the last pair of
// tiles of the row before uses theirs, quarter by quarter into the same registers,
// and the next group's operands likewise around the last row, ahead of which the
// waves meet (`meet`): all of this group's operands are in registers then and the
// next group's copies have landed, so that no wave waits for LDS at a step's
// start.  The promotion of a pair follows while the next one's two chains of four
// instructions run.
//
// Bound by instruction issue and board power: 3.3 VALU instructions to a matrix
// one, the matrix cores busy 0.55 of the time at 2.1 GHz (1.2 PFLOP/s at 4096 x
// 36864 x 7168, 1.77 ms; up to 1.87 on cards that hold less); the LDS reads,
// widening, products and promotions alone reach 0.62 at 2.2, busier orders of them
// hold lower clocks.  Other orders and wave priorities are within 1%.  Tiles of
// 256x256 widen less per product but do not fit the registers (2.35 ms); two stages
// in place of three take 1.96.
template <class C, class Copy, class Meet>
__device__ __forceinline__ void compute_step_exact(const uint8_t* st, const float* sc,
                                                   const uint8_t* st_next, const float* sc_next,
                                                   const FragOffs& fo, ExactState<C>& s,
                                                   v4f (&acc)[C::FM][C::FN], Copy&& issue_copy_n,
                                                   Meet&& meet) {
  static_assert(C::PREMUL && C::FM >= 2 && C::FN == 4, "block-scaled B, four tiles to a row");
  constexpr int NP = 2 * C::FM;  // pairs of tiles
  constexpr int PER_ROW = (C::TILE_LOADS + C::FM - 2) / (C::FM - 1);
  v8i raw_a, raw_b[4];
  raw_b[2] = s.raw_b[0];
  raw_b[3] = s.raw_b[1];
  v4f part[2][2];
  part[1][0] = s.part[0];
  part[1][1] = s.part[1];
  static_for<0, NP>([&](auto t_) {
    constexpr int t = decltype(t_)::value, i = t / 2, h = t % 2;
    constexpr bool last = i == C::FM - 1;
    if constexpr (h == 0 && last) meet();
    if constexpr (h == 0)
      raw_a = load_frag(last ? st_next : st, fo.a_lo, fo.a_hi, last ? 0 : 16 * (i + 1) * 128);
    if constexpr (last) {
      raw_b[2 * h] = load_frag(st_next, fo.b_lo, fo.b_hi, 16 * 2 * h * 128);
      raw_b[2 * h + 1] = load_frag(st_next, fo.b_lo, fo.b_hi, 16 * (2 * h + 1) * 128);
    }
    static_for<0, 4>([&](auto q_) {
      constexpr int q = decltype(q_)::value;
#pragma unroll
      for (int d = 0; d < 2; ++d)
        part[t & 1][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            s.a[q], s.b[2 * h + d][q], q == 0 ? v4f{0.f, 0.f, 0.f, 0.f} : part[t & 1][d], 0, 0, 0);
      // two of the eight promotions of the pair before
      constexpr int u = (t + NP - 1) % NP, ui = u / 2, uj = 2 * (u % 2) + q / 2, r = 2 * (q & 1);
      const float f0 = r == 0 ? s.w.x : s.w.z, f1 = r == 0 ? s.w.y : s.w.w;
      const v4f& pp = part[(t + 1) & 1][q / 2];
      acc[ui][uj][r] = __builtin_fmaf(pp[r], f0, acc[ui][uj][r]);
      acc[ui][uj][r + 1] = __builtin_fmaf(pp[r + 1], f1, acc[ui][uj][r + 1]);
      // operands of the next row or group
      if (t == 0) {
        s.b[2][q] = widen8(raw_b[2][2 * q], raw_b[2][2 * q + 1]);
        s.b[3][q] = widen8(raw_b[3][2 * q], raw_b[3][2 * q + 1]);
      }
      if (last && h == 1) {
        s.b[0][q] = widen8(raw_b[0][2 * q], raw_b[0][2 * q + 1]);
        s.b[1][q] = widen8(raw_b[1][2 * q], raw_b[1][2 * q + 1]);
      }
      if (h == 1) s.a[q] = widen8(raw_a[2 * q], raw_a[2 * q + 1]);
      __builtin_amdgcn_sched_barrier(0);  // LDS reads stay ahead of their use
    });
    if (h == 0) {
      // the row before is promoted: this row's factors, and the next one's
      s.w = s.wn;
      s.wn = *reinterpret_cast<const float4*>(last ? sc_next + fo.sa : sc + fo.sa + 16 * (i + 1));
    }
    if (h == 1 && !last) {
#pragma unroll
      for (int c = i * PER_ROW; c < (i + 1) * PER_ROW && c < C::TILE_LOADS; ++c) issue_copy_n(c);
    }
  });
  s.raw_b[0] = raw_b[2];
  s.raw_b[1] = raw_b[3];
  s.part[0] = part[1][0];
  s.part[1] = part[1][1];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// The LDS arrays of the kernel: one per pipeline stage for the tiles and one
// per stage for the scales (distinct objects, so that the compiler can tell
// the stages apart when it tracks copies in flight).
struct LdsSet {
  uint8_t* st[4];
  float* sc[4];
  float* red;  // E4M3 output: per-wave row maxima [WN][BM]
  float* rcp;  // E4M3 output: per-row reciprocals [BN/128][BM]
};

template <class T, int N>
struct Vec {
  typedef T type __attribute__((ext_vector_type(N)));
};

// The FN values of row r of MFMA row i held by one lane, as the output type:
// fp32, or bf16 packed two per dword (V_CVT_PK_BF16_F32, nearest even).
template <class C, int OUT>
struct RowVals {
  using T = typename std::conditional<OUT == kOutBF16, uint16_t, float>::type;
  typename Vec<T, C::FN>::type v;
  __device__ __forceinline__ RowVals(const v4f (&acc)[C::FM][C::FN], int i, int r) {
    if constexpr (OUT == kOutBF16 && C::FN % 2 == 0) {
      typename Vec<uint32_t, C::FN / 2>::type w;
#pragma unroll
      for (int q = 0; q < C::FN / 2; ++q) w[q] = bf16x2_rne(acc[i][2 * q][r], acc[i][2 * q + 1][r]);
      v = __builtin_bit_cast(typename Vec<T, C::FN>::type, w);
    } else {
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        if constexpr (OUT == kOutBF16) {
          v[j] = f32_to_bf16_rne(acc[i][j][r]);
        } else {
          v[j] = acc[i][j][r];
        }
      }
    }
  }
};

// fp32 or bf16 output.  Lane (g, l) holds rows 16 i + 4 g + r of the wave's
// sub-tile and, through the permuted B staging, the FN consecutive columns
// FN l .. FN l + FN - 1 of the wave's TN columns: one store per row (vector
// when the row start is aligned for it).  A wave whose whole sub-tile lies
// inside C (the common case) stores without per-row tests.
// STREAM: those stores bypass the caches' retention.  Every workgroup of a round
// stores its tile at the same time, and with a second output the bursts are
// larger than the L2s.
template <class C, int OUT, bool STREAM = false>
__device__ __forceinline__ void store_tile(const GemmArgs& p, const TileCoords& t,
                                           const v4f (&acc)[C::FM][C::FN], int wm, int wn,
                                           int lane) {
  using T = typename RowVals<C, OUT>::T;
  using VT = typename Vec<T, C::FN>::type;
  const int g4 = lane >> 4, l16 = lane & 15;
  const int64_t col = t.col0 + wn * C::TN + C::FN * l16;
  const bool vec = C::FN > 1 && reinterpret_cast<uintptr_t>(t.c) % (C::FN * sizeof(T)) == 0 &&
                   p.ldc % C::FN == 0;
  T* const out = reinterpret_cast<T*>(t.c);
  const int64_t wrow0 = t.row0 + wm * C::TM;
  // wave-uniform: every row and column of the wave's sub-tile is inside C
  const bool inside = vec && wrow0 + C::TM <= t.row_end && t.col0 + (wn + 1) * C::TN <= p.N;
  if constexpr (C::FN > 1) {
    if (inside) {
      T* const base = out + (wrow0 + 4 * g4) * p.ldc + col;
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const RowVals<C, OUT> rv(acc, i, r);
          VT* const dst = reinterpret_cast<VT*>(base + (16 * i + r) * p.ldc);
          if constexpr (STREAM) {
            __builtin_nontemporal_store(rv.v, dst);
          } else {
            *dst = rv.v;
          }
        }
        // few addresses at a time (the sums fill the registers)
        if constexpr (STREAM) __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = wrow0 + 16 * i + 4 * g4 + r;
      if (row >= t.row_end) continue;
      const RowVals<C, OUT> rv(acc, i, r);
      T* const dst = out + row * p.ldc + col;
      if constexpr (C::FN > 1) {
        if (vec && col + C::FN <= p.N) {
          *reinterpret_cast<VT*>(dst) = rv.v;
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
        if (col + j < p.N) dst[j] = rv.v[j];
    }
  }
}

// E4M3 output quantized per 1x128 tile along N, the next layer's FP8 input
// (pages: "How online quantization in DeepSeek-V3 differs from delayed
// quantization", item 1, and "How the unified E4M3 format adds to
// DeepSeek-V3's efficiency", section "Fine-grained quantization strategy":
// the same online 1x128 activation quantization, applied to the FP32 output
// before it leaves the kernel).  A row's 128-column tile spans 128 / TN
// waves: each wave reduces its TN columns (lanes, then the 16 lanes of a
// DPP row), the partial maxima meet in LDS, one thread per (row, tile)
// forms the scale and reciprocal exactly as the activation quantizer does,
// and each lane converts and stores its FN consecutive codes per row.
// Requires BN % 128 == 0 and N % 128 == 0 (whole tiles).
template <class C>
__device__ __forceinline__ void store_tile_e4m3(const GemmArgs& p, const TileCoords& t,
                                                const v4f (&acc)[C::FM][C::FN], int wm,
                                                int wn, int lane, float* red, float* rcp) {
  static_assert(C::BN % 128 == 0, "E4M3 output needs whole 128-column tiles per workgroup");
  constexpr int WPB = 128 / C::TN;  // waves across one 128-column tile
  constexpr int NBT = C::BN / 128;  // 128-column tiles per workgroup tile
  const int g4 = lane >> 4, l16 = lane & 15;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < C::FN; ++j) m = fmaxf(m, fabsf(acc[i][j][r]));
      m = max_row16(m);
      if (l16 == 0) red[wn * C::BM + wm * C::TM + 16 * i + 4 * g4 + r] = m;
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < NBT * C::BM; idx += C::THREADS) {
    const int nb = idx / C::BM, rt = idx % C::BM;
    float amax = 0.f;
#pragma unroll
    for (int w = 0; w < WPB; ++w) amax = fmaxf(amax, red[(nb * WPB + w) * C::BM + rt]);
    float s, rr;
    group_scale(amax, s, rr);
    rcp[idx] = rr;
    const int64_t row = t.row0 + rt, cb = t.col0 / 128 + nb;
    if (row < t.row_end && cb * 128 < p.N) p.sc[cb * p.ldsc + row] = s;
  }
  __syncthreads();
  const int64_t col = t.col0 + wn * C::TN + C::FN * l16;
  if (col >= p.N) return;  // the wave's whole 128-column tile is past N
  const int nbw = (wn * C::TN) / 128;
  uint8_t* const out = reinterpret_cast<uint8_t*>(t.c);
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const float4 r4 =
        *reinterpret_cast<const float4*>(rcp + nbw * C::BM + wm * C::TM + 16 * i + 4 * g4);
    const float rv[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = t.row0 + wm * C::TM + 16 * i + 4 * g4 + r;
      if (row >= t.row_end) continue;
      uint8_t* const dst = out + row * p.ldc + col;
      float y[C::FN];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) y[j] = acc[i][j][r] * rv[r];
      if constexpr (C::FN == 1) {
        *dst = (uint8_t)cvt2_e4m3<false>(y[0], 0.f, 0u);
      } else if constexpr (C::FN == 2) {
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)cvt2_e4m3<false>(y[0], y[1], 0u);
      } else {
        static_assert(C::FN % 4 == 0, "FN of 1, 2 or a multiple of 4");
        typename Vec<uint32_t, C::FN / 4>::type w;
#pragma unroll
        for (int q = 0; q < C::FN / 4; ++q) {
          const uint32_t lo = cvt2_e4m3<false>(y[4 * q], y[4 * q + 1], 0u);
          w[q] = cvt2_e4m3<true>(y[4 * q + 2], y[4 * q + 3], lo);
        }
        *reinterpret_cast<typename Vec<uint32_t, C::FN / 4>::type*>(dst) = w;
      }
    }
  }
}

// The K loop of a tile.
template <class C>
__device__ __forceinline__ void k_loop(const GemmArgs& p, const TileCoords& t, const LdsSet& L,
                                       const LoadPlan<C>& lp, const FragOffs& fo, const Rsrc& rs,
                                       int wave, v4f (&acc)[C::FM][C::FN]) {
  const int64_t KB = t.KB;
  // Pipeline: group g lives in LDS stage g % STAGES.  Step kb waits for this
  // wave's copies of group kb (leaving the copies of later groups in flight),
  // meets the other waves at a barrier (so every copy of group kb is visible
  // and every wave has finished reading the stage about to be refilled),
  // refills that stage with group kb + STAGES - 1, then computes group kb.
  // The steady-state loop always refills; the last steps are peeled.
  auto stg = [&](int i) -> uint8_t* { return L.st[i]; };
  auto scl = [&](int i) -> float* { return L.sc[i]; };
  // Group g lives in stage g % STAGES.  The scales of group g are loaded to
  // registers with its tile copies (at step g - STAGES + 1) but written to
  // the stage's scale array only at the end of step g - 1: a register ring of
  // SLEAD = STAGES - 2 scale sets gives their loads the same slack as the
  // tile copies (without it, short steps wait for the scale loads).
  // Every prologue stage is filled (with the last group again when KB is
  // smaller than STAGES - 1; such a stage is never read): a conditional fill
  // would make the compiler assume, at the top of the steady loop, that
  // stage 0 may still be in flight.  The extra copies are issued after every
  // real group, so the drain's waits (which count real groups only) still
  // cover them.
  constexpr int SLEAD = C::STAGES - 2;
  ScaleRegs<C> carry[SLEAD > 0 ? SLEAD : 1];
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) {
    const int64_t g = s < KB ? s : KB - 1;
    ScaleRegs<C> sv;
    load_scales<C>(p, t, lp, g, sv);
    issue_stage<C>(p, rs, lp, g, stg(s), wave);
    if (s == 0) {
      store_scales<C>(scl(0), sv);
    } else {
      carry[s - 1] = sv;
    }
  }
  // end of the step of group k (stage index u = k % STAGES): write the scales
  // of group k + 1, then shift the ring (cur: the scales loaded this step,
  // group k + STAGES - 1)
  auto retire_scales = [&](int u, const ScaleRegs<C>& cur, bool store_next) {
    if constexpr (SLEAD == 0) {
      if (store_next) store_scales<C>(scl((u + 1) % C::STAGES), cur);
    } else {
      if (store_next) store_scales<C>(scl((u + 1) % C::STAGES), carry[0]);
#pragma unroll
      for (int d = 0; d + 1 < SLEAD; ++d) carry[d] = carry[d + 1];
      carry[SLEAD - 1] = cur;
    }
  };

  // wait until at most `later` groups (issued after group kb) are in flight
  auto wait_and_sync = [&](int later) {
    if (C::STAGES > 3 && later >= 2) {
      barrier_after_vmcnt<C::LOADS * (C::STAGES > 3 ? 2 : 0)>();
    } else if (C::STAGES > 2 && later >= 1) {
      barrier_after_vmcnt<C::LOADS * (C::STAGES > 2 ? 1 : 0)>();
    } else {
      barrier_after_vmcnt<0>();
    }
  };

  int64_t kb = 0;
  // steady state: STAGES steps per iteration, each refilling the stage read
  // in the previous step with copies interleaved into its MFMA stream
  for (; kb + 2 * C::STAGES - 2 < KB; kb += C::STAGES) {
#pragma unroll
    for (int u = 0; u < C::STAGES; ++u) {
      wait_and_sync(C::STAGES - 2);
      uint8_t* const nxt = stg((u + C::STAGES - 1) % C::STAGES);
      const int64_t kn = kb + u + C::STAGES - 1;
      ScaleRegs<C> sv;
      load_scales<C>(p, t, lp, kn, sv);
      // keep the scale loads ahead of this step's tile copies (in-order
      // completion then lets their wait leave the tile copies in flight)
      __builtin_amdgcn_sched_barrier(0);
      compute_stage<C, true>(stg(u), scl(u), fo, acc, [&](int c) {
        issue_copy<C>(p, rs, lp, kn, nxt, wave, c);
      });
      retire_scales(u, sv, true);
    }
  }
  // drain: at most 2*STAGES-2 steps remain; unrolled so stage indices stay
  // compile-time constants; any refill is issued before the compute
#pragma unroll
  for (int u = 0; u < 2 * C::STAGES - 2; ++u) {
    const int64_t k = kb + u;
    if (k < KB) {
      const int64_t last = k + C::STAGES - 2 < KB - 1 ? k + C::STAGES - 2 : KB - 1;
      wait_and_sync((int)(last - k));
      uint8_t* const nxt = stg((u + C::STAGES - 1) % C::STAGES);
      const bool refill = k + C::STAGES - 1 < KB;
      ScaleRegs<C> sv{};
      if (refill) {
        load_scales<C>(p, t, lp, k + C::STAGES - 1, sv);
        issue_stage<C>(p, rs, lp, k + C::STAGES - 1, nxt, wave);
      }
      compute_stage<C, false>(stg(u % C::STAGES), scl(u % C::STAGES), fo, acc, [](int) {});
      retire_scales(u % C::STAGES, sv, SLEAD == 0 ? refill : k + 1 < KB);
    }
  }
}

// The K loop with exact products: three LDS stages, group g in stage g % 3.  In
// the step of group k the copies of group k + 2 are issued into the stage of group
// k - 1, which every wave has left when it meets the others in step k - 1; they
// land before the meeting of step k + 1.  Past the last group the copies repeat
// it, into stages that nobody uses, so that all wait counts are constants.
template <class C>
__device__ __forceinline__ void exact_k_loop(const GemmArgs& p, const TileCoords& t,
                                             const LdsSet& L, const LoadPlan<C>& lp,
                                             const FragOffs& fo, const Rsrc& rs, int wave,
                                             v4f (&acc)[C::FM][C::FN]) {
  static_assert(C::STAGES == 3, "three stages");
  const int64_t KB = t.KB;
  auto group = [&](int64_t g) { return g < KB ? g : KB - 1; };
  ScaleRegs<C> ahead;  // scales of the group after the next one
  {
    ScaleRegs<C> sv;
    load_scales<C>(p, t, lp, 0, sv);
    issue_stage<C>(p, rs, lp, 0, L.st[0], wave);
    store_scales<C>(L.sc[0], sv);
    load_scales<C>(p, t, lp, group(1), ahead);
    issue_stage<C>(p, rs, lp, group(1), L.st[1], wave);
  }
  barrier_after_vmcnt<C::LOADS>();
  ExactState<C> s;
  {
    const v8i ra = load_frag(L.st[0], fo.a_lo, fo.a_hi, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) s.a[q] = widen8(ra[2 * q], ra[2 * q + 1]);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const v8i rb = load_frag(L.st[0], fo.b_lo, fo.b_hi, 16 * j * 128);
      if (j >= 2) s.raw_b[j - 2] = rb;
#pragma unroll
      for (int q = 0; q < 4; ++q) s.b[j][q] = widen8(rb[2 * q], rb[2 * q + 1]);
    }
    s.part[0] = s.part[1] = v4f{0.f, 0.f, 0.f, 0.f};
    s.w = float4{0.f, 0.f, 0.f, 0.f};
    s.wn = *reinterpret_cast<const float4*>(L.sc[0] + fo.sa);
  }
  auto step = [&](int64_t k, auto U_) {
    constexpr int U = decltype(U_)::value, N1 = (U + 1) % 3, N2 = (U + 2) % 3;
    ScaleRegs<C> sv;
    const int64_t kn = group(k + 2);
    load_scales<C>(p, t, lp, kn, sv);
    // keep the scale loads ahead of this step's tile copies (in-order
    // completion then lets their wait leave the tile copies in flight)
    __builtin_amdgcn_sched_barrier(0);
    compute_step_exact<C>(
        L.st[U], L.sc[U], L.st[N1], L.sc[N1], fo, s, acc,
        [&](int c) { issue_copy<C>(p, rs, lp, kn, L.st[N2], wave, c); },
        [&] {
          store_scales<C>(L.sc[N1], ahead);
          barrier_after_vmcnt<C::LOADS>();
        });
    ahead = sv;
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  int64_t k = 0;
  for (; k + 3 <= KB; k += 3) {
    step(k, I0{});
    step(k + 1, I1{});
    step(k + 2, I2{});
  }
  if (k < KB) step(k, I0{});
  if (k + 1 < KB) step(k + 1, I1{});
  // the last pair's promotion; the repeated copies land before LDS is used again
  const float f[4] = {s.w.x, s.w.y, s.w.z, s.w.w};
#pragma unroll
  for (int d = 0; d < 2; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[C::FM - 1][2 + d][r] = __builtin_fmaf(s.part[d][r], f[r], acc[C::FM - 1][2 + d][r]);
  wait_vmcnt<0>();
}

// Epilogue of the plain product: the FP32 sums are stored as they are.
struct NoEpilogue {
  static constexpr bool kStream = false;  // see store_tile
  template <class C>
  struct Early {};
  template <class C>
  __device__ __forceinline__ void load(const GemmArgs&, const TileCoords&, int, int, int,
                                       Early<C>&) const {}
  template <class C>
  __device__ __forceinline__ void apply(const GemmArgs&, const TileCoords&,
                                        v4f (&)[C::FM][C::FN], int, int, int,
                                        const Early<C>&) const {}
};

// ep.load<C>(p, t, wm, wn, lane, early) may load operands of its own before the
// K loop; ep.apply<C>(p, t, acc, wm, wn, lane, early) may change a wave's
// finished sums before they are stored.  With GatedB, ep.finish<C, OUT>(p, t,
// acc, wm, wn, lane, LDS) takes the sums and stores all there is.
template <class C, int OUT, class E = NoEpilogue>
__device__ __forceinline__ void block_gemm_body(const GemmArgs& p, const TileCoords& t,
                                                const LdsSet& L, const E& ep = E()) {
  // wave index in an SGPR so that per-wave values stay scalar
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int wm = wave / C::WN, wn = wave % C::WN;

  LoadPlan<C> lp;
  make_plan<C>(p, t, wave, lane, lp);
  const FragOffs fo = frag_offsets<C>(wm, wn, lane);
  const Rsrc rs = make_rsrc_set<C>(p, t);
  typename E::template Early<C> early;
  ep.template load<C>(p, t, wm, wn, lane, early);

  v4f acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  if constexpr (C::EXACT) {
    exact_k_loop<C>(p, t, L, lp, fo, rs, wave, acc);
  } else {
    k_loop<C>(p, t, L, lp, fo, rs, wave, acc);
  }
  if constexpr (C::GATED) {
    ep.template finish<C, OUT>(p, t, acc, wm, wn, lane, L.st[0], L.st[1], L.red, L.rcp);
  } else {
    ep.template apply<C>(p, t, acc, wm, wn, lane, early);
    if constexpr (OUT == kOutE4M3) {
      store_tile_e4m3<C>(p, t, acc, wm, wn, lane, L.red, L.rcp);
    } else {
      store_tile<C, OUT, E::kStream>(p, t, acc, wm, wn, lane);
    }
  }
}

// A tile of a group without K range: C_g = 0 there (fp32 or bf16 output).
template <class C, int OUT>
__device__ __forceinline__ void store_zero_tile(const GemmArgs& p, const TileCoords& t) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  v4f zero[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) zero[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  store_tile<C, OUT>(p, t, zero, wave / C::WN, wave % C::WN, threadIdx.x & 63);
}

// One launch covers the raster of BM x BN tiles.
// Dense and grouped-along-K: when the raster would end in a partial round of
// at most half the compute units' worth of tiles, those last tiles are split
// into two TAIL (half-height) tiles each, so the last round takes half as
// long: workgroups [0, full) take whole tiles, the rest take half tiles.
// Grouped rows: the grid is an upper bound on the tile count (the group
// sizes live on the device); the workgroups past the real count exit at
// once, and a group's last tile-row runs as a TAIL tile when it holds at
// most TAIL::BM rows.  TAIL == C: no half tiles.
// The buffer-resource type exists only for the device; the host pass sees an
// empty kernel (it only needs the launch stub).
template <class C, class TAIL, int SCHED, int OUT, class E>
__device__ __forceinline__ void block_gemm_tile(const GemmArgs& p, int64_t full, const E& ep) {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert((TAIL::THREADS == C::THREADS && TAIL::BN == C::BN && 2 * TAIL::BM == C::BM) ||
                    std::is_same<C, TAIL>::value, "tail tiles are half-height tiles");
  static_assert(SCHED != kGroupK || OUT != kOutE4M3, "grouped-K output is fp32 or bf16");
  constexpr int SB = C::STAGE_BYTES > TAIL::STAGE_BYTES ? C::STAGE_BYTES : TAIL::STAGE_BYTES;
  constexpr int SF = C::SCALE_FLOATS > TAIL::SCALE_FLOATS ? C::SCALE_FLOATS : TAIL::SCALE_FLOATS;
  constexpr int NS = C::STAGES > TAIL::STAGES ? C::STAGES : TAIL::STAGES;
  constexpr bool HALVES = !std::is_same<C, TAIL>::value;
  __shared__ __attribute__((aligned(16))) uint8_t st0[SB];
  __shared__ __attribute__((aligned(16))) uint8_t st1[SB];
  __shared__ __attribute__((aligned(16))) uint8_t st2[NS > 2 ? SB : 16];
  __shared__ __attribute__((aligned(16))) uint8_t st3[NS > 3 ? SB : 16];
  __shared__ __attribute__((aligned(16))) float sc0[SF];
  __shared__ __attribute__((aligned(16))) float sc1[SF];
  __shared__ __attribute__((aligned(16))) float sc2[NS > 2 ? SF : 4];
  __shared__ __attribute__((aligned(16))) float sc3[NS > 3 ? SF : 4];
  constexpr bool Q = OUT == kOutE4M3;
  __shared__ __attribute__((aligned(16))) float red[Q ? C::WN * C::BM : 4];
  __shared__ __attribute__((aligned(16))) float rcp[Q ? C::BN / 128 * C::BM : 4];
  const LdsSet L{{st0, st1, st2, st3}, {sc0, sc1, sc2, sc3}, red, rcp};
  const int64_t bid = blockIdx.x;
  TileCoords t;
  if constexpr (SCHED == kGroupRows) {
    (void)full;
    const int64_t MT = grouped_row_tiles<C>(p);
    const int64_t T = MT * ((p.N + C::BNO - 1) / C::BNO);
    if (bid >= T) return;  // whole workgroup: past the last real tile
    // tiles dealt round-robin over the XCDs (not in contiguous runs): the
    // groups' short last tile-rows and the raster's end then spread evenly
    grouped_tile<C>(p, bid, MT, t);
    if constexpr (HALVES) {
      if (t.row_end - t.row0 <= TAIL::BM) {
        block_gemm_body<TAIL, OUT>(p, t, L, ep);
        return;
      }
    }
    block_gemm_body<C, OUT>(p, t, L, ep);
  } else {
    constexpr int out_bytes = OUT == kOutF32 ? 4 : OUT == kOutBF16 ? 2 : 1;
    auto tile_of = [&](int64_t i) {
      if constexpr (SCHED == kGroupK) {
        kgrouped_tile<C>(p, i, t, out_bytes);
      } else {
        dense_tile<C>(p, i, t);
      }
    };
    // grouped along K: the groups' K lengths differ, so contiguous runs per
    // XCD (equal tile counts) would give the XCDs unequal work; dealing
    // the tiles round-robin gives every XCD tiles of every group
    auto order = [&](int64_t i, int64_t n) {
      return SCHED == kGroupK ? i : xcd_remap(i, n);
    };
    if (bid < full) {
      tile_of(order(bid, full));
      if constexpr (SCHED == kGroupK) {
        if (t.KB == 0) {  // whole workgroup: a group without K range
          store_zero_tile<C, OUT>(p, t);
          return;
        }
      }
      block_gemm_body<C, OUT>(p, t, L, ep);
    } else if constexpr (HALVES) {
      const int64_t j = order(bid - full, (int64_t)gridDim.x - full);
      tile_of(full + j / 2);
      t.row0 += (j & 1) * TAIL::BM;
      if (t.row0 >= t.row_end) return;  // lower half below the last row
      if constexpr (SCHED == kGroupK) {
        if (t.KB == 0) {
          store_zero_tile<TAIL, OUT>(p, t);
          return;
        }
      }
      block_gemm_body<TAIL, OUT>(p, t, L, ep);
    }
  }
#endif
}

template <class C, class TAIL, int SCHED, int OUT>
__global__ __launch_bounds__(C::THREADS) void block_gemm_kernel(GemmArgs p, int64_t full) {
  block_gemm_tile<C, TAIL, SCHED, OUT>(p, full, NoEpilogue());
}

// The dense product with an epilogue (an object of kernel-argument type E).
template <class C, class TAIL, int OUT, class E>
__global__ __launch_bounds__(C::THREADS) void block_gemm_epilogue_kernel(GemmArgs p, int64_t full,
                                                                         E ep) {
  block_gemm_tile<C, TAIL, kDense, OUT>(p, full, ep);
}

// Compute units of the current device, cached per device.  Any thread may
// fill an entry; racing fills store the same value, and the relaxed atomics
// make the race well defined.
inline int device_cus() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
      return 0;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Workgroups of a launch, the first `full` of them on whole tiles (see
// block_gemm_tile); 0 for an empty product, -1 where the grid would be too
// large.
template <class C, int SCHED, class TAIL>
int64_t grid_size(const GemmArgs& args, int64_t& full) {
  const int64_t NT = (args.N + C::BNO - 1) / C::BNO;
  int64_t MT = (args.M + C::BM - 1) / C::BM;
  // grouped rows: every non-empty group adds at most one partial tile-row,
  // and every tile-row holds at least one row
  if (SCHED == kGroupRows) MT = MT + args.G < args.M ? MT + args.G : args.M;
  // grouped K: the same tiles for every group
  const int64_t tiles = MT * NT * (SCHED == kGroupK ? args.G : 1);
  if (tiles <= 0) return 0;
  int64_t blocks = tiles;
  full = tiles;
  if (SCHED != kGroupRows && !std::is_same<C, TAIL>::value) {
    // split the last partial round only when its halves fit in one round
    // (at most half the compute units' worth of tiles): a larger tail would
    // take 1.5 rounds of half tiles, longer than one round of whole tiles
    const int64_t cus = device_cus();
    const int64_t tail = cus > 0 ? tiles % cus : 0;
    if (cus > 0 && tiles > cus && tail != 0 && 2 * tail <= cus) {
      full = tiles - tail;
      blocks = full + 2 * tail;
    }
  }
  return blocks > 0x7FFFFFFF ? -1 : blocks;
}

template <class C, int SCHED, class TAIL = C>
hipError_t launch(const GemmArgs& args, OutKind out, hipStream_t stream) {
  int64_t full = 0;
  const int64_t blocks = grid_size<C, SCHED, TAIL>(args, full);
  if (blocks == 0) return hipSuccess;
  if (blocks < 0) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(C::THREADS);
  switch (out) {
    case kOutF32:
      return launch_kernel(block_gemm_kernel<C, TAIL, SCHED, kOutF32>, grid, block, stream, args,
                           full);
    case kOutBF16:
      return launch_kernel(block_gemm_kernel<C, TAIL, SCHED, kOutBF16>, grid, block, stream,
                           args, full);
    default:
      if constexpr (C::BN % 128 == 0 && !C::ROWB && SCHED != kGroupK) {
        return launch_kernel(block_gemm_kernel<C, TAIL, SCHED, kOutE4M3>, grid, block, stream,
                             args, full);
      } else {
        // E4M3 output needs whole 128-column tiles; row-scaled B (weight
        // gradients) has fp32 and bf16 outputs only
        return hipErrorInvalidConfiguration;
      }
  }
}

// Tile shapes of the dense launches (see gemm.hip).
// BM, BN, waves along M, waves along N, LDS stages, tile-rows per L2 group
using LargeCfg = Cfg<256, 256, 2, 4, 2, 4>;
// half-height tiles: a last partial round of the dense raster, and groups'
// last tile-rows of at most 128 rows
using LargeTail = Cfg<128, 256, 2, 4, 2, 4>;
using Rows32Cfg = Cfg<32, 32, 1, 2, 4, 1>;
using Rows64Cfg = Cfg<64, 128, 1, 4, 4, 1>;

// Tile shape for M > 64: the least estimated time, counted in rounds of
// workgroups (one workgroup per compute unit), a round of 256x256, 128x256
// and 64x128 (four-stage) tiles taking 100, 77 and 40 (relative times per
// round at equal K, measured on MI355X with one or two rounds); the 256x256
// launch runs a last partial round of at most half the compute units as
// 128x256 tiles, half a round.
enum class Tiles { kLarge, kHalf, kSmall };
inline Tiles pick_tiles(const GemmArgs& a) {
  const int64_t cus = device_cus();
  if (cus <= 0) return Tiles::kLarge;
  const int64_t tl = ((a.M + 255) / 256) * ((a.N + 255) / 256);
  const int64_t th = ((a.M + 127) / 128) * ((a.N + 255) / 256);
  const int64_t ts = ((a.M + 63) / 64) * ((a.N + 127) / 128);
  const int64_t tail = tl % cus;
  const int64_t cost_l =
      100 * (tl / cus) + (tail == 0 ? 0 : (tl > cus && 2 * tail <= cus) ? 50 : 100);
  const int64_t cost_h = 77 * ((th + cus - 1) / cus);
  const int64_t cost_s = 40 * ((ts + cus - 1) / cus);
  if (cost_l <= cost_h && cost_l <= cost_s) return Tiles::kLarge;
  return cost_h <= cost_s ? Tiles::kHalf : Tiles::kSmall;
}

}  // namespace gemm
}  // namespace fp8bs
