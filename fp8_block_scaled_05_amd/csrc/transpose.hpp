// Byte transposition in registers, shared by the transposing quantizers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device.hpp"

namespace fp8bs {

// Transpose of an 8x8 byte block: row i is (lo[i], hi[i]) (bytes 0..3, 4..7);
// returns column c as (olo[c], ohi[c]) = bytes c of rows 0..3 and 4..7.
// v_perm_b32 picks each result byte from the 8 bytes {S0 (4..7), S1 (0..3)}.
__device__ __forceinline__ void transpose8x8(const uint32_t (&lo)[8], const uint32_t (&hi)[8],
                                             uint32_t (&olo)[8], uint32_t (&ohi)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t (&src)[8] = c < 4 ? lo : hi;
    const uint32_t b = (uint32_t)(c & 3);
    const uint32_t pick = b | ((4u + b) << 8);  // byte b of S1, then byte b of S0
    const uint32_t r01 = __builtin_amdgcn_perm(src[1], src[0], pick);
    const uint32_t r23 = __builtin_amdgcn_perm(src[3], src[2], pick);
    const uint32_t r45 = __builtin_amdgcn_perm(src[5], src[4], pick);
    const uint32_t r67 = __builtin_amdgcn_perm(src[7], src[6], pick);
    olo[c] = __builtin_amdgcn_perm(r23, r01, 0x05040100u);
    ohi[c] = __builtin_amdgcn_perm(r67, r45, 0x05040100u);
  }
}

// Transpose of 8 rows of 4 bytes: out[c] = bytes c of rows 0..3 and 4..7.
__device__ __forceinline__ void transpose8x4(const uint32_t (&in)[8], u32x2 (&out)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t pick = (uint32_t)c | ((4u + (uint32_t)c) << 8);
    const uint32_t r01 = __builtin_amdgcn_perm(in[1], in[0], pick);
    const uint32_t r23 = __builtin_amdgcn_perm(in[3], in[2], pick);
    const uint32_t r45 = __builtin_amdgcn_perm(in[5], in[4], pick);
    const uint32_t r67 = __builtin_amdgcn_perm(in[7], in[6], pick);
    out[c] = u32x2{__builtin_amdgcn_perm(r23, r01, 0x05040100u),
                   __builtin_amdgcn_perm(r67, r45, 0x05040100u)};
  }
}

}  // namespace fp8bs
