// Register pieces that MXFP8, the block-scaled 8-bit products and AdamW share (gfx950 only).
#pragma once

#include "common.h"

namespace moe {

// Native vectors: HIP's uint4 is a class, which keeps arrays of it out of registers.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 8 bf16 values to fp32.
__device__ __forceinline__ void unpack8(const u32x4_t& w, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// The largest of the 16 lanes of a row, in every one of them: bits of magnitudes, which order as the values do, a
// NaN above all.
__device__ __forceinline__ uint32_t row16_max(uint32_t b) {
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0xB1, 0xf, 0xf, false));    // quad_perm 1,0,3,2
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x4E, 0xf, 0xf, false));    // quad_perm 2,3,0,1
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x124, 0xf, 0xf, false));   // row_ror 4
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x128, 0xf, 0xf, false));   // row_ror 8
  return b;
}

}  // namespace moe
