// Wide stores of 32x32 accumulator blocks, shared by the 8-bit products (gfx950 only).
#pragma once

#include "common.h"

namespace moe {

// Native vectors: HIP's uint4 is a class, which keeps arrays of it out of registers.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ uint32_t bf16pack(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}

// Accumulator block exchange for wide stores.  After the transposed MFMA, lane l holds row l % 32 and,
// for element v, column 8 (v / 4) + 4 (l / 32) + v % 4 of the 32x32 block: a store covers 32 rows
// with 16 bytes each.  v_permlane32_swap of the 4-column pieces of each 16-column half gives lane l
// 8 consecutive columns 16 H + 8 (l / 32) of its row; v_permlane16_swap of the two halves then
// leaves x0 = row l % 16 and x1 = row 16 + l % 16, both at columns 16 ((l / 16) % 2) + 8 (l / 32):
// each 16-byte store covers 16 rows with 64 contiguous bytes.
__device__ __forceinline__ int xcol(int lane) { return 16 * ((lane >> 4) & 1) + 8 * (lane >> 5); }

__device__ __forceinline__ void xchg_block(const f32x16_t& c, float (&x0)[8], float (&x1)[8]) {
  float hv[2][8];
#pragma unroll
  for (int H = 0; H < 2; ++H)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(c[8 * H + e]), __float_as_uint(c[8 * H + 4 + e]),
                                                      false, false);
      hv[H][e] = __uint_as_float(r[0]);
      hv[H][4 + e] = __uint_as_float(r[1]);
    }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(hv[0][e]), __float_as_uint(hv[1][e]), false, false);
    x0[e] = __uint_as_float(r[0]);
    x1[e] = __uint_as_float(r[1]);
  }
}

__device__ __forceinline__ u32x4_t pack8(const float (&v)[8]) {
  u32x4_t w;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = bf16pack(v[2 * e], v[2 * e + 1]);
  return w;
}
__device__ __forceinline__ void unpack8(const u32x4_t& w, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

}  // namespace moe
