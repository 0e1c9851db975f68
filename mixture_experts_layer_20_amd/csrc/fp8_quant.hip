// Quantizers to 8-bit floating point (E4M3) with a float scale for each block of 128.
//
//   scale = max(|v|, 2^-100) / 448 over a block;  code = E4M3(448 v / max |v|), to nearest, ties to even
//
// Activations have a block for 128 elements of a row, weights for 128 x 128: the weights' blocks lie
// square, so the transposed weights that the data gradient multiplies with are the same codes and scales
// in another order, not a second rounding.
//
// The quotient of 448 v, a number of at most 11 bits, by one of 8 bits is either a number of at most 5 bits (a
// code, or the middle of two) or at least 2^-13 of itself away from every such number.  So it is formed as v
// times the rounded 448 / max |v|, which is off by 2^-23, and rounded to 17 bits: the 5-bit numbers come out
// exactly, the others on their own side of them, and the codes are those of the exact quotient.
#include "train_step.h"

#include "lanes.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int BLK = 128;
constexpr float TOP = 448.0f;
constexpr float TINY = 0x1p-100f;

// Bits of the largest magnitude of 8 bf16 values (as fp32 bits; a NaN is above all).
__device__ __forceinline__ uint32_t max8(const u32x4_t& w) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) m = max(m, max((w[q] & 0x7fffu) << 16, w[q] & 0x7fff0000u));
  return m;
}

// A block's largest magnitude as it is divided by, and its scale: NaN where the block has a NaN or an
// infinity, so that every product with it is NaN.
__device__ __forceinline__ float block_top(uint32_t bits) { return fmaxf(__uint_as_float(bits), TINY); }
__device__ __forceinline__ float block_scale(uint32_t bits) {
  return bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : block_top(bits) / TOP;
}

__device__ __forceinline__ float quotient(uint32_t bits, float inv) {
  return __uint_as_float((__float_as_uint(__uint_as_float(bits) * inv) + 0x40u) & ~0x7fu);
}
__device__ __forceinline__ u32x2_t codes8(const u32x4_t& w, float inv) {
  u32x2_t c;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(w[2 * q] << 16, inv), quotient(w[2 * q] & 0xffff0000u, inv), 0, false);
    c[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient(w[2 * q + 1] << 16, inv),
                                                     quotient(w[2 * q + 1] & 0xffff0000u, inv), lo, true);
  }
  return c;
}

// Rows: 8 elements a lane, 16 lanes a block.  Bound by memory: 65536 x 2048 84 us, 4.8 TB/s (a copy 5.2); with a
// division for each element, and 64-bit ones for each lane's place, it was bound by what it computed, 100 us.
__global__ __launch_bounds__(256) void fp8_quant_rows_kernel(const bf16_t* __restrict__ x, long long R, int K,
                                                             long long ldx, uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  const int nch = K >> 3;   // a multiple of 16
  const long long total = R * nch, stride = (long long)gridDim.x * 256;
  long long i = (long long)blockIdx.x * 256 + threadIdx.x, r = i / nch;
  int c = (int)(i - r * nch);
  const long long rows = stride / nch;
  const int cols = (int)(stride - rows * nch);
  for (; i < total; i += stride) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + r * ldx + (long long)c * 8);
    const uint32_t bits = row16_max(max8(v));
    *reinterpret_cast<u32x2_t*>(codes + r * K + (long long)c * 8) = codes8(v, TOP / block_top(bits));
    if ((c & 15) == 0) scales[(long long)(c >> 4) * R + r] = block_scale(bits);
    r += rows;   // on by `stride` chunks
    c += cols;
    if (c >= nch) {
      c -= nch;
      ++r;
    }
  }
}

// Weights: one 128 x 128 block a workgroup; the codes also transposed, through LDS.  64 x 2048 x 1024 with both
// forms 107 us, 5.0 TB/s.
__global__ __launch_bounds__(256) void fp8_quant_weights_kernel(const bf16_t* __restrict__ w, int N, int K,
                                                                uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                                uint8_t* __restrict__ codes_t, float* __restrict__ scales_t) {
  __shared__ uint32_t top_s[4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[BLK][BLK + 16];
  const int nb = N / BLK, kb = K / BLK;
  const long long blk = blockIdx.x;
  const int g = (int)(blk / ((long long)nb * kb)), rem = (int)(blk - (long long)g * nb * kb);
  const int bn = rem / kb, bk = rem - bn * kb;
  const int row = threadIdx.x >> 4, c = threadIdx.x & 15;   // rows row + 16 i, 8 elements at 8 c
  const bf16_t* src = w + ((long long)g * N + (long long)bn * BLK) * K + (long long)bk * BLK + 8 * c;
  u32x4_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const u32x4_t*>(src + (long long)(row + 16 * i) * K);
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) bits = max(bits, max8(v[i]));
  bits = row16_max(bits);
  bits = max(bits, (uint32_t)__shfl_xor((int)bits, 16, 64));
  bits = max(bits, (uint32_t)__shfl_xor((int)bits, 32, 64));
  if ((threadIdx.x & 63) == 0) top_s[threadIdx.x >> 6] = bits;
  __syncthreads();
  bits = max(max(top_s[0], top_s[1]), max(top_s[2], top_s[3]));
  const float inv = TOP / block_top(bits);
  uint8_t* dst = codes + ((long long)g * N + (long long)bn * BLK) * K + (long long)bk * BLK + 8 * c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const u32x2_t q = codes8(v[i], inv);
    *reinterpret_cast<u32x2_t*>(dst + (long long)(row + 16 * i) * K) = q;
    if (codes_t) *reinterpret_cast<u32x2_t*>(&tile[row + 16 * i][8 * c]) = q;
  }
  if (threadIdx.x == 0) {
    scales[((long long)g * nb + bn) * kb + bk] = block_scale(bits);
    if (codes_t) scales_t[((long long)g * kb + bk) * nb + bn] = block_scale(bits);
  }
  if (!codes_t) return;
  __syncthreads();
  // transposed: column `col` of the block, rows 64 half .. + 63
  const int col = threadIdx.x >> 1, half = threadIdx.x & 1;
  uint8_t* to = codes_t + ((long long)g * K + (long long)bk * BLK + col) * N + (long long)bn * BLK + 64 * half;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    u32x4_t o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 64 * half + 16 * q + 4 * e;
      o[e] = tile[r][col] | ((uint32_t)tile[r + 1][col] << 8) | ((uint32_t)tile[r + 2][col] << 16) |
             ((uint32_t)tile[r + 3][col] << 24);
    }
    *reinterpret_cast<u32x4_t*>(to + 16 * q) = o;
  }
}

}  // namespace

hipError_t launch_fp8_quant_rows(const void* x, long long R, int K, long long ldx, uint8_t* codes, float* scales,
                                 hipStream_t s) {
  const long long total = R * (K / 8);
  if (total == 0) return hipSuccess;
  const int blocks = (int)std::min<long long>((total + 255) / 256, 256LL * 16);
  fp8_quant_rows_kernel<<<dim3(blocks), dim3(256), 0, s>>>(reinterpret_cast<const bf16_t*>(x), R, K, ldx, codes, scales);
  return hipGetLastError();
}

hipError_t launch_fp8_quant_weights(const void* w, int G, int N, int K, uint8_t* codes, float* scales, uint8_t* codes_t,
                                    float* scales_t, hipStream_t s) {
  const long long blocks = (long long)G * (N / BLK) * (K / BLK);
  fp8_quant_weights_kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(reinterpret_cast<const bf16_t*>(w), N, K, codes,
                                                                        scales, codes_t, scales_t);
  return hipGetLastError();
}

}  // namespace moe
