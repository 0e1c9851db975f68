// Products in 8-bit floating point with a float scale for each block of 128, and their quantizers.
//
//   scale = max(|v|, 2^-100) / 448 over a block;  code = E4M3(448 v / max |v|), to nearest, ties to even
//   C[m, n] = sum_b sa[m, b] sb[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
//
// Activations have a block for 128 elements of a row, weights for 128 x 128: the weights' blocks lie
// square, so the transposed weights that the data gradient multiplies with are the same codes and scales
// in another order, not a second rounding.
//
// A bf16 v times 448 is exact in fp32 (8 + 3 bits), and the quotient of an 11-bit by an 8-bit number is
// either a number of at most 5 bits, where two codes meet, or further than 2^-14 of itself from every such
// number: rounding the quotient to fp32 first changes no code.
//
// The matrix instruction multiplies E4M3 codes exactly and adds in fp32; a block's 128 products per output
// go through two instructions of depth 64 from a zero accumulator, whose result is scaled and added.
#include "train_step.h"

#include "mxfp8.h"

#include <algorithm>

namespace moe {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int BLK = 128;
constexpr float TOP = 448.0f;
constexpr float TINY = 0x1p-100f;
constexpr int ONE = 0x7f7f7f7f;   // scale bytes of the matrix instruction: 2^0

__device__ __forceinline__ uint32_t row16_max(uint32_t b) {   // of a row of 16 lanes
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0xB1, 0xf, 0xf, false));    // quad_perm 1,0,3,2
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x4E, 0xf, 0xf, false));    // quad_perm 2,3,0,1
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x124, 0xf, 0xf, false));   // row_ror 4
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x128, 0xf, 0xf, false));   // row_ror 8
  return b;
}

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

__device__ __forceinline__ float quotient(uint32_t bits, float top) {
  return fminf(fmaxf(__uint_as_float(bits) * TOP / top, -TOP), TOP);
}
__device__ __forceinline__ u32x2_t codes8(const u32x4_t& w, float top) {
  u32x2_t c;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(w[2 * q] << 16, top), quotient(w[2 * q] & 0xffff0000u, top), 0, false);
    c[q] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient(w[2 * q + 1] << 16, top),
                                                     quotient(w[2 * q + 1] & 0xffff0000u, top), lo, true);
  }
  return c;
}

// Rows: 8 elements a lane, 16 lanes a block.
__global__ __launch_bounds__(256) void fp8_quant_rows_kernel(const bf16_t* __restrict__ x, long long R, int K,
                                                             long long ldx, uint8_t* __restrict__ codes,
                                                             float* __restrict__ scales) {
  const int nch = K >> 3;   // a multiple of 16
  const long long total = R * nch, stride = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
    const long long r = i / nch;
    const int c = (int)(i - r * nch);
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + r * ldx + (long long)c * 8);
    const uint32_t bits = row16_max(max8(v));
    *reinterpret_cast<u32x2_t*>(codes + r * K + (long long)c * 8) = codes8(v, block_top(bits));
    if ((c & 15) == 0) scales[(long long)(c >> 4) * R + r] = block_scale(bits);
  }
}

// Weights: one 128 x 128 block a workgroup; the codes also transposed, through LDS.
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
  const float top = block_top(bits);
  uint8_t* dst = codes + ((long long)g * N + (long long)bn * BLK) * K + (long long)bk * BLK + 8 * c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const u32x2_t q = codes8(v[i], top);
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

// ---- Products: 128 x 128 tiles ------------------------------------------------------------------
// Four waves, 64 x 64 each; K goes in blocks of 128 through a double-buffered LDS tile, 16-byte chunks
// XOR-swizzled by (row >> 1) & 7.  The weights are the instruction's first operand, so a lane's
// accumulators hold 4 consecutive output columns of one row: its row's scale is one register.
constexpr int TB = 128;
constexpr int OPBYTES = TB * TB;

__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ uint32_t bf16pack(float a, float b) {
  return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}

// The group of row tile mt and its rows, from the group offsets: rows of a group in tiles of TB, groups in
// order; false past the last.  A wave's lanes count 64 groups at a time.
__device__ __forceinline__ bool find_rows(const int32_t* offsets, int G, int M, int mt, int& g, int& m0, int& m_end) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int g0 = 0; g0 < G; g0 += 64) {
    const int q = g0 + lane;
    int r0 = 0, r1 = 0;
    if (q < G) {
      r0 = min(max(offsets[q], 0), M);
      r1 = min(max(offsets[q + 1], r0), M);
    }
    const int n = (r1 - r0 + TB - 1) / TB;
    int sum = n;   // tiles of the lanes up to this one
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(sum, off, 64);
      if (lane >= off) sum += o;
    }
    const int all = __shfl(sum, 63, 64);
    if (mt < before + all) {
      const unsigned long long later = __ballot(before + sum > mt);
      const int at = __ffsll((long long)later) - 1;
      g = g0 + at;
      m0 = __shfl(r0, at, 64) + (mt - before - __shfl(sum - n, at, 64)) * TB;
      m_end = __shfl(r1, at, 64);
      return true;
    }
    before += all;
  }
  return false;
}

__device__ __forceinline__ i32x8_t read_frag(const uint8_t* tile, int row, int s, int h) {
  const uint8_t* base = tile + row * TB;
  const int sw = swz(row);
  const u32x4_t p = *reinterpret_cast<const u32x4_t*>(base + 16 * ((4 * s + h) ^ sw));
  const u32x4_t q = *reinterpret_cast<const u32x4_t*>(base + 16 * ((4 * s + 2 + h) ^ sw));
  i32x8_t r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = (int)p[j];
    r[4 + j] = (int)q[j];
  }
  return r;
}

template <int EPI>
__global__ __launch_bounds__(256, 2) void fp8_gemm_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][OPBYTES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, li = lane & 31, h = lane >> 5;
  constexpr int OC = EPI == MX_EPI_SWIGLU ? 64 : 128;   // the SwiGLU tile: 64 gate and 64 up columns
  const int NT = p.N / OC;
  const int nt = blockIdx.x % NT;
  int g, m0, m_end;
  if (!find_rows(p.offsets, p.G, p.M, blockIdx.x / NT, g, m0, m_end)) return;
  const int nk = p.K / TB;
  const bool split = EPI != MX_EPI_SWIGLU && p.b2 != nullptr;
  const int K1 = split ? p.ksplit : p.K, K2 = EPI == MX_EPI_SWIGLU ? p.K : p.K - K1;

  // Loads: rows (tid >> 3) + 32 j, 16-byte chunk tid & 7, of both operands.
  const int lrow = tid >> 3, lch = tid & 7;
  const uint8_t* ga[4];
  const uint8_t* gb[4];
  const uint8_t* gb2[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = lrow + 32 * j;
    ga[j] = p.a + (long long)min(m0 + r, m_end - 1) * p.K + 16 * lch;
    if constexpr (EPI == MX_EPI_SWIGLU) {
      const long long br = (long long)g * p.N + nt * 64 + (r >> 6) * 32 + (r & 31);
      gb[j] = (((r >> 5) & 1) ? p.b2 : p.b) + br * p.K + 16 * lch;
      gb2[j] = gb[j];
    } else {
      const long long br = (long long)g * p.N + nt * TB + r;
      gb[j] = p.b + br * K1 + 16 * lch;
      gb2[j] = split ? p.b2 + br * K2 + 16 * lch - K1 : gb[j];
    }
  }
  const int lofs = lrow * TB + 16 * (lch ^ swz(lrow));
  // Scales: one of each of the lane's two rows, one of each of the wave's column blocks of 128.
  const float* sa_p[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) sa_p[i] = p.as + min(m0 + wm * 64 + i * 32 + li, m_end - 1);
  const long long nblk = (long long)g * (p.N / BLK) + (EPI == MX_EPI_SWIGLU ? nt / 2 : nt);
  const float* sb_p = p.bs + nblk * (K1 / BLK);
  const float* sb2_p = p.bs2 ? p.bs2 + nblk * (K2 / BLK) : nullptr;

  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  u32x4_t ra[4], rb[4];
  auto fetch = [&](int kt) {
    const int off = kt * TB;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ra[j] = *reinterpret_cast<const u32x4_t*>(ga[j] + off);
      rb[j] = *reinterpret_cast<const u32x4_t*>((off >= K1 ? gb2[j] : gb[j]) + off);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<u32x4_t*>(&lds[buf][0][lofs + 32 * TB * j]) = ra[j];
      *reinterpret_cast<u32x4_t*>(&lds[buf][1][lofs + 32 * TB * j]) = rb[j];
    }
  };
  fetch(0);
  store(0);
  __syncthreads();
  for (int kt = 0; kt < nk; ++kt) {
    const int cur = kt & 1;
    if (kt + 1 < nk) fetch(kt + 1);
    float sa[2], sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) sa[i] = sa_p[i][(long long)kt * p.M];
    if constexpr (EPI == MX_EPI_SWIGLU) {
      sb[0] = sb_p[kt];
      sb[1] = sb2_p[kt];
    } else {
      sb[0] = sb[1] = kt * TB >= K1 ? sb2_p[kt - K1 / TB] : sb_p[kt];
    }
    f32x16_t part[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      i32x8_t fa[2], fb[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        fa[q] = read_frag(lds[cur][0], wm * 64 + q * 32 + li, s, h);
        fb[q] = read_frag(lds[cur][1], wn * 64 + q * 32 + li, s, h);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (s == 0) {
#pragma unroll
            for (int r = 0; r < 16; ++r) part[i][j][r] = 0.f;
          }
          part[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], part[i][j], 0, 0, 0, ONE, 0, ONE);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = sa[i] * sb[j];
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] += f * part[i][j][r];
      }
    if (kt + 1 < nk) store(cur ^ 1);
    __syncthreads();
  }

  // Epilogue: lane holds row li of each 32-row block, columns 8 (r / 4) + 4 h + r % 4.
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = m0 + wm * 64 + i * 32 + li;
    if (row >= m_end) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (EPI == MX_EPI_SWIGLU) {
        const long long o = (long long)row * p.N + nt * 64 + wn * 32 + 8 * q + 4 * h;
        float hv[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float a = acc[i][0][4 * q + r];
          hv[r] = a * sigmoid_f32(a) * acc[i][1][4 * q + r];
        }
        auto put = [&](void* out, float v0, float v1, float v2, float v3) {
          *reinterpret_cast<uint2*>(reinterpret_cast<bf16_t*>(out) + o) = make_uint2(bf16pack(v0, v1), bf16pack(v2, v3));
        };
        if (p.out0) put(p.out0, acc[i][0][4 * q], acc[i][0][4 * q + 1], acc[i][0][4 * q + 2], acc[i][0][4 * q + 3]);
        if (p.out1) put(p.out1, acc[i][1][4 * q], acc[i][1][4 * q + 1], acc[i][1][4 * q + 2], acc[i][1][4 * q + 3]);
        put(p.out2, hv[0], hv[1], hv[2], hv[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = nt * TB + wn * 64 + j * 32 + 8 * q + 4 * h;
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = acc[i][j][4 * q + r];
          if constexpr (EPI == MX_EPI_SWIGLU_BWD) {
            const long long o = (long long)row * p.N + col;
            const uint2 av = *reinterpret_cast<const uint2*>(reinterpret_cast<const bf16_t*>(p.aux0) + o);
            const uint2 bv = *reinterpret_cast<const uint2*>(reinterpret_cast<const bf16_t*>(p.aux1) + o);
            const uint32_t aw[2] = {av.x, av.y}, bw[2] = {bv.x, bv.y};
            float da[4], db[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float a = bf16_to_f32((bf16_t)(aw[r >> 1] >> (16 * (r & 1))));
              const float bb = bf16_to_f32((bf16_t)(bw[r >> 1] >> (16 * (r & 1))));
              const float sg = sigmoid_f32(a);
              da[r] = v[r] * bb * sg * (1.0f + a * (1.0f - sg));
              db[r] = v[r] * a * sg;
            }
            bf16_t* dab = reinterpret_cast<bf16_t*>(p.out0) + (long long)row * (2 * p.N);
            *reinterpret_cast<uint2*>(dab + col) = make_uint2(bf16pack(da[0], da[1]), bf16pack(da[2], da[3]));
            *reinterpret_cast<uint2*>(dab + p.N + col) = make_uint2(bf16pack(db[0], db[1]), bf16pack(db[2], db[3]));
          } else {
            *reinterpret_cast<uint2*>(reinterpret_cast<bf16_t*>(p.out0) + (long long)row * p.N + col) =
                make_uint2(bf16pack(v[0], v[1]), bf16pack(v[2], v[3]));
          }
        }
      }
    }
  }
}

template <int EPI>
hipError_t launch_tiles(const Fp8GemmArgs& a, hipStream_t s) {
  const long long rows = (a.M + TB - 1) / TB + std::min(a.G, a.M);
  const long long tiles = rows * (a.N / (EPI == MX_EPI_SWIGLU ? 64 : 128));
  fp8_gemm_kernel<EPI><<<dim3((unsigned)tiles), dim3(256), 0, s>>>(a);
  return hipGetLastError();
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

size_t fp8_gemm_ws_bytes(int G, long long M, long long N, long long K) {
  (void)G; (void)M; (void)N; (void)K;
  return 0;
}

hipError_t launch_fp8_gemm(int epi, const Fp8GemmArgs& a, hipStream_t s) {
  if (a.M == 0) return hipSuccess;
  switch (epi) {
    case MX_EPI_SWIGLU: return launch_tiles<MX_EPI_SWIGLU>(a, s);
    case MX_EPI_SWIGLU_BWD: return launch_tiles<MX_EPI_SWIGLU_BWD>(a, s);
    default: return launch_tiles<MX_EPI_STORE>(a, s);
  }
}

}  // namespace moe
