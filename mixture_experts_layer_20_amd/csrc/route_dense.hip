// Products of a dense logit gradient G [T, E] (fp32): dw = G^T x [E, d] and dx = G w [T, d].
//
// Both are out[n, c] = sum_k P[k, c] Q[k, n] with P = x or w as it lies, on the fp32 matrix instruction (16 x 16
// x 4), so nothing is rounded but the sums.  P is its first operand: a lane's four results are neighbouring
// columns of one output row.  A wave forms 64 x 64 outputs from 4 + 4 loads of a dword for 16 matrix
// instructions (512 cycles of its SIMD), straight from memory: the four waves of a workgroup, side by side in
// c, read the same Q through the CU's cache.
//
// dw sums over T tokens for few outputs: T goes in parts to about 2048 waves, two for each SIMD, of 32 tokens or
// more, whose sums are added in order.  T 1537, d 1000, E 60 in fp32: both products 17 us in one launch (12 + 13
// in two) and 4 for the parts' join, against 54 + 27 + 4 with vector multiply-adds of one column a thread; 14 MB
// and 0.4 GFLOP are 3 us.  What bounds it is the latency of the 15 steps of 4 that a wave of dx takes, 4 of them
// in flight (with the next 4 loaded while 4 are multiplied: 20 us).
#include "train_step.h"

#include <algorithm>

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int TILE = 64;     // outputs of a wave, each way
constexpr int AHEAD = 4;     // steps of 4 of k in flight

int dw_splits(long long T, long long d, int E) {
  const long long tiles = ceil_div(d, TILE) * (long long)ceil_div(E, TILE);
  return (int)std::max(1LL, std::min<long long>(ceil_div(T, 32), 2048 / tiles));
}

// DW: Q = G, k the tokens of a part, out the parts' sums [parts, E, d]; else Q[k, n] = G[n, k], out dx.
template <typename T, bool DW>
__device__ __forceinline__ void dense_product(const float* G, const T* P, int ntok, int d, int E, int block, int part,
                                              int parts, void* out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, q = lane >> 4;
  const int cols = (d + 4 * TILE - 1) / (4 * TILE);
  const int c0 = (block % cols * 4 + wave) * TILE, n0 = block / cols * TILE;
  if (c0 >= d) return;
  const int N = DW ? E : ntok, K = DW ? ntok : E;
  const int kb = (int)((long long)K * part / parts), ke = (int)((long long)K * (part + 1) / parts);
  f32x4_t acc[4][4];   // c, n
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int c[4], n[4];   // loads past the edges take the last column, whose products are dropped
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = min(c0 + 16 * i + li, d - 1);
    n[i] = min(n0 + 16 * i + li, N - 1);
  }
  for (int k0 = kb; k0 < ke; k0 += 4 * AHEAD) {
    float p[AHEAD][4], g[AHEAD][4];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int k = min(k0 + 4 * u + q, ke - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[u][i] = to_f32<T>(P[(size_t)k * d + c[i]]);
        g[u][i] = DW ? G[(size_t)k * E + n[i]] : G[(size_t)n[i] * E + k];
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const bool in = k0 + 4 * u + q < ke;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[u][i] = in ? p[u][i] : 0.0f;
        g[u][i] = in ? g[u][i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(p[u][i], g[u][j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = n0 + 16 * j + li;
    if (row >= N) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = c0 + 16 * i + 4 * q;   // d is a multiple of 8
      if (col >= d) continue;
      const f32x4_t v = acc[i][j];
      if constexpr (DW) {
        *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + ((size_t)part * E + row) * d + col) = v;
      } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + (size_t)row * d + col) = v;
      } else {
        const uint32_t lo = (uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16);
        const uint32_t hi = (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16);
        *reinterpret_cast<uint2*>(reinterpret_cast<bf16_t*>(out) + (size_t)row * d + col) = make_uint2(lo, hi);
      }
    }
  }
}

// Both in one launch, dw's workgroups first: neither fills the CUs by itself where the tokens are few.
template <typename T>
__global__ __launch_bounds__(256) void dense_products_kernel(const float* G, const T* x, const T* w, int ntok, int d, int E,
                                                             int dw_blocks, int parts, float* sums, T* dx) {
  const int b = blockIdx.x;
  if (b < dw_blocks) {
    const int tiles = dw_blocks / parts;
    dense_product<T, true>(G, x, ntok, d, E, b % tiles, b / tiles, parts, sums);
  } else {
    dense_product<T, false>(G, w, ntok, d, E, b - dw_blocks, 0, 1, dx);
  }
}

// The parts' sums in order; no part (no token): zeros.
__global__ __launch_bounds__(256) void dense_join_kernel(const float* parts, int count, int n, float* dw) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float s = 0.0f;
#pragma unroll 8
  for (int p = 0; p < count; ++p) s += parts[(size_t)p * n + i];
  dw[i] = s;
}

template <typename T>
hipError_t launch_products(const float* G, const T* x, const T* w, int ntok, int d, int E, float* dw, T* dx, float* parts,
                           hipStream_t s) {
  const int count = ntok > 0 ? dw_splits(ntok, d, E) : 0;
  if (ntok > 0) {
    const int cols = ceil_div(d, 4 * TILE);
    const int dw_blocks = cols * ceil_div(E, TILE) * count, dx_blocks = cols * ceil_div(ntok, TILE);
    dense_products_kernel<T><<<dim3((unsigned)dw_blocks + dx_blocks), dim3(256), 0, s>>>(G, x, w, ntok, d, E, dw_blocks, count, parts, dx);
  }
  dense_join_kernel<<<dim3(ceil_div((long long)E * d, 256)), dim3(256), 0, s>>>(parts, count, E * d, dw);
  return hipGetLastError();
}

}  // namespace

size_t router_dense_bwd_ws_bytes(long long T, long long d, int E) {
  return T > 0 ? (size_t)dw_splits(T, d, E) * E * d * sizeof(float) : 0;
}

// Both products in one grid of fewer than 2^24 workgroups, dw's elements counted in an int.
bool router_dense_bwd_fits(long long T, long long d, int E) {
  const long long cols = (d + 4 * TILE - 1) / (4 * TILE), etiles = (E + TILE - 1) / TILE;
  const long long dw_blocks = T > 0 ? cols * etiles * dw_splits(T, d, E) : 0;
  return E * d < 1LL << 31 && dw_blocks + cols * ((T + TILE - 1) / TILE) < 1LL << 24;
}

hipError_t launch_router_dense_bwd(const float* G, const void* x, const void* w, int T, int d, int E, bool bf16,
                                   float* dw, void* dx, void* ws, hipStream_t s) {
  float* parts = reinterpret_cast<float*>(ws);
  if (bf16)
    return launch_products<bf16_t>(G, reinterpret_cast<const bf16_t*>(x), reinterpret_cast<const bf16_t*>(w), T, d, E, dw,
                                   reinterpret_cast<bf16_t*>(dx), parts, s);
  return launch_products<float>(G, reinterpret_cast<const float*>(x), reinterpret_cast<const float*>(w), T, d, E, dw,
                                reinterpret_cast<float*>(dx), parts, s);
}

}  // namespace moe
