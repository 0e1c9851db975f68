// Softmax cross entropy over a vocabulary and its gradient, in pieces of the vocabulary.
//
//   l = h w^T (T x V),  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l[t, target_t]
//   P = dloss_t (exp(l_tv - lse_t) - [v = target_t]),  dh = P w,  dw = P^T h
//
// The logits are never stored.  Forward: each tile of the product keeps, per row, the maximum and
// the sum of exponentials of each 64 of its columns; a second kernel joins a row's parts in order.  Backward: the product is formed again one piece of
// the vocabulary at a time, its epilogue writes P of the piece (in the storage type: the operand of
// the two gradient products), and dh accumulates over the pieces in fp32.
// A target outside [0, V) marks a row without loss: loss 0, P = 0 exactly.
#include "vocab_loss.h"

#include <algorithm>

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

using namespace vocab;

// ---------------------------------------------------------------------------------------------
// 128x128 tiles, four waves of 64x64, operands staged through registers: any T, V and d (a multiple
// of 8), both types.

constexpr int TM = 128, TN = 128, NT = 256;

template <typename T> struct Cfg;
template <> struct Cfg<bf16_t> {
  static constexpr int BK = 32, E = 8, LD = BK + 8;   // E: elements of a 16-byte chunk
};
template <> struct Cfg<float> {
  static constexpr int BK = 16, E = 4, LD = BK + 4;
};

// Operand chunk c (0..511) of the K step at k0 into its LDS tile [128][LD].  KC: rows of K
// consecutive elements; otherwise K rows of consecutive tile rows.  Elements outside are zero.
template <typename T, bool KC>
struct Stage {
  static constexpr int E = Cfg<T>::E, BK = Cfg<T>::BK, LD = Cfg<T>::LD;
  u32x4_t v[2];
  __device__ __forceinline__ void load(const T* base, size_t ld, int row0, int rows, int k0, int K) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = threadIdx.x + i * NT;
      const int r = KC ? c / (BK / E) : (c % (TM / E)) * E;
      const int k = k0 + (KC ? (c % (BK / E)) * E : c / (TM / E));
      v[i] = u32x4_t{0, 0, 0, 0};
      if (row0 + r < rows && k < K) v[i] = *reinterpret_cast<const u32x4_t*>(KC ? base + (size_t)(row0 + r) * ld + k : base + (size_t)k * ld + row0 + r);
    }
  }
  __device__ __forceinline__ void store(T* lds) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = threadIdx.x + i * NT;
      if constexpr (KC) {
        *reinterpret_cast<u32x4_t*>(lds + (c / (BK / E)) * LD + (c % (BK / E)) * E) = v[i];
      } else {
        const int r = (c % (TM / E)) * E, k = c / (TM / E);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if constexpr (E == 8) lds[(r + e) * LD + k] = (bf16_t)(v[i][e / 2] >> (16 * (e & 1)));
          else lds[(r + e) * LD + k] = __uint_as_float(v[i][e]);
        }
      }
    }
  }
};

__device__ __forceinline__ void store4(bf16_t* p, const float (&v)[4]) {
  uint2 w;
  w.x = (uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16);
  w.y = (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16);
  *reinterpret_cast<uint2*>(p) = w;
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// MODE's operands.  STATS, GRAD: rows of h against words of the piece, K = d.  DH: rows of P against
// columns of w, K = the piece's words.  DW: the piece's words against columns of h, K = T.
template <typename T, int MODE>
__global__ __launch_bounds__(NT) void vocab_tile_kernel(VocabArgs p) {
  constexpr int BK = Cfg<T>::BK, LD = Cfg<T>::LD;
  __shared__ __attribute__((aligned(16))) T sa[TM * LD];
  __shared__ __attribute__((aligned(16))) T sb[TN * LD];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave >> 1, wn = wave & 1;
  const T* h = reinterpret_cast<const T*>(p.h);
  const T* w = reinterpret_cast<const T*>(p.w) + (size_t)p.v0 * p.d;
  const T* P = reinterpret_cast<const T*>(p.p);
  constexpr bool LOGITS = MODE == VL_STATS || MODE == VL_GRAD;
  const int M = MODE == VL_DW ? p.vn : p.T;
  const int N = LOGITS ? p.vn : p.d;
  // P's columns past the piece's words are zero up to the next multiple of 8
  const int K = LOGITS ? p.d : (MODE == VL_DH ? p.vn : p.T);
  const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TN;

  f32x16_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  Stage<T, MODE != VL_DW> a;
  Stage<T, LOGITS> b;
  auto load = [&](int k0) {
    if constexpr (LOGITS) {
      a.load(h, p.d, m0, M, k0, K);
      b.load(w, p.d, n0, N, k0, K);
    } else if constexpr (MODE == VL_DH) {
      a.load(P, p.ldp, m0, M, k0, K);
      b.load(w, p.d, n0, N, k0, K);
    } else {
      a.load(P, p.ldp, m0, M, k0, K);
      b.load(h, p.d, n0, N, k0, K);
    }
  };
  load(0);
  for (int k0 = 0; k0 < K; k0 += BK) {
    __syncthreads();
    a.store(sa);
    b.store(sb);
    __syncthreads();
    if (k0 + BK < K) load(k0 + BK);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int s = 0; s < BK / 16; ++s) {
        bf16x8_t fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          fa[i] = *reinterpret_cast<const bf16x8_t*>(sa + (wm * 64 + i * 32 + (lane & 31)) * LD + s * 16 + (lane >> 5) * 8);
          fb[i] = *reinterpret_cast<const bf16x8_t*>(sb + (wn * 64 + i * 32 + (lane & 31)) * LD + s * 16 + (lane >> 5) * 8);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int s = 0; s < BK / 2; ++s) {
        float fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          fa[i] = sa[(wm * 64 + i * 32 + (lane & 31)) * LD + s * 2 + (lane >> 5)];
          fb[i] = sb[(wn * 64 + i * 32 + (lane & 31)) * LD + s * 2 + (lane >> 5)];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
      }
    }
  }

  // Lane l holds row l % 32 of block i and, in element v, column 8 (v / 4) + 4 (l / 32) + v % 4 of
  // block j.
  if constexpr (MODE == VL_STATS) {
    const int c0 = n0 + wn * 64;   // this wave's part: 64 words
    if (c0 >= N) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = m0 + wm * 64 + i * 32 + (lane & 31);
      float mx = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (c0 + j * 32 + 8 * (e / 4) + 4 * (lane >> 5) + e % 4 >= N) acc[i][j][e] = -__builtin_inff();
          mx = fmaxf(mx, acc[i][j][e]);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      float sm = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) sm += expf(acc[i][j][e] - mx);
      sm += __shfl_xor(sm, 32, 64);
      if (lane < 32 && row < M) p.part[(size_t)((p.v0 + c0) / WORDS_PER_PART) * p.T + row] = make_float2(mx, sm);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = m0 + wm * 64 + i * 32 + (lane & 31);
    if (row >= M) continue;
    float lse = 0.0f, dl = 0.0f;
    int tgt = -1;
    if constexpr (MODE == VL_GRAD) {
      lse = p.lse[row];
      tgt = p.target[row];
      dl = tgt >= 0 && tgt < p.V ? p.dloss[row] : 0.0f;
      tgt -= p.v0;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + wn * 64 + j * 32 + 8 * g + 4 * (lane >> 5);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
        if constexpr (MODE == VL_GRAD) {
          if (n >= p.ldp) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float q = expf(v[e] - lse) - (n + e == tgt ? 1.0f : 0.0f);
            v[e] = dl == 0.0f || n + e >= N ? 0.0f : dl * q;
          }
          store4(reinterpret_cast<T*>(p.p) + (size_t)row * p.ldp + n, v);
        } else {
          if (n >= N) continue;   // N = d, a multiple of 8
          if constexpr (MODE == VL_DH) {
            float* acc_row = p.dh_acc + (size_t)row * p.d + n;
            if (!p.first) {
              const float4 o = *reinterpret_cast<const float4*>(acc_row);
              v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
            }
            if (p.last) store4(reinterpret_cast<T*>(p.dh) + (size_t)row * p.d + n, v);
            else store4(acc_row, v);
          } else {
            store4(reinterpret_cast<T*>(p.dw) + (size_t)(p.v0 + row) * p.d + n, v);
          }
        }
      }
  }
}

int parts_of(long long V) { return (int)((V + WORDS_PER_PART - 1) / WORDS_PER_PART); }

// Joins a row's parts and forms the target's logit as a product of its own, which spares the tiles a
// search for it (2 T d elements read beside the product's V d).  JR rows per workgroup, the parts of
// a row dealt to its NT / JR threads and joined in a fixed tree.
__device__ __forceinline__ float2 join_parts(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  // a part of nothing has a maximum of -inf and adds nothing
  const float u = a.x == m ? a.y : a.y * expf(a.x - m), v = b.x == m ? b.y : b.y * expf(b.x - m);
  return make_float2(m, u + v);
}
template <typename T, int JR>
__global__ __launch_bounds__(NT) void vocab_lse_kernel(VocabArgs p, int parts, float* loss, float* lse) {
  constexpr int TPR = NT / JR, NWV = NT / 64;
  __shared__ float2 sl[NWV][JR];
  __shared__ float dots[NWV][JR];
  const int r0 = blockIdx.x * JR, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  {
    // consecutive threads take consecutive rows: a part's statistics are contiguous over the rows
    const int r = threadIdx.x % JR, row = min(r0 + r, p.T - 1);
    const float2* part = p.part + row;
    float2 acc = make_float2(-__builtin_inff(), 0.0f);
    int i = threadIdx.x / JR;
    for (; i + 3 * TPR < parts; i += 4 * TPR) {
      float2 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = part[(size_t)(i + u * TPR) * p.T];
      acc = join_parts(acc, join_parts(join_parts(v[0], v[1]), join_parts(v[2], v[3])));
    }
    for (; i < parts; i += TPR) acc = join_parts(acc, part[(size_t)i * p.T]);
#pragma unroll
    for (int off = 32; off >= JR; off >>= 1)
      acc = join_parts(acc, make_float2(__shfl_xor(acc.x, off, 64), __shfl_xor(acc.y, off, 64)));
    if (lane < JR) sl[wave][lane] = acc;
  }
  {
    // consecutive threads share a row: TPR of them, 16 bytes each
    const int r = threadIdx.x / TPR, s = threadIdx.x % TPR, row = min(r0 + r, p.T - 1);
    const int t = p.target[row];
    constexpr int E = 16 / sizeof(T);
    float a = 0.0f;
    if (t >= 0 && t < p.V) {
      const T* h = reinterpret_cast<const T*>(p.h) + (size_t)row * p.d;
      const T* w = reinterpret_cast<const T*>(p.w) + (size_t)t * p.d;
      for (int c = s * E; c < p.d; c += TPR * E) {
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(h + c), y = *reinterpret_cast<const u32x4_t*>(w + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (E == 8) {
            a += __uint_as_float(x[e] << 16) * __uint_as_float(y[e] << 16);
            a += __uint_as_float(x[e] & 0xffff0000u) * __uint_as_float(y[e] & 0xffff0000u);
          } else {
            a += __uint_as_float(x[e]) * __uint_as_float(y[e]);
          }
        }
      }
    }
#pragma unroll
    for (int off = (TPR < 64 ? TPR : 64) / 2; off >= 1; off >>= 1) a += __shfl_xor(a, off, 64);
    if (lane % TPR == 0) dots[wave][r] = a;   // TPR > 64: one partial per wave
  }
  __syncthreads();
  const int r = threadIdx.x, row = r0 + r;
  if (r >= JR || row >= p.T) return;
  float2 acc = sl[0][r];
#pragma unroll
  for (int w = 1; w < NWV; ++w) acc = join_parts(acc, sl[w][r]);
  float dot = 0.0f;
  if constexpr (TPR > 64) {
    for (int w = 0; w < NWV; ++w) dot += dots[w][0];
  } else {
    dot = dots[r * TPR / 64][r];
  }
  const float l = acc.x + logf(acc.y);
  const int t = p.target[row];
  lse[row] = l;
  loss[row] = t >= 0 && t < p.V ? l - dot : 0.0f;
}

// As many rows per workgroup as still fill the CUs: few rows have their parts dealt to more threads.
template <typename T>
hipError_t launch_lse(const VocabArgs& p, float* loss, float* lse, hipStream_t s) {
  const int parts = parts_of(p.V);
  if (p.T >= 16 * NUM_CUS) vocab_lse_kernel<T, 16><<<dim3(ceil_div(p.T, 16)), dim3(NT), 0, s>>>(p, parts, loss, lse);
  else if (p.T >= 4 * NUM_CUS) vocab_lse_kernel<T, 4><<<dim3(ceil_div(p.T, 4)), dim3(NT), 0, s>>>(p, parts, loss, lse);
  else vocab_lse_kernel<T, 1><<<dim3(p.T), dim3(NT), 0, s>>>(p, parts, loss, lse);
  return hipGetLastError();
}

template <typename T>
__global__ __launch_bounds__(NT) void fill_zero_kernel(T* p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * NT + threadIdx.x; i < n; i += (size_t)gridDim.x * NT) p[i] = T(0);
}

// Words per piece of the backward, a multiple of 256: pieces of one size, P of about 2^26 elements
// and at least 4096 words.
int piece_words(long long T, long long V) {
  const long long want = std::max<long long>(4096, (1LL << 26) / std::max<long long>(T, 1));
  const long long pieces = (V + want - 1) / want;
  return (int)(((V + pieces - 1) / pieces + 255) / 256 * 256);
}

bool use_pipe(int T, int d, int V, bool bf16) { return bf16; }

template <typename T, int MODE>
hipError_t launch_tiles(const VocabArgs& p, hipStream_t s) {
  const int M = MODE == VL_DW ? p.vn : p.T;
  const int N = MODE == VL_DW || MODE == VL_DH ? p.d : (MODE == VL_GRAD ? std::min(p.ldp, ceil_div(p.vn, 8) * 8) : p.vn);
  hipLaunchKernelGGL((vocab_tile_kernel<T, MODE>), dim3(ceil_div(N, TN), ceil_div(M, TM)), dim3(NT), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t loss_fwd(VocabArgs p, float* loss, float* lse, void* ws, hipStream_t s) {
  p.part = reinterpret_cast<float2*>(ws);
  p.v0 = 0;
  p.vn = p.V;
  const hipError_t e = use_pipe(p.T, p.d, p.V, sizeof(T) == 2) ? launch_pipe(VL_STATS, p, s) : launch_tiles<T, VL_STATS>(p, s);
  if (e != hipSuccess) return e;
  return launch_lse<T>(p, loss, lse, s);
}

// Bytes of the accumulated dh.
size_t acc_bytes(int T, int d, int V, bool bf16) {
  return align256(use_pipe(T, d, V, bf16) ? pipe_acc_bytes(T, d, piece_words(T, V)) : (size_t)T * d * 4);
}

template <typename T>
hipError_t loss_bwd(VocabArgs p, void* ws, hipStream_t s) {
  if (p.T == 0) {
    const size_t n = (size_t)p.V * p.d;
    fill_zero_kernel<T><<<dim3((unsigned)std::min<size_t>((n + NT - 1) / NT, 8192)), dim3(NT), 0, s>>>((T*)p.dw, n);
    return hipGetLastError();
  }
  const int words = piece_words(p.T, p.V);
  const bool pipe = use_pipe(p.T, p.d, p.V, sizeof(T) == 2);
  p.ldp = words;
  p.dh_acc = reinterpret_cast<float*>(ws);
  p.p = reinterpret_cast<char*>(ws) + acc_bytes(p.T, p.d, p.V, sizeof(T) == 2);
  for (int v0 = 0; v0 < p.V; v0 += words) {
    p.v0 = v0;
    p.vn = std::min(words, p.V - v0);
    p.first = v0 == 0;
    p.last = v0 + words >= p.V;
    hipError_t e = pipe ? launch_pipe(VL_GRAD, p, s) : launch_tiles<T, VL_GRAD>(p, s);
    if (e == hipSuccess) e = pipe ? launch_pipe(VL_DH, p, s) : launch_tiles<T, VL_DH>(p, s);
    if (e == hipSuccess) e = pipe ? launch_pipe(VL_DW, p, s) : launch_tiles<T, VL_DW>(p, s);
    if (e != hipSuccess) return e;
  }
  return pipe ? launch_pipe_join(p, s) : hipSuccess;
}

}  // namespace

size_t vocab_loss_ws_bytes(long long T, long long d, long long V, bool bf16) {
  return (size_t)T * parts_of(V) * sizeof(float2);
}

hipError_t launch_vocab_loss(const void* h, const void* w, const int32_t* target, int T, int d, int V, bool bf16,
                             float* loss, float* lse, void* ws, hipStream_t s) {
  VocabArgs p{};
  p.h = h; p.w = w; p.target = target; p.T = T; p.d = d; p.V = V;
  return bf16 ? loss_fwd<bf16_t>(p, loss, lse, ws, s) : loss_fwd<float>(p, loss, lse, ws, s);
}

size_t vocab_loss_bwd_ws_bytes(long long T, long long d, long long V, bool bf16) {
  if (T <= 0) return 0;
  return acc_bytes((int)T, (int)d, (int)V, bf16) + (size_t)T * piece_words(T, V) * (bf16 ? 2 : 4);
}

hipError_t launch_vocab_loss_bwd(const void* h, const void* w, const int32_t* target, const float* lse,
                                 const float* dloss, int T, int d, int V, bool bf16, void* dh, void* dw, void* ws,
                                 hipStream_t s) {
  VocabArgs p{};
  p.h = h; p.w = w; p.target = target; p.lse = lse; p.dloss = dloss; p.T = T; p.d = d; p.V = V; p.dh = dh; p.dw = dw;
  return bf16 ? loss_bwd<bf16_t>(p, ws, s) : loss_bwd<float>(p, ws, s);
}

}  // namespace moe
