// Softmax cross entropy over a vocabulary and its gradient, in pieces of the vocabulary.
//
//   l = h w^T (T x V),  lse_t = log sum_v exp(l_tv),  loss_t = lse_t - l[t, target_t]
//   P = (dloss_t / s) (exp(l_tv - lse_t) - [v = target_t]),  dh = s P w,  dw = s P^T h
//
// The logits are never stored.  Forward: each tile of the product keeps, per row, the maximum and
// the sum of exponentials of each 64 (or 32) of its columns; a second kernel joins a row's parts in a
// fixed order.  Backward: the product is formed again one piece of the vocabulary at a time, its
// epilogue writes P of the piece (in the storage type: the operand of the two gradient products; one
// more rounding of its elements than an fp32 P would have, at four times the products' rate), and dh
// accumulates over the pieces in fp32.
// s is the largest |dloss| of a row with a loss.  Of the mean's gradient, where every dloss is 1 / n,
// the target's element of P is then near -1, not near -1 / n, whose rounding to bf16 would be the same
// in every row and add up in dw: at 8192 x 4096 x 65536 the gradients are 0.19% off the exact ones
// instead of 0.27% (0.17% is the rounding of the outputs themselves).
// A target outside [0, V) marks a row without loss: loss 0, P = 0 exactly.
#include "vocab_loss.h"

#include <algorithm>
#include <cmath>
#include <initializer_list>

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

using namespace vocab;

constexpr int NT = 256;

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
hipError_t launch_lse(const VocabArgs& p, int parts, float* loss, float* lse, hipStream_t s) {
  if (p.T >= 16 * NUM_CUS) vocab_lse_kernel<T, 16><<<dim3(ceil_div(p.T, 16)), dim3(NT), 0, s>>>(p, parts, loss, lse);
  else if (p.T >= 4 * NUM_CUS) vocab_lse_kernel<T, 4><<<dim3(ceil_div(p.T, 4)), dim3(NT), 0, s>>>(p, parts, loss, lse);
  else vocab_lse_kernel<T, 1><<<dim3(p.T), dim3(NT), 0, s>>>(p, parts, loss, lse);
  return hipGetLastError();
}

// The largest finite |dloss| of a row with a loss, 1 if there is none.
__global__ __launch_bounds__(1024) void vocab_scale_kernel(VocabArgs p, float* scale) {
  __shared__ float red[16];
  float m = 0.0f;
#pragma unroll 4
  for (int t = threadIdx.x; t < p.T; t += 1024) m = fmaxf(m, dloss_size(p, t));
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < 16; ++i) m = fmaxf(m, red[i]);
    *scale = m > 0.0f ? m : 1.0f;
  }
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

// Which tiles a product takes: 64x64, 128x128 (vocab_loss_tile.hip) or, bf16 only, 256x256
// (vocab_loss_pipe.hip), by an estimate of each in us, straight lines through the times of some 20 shapes
// that they meet within 6-16%: of the tile kernels the work per CU, n tiles of s steps of K, of the
// pipelined kernel the rounds of its workgroups, one per CU.  Measured forward kernels, 64, 128 and 256 (us):
// 100 tokens x 8000 words x d 4096: 20.8, 36.7, 54.3; 1000 x 4000 x 1000: 22.3, 17.0, 28.6;
// 2000 x 4000 x 1000: 41.3, 27.8, 29.0; 3000 x 20000 x 128: 56, 54, 28; 184 x 30594 x 3784: 137, 100, 102.
enum Tiles { SMALL, LARGE, PIPE };

// n: tiles per CU; K of a tile.
struct Load {
  double n;
  int k;
};
Load tile_load(int M, int N, int K, int splits, bool large) {
  return Load{(double)tile_count(M, N, large) * splits / NUM_CUS, ceil_div(K, splits)};
}
// fp32 is bound by the matrix cores: 0.0198 us of a CU for each k of a 64x64 tile, 0.069 of a 128x128
// one, of which two run together and end together.
double f32_us(Load a, Load b, bool large) {
  const double n = a.n + b.n, k = (a.n * a.k + b.n * b.k) / n;
  if (!large) return 4.0 + 0.0198 * std::min(std::ceil(n), n + 0.5) * k;
  return 6.0 + 0.069 * (n <= 1 ? 1 : 2 * std::ceil(n / 2)) * k;
}

Tiles logits_tiles(int T, int d, int words, bool bf16) {
  const Load s = tile_load(T, words, d, 1, false), l = tile_load(T, words, d, 1, true);
  const bool one_row = T <= 64;   // of 64x64 tiles: large ones would be half empty
  if (!bf16) return !one_row && f32_us(l, Load{0, 0}, true) < f32_us(s, Load{0, 0}, false) ? LARGE : SMALL;
  double best = 3.3 + 0.6 * std::max(s.n, 0.9) * (ceil_div(d, 128) + 0.35);
  Tiles tiles = SMALL;
  const double large = 5.4 + 0.65 * std::max(l.n, 0.75) * (ceil_div(d, 64) + 3.1);
  if (!one_row && large < best) best = large, tiles = LARGE;
  const int rounds = ceil_div((long long)ceil_div(T, 256) * ceil_div(words, 256), NUM_CUS);
  return 3.2 + rounds * (3.7 + 1.3 * ceil_div(d, 64)) < best ? PIPE : tiles;
}

// dh and dw: both in tiles of one size run as one launch.
struct GradTiles {
  Tiles dh, dw;
};
GradTiles grad_tiles(int T, int d, int words, bool bf16) {
  const auto join_us = [](double partials) { return partials > 0 ? 3.0 + partials * 4 / 6.4e6 : 0.0; };
  GradTiles plan{SMALL, SMALL};
  double best = 0;
  for (Tiles dh : {SMALL, LARGE, PIPE})
    for (Tiles dw : {SMALL, LARGE, PIPE}) {
      if (dh != PIPE && dw != PIPE ? dh != dw : !bf16) continue;
      double us = 0, sums = 0;   // sums: elements of the partial products that the tiles' join reads
      Load tile[2] = {};
      bool large = false;
      const auto add = [&](Load& to, int M, int N, int K, Tiles t) {
        large = t == LARGE;
        const int splits = tile_splits(M, N, K, large);
        to = tile_load(M, N, K, splits, large);
        if (splits > 1) sums += (double)splits * M * N;
      };
      if (dh == PIPE) {
        const int splits = pipe_dh_splits(T, d, words);
        const int rounds = ceil_div((long long)ceil_div(T, 256) * ceil_div(d, 256) * splits, NUM_CUS);
        us += 1.1 + rounds * (2.9 + 1.87 * ceil_div(ceil_div(words, splits), 64)) + join_us((double)splits * T * d);
      } else {
        add(tile[0], T, d, words, dh);
      }
      if (dw == PIPE) {
        const int splits = pipe_dw_splits(T, d, words);
        const int rounds = ceil_div((long long)ceil_div(words, 256) * ceil_div(d, 256) * splits, NUM_CUS);
        us += rounds * (9.7 + 1.47 * ceil_div(ceil_div(T, splits), 64)) + (splits > 1 ? join_us((double)splits * words * d) : 0.0);
      } else {
        add(tile[1], words, d, T, dw);
      }
      if (dh != PIPE || dw != PIPE) {
        if (!bf16) {
          us += f32_us(tile[0], tile[1], large);
        } else {
          us += large ? 6.2 : 4.5;
          for (const Load& t : tile) us += large ? 0.55 * t.n * (ceil_div(t.k, 64) + 6) : 0.565 * t.n * (ceil_div(t.k, 128) + 0.6);
        }
        us += join_us(sums);
      }
      if (best == 0 || us < best) best = us, plan = GradTiles{dh, dw};
    }
  return plan;
}

hipError_t launch_product(Tiles tiles, int mode, VocabArgs p, bool bf16, hipStream_t s) {
  p.large = tiles == LARGE;
  return tiles == PIPE ? launch_pipe(mode, p, s) : launch_tile(mode, p, bf16, s);
}

template <typename T>
hipError_t loss_fwd(VocabArgs p, float* loss, float* lse, void* ws, hipStream_t s) {
  constexpr bool bf16 = sizeof(T) == 2;
  p.part = reinterpret_cast<float2*>(ws);
  p.v0 = 0;
  p.vn = p.V;
  const Tiles tiles = logits_tiles(p.T, p.d, p.V, bf16);
  const hipError_t e = launch_product(tiles, VL_STATS, p, bf16, s);
  if (e != hipSuccess) return e;
  return launch_lse<T>(p, ceil_div(p.V, tiles == PIPE ? PIPE_PART : TILE_PART), loss, lse, s);
}

// The workspace of the backward: the scale, dh's accumulators, dw's partial products (where its rows
// are split; the last piece may be narrower and split further), then P.
struct BwdSpace {
  size_t scale = 256, dh, dw, p;
  size_t total() const { return scale + dh + dw + p; }
};
BwdSpace bwd_space(int T, int d, int V, bool bf16) {
  const int words = piece_words(T, V), wide = std::min(words, V), last = V - (V - 1) / words * words;
  const GradTiles tiles = grad_tiles(T, d, words, bf16);
  BwdSpace s;
  s.dh = align256(tiles.dh == PIPE ? pipe_dh_bytes(T, d, words) : tile_acc_bytes(T, d, words, tiles.dh == LARGE));
  s.dw = 0;
  for (int vn : {wide, last}) {
    const bool large = tiles.dw == LARGE;
    const size_t tile = tile_splits(vn, d, T, large) > 1 ? tile_acc_bytes(vn, d, T, large) : 0;
    s.dw = std::max(s.dw, align256(tiles.dw == PIPE ? pipe_dw_bytes(T, d, vn) : tile));
  }
  s.p = (size_t)T * words * (bf16 ? 2 : 4);
  return s;
}

template <typename T>
hipError_t loss_bwd(VocabArgs p, void* ws, hipStream_t s) {
  if (p.T == 0) {
    const size_t n = (size_t)p.V * p.d;
    fill_zero_kernel<T><<<dim3((unsigned)std::min<size_t>((n + NT - 1) / NT, 8192)), dim3(NT), 0, s>>>((T*)p.dw, n);
    return hipGetLastError();
  }
  constexpr bool bf16 = sizeof(T) == 2;
  const int words = piece_words(p.T, p.V);
  const GradTiles tiles = grad_tiles(p.T, p.d, words, bf16);
  const BwdSpace space = bwd_space(p.T, p.d, p.V, bf16);
  p.ldp = words;
  char* at = reinterpret_cast<char*>(ws);
  float* scale = reinterpret_cast<float*>(at);
  p.scale = scale;
  p.dh_acc = reinterpret_cast<float*>(at += space.scale);
  p.dw_acc = reinterpret_cast<float*>(at += space.dh);
  p.p = at += space.dw;
  hipError_t e = hipSuccess;
  if (p.T <= SCALE_ROWS && logits_tiles(p.T, p.d, std::min(words, p.V), bf16) != PIPE) {
    p.scale_out = scale;   // the first piece's tiles find it
  } else {
    vocab_scale_kernel<<<dim3(1), dim3(1024), 0, s>>>(p, scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  for (int v0 = 0; v0 < p.V; v0 += words) {
    p.v0 = v0;
    p.vn = std::min(words, p.V - v0);
    p.first = v0 == 0;
    p.last = v0 + words >= p.V;
    e = launch_product(logits_tiles(p.T, p.d, p.vn, bf16), VL_GRAD, p, bf16, s);
    if (e != hipSuccess) return e;
    p.scale_out = nullptr;
    if (tiles.dh != PIPE && tiles.dw != PIPE) {
      p.large = tiles.dh == LARGE;
      e = launch_tile_pair(p, bf16, s);
    } else {
      e = launch_product(tiles.dh, VL_DH, p, bf16, s);
      if (e == hipSuccess) e = launch_product(tiles.dw, VL_DW, p, bf16, s);
      p.large = tiles.dh == LARGE;
      if (e == hipSuccess && p.last) e = tiles.dh == PIPE ? launch_pipe_join(p, s) : launch_tile_join(p, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t vocab_loss_ws_bytes(long long T, long long d, long long V, bool bf16) {
  return (size_t)T * ceil_div(V, logits_tiles((int)T, (int)d, (int)V, bf16) == PIPE ? PIPE_PART : TILE_PART) * sizeof(float2);
}

hipError_t launch_vocab_loss(const void* h, const void* w, const int32_t* target, int T, int d, int V, bool bf16,
                             float* loss, float* lse, void* ws, hipStream_t s) {
  VocabArgs p{};
  p.h = h; p.w = w; p.target = target; p.T = T; p.d = d; p.V = V;
  return bf16 ? loss_fwd<bf16_t>(p, loss, lse, ws, s) : loss_fwd<float>(p, loss, lse, ws, s);
}

VocabPlan vocab_loss_plan(int T, int d, int V, bool bf16) {
  VocabPlan plan{};
  if (T == 0) return plan;
  const auto side = [](Tiles t) { return t == PIPE ? 256 : t == LARGE ? 128 : 64; };
  VocabArgs p{};
  p.T = T; p.d = d; p.V = V;
  p.ldp = piece_words(T, V);
  p.vn = std::min(p.ldp, V);
  p.first = true;
  p.last = p.vn == V;
  plan.piece_words = p.ldp;
  plan.pieces = ceil_div(V, p.ldp);
  plan.fwd_tile = side(logits_tiles(T, d, V, bf16));
  plan.logits_tile = side(logits_tiles(T, d, p.vn, bf16));
  const GradTiles tiles = grad_tiles(T, d, p.ldp, bf16);
  plan.dh_tile = side(tiles.dh);
  plan.dw_tile = side(tiles.dw);
  const auto ks = [&](Tiles t, int mode) {
    p.large = t == LARGE;
    return t == PIPE ? pipe_ks(mode, p) : tile_ks(mode, p, bf16);
  };
  plan.dh_splits = ks(tiles.dh, VL_DH);
  plan.dw_splits = ks(tiles.dw, VL_DW);
  return plan;
}

size_t vocab_loss_bwd_ws_bytes(long long T, long long d, long long V, bool bf16) {
  if (T <= 0) return 0;
  return bwd_space((int)T, (int)d, (int)V, bf16).total();
}

hipError_t launch_vocab_loss_bwd(const void* h, const void* w, const int32_t* target, const float* lse,
                                 const float* dloss, int T, int d, int V, bool bf16, void* dh, void* dw, void* ws,
                                 hipStream_t s) {
  VocabArgs p{};
  p.h = h; p.w = w; p.target = target; p.lse = lse; p.dloss = dloss; p.T = T; p.d = d; p.V = V; p.dh = dh; p.dw = dw;
  return bf16 ? loss_bwd<bf16_t>(p, ws, s) : loss_bwd<float>(p, ws, s);
}

}  // namespace moe
