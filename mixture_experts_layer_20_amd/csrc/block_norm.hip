// Norms before and after the MoE block, with the block's gate and residual scale, and their backward.
//
//   before   xn  = x r w,                     r = 1 / sqrt(mean_j x_j^2 + eps)
//   after    out = a x + g * (y r w),         r = 1 / sqrt(mean_j y_j^2 + eps)
// The block's output y comes as a tensor, or is the layer's weighted combine, summed here: the
// normalised row is then read once from the experts' rows and never stored.
//
// Backward, with n = y r (or x r) and u = w * g * dout (or w * dxn):
//   dy = r (u - n mean_j(u_j n_j)),  dg_s = w * S_s,  dw = sum_s g_s * S_s,
//   S_s = sum over the rows t of gate row s of dout_t * n_t
// so one column sum S per gate row gives both parameter gradients.
//
// Every sum, norm and statistic is fp32; a value is rounded to the storage type once, at its store.
//
// Bound by memory.  A row lies in the registers of a wave (d <= 1024), else of a workgroup of up to
// 1024 lanes, from its loads to its stores, so each tensor passes once.  8192 x 4096 bf16, top-4 and a
// shared expert: before 21 us (134 MB, 6.3 TB/s), combine and after 73 us (470 MB, 6.4 TB/s), with the
// combined rows kept for the backward 89 us (537 MB, 6.0 TB/s; 97 us for as many bytes at 16384 x 2048).
// 16384 x 2048 bf16: before 24 us, after 35 us (201 MB, 5.7 TB/s), their backward 44 us (268 MB, 6.1
// TB/s) and 33 us (201 MB, 6.1 TB/s) and 6.4 us each for the join of the column sums.  A device copy
// moves 5.1 TB/s; what is above it comes from the last-level cache.
#include "block_step.h"

#include <algorithm>

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// 8 consecutive elements, as loaded and widened.  load_once: a stream that nothing reads again soon (a
// nontemporal load: the experts' rows at 6.6 TB/s instead of 4.9).  Stores are nontemporal: the four
// calls of a forward and backward pass at 16384 x 2048 take 140 us with them and 161 without, where
// the inputs they read in common then stay in the last-level cache; inside the layer, with its
// products between the calls, both take the same time.
template <typename T> struct Seg8;
template <> struct Seg8<bf16_t> {
  u32x4_t w;
  __device__ __forceinline__ void load(const bf16_t* p) { w = *reinterpret_cast<const u32x4_t*>(p); }
  __device__ __forceinline__ void load_once(const bf16_t* p) {
    w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  }
  __device__ __forceinline__ void zero() { w = u32x4_t{0, 0, 0, 0}; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ void put(bf16_t* p, const float (&v)[8]) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (uint32_t)f32_to_bf16(v[2 * i]) | ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16);
    __builtin_nontemporal_store(r, reinterpret_cast<u32x4_t*>(p));
  }
};
template <> struct Seg8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void load_once(const float* p) { load(p); }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ static __forceinline__ void put(float* p, const float (&v)[8]) {
    __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4_t*>(p));
    __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4_t*>(p) + 1);
  }
};

__device__ __forceinline__ void load4(const bf16_t* p, float (&v)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}

constexpr int NT = 256;   // threads of a workgroup, or L where a row takes more
template <int L>
constexpr int threads() { return L < NT ? NT : L; }

// Sum over the L lanes that share a row (L = 64: a wave; otherwise the workgroup, one row at a time).
// `red` holds one value per wave and slot; two slots alternate, so one barrier per sum is enough.
template <int L>
__device__ __forceinline__ float row_sum(float s, float (&red)[2][16], int& slot) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < L / 64; i += 4)
      s += (red[slot][i] + red[slot][i + 1]) + (red[slot][i + 2] + red[slot][i + 3]);
    slot ^= 1;
  }
  return s;
}

// Lane `lane` of the L lanes of a row holds the 8-element segments lane + i L, i < NV.
struct Cols {
  int c;
  bool in;
};
template <int L>
__device__ __forceinline__ Cols cols(int lane, int i, int d) {
  const int c = 8 * (lane + i * L);
  return Cols{c, c < d};
}

template <typename T, int L, int NV>
__global__ __launch_bounds__(threads<L>()) void norm_in_kernel(const T* x, const T* w, int rows, int d, float eps, T* xn,
                                                     float* rstd) {
  __shared__ float red[2][16];
  const int lane = threadIdx.x % L;
  int slot = 0;
  // (a wave, or a workgroup whose row sum has barriers, leaves the loop as a whole)
  for (int t = blockIdx.x * (threads<L>() / L) + threadIdx.x / L; t < rows; t += gridDim.x * (threads<L>() / L)) {
    Seg8<T> xr[NV], wr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols k = cols<L>(lane, i, d);
      if (k.in) {
        xr[i].load(x + (size_t)t * d + k.c);
        wr[i].load(w + k.c);
      } else {
        xr[i].zero();
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8];
      xr[i].get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[e] * v[e];
    }
    const float r = 1.0f / sqrtf(row_sum<L>(s, red, slot) / (float)d + eps);
    if (rstd && lane == 0) rstd[t] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols k = cols<L>(lane, i, d);
      if (!k.in) continue;
      float v[8], wv[8];
      xr[i].get(v);
      wr[i].get(wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * r * wv[e];
      Seg8<T>::put(xn + (size_t)t * d + k.c, v);
    }
  }
}

// The norm after the block.  COMBINE: y is the layer's weighted combine of k rows of y_perm and the
// shared expert's row, summed in fp32 in the order of combine_kernel (slots, then the shared row) and
// normalised unrounded; y_out (if given) gets it rounded, for the backward.  Up to four expert rows
// are loaded before the first is used, and the residual, weight and gate before the row's statistic
// is known.
template <typename T, int L, int NV, bool COMBINE>
__global__ __launch_bounds__(threads<L>()) void norm_out_kernel(const T* y, const float* topk_gate, const int32_t* dest_pos,
                                                      const T* shared, int k, const T* x, const T* w, const T* gate,
                                                      int gate_rows, float res_scale, int rows, int d, float eps,
                                                      T* y_out, T* out, float* rstd) {
  __shared__ float red[2][16];
  const int lane = threadIdx.x % L;
  int slot = 0;
  for (int t = blockIdx.x * (threads<L>() / L) + threadIdx.x / L; t < rows; t += gridDim.x * (threads<L>() / L)) {
    float yv[NV][8];
    Seg8<T> xr[NV], wr[NV], gr[NV], sr[NV];
    const T* grow = gate ? gate + (size_t)(t / gate_rows) * d : nullptr;
    auto load = [&](Seg8<T> (&r)[NV], const T* from) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Cols q = cols<L>(lane, i, d);
        if (q.in) r[i].load(from + q.c);
        else r[i].zero();
      }
    };
    if constexpr (COMBINE) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) yv[i][e] = 0.0f;
      constexpr int G = 4;   // rows in flight
      for (int j0 = 0; j0 < k; j0 += G) {
        Seg8<T> r[G][NV];
        float g[G];
#pragma unroll
        for (int u = 0; u < G; ++u)
          if (j0 + u < k) {
            g[u] = topk_gate[(size_t)t * k + j0 + u];
            const T* row = y + (size_t)dest_pos[(size_t)t * k + j0 + u] * d;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              const Cols q = cols<L>(lane, i, d);
              if (q.in) r[u][i].load_once(row + q.c);
              else r[u][i].zero();
            }
          }
        if (j0 == 0) {
          if (shared) load(sr, shared + (size_t)t * d);
          load(xr, x + (size_t)t * d);
        }
#pragma unroll
        for (int u = 0; u < G; ++u)
          if (j0 + u < k) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              float v[8];
              r[u][i].get(v);
#pragma unroll
              for (int e = 0; e < 8; ++e) yv[i][e] += g[u] * v[e];
            }
          }
      }
      if (shared) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float v[8];
          sr[i].get(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) yv[i][e] += v[e];
        }
      }
      if (y_out) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const Cols q = cols<L>(lane, i, d);
          if (q.in) Seg8<T>::put(y_out + (size_t)t * d + q.c, yv[i]);
        }
      }
    } else {
      load(sr, y + (size_t)t * d);
      load(xr, x + (size_t)t * d);
#pragma unroll
      for (int i = 0; i < NV; ++i) sr[i].get(yv[i]);
    }
    load(wr, w);
    if (grow) load(gr, grow);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += yv[i][e] * yv[i][e];
    const float r = 1.0f / sqrtf(row_sum<L>(s, red, slot) / (float)d + eps);
    if (rstd && lane == 0) rstd[t] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols q = cols<L>(lane, i, d);
      if (!q.in) continue;
      float xv[8], wv[8], o[8];
      xr[i].get(xv);
      wr[i].get(wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = yv[i][e] * r * wv[e];
      if (grow) {
        gr[i].get(wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= wv[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += res_scale * xv[e];
      Seg8<T>::put(out + (size_t)t * d + q.c, o);
    }
  }
}

// Row block of the backward: workgroup b owns rows b R .. min(T, (b + 1) R), walked piece by piece
// (a piece: the block's rows of one gate row).  At a piece's end the column sum S of its rows goes
//   to dgate directly when the gate row lies inside the block,
//   else to the block's `head` partial (the gate row began before the block or at its start) or its
//   `tail` partial (it began inside and goes on in the next block): a block has at most one of each.
// Gated by several gate rows (MULTI), the block's dw is summed over its pieces; otherwise the one
// column sum S, or its join over the blocks, gives both.
struct BwdArgs {
  int rows, d, R, gate_rows;
  float res_scale;
  float* part;   // [3][blocks][d]: dw partials (MULTI), head (the only ones otherwise), tail
  float* dw;
  float* dgate;
  int row_blocks;   // workgroups behind these take the column sums, if there are any
};

// Few rows: the column sums need each row's rstd alone, which is given, so workgroups beside those of
// the rows form them, 16 columns each, from a second reading of the rows, and no join follows.
template <typename T, int TH>
__device__ __forceinline__ void column_sums(const T* dout, const T* y, const T* w, const T* gate, const float* rstd,
                                            const BwdArgs& p) {
  constexpr int SL = TH / 4;
  __shared__ float red[SL][16 + 1];
  const int d = p.d, slice = threadIdx.x / 4, x = threadIdx.x % 4 * 4;
  const int c = ((int)blockIdx.x - p.row_blocks) * 16 + x;
  const bool in = c < d;   // d is a multiple of 8
  float dw[4] = {0, 0, 0, 0};
  for (int t0 = 0, seg = 0; t0 < p.rows; ++seg) {
    const int t1 = gate ? (int)min((long long)p.rows, (long long)t0 + p.gate_rows) : p.rows;
    float S[4] = {0, 0, 0, 0};
    if (in) {
#pragma unroll 4
      for (int t = t0 + slice; t < t1; t += SL) {
        float n[4], g[4];
        load4(y + (size_t)t * d + c, n);
        load4(dout + (size_t)t * d + c, g);
        const float r = rstd[t];
#pragma unroll
        for (int e = 0; e < 4; ++e) S[e] += g[e] * (n[e] * r);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[slice][x + e] = S[e];
#pragma unroll
    for (int off = SL / 2; off >= 1; off >>= 1) {
      __syncthreads();
      if (slice < off) {
#pragma unroll
        for (int e = 0; e < 4; ++e) red[slice][x + e] += red[slice + off][x + e];
      }
    }
    if (slice == 0 && in) {
      float wv[4], gv[4];
      if (gate) {
        load4(w + c, wv);
        load4(gate + (size_t)seg * d + c, gv);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = red[0][x + e];
        dw[e] += gate ? gv[e] * v : v;
        if (gate) p.dgate[(size_t)seg * d + c + e] = wv[e] * v;
      }
    }
    __syncthreads();
    t0 = t1;
  }
  if (slice == 0 && in) {
#pragma unroll
    for (int e = 0; e < 4; ++e) p.dw[c + e] = dw[e];
  }
}

// IN: dxn (as dout), x (as y), dres.  Otherwise: dout, y, gate.  The next row is loaded while the
// current one is reduced: without it the loads of a row waited for the statistic of the row before.
template <typename T, int L, int NV, bool IN, bool MULTI>
__global__ __launch_bounds__(threads<L>()) void norm_bwd_kernel(const T* dout, const T* y, const T* w, const T* gate,
                                                                const T* dres, const float* rstd, T* dy, BwdArgs p) {
  constexpr int NS = threads<L>() / L;   // rows in flight of a workgroup
  constexpr bool AHEAD = L < 1024;       // (a workgroup of 1024 has 128 registers a lane: no room)
  __shared__ float red[2][16];
  extern __shared__ float sums[];   // [NS - 1][8 NV L] column sums of the other waves (L = 64)
  const int lane = threadIdx.x % L, me = threadIdx.x / L;
  const int d = p.d;
  if ((int)blockIdx.x >= p.row_blocks) return column_sums<T, threads<L>()>(dout, y, w, gate, rstd, p);
  const int r0 = blockIdx.x * p.R, r1 = min(p.rows, r0 + p.R);
  const int blocks = p.row_blocks;
  const bool sums_here = (int)gridDim.x == blocks;
  const float inv_d = 1.0f / (float)d;
  int slot = 0;
  struct Row {
    Seg8<T> y[NV], g[NV], e[IN ? NV : 1];
    float r;
  };
  auto load = [&](Row& q, int t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols c = cols<L>(lane, i, d);
      if (c.in) {
        q.y[i].load(y + (size_t)t * d + c.c);
        q.g[i].load(dout + (size_t)t * d + c.c);
        if constexpr (IN) {
          if (dres) q.e[i].load(dres + (size_t)t * d + c.c);
        }
      } else {
        q.y[i].zero();
        q.g[i].zero();
      }
    }
    q.r = rstd[t];
  };
  float dwacc[MULTI ? NV : 1][8] = {};
  for (int p0 = r0; p0 < r1;) {
    const int seg = gate ? p0 / p.gate_rows : 0;
    const long long seg_end = MULTI ? (long long)(seg + 1) * p.gate_rows : (long long)p.rows;
    const int p1 = (int)min((long long)r1, seg_end);
    float gw[NV][8], S[NV][8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const Cols q = cols<L>(lane, i, d);
      Seg8<T> sg;
      sg.zero();
      if (q.in) sg.load(w + q.c);
      sg.get(gw[i]);
      if (gate && q.in) {
        float gv[8];
        sg.load(gate + (size_t)seg * d + q.c);
        sg.get(gv);
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[i][e] *= gv[e];
      }
    }
    Row cur, next;
    if (AHEAD && p0 + me < p1) load(next, p0 + me);
    for (int t = p0 + me; t < p1; t += NS) {
      if constexpr (AHEAD) {
        cur = next;
        if (t + NS < p1) load(next, t + NS);
      } else {
        load(cur, t);
      }
      const float r = cur.r;
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float n[8], g[8];
        cur.y[i].get(n);
        cur.g[i].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          n[e] *= r;
          S[i][e] += g[e] * n[e];
          dot += g[e] * gw[i][e] * n[e];
        }
      }
      const float m = row_sum<L>(dot, red, slot) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Cols q = cols<L>(lane, i, d);
        if (!q.in) continue;
        float n[8], g[8];
        cur.y[i].get(n);
        cur.g[i].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = r * (g[e] * gw[i][e] - n[e] * r * m);
        if constexpr (IN) {
          if (dres) {
            float v[8];
            cur.e[i].get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] += p.res_scale * v[e];
          }
        }
        Seg8<T>::put(dy + (size_t)t * d + q.c, g);
      }
    }
    p0 = p1;
    if (!sums_here) continue;
    // S over the workgroup's waves, into wave 0 (L = 64)
    if constexpr (NS > 1) {
      if (me > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) sums[((me - 1) * NV * 8 + i * 8 + e) * L + lane] = S[i][e];
      }
      __syncthreads();
      if (me == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int o = 0; o < NS - 1; ++o) S[i][e] += sums[(o * NV * 8 + i * 8 + e) * L + lane];
      }
      __syncthreads();
    }
    if (me == 0) {
      const long long seg_begin = MULTI ? (long long)seg * p.gate_rows : 0;
      const bool whole = seg_begin >= r0 && min(seg_end, (long long)p.rows) <= r1;
      float* head = p.part + ((size_t)(seg_begin <= r0 ? 1 : 2) * blocks + blockIdx.x) * d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Cols q = cols<L>(lane, i, d);
        if (!q.in) continue;
        if (!whole) Seg8<float>::put(head + q.c, S[i]);
        if (!MULTI && !whole) continue;   // the join forms dw and dgate from the blocks' sums
        Seg8<T> sg;
        float wv[8], gv[8];
        sg.load(w + q.c);
        sg.get(wv);
        if (gate) {
          sg.load(gate + (size_t)seg * d + q.c);
          sg.get(gv);
        }
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = wv[e] * S[i][e];
        if (whole && gate) Seg8<float>::put(p.dgate + (size_t)seg * d + q.c, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = gate ? gv[e] * S[i][e] : S[i][e];
        if constexpr (MULTI) {
#pragma unroll
          for (int e = 0; e < 8; ++e) dwacc[i][e] += o[e];
        } else {
          Seg8<float>::put(p.dw + q.c, o);
        }
      }
    }
  }
  if constexpr (MULTI) {
    if (me == 0 && sums_here) {
      float* to = blocks == 1 ? p.dw : p.part + (size_t)blockIdx.x * d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const Cols q = cols<L>(lane, i, d);
        if (q.in) Seg8<float>::put(to + q.c, dwacc[i]);
      }
    }
  }
}

// Joins the row blocks' partials in a fixed order, 16 columns by 64 slices of the blocks per
// workgroup.  One gate row or none: dw = gate S and dgate = w S of the joined sum.  Several (MULTI):
// blockIdx.y = 0 joins dw; the others dgate, one gate row each where there are few gate rows
// (y = row + 1), else the gate row that the end of block y - 1 cuts, if that is its first cut.
template <typename T, bool MULTI>
__global__ __launch_bounds__(NT) void norm_bwd_join_kernel(const T* w, const T* gate, BwdArgs p, int blocks, bool by_row) {
  constexpr int SL = NT / 4;
  __shared__ float red[SL][16 + 1];
  const int d = p.d;
  const int c = blockIdx.x * 16 + (threadIdx.x % 4) * 4, slice = threadIdx.x / 4;
  int b0 = 0, b1 = blocks;   // blocks whose partials are added
  int seg = 0;
  long long seg_begin = 0;
  if (MULTI && blockIdx.y > 0) {
    seg = by_row ? blockIdx.y - 1 : (int)((long long)blockIdx.y * p.R - 1) / p.gate_rows;   // block y - 1's last row
    seg_begin = (long long)seg * p.gate_rows;
    const long long seg_last = min((long long)p.rows, seg_begin + p.gate_rows) - 1;
    b0 = (int)(seg_begin / p.R);
    b1 = (int)(seg_last / p.R) + 1;
    if (b1 - b0 < 2) return;                                 // inside one block: written there
    if (!by_row && b0 != (int)blockIdx.y - 1) return;        // an earlier cut handles it
  }
  float a[4] = {0, 0, 0, 0};
  if (c < d) {
    const bool dw = MULTI && blockIdx.y == 0;
#pragma unroll 4
    for (int b = b0 + slice; b < b1; b += SL) {
      const int kind = dw ? 0 : (seg_begin <= (long long)b * p.R ? 1 : 2);
      const float4 v = *reinterpret_cast<const float4*>(p.part + ((size_t)kind * blocks + b) * d + c);
      a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) red[slice][(threadIdx.x % 4) * 4 + e] = a[e];
  __syncthreads();
  // 16 threads per column add 4 slices each, then a tree
  const int col = threadIdx.x / 16, part = threadIdx.x % 16;
  float s = (red[part][col] + red[part + 16][col]) + (red[part + 32][col] + red[part + 48][col]);
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
  const int at = blockIdx.x * 16 + col;
  if (part != 0 || at >= d) return;
  if (MULTI && blockIdx.y == 0) {
    p.dw[at] = s;
  } else if (MULTI) {
    p.dgate[(size_t)seg * d + at] = to_f32<T>(w[at]) * s;
  } else {
    p.dw[at] = gate ? to_f32<T>(gate[at]) * s : s;
    if (gate) p.dgate[at] = to_f32<T>(w[at]) * s;
  }
}

__global__ __launch_bounds__(NT) void zero_f32_kernel(float* p, int n) {
  const int i = blockIdx.x * NT + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// Lanes per row and segments per lane for a width of d.  At most two segments a lane: with four the
// backward's registers spilled (fp32: 200 of them).
template <typename F>
hipError_t by_width(int d, F&& f) {
  if (d <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  if (d <= 1024) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (d <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  if (d <= 4096) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  if (d <= 8192) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

// One workgroup for each turn of rows, as far as a grid of 2^32 threads goes.
int fwd_blocks(int T, int rows) { return std::min(ceil_div(T, rows), 1 << 20); }

// Rows per workgroup of the backward: about BLOCKS workgroups, at least one row per wave or
// workgroup that walks rows.
constexpr int BLOCKS = 1024;
int bwd_rows(long long T, int d) {
  const int ns = d <= 1024 ? 4 : 1;
  const long long r = (T + BLOCKS - 1) / BLOCKS;
  return (int)std::max<long long>(ns, (r + ns - 1) / ns * ns);
}

// Few rows: column sums beside the rows instead of partials and their join.  Forward and backward, a
// call after the other (us): 61 rows x 2048 30.3 -> 26.3, 512 x 4096 32.7 -> 26.3, 1024 x 1024 29.7 ->
// 27.0; but 1024 x 4096 44.9 -> 46.4, 2048 x 1000 in fp32 29.7 -> 36.4, 200 x 16384 40.7 -> 46.8.  Gate
// rows are walked one after the other: 512 x 1000 with 4 of them 26.2 -> 23.9, 1000 x 1000 with 8 26.1 ->
// 33.2.
bool few_rows(long long T, int d) { return T <= 1024 && T * d <= 1 << 21; }

template <typename T, bool IN, bool MULTI>
hipError_t norm_bwd_rows(const T* dout, const T* y, const T* w, const T* gate, const T* dres, const float* rstd, T* dy,
                         BwdArgs p, hipStream_t s) {
  const int blocks = ceil_div(p.rows, p.R);
  const int gate_rows = MULTI ? ceil_div(p.rows, p.gate_rows) : 0;
  const int columns = blocks > 1 && gate_rows <= 4 && few_rows(p.rows, p.d) ? ceil_div(p.d, 16) : 0;
  p.row_blocks = blocks;
  hipError_t e = by_width(p.d, [&](auto L, auto NV) {
    constexpr int th = threads<decltype(L)::value>(), ns = th / decltype(L)::value;
    const size_t lds = (size_t)(ns - 1) * 8 * decltype(NV)::value * decltype(L)::value * sizeof(float);
    hipLaunchKernelGGL((norm_bwd_kernel<T, decltype(L)::value, decltype(NV)::value, IN, MULTI>), dim3(blocks + columns), dim3(th),
                       lds, s, dout, y, w, gate, dres, rstd, dy, p);
    return hipGetLastError();
  });
  if (e != hipSuccess || blocks == 1 || columns > 0) return e;
  const bool by_row = gate_rows < blocks;
  norm_bwd_join_kernel<T, MULTI><<<dim3(ceil_div(p.d, 16), 1 + (MULTI ? (by_row ? gate_rows : blocks - 1) : 0)), dim3(NT), 0,
                                   s>>>(w, gate, p, blocks, by_row);
  return hipGetLastError();
}

template <typename T, bool IN>
hipError_t norm_bwd(const T* dout, const T* y, const T* w, const T* gate, const T* dres, const float* rstd, T* dy,
                    BwdArgs p, hipStream_t s) {
  if (p.rows == 0) {
    zero_f32_kernel<<<dim3(ceil_div(p.d, NT)), dim3(NT), 0, s>>>(p.dw, p.d);
    return hipGetLastError();
  }
  p.R = bwd_rows(p.rows, p.d);
  if constexpr (!IN) {
    if (gate && p.gate_rows < p.rows) return norm_bwd_rows<T, IN, true>(dout, y, w, gate, dres, rstd, dy, p, s);
  }
  return norm_bwd_rows<T, IN, false>(dout, y, w, gate, dres, rstd, dy, p, s);
}

}  // namespace

hipError_t launch_norm_in(const void* x, const void* w, int T, int d, float eps, bool bf16, void* xn, float* rstd,
                          hipStream_t s) {
  auto go = [&](auto tag) {
    typedef decltype(tag) E;
    auto run = [&](auto L, auto NV) {
      hipLaunchKernelGGL((norm_in_kernel<E, decltype(L)::value, decltype(NV)::value>),
                         dim3(fwd_blocks(T, threads<decltype(L)::value>() / decltype(L)::value)),
                         dim3(threads<decltype(L)::value>()), 0, s, (const E*)x, (const E*)w, T, d, eps,
                         (E*)xn, rstd);
      return hipGetLastError();
    };
    // a wave per row as far as its registers go: 24.3 us against 27.6 at 16384 x 2048
    if (d > 1024 && d <= 2048) return run(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    return by_width(d, run);
  };
  return bf16 ? go(bf16_t{}) : go(float{});
}

hipError_t launch_norm_out(const void* y, const float* topk_gate, const int32_t* dest_pos, const void* shared, int k,
                           const void* x, const void* w, const void* gate, int gate_rows, float res_scale, float eps,
                           int T, int d, bool bf16, void* y_out, void* out, float* rstd, hipStream_t s) {
  auto go = [&](auto tag, auto comb) {
    typedef decltype(tag) E;
    return by_width(d, [&](auto L, auto NV) {
      hipLaunchKernelGGL((norm_out_kernel<E, decltype(L)::value, decltype(NV)::value, decltype(comb)::value>),
                         dim3(fwd_blocks(T, threads<decltype(L)::value>() / decltype(L)::value)),
                         dim3(threads<decltype(L)::value>()), 0, s, (const E*)y, topk_gate, dest_pos,
                         (const E*)shared, k, (const E*)x, (const E*)w, (const E*)gate, gate_rows, res_scale, T, d, eps,
                         (E*)y_out, (E*)out, rstd);
      return hipGetLastError();
    });
  };
  if (dest_pos) return bf16 ? go(bf16_t{}, std::true_type{}) : go(float{}, std::true_type{});
  return bf16 ? go(bf16_t{}, std::false_type{}) : go(float{}, std::false_type{});
}

size_t norm_bwd_ws_bytes(long long T, int d) {
  if (T <= 0) return 0;
  return (size_t)3 * ((T + bwd_rows(T, d) - 1) / bwd_rows(T, d)) * d * sizeof(float);
}

hipError_t launch_norm_in_bwd(const void* dxn, const void* x, const void* w, const float* rstd, const void* dres,
                              float res_scale, int T, int d, bool bf16, void* dx, float* dw, void* ws, hipStream_t s) {
  BwdArgs p{T, d, 0, 1, res_scale, (float*)ws, dw, nullptr};
  if (bf16)
    return norm_bwd<bf16_t, true>((const bf16_t*)dxn, (const bf16_t*)x, (const bf16_t*)w, nullptr, (const bf16_t*)dres,
                                  rstd, (bf16_t*)dx, p, s);
  return norm_bwd<float, true>((const float*)dxn, (const float*)x, (const float*)w, nullptr, (const float*)dres, rstd,
                               (float*)dx, p, s);
}

hipError_t launch_norm_out_bwd(const void* dout, const void* y, const void* w, const void* gate, int gate_rows,
                               const float* rstd, int T, int d, bool bf16, void* dy, float* dw, float* dgate, void* ws,
                               hipStream_t s) {
  BwdArgs p{T, d, 0, gate_rows, 0.0f, (float*)ws, dw, dgate};
  if (bf16)
    return norm_bwd<bf16_t, false>((const bf16_t*)dout, (const bf16_t*)y, (const bf16_t*)w, (const bf16_t*)gate, nullptr,
                                   rstd, (bf16_t*)dy, p, s);
  return norm_bwd<float, false>((const float*)dout, (const float*)y, (const float*)w, (const float*)gate, nullptr, rstd,
                                (float*)dy, p, s);
}

}  // namespace moe
