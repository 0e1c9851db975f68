// The products of the vocabulary loss (vocab_loss.hip has the formulas) in tiles of 64x64 or 128x128,
// both types: fp32, and bf16 where the 256x256 tiles of vocab_loss_pipe.hip fill the CUs badly.
//
// A workgroup of 4 waves takes one tile, RB x RB blocks of 32x32 per wave; two or four workgroups share
// a CU.  K goes through two LDS stages of 256 or 128 bytes per row and operand (64 bf16 or 32 fp32
// values in 128 bytes), filled by direct-to-LDS loads two steps ahead (four stages are no faster).  An
// operand contiguous along K is kept [64 rows][256 or 128 bytes], 16-byte chunks XOR-swizzled by the
// row; one contiguous along its rows is kept [k][64 rows] and read transposed (bf16) or value by value
// (fp32).  fp32 products run on v_mfma_f32_32x32x2_f32, which multiplies and adds in fp32; the two k of
// an instruction are 4 apart, so one 16-byte read feeds four of them.
// Rows past the end are read clamped and not stored, K and columns past the end read zeros.
//
// Large fp32 products run at 122-125 TFLOP/s in 128x128 tiles and 101-111 in 64x64 ones (a library
// product: 139), bound by the matrix cores.  A bf16 tile of 128x128 reads half as much LDS for each
// matrix instruction: 1500 tokens x 5000 words x d 3000 forward 64.5 us (700 TFLOP/s) against 126.  Few
// rows run at the rate of the words' stream: 7 tokens x 50021 words x d 2048 in 43 us (205 MB, 4.8
// TB/s).  Small products are bound by the latency of their few steps.
#include "vocab_loss.h"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace vocab {
namespace {

constexpr int TS = 64;                  // tile rows and columns of RB = 1
constexpr int NT = 256;
constexpr int JOIN_FEW = 32768;         // vectors of a join whose splits are dealt to 16 slices
// NF: fragment groups of a stage, 16 bf16 or 8 fp32 k each, so 32 NF bytes of a row.
constexpr int row_bytes(int nf) { return 32 * nf; }
constexpr int loads(int nf) { return nf / 2; }           // direct loads per wave, stage and operand
constexpr int op_bytes(int nf) { return 64 * row_bytes(nf); }

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) void gvoid_t;
typedef __attribute__((address_space(3))) void lvoid_t;

__device__ __attribute__((aligned(16))) uint4 g_zeros[4];

template <int MODE> struct Tr {
  static constexpr bool a_kc = MODE != VL_DW;
  static constexpr bool b_kc = MODE == VL_STATS || MODE == VL_GRAD;
};

__device__ __forceinline__ uint32_t lds_addr_of(const void* ptr) {
  return (uint32_t)(uintptr_t)((const __attribute__((address_space(3))) char*)ptr);
}

// Rows of 256 bytes: 16 rows read at one chunk hit 16 bank groups; of 128 bytes: two rows share one.
template <int NF>
__device__ __forceinline__ int swizzle(int row) {
  return NF == 8 ? row & 15 : (row >> 1) & 7;
}

// One operand's part of a stage: where each lane's loads read, and the LDS layout.  ONCE: the operand
// is read by this tile alone (nontemporal loads).
template <typename T, bool KC, int NF, bool ONCE>
struct Operand {
  static constexpr int ROWB = row_bytes(NF), LP = loads(NF);
  static constexpr int E = 16 / sizeof(T), BK = ROWB / sizeof(T);
  static constexpr int CPR = KC ? ROWB / 16 : 64 / E;   // 16-byte chunks of an LDS row
  const char* src[LP];
  int k[LP];       // first k of the lane's piece, from the tile's first
  bool in[LP];     // columns inside (not KC)

  __device__ __forceinline__ static int logical(int row, int chunk) {
    if constexpr (KC) return chunk ^ swizzle<NF>(row);
    else if constexpr (E == 8) return chunk ^ (((row >> 1) & 1) << 2);
    else return chunk ^ (((row >> 2) & 1) << 3);
  }
  // base: element (row 0, k 0) of the operand; r0, k0: the tile's first row and k.
  __device__ __forceinline__ void init(const T* base, size_t ld, int r0, int rows, int k0, int wave, int lane) {
#pragma unroll
    for (int j = 0; j < LP; ++j) {
      const int q = (wave * LP + j) * 64 + lane;
      const int row = q / CPR, c = logical(row, q % CPR) * E;
      if constexpr (KC) {
        src[j] = reinterpret_cast<const char*>(base + (size_t)min(r0 + row, rows - 1) * ld + k0 + c);
        k[j] = c;
        in[j] = true;
      } else {
        in[j] = r0 + c < rows;
        src[j] = reinterpret_cast<const char*>(base + (size_t)(k0 + row) * ld + (in[j] ? r0 + c : 0));
        k[j] = row;
      }
    }
  }
  // The stage whose first k is `at`, of k_end in the tile; then the sources move one stage on.
  __device__ __forceinline__ void issue(char* lds, int at, int k_end, size_t ld, int wave) {
#pragma unroll
    for (int j = 0; j < LP; ++j) {
      const char* from = in[j] && at + k[j] < k_end ? src[j] : reinterpret_cast<const char*>(g_zeros);
      __builtin_amdgcn_global_load_lds((gvoid_t*)from, (lvoid_t*)(lds + (wave * LP + j) * 1024), 16, 0, ONCE ? 2 : 0);
      src[j] += KC ? (size_t)ROWB : (size_t)BK * ld * sizeof(T);
    }
  }
};

// A wave's fragments of a stage.  Group s, lane l: row l % 32 of the block and, bf16: k 16 s + 8 (l / 32)
// + 0..7; fp32: k 8 s + 4 (l / 32) + 0..3.
template <typename T, bool KC, int NF>
struct Frags {
  static constexpr int E = 16 / sizeof(T), ROWB = row_bytes(NF);
  u32x4_t v[NF];
  u32x2_t h[NF][2];   // bf16, not KC: two transposed reads of 4 k

  __device__ __forceinline__ void read(uint32_t base, int rb, int lane) {
    if constexpr (KC) {
      const int row = rb + (lane & 31);
      const uint32_t a = base + row * ROWB + (((lane >> 5) ^ swizzle<NF>(row)) << 4);
#pragma unroll
      for (int s = 0; s < NF; ++s) asm volatile("ds_read_b128 %0, %1" : "=v"(v[s]) : "v"(a ^ (uint32_t)(32 * s)));
    } else if constexpr (E == 8) {
      const int b = lane >> 4, c = (lane & 15) >> 2, k = (b >> 1) * 8 + c, col = rb + 16 * (b & 1) + 4 * (lane & 3);
      const uint32_t a = base + k * 128 + (((col >> 3) ^ (((k >> 1) & 1) << 2)) << 4) + (col & 7) * 2;
#pragma unroll
      for (int s = 0; s < NF; ++s) {
        asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(h[s][0]) : "v"(a), "i"(2048 * s));
        asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(h[s][1]) : "v"(a), "i"(2048 * s + 512));
      }
    } else {
      const int col = rb + (lane & 31), half = lane >> 5;
      const uint32_t a = base + half * 1024 + (((col >> 2) ^ (half << 3)) << 4) + (col & 3) * 4;
#pragma unroll
      for (int s = 0; s < NF; ++s) {
        uint32_t x0, x1, x2, x3;
        asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(x0) : "v"(a), "i"(2048 * s));
        asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(x1) : "v"(a), "i"(2048 * s + 256));
        asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(x2) : "v"(a), "i"(2048 * s + 512));
        asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(x3) : "v"(a), "i"(2048 * s + 768));
        f[s][0] = x0; f[s][1] = x1; f[s][2] = x2; f[s][3] = x3;
      }
    }
  }
  uint32_t f[NF][4];   // fp32, not KC

  // After a wait: the values are in-out operands here, so no use of them moves above it.
  __device__ __forceinline__ void landed() {
#pragma unroll
    for (int s = 0; s < NF; ++s) {
      if constexpr (KC) asm volatile("" : "+v"(v[s]));
      else if constexpr (E == 8) asm volatile("" : "+v"(h[s][0]), "+v"(h[s][1]));
      else asm volatile("" : "+v"(f[s][0]), "+v"(f[s][1]), "+v"(f[s][2]), "+v"(f[s][3]));
    }
  }
  __device__ __forceinline__ bf16x8_t get16(int s) const {
    if constexpr (KC) return __builtin_bit_cast(bf16x8_t, v[s]);
    const u32x4_t u = {h[s][0].x, h[s][0].y, h[s][1].x, h[s][1].y};
    return __builtin_bit_cast(bf16x8_t, u);
  }
  __device__ __forceinline__ float get32(int s, int e) const {
    return __uint_as_float(KC ? v[s][e] : f[s][e]);
  }
};

constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | 0xf70; }   // vmcnt alone
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(N));
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

__device__ __forceinline__ void store4(bf16_t* p, const float (&v)[4]) {
  u32x2_t w;
  w.x = (uint32_t)f32_to_bf16(v[0]) | ((uint32_t)f32_to_bf16(v[1]) << 16);
  w.y = (uint32_t)f32_to_bf16(v[2]) | ((uint32_t)f32_to_bf16(v[3]) << 16);
  *reinterpret_cast<u32x2_t*>(p) = w;
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// How a product is cut: splits of K, K per split, whether the tiles store the result itself (else
// partial products, which a join adds up).
struct Cut {
  int ks, kchunk;
  bool direct;
};

// The largest finite |dloss| of a row with a loss, 1 if there is none, for at most SCALE_ROWS rows.
__device__ __forceinline__ float scale_of_rows(const VocabArgs& p) {
  __shared__ float red[NT / 64];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < SCALE_ROWS / NT; ++i) {
    const int t = threadIdx.x + i * NT;
    if (t < p.T) m = fmaxf(m, dloss_size(p, t));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  return m > 0.0f ? m : 1.0f;
}

// One tile.  Workgroup `block` of the product runs on XCD block % 8: each XCD walks one run of the tile
// order, rows first, so the tiles that read one panel of the large operand run together.
template <typename T, int MODE, int NF, bool ONCE, int RB>
__device__ __forceinline__ void run_tile(const VocabArgs& p, const Cut& cut, int block, char* lds) {
  constexpr bool AK = Tr<MODE>::a_kc, BKC = Tr<MODE>::b_kc;
  constexpr int BK = row_bytes(NF) / sizeof(T), LP = loads(NF), OPB = op_bytes(NF), STAGE = 2 * RB * OPB;
  constexpr int TR = TS * RB;   // the tile's rows and columns
  const int ks = cut.ks, kchunk = cut.kchunk;
  const bool direct = cut.direct;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave >> 1, wn = wave & 1;
  constexpr bool LOGITS = MODE == VL_STATS || MODE == VL_GRAD;
  const int M = MODE == VL_DW ? p.vn : p.T;
  const int N = LOGITS ? p.vn : p.d;
  const int K = LOGITS ? p.d : (MODE == VL_DH ? p.vn : p.T);
  const T* h = reinterpret_cast<const T*>(p.h);
  const T* w = reinterpret_cast<const T*>(p.w) + (size_t)p.v0 * p.d;
  const T* P = reinterpret_cast<const T*>(p.p);
  const T* abase = LOGITS ? h : P;
  const T* bbase = MODE == VL_DW ? h : w;
  const size_t lda = LOGITS ? p.d : p.ldp, ldb = p.d;

  const int MT = (M + TR - 1) / TR, NTL = (N + TR - 1) / TR, total = MT * NTL * ks;
  const int per = (total + 7) >> 3;
  const int L = (block & 7) * per + (block >> 3);
  if ((block >> 3) >= per || L >= total) return;
  const int split = L / (MT * NTL), l = L - split * (MT * NTL);
  const int nt = l / MT, mt = l - nt * MT;
  const int m0 = mt * TR, n0 = nt * TR;
  const int k0 = split * kchunk, k_end = min(K - k0, kchunk);
  const int nk = (k_end + BK - 1) / BK;

  // An operand is RB blocks of 64 rows; a wave reads one of them whole (RB = 2) or half of it.
  Operand<T, AK, NF, false> oa[RB];
  Operand<T, BKC, NF, ONCE> ob[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    oa[b].init(abase, lda, m0 + TS * b, M, k0, wave, lane);
    ob[b].init(bbase, ldb, n0 + TS * b, N, k0, wave, lane);
  }
  auto issue = [&](char* slot, int at) {
#pragma unroll
    for (int b = 0; b < RB; ++b) oa[b].issue(slot + b * OPB, at, k_end, lda, wave);
#pragma unroll
    for (int b = 0; b < RB; ++b) ob[b].issue(slot + (RB + b) * OPB, at, k_end, ldb, wave);
  };
  // Past the last stage the loads read zeros into slots that nobody reads.
#pragma unroll
  for (int s = 0; s < 2; ++s) issue(lds + s * STAGE, s * BK);
  f32x16_t acc[RB][RB];
#pragma unroll
  for (int a = 0; a < RB; ++a)
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.0f;
  const uint32_t lds0 = lds_addr_of(lds);
  for (int j = 0; j < nk; ++j) {
    char* slot = lds + (j & 1) * STAGE;
    const uint32_t sb = lds0 + (j & 1) * STAGE;
    wait_vm<2 * LP * RB>();   // stage j has landed, stage j + 1 may be in flight
    barrier();
    Frags<T, AK, NF> fa[RB];
    Frags<T, BKC, NF> fb[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      fa[b].read(sb + (RB == 1 ? 0 : wm * OPB), RB == 1 ? wm * 32 : b * 32, lane);
      fb[b].read(sb + (RB == 1 ? OPB : (RB + wn) * OPB), RB == 1 ? wn * 32 : b * 32, lane);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      fa[b].landed();
      fb[b].landed();
    }
    barrier();           // every wave has read stage j
    issue(slot, (j + 2) * BK);
#pragma unroll
    for (int s = 0; s < NF; ++s) {
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int a = 0; a < RB; ++a)
#pragma unroll
          for (int b = 0; b < RB; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[b].get16(s), fa[a].get16(s), acc[a][b], 0, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int a = 0; a < RB; ++a)
#pragma unroll
            for (int b = 0; b < RB; ++b)
              acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[b].get32(s, e), fa[a].get32(s, e), acc[a][b], 0, 0, 0);
      }
    }
  }
  wait_vm<0>();   // no direct load may still be writing when the workgroup's LDS is released

  // Lane l holds row l % 32 of a block and, in element e, column 8 (e / 4) + 4 (l / 32) + e % 4.
  const int half = lane >> 5;
  float scale = 1.0f;
  if constexpr (MODE == VL_GRAD) {
    if (p.scale_out) {   // few rows: every tile finds the scale itself, one writes it for the kernels after
      scale = scale_of_rows(p);
      if (L == 0 && threadIdx.x == 0) *p.scale_out = scale;
    } else {
      scale = *p.scale;
    }
  }
  const float out_scale = (MODE == VL_DH || MODE == VL_DW) && direct ? *p.scale : 1.0f;   // else the join scales
#pragma unroll
  for (int a = 0; a < RB; ++a) {
    const int row = m0 + wm * 32 * RB + a * 32 + (lane & 31);
    float lse = 0.0f, dl = 0.0f;
    int tgt = -1;
    if constexpr (MODE == VL_GRAD) {
      if (row < M) {
        lse = p.lse[row];
        tgt = p.target[row];
        dl = tgt >= 0 && tgt < p.V ? p.dloss[row] / scale : 0.0f;
        tgt -= p.v0;
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int c0 = n0 + wn * 32 * RB + b * 32;
      f32x16_t& x = acc[a][b];
      if constexpr (MODE == VL_STATS) {
        if (c0 >= N) continue;
        float mx = -__builtin_inff();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (c0 + 8 * (e >> 2) + 4 * half + (e & 3) >= N) x[e] = -__builtin_inff();
          mx = fmaxf(mx, x[e]);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        // of an infinite maximum: words that are all -inf add nothing, one of +inf makes the sum infinite
        const float m = fabsf(mx) < __builtin_inff() ? mx : 0.0f;
        float sm = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) sm += expf(x[e] - m);
        sm += __shfl_xor(sm, 32, 64);
        if (half == 0 && row < M) p.part[(size_t)((p.v0 + c0) / TILE_PART) * p.T + row] = make_float2(mx, sm);
        continue;
      }
      if (row >= M) continue;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = c0 + 8 * g + 4 * half;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = x[4 * g + e] * out_scale;
        if constexpr (MODE == VL_GRAD) {   // columns up to the tile's end, inside P's row of a multiple of 256
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float q = expf(v[e] - lse) - (n + e == tgt ? 1.0f : 0.0f);
            v[e] = dl == 0.0f || n + e >= N ? 0.0f : dl * q;
          }
          store4(reinterpret_cast<T*>(p.p) + (size_t)row * p.ldp + n, v);
        } else if (n < N) {   // N = d, a multiple of 8
          if constexpr (MODE == VL_DH) {
            if (direct) {
              store4(reinterpret_cast<T*>(p.dh) + (size_t)row * p.d + n, v);
            } else {   // dh: partial product `split` of the pieces so far
              float* to = p.dh_acc + ((size_t)split * p.T + row) * p.d + n;
              if (!p.first) {
                const float4 o = *reinterpret_cast<const float4*>(to);
                v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
              }
              store4(to, v);
            }
          } else if (direct) {
            store4(reinterpret_cast<T*>(p.dw) + (size_t)(p.v0 + row) * p.d + n, v);
          } else {
            store4(p.dw_acc + ((size_t)split * M + row) * p.d + n, v);
          }
        }
      }
    }
  }
}

template <typename T, int MODE, int NF, bool ONCE, int RB>
__global__ __launch_bounds__(NT, NF * RB == 8 ? 2 : 4) void vocab_tile_kernel(VocabArgs p, Cut cut) {
  __shared__ __attribute__((aligned(1024))) char lds[4 * RB * op_bytes(NF)];
  run_tile<T, MODE, NF, ONCE, RB>(p, cut, blockIdx.x, lds);
}

// dh's and dw's products side by side: neither needs the other, and of few rows and words neither
// fills the CUs alone (257 x 256 against 1000 words in fp32: 10 us together, 10 us each apart).
template <typename T, int RB>
__global__ __launch_bounds__(NT, RB == 2 ? 2 : 4) void vocab_tile_pair_kernel(VocabArgs p, Cut dh, Cut dw, int dh_blocks) {
  __shared__ __attribute__((aligned(1024))) char lds[4 * RB * op_bytes(4)];
  if ((int)blockIdx.x < dh_blocks) run_tile<T, VL_DH, 4, false, RB>(p, dh, blockIdx.x, lds);
  else run_tile<T, VL_DW, 4, false, RB>(p, dw, blockIdx.x - dh_blocks, lds);
}

// out = the scaled sum of ks partial products of n elements in a fixed order, rounded; two such sums in
// one launch (n = 0: none).
template <typename T>
struct Join {
  const float* parts;
  T* out;
  size_t n;   // a multiple of 8
  int ks;
};
// SL slices of the splits are summed side by side, then joined in order: 16 where the outputs are few
// and the splits many, whose loads then overlap (forward and backward, us): 1 x 100000 words x d 128,
// 256 splits, 68.6 -> 57.4; 6 x 18673 x 376 41.0 -> 36.7; 100 x 60000 x 256 63.7 -> 61.1.
template <typename T, int SL>
__global__ __launch_bounds__(NT) void vocab_tile_join_kernel(Join<T> a, Join<T> b, const float* scale) {
  constexpr int VPB = NT / SL;   // vectors of 4 of a workgroup at a time
  __shared__ float4 red[SL > 1 ? SL - 1 : 1][VPB];
  const int slice = threadIdx.x / VPB, x = threadIdx.x % VPB;
  const size_t vectors = (a.n + b.n) / 4;
  for (size_t v0 = (size_t)blockIdx.x * VPB; v0 < vectors; v0 += (size_t)gridDim.x * VPB) {
    const size_t i = (v0 + x) * 4;
    const bool in = v0 + x < vectors;
    const Join<T>& j = i < a.n ? a : b;
    const size_t at = i < a.n ? i : i - a.n;
    float v[4] = {0, 0, 0, 0};
    if (in) {
      const int per = SL == 1 ? j.ks : (j.ks + SL - 1) / SL, s1 = min(j.ks, (slice + 1) * per);
#pragma unroll 4
      for (int s = slice * per; s < s1; ++s) {
        const float4 o = *reinterpret_cast<const float4*>(j.parts + s * j.n + at);
        v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
      }
    }
    if constexpr (SL > 1) {
      if (slice > 0) red[slice - 1][x] = make_float4(v[0], v[1], v[2], v[3]);
      __syncthreads();
      if (slice == 0) {
#pragma unroll
        for (int s = 0; s < SL - 1; ++s) {
          const float4 o = red[s][x];
          v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
        }
      }
      __syncthreads();
    }
    if (in && slice == 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= *scale;
      store4(j.out + at, v);
    }
  }
}
template <typename T>
hipError_t launch_join(const Join<T>& a, const Join<T>& b, const float* scale, hipStream_t s) {
  if (a.n + b.n == 0) return hipSuccess;
  auto run = [&](auto kernel, int vpb) {
    kernel<<<dim3((unsigned)std::min<size_t>(((a.n + b.n) / 4 + vpb - 1) / vpb, 1 << 20)), dim3(NT), 0, s>>>(a, b, scale);
    return hipGetLastError();
  };
  if ((a.n + b.n) / 4 <= JOIN_FEW && std::max(a.n ? a.ks : 0, b.n ? b.ks : 0) >= 16) return run(vocab_tile_join_kernel<T, 16>, NT / 16);
  return run(vocab_tile_join_kernel<T, 1>, NT);
}

// K per split of dh or dw, a multiple of a stage; dh's is the same for every piece of a call.
template <typename T>
int split_chunk(int M, int N, int K, bool large) {
  constexpr int BK = 256 / sizeof(T);
  return ceil_div(ceil_div(K, tile_splits(M, N, K, large)), BK) * BK;
}

template <typename T>
Cut cut_of(int mode, const VocabArgs& p) {
  Cut c{1, p.d, true};
  if (mode == VL_DH) {
    c.kchunk = split_chunk<T>(p.T, p.d, p.ldp, p.large);
    c.ks = ceil_div(p.vn, c.kchunk);
    c.direct = c.ks == 1 && p.first && p.last;   // dh of several pieces is accumulated in fp32
  } else if (mode == VL_DW) {
    c.kchunk = split_chunk<T>(p.vn, p.d, p.T, p.large);
    c.ks = ceil_div(p.T, c.kchunk);
    c.direct = c.ks == 1;
  }
  return c;
}

// Workgroups of a product, a multiple of the XCDs.
unsigned blocks_of(int mode, const VocabArgs& p, const Cut& c) {
  const int M = mode == VL_DW ? p.vn : p.T, N = mode == VL_DW || mode == VL_DH ? p.d : p.vn;
  return (unsigned)((tile_count(M, N, p.large) * c.ks + 7) / 8 * 8);
}

template <typename T>
Join<T> join_dw(const VocabArgs& p, const Cut& c) {
  return Join<T>{p.dw_acc, reinterpret_cast<T*>(p.dw) + (size_t)p.v0 * p.d, c.direct ? 0 : (size_t)p.vn * p.d, c.ks};
}
// The sum over all pieces: the first one, the widest, used every split.
template <typename T>
Join<T> join_dh(const VocabArgs& p) {
  const int wide = std::min(p.V, p.ldp), ks = ceil_div(wide, split_chunk<T>(p.T, p.d, p.ldp, p.large));
  return Join<T>{p.dh_acc, reinterpret_cast<T*>(p.dh), ks == 1 && p.V <= p.ldp ? 0 : (size_t)p.T * p.d, ks};
}

template <typename T, int MODE>
hipError_t launch(const VocabArgs& p, hipStream_t s) {
  const Cut c = cut_of<T>(MODE, p);
  const dim3 grid(blocks_of(MODE, p, c));
  // 256 bytes of each word's row at a time where a single row tile reads the words once (bound by that
  // stream), 128 otherwise (four workgroups per CU): 64 tokens x 12485 words x d 3472 forward 26.6 us
  // against 33.3, 500 x 4000 x 2048 21.3 against 19.7.
  // That stream is nontemporal in the forward where it would displace most of the last-level cache:
  // 7 tokens against 205 MB of words 45.5 us instead of 52.5; 87 MB, which the backward then finds in
  // the cache, would take 12 us longer there.
  constexpr bool LOGITS = MODE == VL_STATS || MODE == VL_GRAD;
  auto run = [&](auto nf, auto once, auto rb) {
    hipLaunchKernelGGL((vocab_tile_kernel<T, MODE, decltype(nf)::value, decltype(once)::value, decltype(rb)::value>), grid,
                       dim3(NT), 0, s, p, c);
  };
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 4> Short;
  typedef std::integral_constant<int, LOGITS ? 8 : 4> Stream;
  typedef std::integral_constant<bool, MODE == VL_STATS> Once;
  if (LOGITS && p.T <= TS && (size_t)p.vn * p.d * sizeof(T) >= size_t(128) << 20) run(Stream{}, Once{}, One{});
  else if (LOGITS && p.T <= TS) run(Stream{}, std::false_type{}, One{});
  else if (p.large) run(Short{}, std::false_type{}, std::integral_constant<int, 2>{});
  else run(Short{}, std::false_type{}, One{});
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || MODE != VL_DW) return e;
  return launch_join(join_dw<T>(p, c), Join<T>{}, p.scale, s);
}

// dh or dw alone: bf16, where the other one takes the 256x256 tiles.
template <typename T>
hipError_t launch_mode(int mode, const VocabArgs& p, hipStream_t s) {
  if (mode == VL_STATS) return launch<T, VL_STATS>(p, s);
  if (mode == VL_GRAD) return launch<T, VL_GRAD>(p, s);
  if constexpr (sizeof(T) == 2) {
    if (mode == VL_DH) return launch<T, VL_DH>(p, s);
    if (mode == VL_DW) return launch<T, VL_DW>(p, s);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_both(const VocabArgs& p, hipStream_t s) {
  const Cut dh = cut_of<T>(VL_DH, p), dw = cut_of<T>(VL_DW, p);
  const unsigned nh = blocks_of(VL_DH, p, dh), nw = blocks_of(VL_DW, p, dw);
  auto kernel = p.large ? vocab_tile_pair_kernel<T, 2> : vocab_tile_pair_kernel<T, 1>;
  hipLaunchKernelGGL(kernel, dim3(nh + nw), dim3(NT), 0, s, p, dh, dw, (int)nh);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_join(join_dw<T>(p, dw), p.last ? join_dh<T>(p) : Join<T>{}, p.scale, s);
}

}  // namespace

long long tile_count(int M, int N, bool large) {
  const int ts = large ? 2 * TS : TS;
  return (long long)ceil_div(M, ts) * ceil_div(N, ts);
}

// Splits of the K of an M x N product: as many as fill two workgroups per CU, at least 256 k each.
int tile_splits(int M, int N, int K, bool large) {
  return (int)std::max<long long>(1, std::min<long long>(2 * NUM_CUS / tile_count(M, N, large), K / 256));
}

size_t tile_acc_bytes(int M, int N, int K, bool large) { return (size_t)tile_splits(M, N, K, large) * M * N * sizeof(float); }

int tile_ks(int mode, const VocabArgs& p, bool bf16) {
  return bf16 ? cut_of<bf16_t>(mode, p).ks : cut_of<float>(mode, p).ks;
}

hipError_t launch_tile(int mode, const VocabArgs& p, bool bf16, hipStream_t s) {
  return bf16 ? launch_mode<bf16_t>(mode, p, s) : launch_mode<float>(mode, p, s);
}

hipError_t launch_tile_pair(const VocabArgs& p, bool bf16, hipStream_t s) {
  return bf16 ? launch_both<bf16_t>(p, s) : launch_both<float>(p, s);
}

hipError_t launch_tile_join(const VocabArgs& p, hipStream_t s) {
  return launch_join(join_dh<bf16_t>(p), Join<bf16_t>{}, p.scale, s);
}

}  // namespace vocab
}  // namespace moe
