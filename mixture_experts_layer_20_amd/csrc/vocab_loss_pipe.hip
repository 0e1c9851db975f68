// Pipelined bf16 products of the vocabulary loss for gfx950, 256x256 tiles, with the loss's
// epilogues (vocab_loss.hip has the formulas):
//   VL_STATS  l = h w^T of all words -> maximum and sum of exponentials of each row's 64-word groups
//   VL_GRAD   l of the piece's words again -> P = dloss / s (exp(l - lse) - [word = target]), bf16
//   VL_DH     P w: accumulated over the pieces in fp32
//   VL_DW     P^T h: the piece's rows of dw
//
// One workgroup per CU, 8 waves in a 2x4 grid, 128x64 per wave (4x2 blocks of
// v_mfma_f32_32x32x16_bf16), K in steps of 64 through two 64 KiB LDS stages that direct-to-LDS loads
// fill two steps ahead, across tile boundaries.  An operand that is contiguous along K is kept
// [row][64 k] (128-byte rows, 16-byte chunks XOR-swizzled) and read with ds_read_b128; one that is
// contiguous along its rows is kept [64 k][256 rows] and read transposed with ds_read_b64_tr_b16.  A
// K step is four phases of 8 MFMAs; every fragment read and every load is placed between two MFMAs.
// The same scheme as the grouped GEMM's, for one dense product of any size: rows past the end are
// read clamped and dropped at the store, K and columns past the end read a page of zeros.
//
// Bound by the matrix cores, whose rate the board's power limits: the 8192 x 4096 x 65536 logits of
// normal data take 3.38 ms (1300 TFLOP/s, the matrix cores busy for 74%), of all-zero data 2.61 ms; a
// library product of the same operands, which writes the logits instead of reading them off, takes
// 3.04 and 2.32 ms.  Of the 3.38 ms some 0.10 are outside the K loop.  P, dh and dw of a piece of 8192
// words: 0.446, 0.451 and 0.424 ms (1230, 1220 and 1300 TFLOP/s).  At 1031 x 1000 x 50021 a fifth of
// the tiles' rows is empty and the four products take 133-169 us each (610-780 TFLOP/s).
#include "vocab_loss.h"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace vocab {
namespace {

constexpr int BM = 256, BN = 256, BKS = 64;
constexpr int NW = 8, NTH = 64 * NW, WGN = 4;
constexpr int MI = 4, NI = 2;           // 32x32 blocks of a wave
constexpr int LP = 4;                   // direct loads (1 KiB) per wave, stage and operand
constexpr int OPB = 256 * BKS * 2;      // one operand's part of a stage
constexpr int STAGE = 2 * OPB;
constexpr int BAND = 4;                 // row tiles walked together (2, 8, 16 and 32 are no faster)
constexpr float LOG2E = 1.44269504088896340736f;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) void gvoid_t;
typedef __attribute__((address_space(3))) void lvoid_t;

__device__ __attribute__((aligned(16))) uint4 g_zeros[64];

constexpr int VL_DW_SPLIT = 4;   // VL_DW with its K split: partial products to the workspace

template <int MODE> struct Tr {
  static constexpr bool a_kc = MODE != VL_DW && MODE != VL_DW_SPLIT;
  static constexpr bool b_kc = MODE == VL_STATS || MODE == VL_GRAD;
};

__device__ __forceinline__ uint32_t lds_addr_of(const void* ptr) {
  return (uint32_t)(uintptr_t)((const __attribute__((address_space(3))) char*)ptr);
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <typename T>
__device__ __forceinline__ T* uniform_ptr(T* ptr) {
  const uint64_t v = (uint64_t)(uintptr_t)ptr;
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return (T*)(uintptr_t)((hi << 32) | lo);
}

// ---- Geometry ------------------------------------------------------------------------------
// The product C[m, n] = sum_k A(m, k) B(n, k) of a mode, its tiles and its split of K.
struct Geo {
  const char* a;
  const char* b;
  int lda, ldb;        // row lengths of the stored operands, elements
  int M, N, K;
  int MT, NT, ks, kchunk, total;
};

struct Tile {
  int m0, n0, k0, k1, nk, slab;   // slab: the tile's number over all splits (VL_DH accumulators)
  bool half;                       // at most 128 rows: the second row half of waves issues loads only
};

template <int MODE>
__device__ __forceinline__ Geo geometry(const VocabArgs& p, int ks, int kchunk) {
  Geo g;
  const char* w = reinterpret_cast<const char*>(p.w) + (size_t)p.v0 * p.d * 2;
  const char* h = reinterpret_cast<const char*>(p.h);
  const char* P = reinterpret_cast<const char*>(p.p);
  if constexpr (MODE == VL_STATS || MODE == VL_GRAD) {
    g.a = h; g.lda = p.d; g.b = w; g.ldb = p.d; g.M = p.T; g.N = p.vn; g.K = p.d;
  } else if constexpr (MODE == VL_DH) {
    g.a = P; g.lda = p.ldp; g.b = w; g.ldb = p.d; g.M = p.T; g.N = p.d; g.K = p.vn;
  } else {
    g.a = P; g.lda = p.ldp; g.b = h; g.ldb = p.d; g.M = p.vn; g.N = p.d; g.K = p.T;
  }
  g.MT = (g.M + BM - 1) / BM;
  g.NT = (g.N + BN - 1) / BN;
  g.ks = ks;
  g.kchunk = kchunk;
  g.total = g.MT * g.NT * ks;
  return g;
}

// Tile order: split by split; inside a split bands of BAND row tiles, column by column, so the 32
// workgroups of an XCD read 4 row panels and 8 column panels at a time.
__device__ __forceinline__ Tile decode(const Geo& g, int L) {
  Tile t;
  const int per = g.MT * g.NT;
  const int split = L / per;
  const int l = L - split * per;
  const int b = l / (BAND * g.NT);
  const int mb = min(BAND, g.MT - b * BAND);
  const int r = l - b * BAND * g.NT;
  const int nt = r / mb, mt = b * BAND + (r - nt * mb);
  t.m0 = mt * BM;
  t.n0 = nt * BN;
  t.k0 = split * g.kchunk;
  t.k1 = min(g.K, t.k0 + g.kchunk);
  t.nk = (t.k1 - t.k0 + BKS - 1) / BKS;
  t.slab = (split * g.MT + mt) * g.NT + nt;
  t.half = g.M - t.m0 <= BM / 2;
  return t;
}

// ---- Loads ---------------------------------------------------------------------------------
// Load j (0..3) of wave w fills the 1 KiB slot 4 w + j of its operand.  KC: rows 8 (4 w + j) + lane / 8,
// chunk lane % 8 of the 128-byte row holding the logical chunk (lane % 8) ^ swizzle(row).  MC: k rows
// 2 (4 w + j) + lane / 32, 16-byte chunk lane % 32 of the 512-byte row holding the logical chunk
// (lane % 32) ^ 4 (k % 4).
__device__ __forceinline__ int kc_swz(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int kc_col(int j, int lane) { return ((lane & 7) ^ (4 * (j & 1) + (lane >> 4))) * 8; }
__device__ __forceinline__ int mc_krow(int j, int wave, int lane) { return 2 * (LP * wave + j) + (lane >> 5); }
__device__ __forceinline__ int mc_col(int j, int lane) { return ((lane & 31) ^ ((2 * (j & 1) + (lane >> 5)) << 2)) * 8; }

struct Offs {
  uint32_t a[LP], b[LP];   // byte offsets from the stage's bases
};

struct Source {
  const char* sa;
  const char* sb;
  int k_left;      // K elements from the stage's start to the tile's end
  bool edge;       // columns past the end (operands contiguous along their rows)
};

struct Producer {
  Tile t;
  int i, k;        // tile list position, K step
  Offs o;
  Source s;
};

template <bool KC>
__device__ __forceinline__ void operand_offsets(uint32_t (&o)[LP], int ld, int rows_left, int wave, int lane) {
#pragma unroll
  for (int j = 0; j < LP; ++j) {
    if constexpr (KC) {
      const int row = min(8 * (LP * wave + j) + (lane >> 3), rows_left - 1);
      o[j] = ((uint32_t)row * (uint32_t)ld + (uint32_t)kc_col(j, lane)) * 2u;
    } else {
      o[j] = ((uint32_t)mc_krow(j, wave, lane) * (uint32_t)ld + (uint32_t)mc_col(j, lane)) * 2u;
    }
  }
}

template <int MODE>
__device__ __forceinline__ void set_tile(Producer& pr, const Geo& g, const Tile& t, int i, int wave, int lane) {
  pr.t = t;
  pr.i = i;
  pr.k = 0;
  operand_offsets<Tr<MODE>::a_kc>(pr.o.a, g.lda, g.M - t.m0, wave, lane);
  operand_offsets<Tr<MODE>::b_kc>(pr.o.b, g.ldb, g.N - t.n0, wave, lane);
  const size_t ao = Tr<MODE>::a_kc ? (size_t)t.m0 * g.lda + t.k0 : (size_t)t.k0 * g.lda + t.m0;
  const size_t bo = Tr<MODE>::b_kc ? (size_t)t.n0 * g.ldb + t.k0 : (size_t)t.k0 * g.ldb + t.n0;
  pr.s.sa = uniform_ptr(g.a + ao * 2);
  pr.s.sb = uniform_ptr(g.b + bo * 2);
  pr.s.k_left = t.k1 - t.k0;
  pr.s.edge = (!Tr<MODE>::a_kc && g.M - t.m0 < BM) || (!Tr<MODE>::b_kc && g.N - t.n0 < BN);
}

// The stream's position in scalar registers: the compiler does not always see that it is the same in
// every lane, and would then keep it per lane and branch on masks.
__device__ __forceinline__ void scalar(Producer& pr, int& j) {
  pr.k = uniform(pr.k);
  pr.i = uniform(pr.i);
  pr.t.nk = uniform(pr.t.nk);
  pr.s.k_left = uniform(pr.s.k_left);
  pr.s.sa = uniform_ptr(pr.s.sa);
  pr.s.sb = uniform_ptr(pr.s.sb);
  j = uniform(j);
}

// The next stage of the stream; past the last one it stays there (valid memory, into slots that
// nobody reads again).
template <int MODE>
__device__ __forceinline__ void advance(Producer& pr, const Geo& g, int hi, int step, int wave, int lane) {
  if (pr.k + 1 < pr.t.nk) {
    ++pr.k;
    pr.s.sa += Tr<MODE>::a_kc ? (size_t)BKS * 2 : (size_t)BKS * 2 * g.lda;
    pr.s.sb += Tr<MODE>::b_kc ? (size_t)BKS * 2 : (size_t)BKS * 2 * g.ldb;
    pr.s.k_left -= BKS;
  } else if (pr.i + step < hi) {
    set_tile<MODE>(pr, g, decode(g, pr.i + step), pr.i + step, wave, lane);
  }
}

// EXACT: every tile and K step of the product is whole, so no piece needs a check.
template <int MODE, bool EXACT, int IDX>
__device__ __forceinline__ void issue(char* stage, const Producer& pr, const Geo& g, int wave, int lane) {
  constexpr bool A_OP = IDX < LP;
  constexpr int J = IDX % LP;
  constexpr bool KC = A_OP ? Tr<MODE>::a_kc : Tr<MODE>::b_kc;
  lvoid_t* to = (lvoid_t*)(stage + (A_OP ? 0 : OPB) + (LP * wave + J) * 1024);
  const char* src = (A_OP ? pr.s.sa : pr.s.sb) + (A_OP ? pr.o.a[J] : pr.o.b[J]);
  if (!EXACT && (pr.s.edge || pr.s.k_left < BKS)) {   // the same in every lane
    bool in;
    if constexpr (KC) in = kc_col(J, lane) < pr.s.k_left;
    else in = mc_krow(J, wave, lane) < pr.s.k_left && mc_col(J, lane) < (A_OP ? g.M - pr.t.m0 : g.N - pr.t.n0);
    const char* from = in ? src : reinterpret_cast<const char*>(g_zeros);
    __builtin_amdgcn_global_load_lds((gvoid_t*)from, to, 16, 0, 0);
  } else {
    __builtin_amdgcn_global_load_lds((gvoid_t*)src, to, 16, 0, 0);
  }
}

template <int MODE, bool EXACT, int IDX>
__device__ __forceinline__ void issue_all(char* stage, const Producer& pr, const Geo& g, int wave, int lane) {
  if constexpr (IDX < 2 * LP) {
    issue<MODE, EXACT, IDX>(stage, pr, g, wave, lane);
    issue_all<MODE, EXACT, IDX + 1>(stage, pr, g, wave, lane);
  }
}

// ---- Fragments -----------------------------------------------------------------------------
template <bool KC, int NB> struct Frag;
template <int NB> struct Frag<true, NB> {
  static constexpr int READS = NB;
  bf16x8_t v[NB];
  template <int R>
  __device__ __forceinline__ void read_one(uint32_t addr) {
    asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v[R]) : "v"(addr), "i"(4096 * R));
  }
  __device__ __forceinline__ bf16x8_t get(int i) const { return v[i]; }
  __device__ __forceinline__ void landed() {
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(v[i]));
  }
};
template <int NB> struct Frag<false, NB> {
  static constexpr int READS = 2 * NB;
  u32x2_t h[2][NB];
  template <int R>
  __device__ __forceinline__ void read_one(uint32_t addr) {
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(h[R & 1][R >> 1]) : "v"(addr ^ (uint32_t)((R >> 1) << 6)), "i"((R & 1) * 2048));
  }
  __device__ __forceinline__ bf16x8_t get(int i) const {
    const u32x4_t u = {h[0][i].x, h[0][i].y, h[1][i].x, h[1][i].y};
    return __builtin_bit_cast(bf16x8_t, u);
  }
  __device__ __forceinline__ void landed() {
#pragma unroll
    for (int i = 0; i < NB; ++i) asm volatile("" : "+v"(h[0][i]), "+v"(h[1][i]));
  }
};
template <int MODE> using FragA = Frag<Tr<MODE>::a_kc, MI>;
template <int MODE> using FragB = Frag<Tr<MODE>::b_kc, NI>;

template <int MODE>
__device__ __forceinline__ void frag_wait(FragA<MODE>& a, FragB<MODE>& b) {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  a.landed();
  b.landed();
}

// LDS address of a lane's first fragment read, block row rb, substep 0 (substep s: sub_addr).  The
// transposed read takes 16-lane groups: group b covers columns rb + 16 (b & 1) + [0, 16) of k rows
// 8 (b >> 1) + [0, 8), lane 4 c + q of it pointing at k row c, columns 4 q.
template <bool KC>
__device__ __forceinline__ uint32_t frag_base(uint32_t base, int rb, int lane) {
  if constexpr (KC) {
    const int row = rb + (lane & 31);
    return base + row * 128 + (((lane >> 5) ^ kc_swz(row)) << 4);
  } else {
    const int b = lane >> 4, j = lane & 15, c = j >> 2, q = j & 3;
    const int k = (b >> 1) * 8 + c;
    const int col = rb + 16 * (b & 1) + 4 * q;
    return base + k * 512 + (((col >> 3) ^ ((k & 3) << 2)) << 4) + (col & 7) * 2;
  }
}
template <bool KC, int S>
__device__ __forceinline__ uint32_t sub_addr(uint32_t base, uint32_t sb) {
  if constexpr (KC) return (base + sb) ^ (uint32_t)(32 * S);
  else return base + sb + (uint32_t)(8192 * S);
}

// ---- K step --------------------------------------------------------------------------------
constexpr int SLOTS = MI * NI;

template <int MODE, int R>
__device__ __forceinline__ void read_slot(FragA<MODE>& a, FragB<MODE>& b, uint32_t ra, uint32_t rb) {
  if constexpr (R < FragA<MODE>::READS) a.template read_one<R>(ra);
  else if constexpr (R < FragA<MODE>::READS + FragB<MODE>::READS) b.template read_one<R - FragA<MODE>::READS>(rb);
}
template <int MODE, int R>
__device__ __forceinline__ void read_all(FragA<MODE>& a, FragB<MODE>& b, uint32_t ra, uint32_t rb) {
  if constexpr (R < FragA<MODE>::READS + FragB<MODE>::READS) {
    read_slot<MODE, R>(a, b, ra, rb);
    read_all<MODE, R + 1>(a, b, ra, rb);
  }
}

// One phase: the MFMAs of the current substep, between them the fragment reads of the next one and
// (LOADS) the loads of the stage two steps ahead.  ACT = false: a wave without rows, loads only.
template <int MODE, bool EXACT, bool ACT, bool LOADS, int Q>
__device__ __forceinline__ void phase(f32x16_t (&acc)[MI][NI], const FragA<MODE>& ac, const FragB<MODE>& bc,
                                      FragA<MODE>& an, FragB<MODE>& bn, uint32_t ra, uint32_t rb, char* stage,
                                      const Producer& pr, const Geo& g, int wave, int lane) {
  if constexpr (Q < SLOTS) {
    if constexpr (ACT) {
      constexpr int i = Q / NI, j = Q % NI;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bc.get(j), ac.get(i), acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      read_slot<MODE, Q>(an, bn, ra, rb);
      read_slot<MODE, Q + SLOTS>(an, bn, ra, rb);
    }
    if constexpr (LOADS) issue<MODE, EXACT, Q>(stage, pr, g, wave, lane);
    __builtin_amdgcn_sched_barrier(0);
    phase<MODE, EXACT, ACT, LOADS, Q + 1>(acc, ac, bc, an, bn, ra, rb, stage, pr, g, wave, lane);
  }
}

constexpr int waitcnt_vm(int n) { return (n & 15) | ((n >> 4) << 14) | 0x70; }
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(N));
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

// Stores that every epilogue issues at least, after the last stage loads before it.
template <int MODE>
constexpr int epilogue_stores() { return MODE == VL_STATS ? 0 : 16; }

template <int MODE, bool EXACT, bool ACT>
__device__ __forceinline__ void kstep(f32x16_t (&acc)[MI][NI], uint32_t fa, uint32_t fb, FragA<MODE>& a0,
                                      FragB<MODE>& b0, FragA<MODE>& a1, FragB<MODE>& b1, int j, bool after_epilogue,
                                      Producer& pr, const Geo& g, int hi, int step, int wave, int lane, char* lds) {
  constexpr bool AK = Tr<MODE>::a_kc, BK = Tr<MODE>::b_kc;
  const uint32_t sb = (j & 1) * STAGE, sn = ((j + 1) & 1) * STAGE;
  phase<MODE, EXACT, ACT, false, 0>(acc, a0, b0, a1, b1, sub_addr<AK, 1>(fa, sb), sub_addr<BK, 1>(fb, sb), nullptr, pr, g, wave, lane);
  if constexpr (ACT) frag_wait<MODE>(a1, b1);
  phase<MODE, EXACT, ACT, false, 0>(acc, a1, b1, a0, b0, sub_addr<AK, 2>(fa, sb), sub_addr<BK, 2>(fb, sb), nullptr, pr, g, wave, lane);
  if constexpr (ACT) frag_wait<MODE>(a0, b0);
  phase<MODE, EXACT, ACT, false, 0>(acc, a0, b0, a1, b1, sub_addr<AK, 3>(fa, sb), sub_addr<BK, 3>(fb, sb), nullptr, pr, g, wave, lane);
  if constexpr (ACT) frag_wait<MODE>(a1, b1);
  // Stage j + 1 has landed (the first step after an epilogue: only that epilogue's stores may still
  // be out, which were issued after the stage's loads), and every wave is done with slot j & 1.
  if (after_epilogue) wait_vm<epilogue_stores<MODE>()>();
  else wait_vm<0>();
  barrier();
  phase<MODE, EXACT, ACT, true, 0>(acc, a1, b1, a0, b0, sub_addr<AK, 0>(fa, sn), sub_addr<BK, 0>(fb, sn), lds + sb, pr, g, wave, lane);
  advance<MODE>(pr, g, hi, step, wave, lane);
  if constexpr (ACT) frag_wait<MODE>(a0, b0);
}

// ---- Epilogues -----------------------------------------------------------------------------
// An accumulator block is the transpose of the output block: lane l holds output row l % 32 and, in
// element e, column 8 (e / 4) + 4 (l / 32) + e % 4.
__device__ __forceinline__ int block_col(int e, int lane) { return 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3); }

__device__ __forceinline__ float other_half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Maximum and sum of exponentials of the wave's 64 columns, per row.
__device__ __forceinline__ void stats_epilogue(const VocabArgs& p, const Geo& g, f32x16_t (&acc)[MI][NI], int row0,
                                               int col0, int lane) {
  if (col0 >= g.N) return;
  if (g.N - col0 < 64) {         // words past the end
    asm volatile("");
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (col0 + 32 * j + block_col(e, lane) >= g.N) acc[i][j][e] = -__builtin_inff();
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    float mx = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        mx = fmaxf(mx, acc[i][j][e]);
      }
    mx = other_half_max(mx);
    // of an infinite maximum: words that are all -inf add nothing, one of +inf makes the sum infinite
    float m2 = mx * LOG2E;
    if (!(fabsf(m2) < __builtin_inff())) m2 = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) s += __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], LOG2E, -m2));
    s = other_half_sum(s);
    const int row = row0 + 32 * i + (lane & 31);
    if (lane < 32 && row < g.M) p.part[(size_t)((p.v0 + col0) / PIPE_PART) * p.T + row] = make_float2(mx, s);
  }
}

struct OutWin {
  __amdgpu_buffer_rsrc_t r;
  uint32_t row_bytes;
  int cols;   // columns of the window inside the output
};
// Rows past the window's are dropped by the buffer's size; pieces of 8 columns past `cols` by an
// offset beyond any size.
__device__ __forceinline__ OutWin out_win(void* base, size_t elem, int rows, int ld, int cols) {
  OutWin w;
  w.row_bytes = (uint32_t)uniform(ld * 2);
  w.cols = cols;
  char* b = uniform_ptr(reinterpret_cast<char*>(base) + elem * 2);
  w.r = __builtin_amdgcn_make_buffer_rsrc(b, 0, uniform(max(rows, 0) * (int)w.row_bytes), 0x00020000);
  return w;
}

__device__ __forceinline__ u32x4_t pack8(const float (&x)[8]) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 b16x2_t __attribute__((ext_vector_type(2)));
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2_t v = {x[2 * i], x[2 * i + 1]};
    w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b16x2_t));
  }
  return w;
}

// Half H of a block as 8 consecutive columns 16 H + 8 (l / 32) + 0..7 of row l % 32.
__device__ __forceinline__ void block_half(const f32x16_t& c, int h, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(c[8 * h + e]), __float_as_uint(c[8 * h + 4 + e]), false, false);
    x[e] = __uint_as_float(r[0]);
    x[4 + e] = __uint_as_float(r[1]);
  }
}
__device__ __forceinline__ void swap16(const u32x4_t& a, const u32x4_t& b, u32x4_t& r0, u32x4_t& r1) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto r = __builtin_amdgcn_permlane16_swap(a[e], b[e], false, false);
    r0[e] = r[0];
    r1[e] = r[1];
  }
}

// Two neighbouring blocks as whole 128-byte rows: after swap16 each block has rows 0..15 and 16..31
// (lane l: row l % 16, 16 bytes at column 16 (l / 16 % 2) + 8 (l / 32)); a rotation by 8 lanes of
// block 1's pieces and a select on lane bit 3 pair the blocks into rows 0..7 and 8..15.
template <bool NT>
__device__ __forceinline__ void st_rows128(const OutWin& w, int br, const float (&x0)[2][8], const float (&x1)[2][8],
                                           int lane) {
  constexpr int AUX = NT ? 2 : 0;
  u32x4_t a[2], c[2];
  swap16(pack8(x0[0]), pack8(x0[1]), a[0], a[1]);
  swap16(pack8(x1[0]), pack8(x1[1]), c[0], c[1]);
  const bool hi8 = (lane & 8) != 0;
  const int cx = 16 * ((lane >> 4) & 1) + 8 * (lane >> 5);
  const int ca = cx + (hi8 ? 32 : 0), cb = cx + (hi8 ? 0 : 32);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    u32x4_t A, B;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t t = (uint32_t)__builtin_amdgcn_mov_dpp((int)c[q][e], 0x128, 0xf, 0xf, false);
      A[e] = hi8 ? t : a[q][e];
      B[e] = hi8 ? a[q][e] : t;
    }
    const int r = br + (lane & 7) + 16 * q;
    const int oa = ca < w.cols ? (int)(r * w.row_bytes) + ca * 2 : 0x7ffffff0;
    const int ob = cb < w.cols ? (int)((r + 8) * w.row_bytes) + cb * 2 : 0x7ffffff0;
    __builtin_amdgcn_raw_buffer_store_b128(A, w.r, oa, 0, AUX);
    __builtin_amdgcn_raw_buffer_store_b128(B, w.r, ob, 0, AUX);
  }
}
template <int I, bool NT>
__device__ __forceinline__ void store_rows(const OutWin& w, const f32x16_t (&acc)[MI][NI], int lane) {
  if constexpr (I < MI) {
    float v0[2][8], v1[2][8];
    block_half(acc[I][0], 0, v0[0]);
    block_half(acc[I][0], 1, v0[1]);
    block_half(acc[I][1], 0, v1[0]);
    block_half(acc[I][1], 1, v1[1]);
    st_rows128<NT>(w, 32 * I, v0, v1, lane);
    store_rows<I + 1, NT>(w, acc, lane);
  }
}

// Logits to P, in place.  A row without loss has lse = +inf and dl = 0: exactly zero.
__device__ __forceinline__ void grad_epilogue(const VocabArgs& p, const Geo& g, f32x16_t (&acc)[MI][NI], int row0,
                                              int col0, int lane) {
  const float scale = *p.scale;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int row = row0 + 32 * i + (lane & 31);
    int tgt = -1;
    float l2 = __builtin_inff(), dl = 0.0f;
    if (row < g.M) {
      tgt = p.target[row];
      if (tgt >= 0 && tgt < p.V) {
        dl = p.dloss[row] / scale;
        l2 = dl == 0.0f ? l2 : p.lse[row] * LOG2E;
      }
    }
    const int tc = tgt - p.v0 - col0;   // the target's column in the wave's 64
    const bool mine = dl != 0.0f && tc >= 0 && tc < 64;
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = dl * __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], LOG2E, -l2));
    if (__ballot(mine) != 0) {   // one wave in eight has a target at 128 rows x 64 of 65536 words
      asm volatile("");          // a branch, not 32 selects for everybody
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (mine && 32 * j + block_col(e, lane) == tc) acc[i][j][e] -= dl;
        }
    }
  }
  if (g.N - col0 < 64) {         // words past the piece's end
    asm volatile("");
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (col0 + 32 * j + block_col(e, lane) >= g.N) acc[i][j][e] = 0.0f;
  }
}

// The wave's accumulators in the workspace: 128 x 64 floats, one KiB per store of 4 elements.
__device__ __forceinline__ f32x4_t* acc_slab(float* acc, const Tile& t, int wave) {
  return reinterpret_cast<f32x4_t*>(acc) + ((size_t)t.slab * NW + wave) * (MI * NI * 4 * 64);
}
__device__ __forceinline__ void store_slab(f32x4_t* to, const f32x16_t (&acc)[MI][NI]) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        to[((i * NI + j) * 4 + q) * 64] = f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
}

template <int MODE>
__device__ __forceinline__ void epilogue(const VocabArgs& p, const Geo& g, f32x16_t (&acc)[MI][NI], const Tile& t,
                                         int wm, int wn, int wave, int lane) {
  const int row0 = t.m0 + wm * 32 * MI, col0 = t.n0 + wn * 32 * NI;
  const int rows = min(32 * MI, g.M - row0);
  if constexpr (MODE == VL_STATS) {
    stats_epilogue(p, g, acc, row0, col0, lane);
  } else if constexpr (MODE == VL_GRAD) {
    grad_epilogue(p, g, acc, row0, col0, lane);
    store_rows<0, false>(out_win(p.p, (size_t)row0 * p.ldp + col0, rows, p.ldp, 64), acc, lane);
  } else if constexpr (MODE == VL_DH) {
    store_slab(acc_slab(p.dh_acc, t, wave) + lane, acc);
  } else if constexpr (MODE == VL_DW_SPLIT) {
    store_slab(acc_slab(p.dw_acc, t, wave) + lane, acc);
  } else {
    const float scale = *p.scale;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] *= scale;
    store_rows<0, true>(out_win(p.dw, ((size_t)p.v0 + row0) * p.d + col0, rows, p.d, g.N - col0), acc, lane);
  }
}

template <int MODE, bool EXACT, bool ACT>
__device__ __forceinline__ void run_tile(const VocabArgs& p, const Geo& g, const Tile& t, uint32_t fa, uint32_t fb,
                                         FragA<MODE>& a0, FragB<MODE>& b0, FragA<MODE>& a1, FragB<MODE>& b1, int& j,
                                         bool& after_epilogue, Producer& pr, int hi, int step, int wm, int wn, int wave,
                                         int lane, char* lds) {
  f32x16_t acc[MI][NI];
  if (MODE == VL_DH && !p.first) {
    const f32x4_t* from = acc_slab(p.dh_acc, t, wave) + lane;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int jj = 0; jj < NI; ++jj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4_t v = from[((i * NI + jj) * 4 + q) * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][jj][4 * q + e] = v[e];
        }
  } else {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int jj = 0; jj < NI; ++jj)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][jj][e] = 0.0f;
  }
  for (int k = 0; k < t.nk; ++k, ++j) {
    scalar(pr, j);
    kstep<MODE, EXACT, ACT>(acc, fa, fb, a0, b0, a1, b1, j, after_epilogue, pr, g, hi, step, wave, lane, lds);
    after_epilogue = false;
  }
  // per-lane addressing of the epilogue is computed here, not kept in registers through the K loop
  asm volatile("v_mov_b32 %0, %0" : "+v"(lane));
  epilogue<MODE>(p, g, acc, t, wm, wn, wave, lane);
  after_epilogue = true;
}

template <int MODE, bool EXACT>
__global__ __launch_bounds__(NTH, 1) void vocab_pipe_kernel(VocabArgs p, int ks, int kchunk) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave / WGN, wn = wave % WGN;
  const Geo g = geometry<MODE>(p, ks, kchunk);
  const uint32_t lds0 = lds_addr_of(lds);
  const uint32_t fa = frag_base<Tr<MODE>::a_kc>(lds0, wm * 32 * MI, lane);
  const uint32_t fb = frag_base<Tr<MODE>::b_kc>(lds0 + OPB, wn * 32 * NI, lane);

  // Workgroup b runs on XCD b % 8: each XCD walks one run of the tile order.
  const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
  const int per = (g.total + 7) >> 3;
  const int hi = min(g.total, (xcd + 1) * per);
  int i = xcd * per + (blockIdx.x >> 3);
  if (i >= hi) return;

  Producer pr;
  set_tile<MODE>(pr, g, decode(g, i), i, wave, lane);
  Tile t = pr.t;
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    issue_all<MODE, EXACT, 0>(lds + s * STAGE, pr, g, wave, lane);
    advance<MODE>(pr, g, hi, step, wave, lane);
  }
  wait_vm<2 * LP>();   // the first stage has landed
  barrier();
  FragA<MODE> a0, a1;
  FragB<MODE> b0, b1;
  int j = 0;
  bool after_epilogue = false;
  for (;;) {
    if (t.half && wm == 1) {
      run_tile<MODE, EXACT, false>(p, g, t, fa, fb, a0, b0, a1, b1, j, after_epilogue, pr, hi, step, wm, wn, wave, lane, lds);
    } else {
      const uint32_t sb = (j & 1) * STAGE;
      read_all<MODE, 0>(a0, b0, sub_addr<Tr<MODE>::a_kc, 0>(fa, sb), sub_addr<Tr<MODE>::b_kc, 0>(fb, sb));
      frag_wait<MODE>(a0, b0);
      run_tile<MODE, EXACT, true>(p, g, t, fa, fb, a0, b0, a1, b1, j, after_epilogue, pr, hi, step, wm, wn, wave, lane, lds);
    }
    i += step;
    if (i >= hi) break;
    t = decode(g, i);
  }
  wait_vm<0>();   // no direct load may still be writing when the workgroup's LDS is released
}

// out [M, N] = the scaled sum of the splits' accumulators, rounded.  A thread takes 4 columns of a row.
__global__ __launch_bounds__(256) void vocab_join_kernel(const float* acc, bf16_t* out, int M, int N, int ks, const float* scale) {
  const int MT = (M + BM - 1) / BM, NT = (N + BN - 1) / BN;
  const int per = MI * NI * 4 * 64;   // vectors of a wave
  const size_t slabs = (size_t)MT * NT * NW * per;
  for (size_t at = (size_t)blockIdx.x * 256 + threadIdx.x; at < slabs; at += (size_t)gridDim.x * 256) {
    const int lane = at % 64, q = at / 64 % 4, blk = at / 256 % (MI * NI), wave = at / per % NW;
    const int tile = (int)(at / ((size_t)per * NW));
    const int row = tile / NT * BM + wave / WGN * 32 * MI + blk / NI * 32 + (lane & 31);
    const int col = tile % NT * BN + wave % WGN * 32 * NI + blk % NI * 32 + 8 * q + 4 * (lane >> 5);
    if (row >= M || col >= N) continue;
    const f32x4_t* from = reinterpret_cast<const f32x4_t*>(acc) + at;
    f32x4_t s = from[0];
    for (int k = 1; k < ks; ++k) s += from[(size_t)k * slabs];
    s *= *scale;
    u32x2_t w;
    w.x = (uint32_t)f32_to_bf16(s[0]) | ((uint32_t)f32_to_bf16(s[1]) << 16);
    w.y = (uint32_t)f32_to_bf16(s[2]) | ((uint32_t)f32_to_bf16(s[3]) << 16);
    *reinterpret_cast<u32x2_t*>(out + (size_t)row * N + col) = w;
  }
}
hipError_t launch_join(const float* acc, bf16_t* out, int M, int N, int ks, const float* scale, hipStream_t s) {
  const size_t vectors = (size_t)ceil_div(M, BM) * ceil_div(N, BN) * (BM * BN / 4);
  hipLaunchKernelGGL(vocab_join_kernel, dim3((unsigned)std::min<size_t>(vectors / 256, 1 << 20)), dim3(256), 0, s, acc, out, M, N, ks, scale);
  return hipGetLastError();
}

// K per split of dh or dw: a multiple of the K step; dh's is the same for every piece of a call.
int split_chunk(int K, int splits) { return ceil_div(ceil_div(K, splits), BKS) * BKS; }

template <int MODE>
hipError_t launch(const VocabArgs& p, int M, int N, int K, int kchunk, hipStream_t s) {
  const int ks = ceil_div(K, kchunk);
  const long long total = (long long)ceil_div(M, BM) * ceil_div(N, BN) * ks;
  const int grid = (int)std::min<long long>((total + 7) / 8 * 8, NUM_CUS);
  const bool exact = K % BKS == 0 && (MODE == VL_STATS || MODE == VL_GRAD || (N % BN == 0 && (MODE == VL_DH || M % BM == 0)));
  if (exact) hipLaunchKernelGGL((vocab_pipe_kernel<MODE, true>), dim3(grid), dim3(NTH), 0, s, p, ks, kchunk);
  else hipLaunchKernelGGL((vocab_pipe_kernel<MODE, false>), dim3(grid), dim3(NTH), 0, s, p, ks, kchunk);
  return hipGetLastError();
}

}  // namespace

namespace {
// As many splits as the CUs hold beside the output tiles, at least least_k k each.
int splits(int M, int N, int K, int least_k) {
  const long long tiles = (long long)ceil_div(M, BM) * ceil_div(N, BN);
  return (int)std::max<long long>(1, std::min<long long>(NUM_CUS / tiles, K / least_k));
}
size_t acc_bytes(int M, int N, int ks) { return (size_t)ks * ceil_div(M, BM) * ceil_div(N, BN) * BM * BN * sizeof(float); }
}  // namespace

// dh passes through fp32 memory anyway (it is accumulated over the pieces); dw only where its sum is
// split, which pays from some 1500 rows per split on: 5000 rows x d 400 x 40000 words, forward and
// backward, 1220 -> 1036 us; 2048 x 1024 x 8000 split in two 176 -> 182.
int pipe_dh_splits(int T, int d, int words) { return splits(T, d, words, 512); }
int pipe_dw_splits(int T, int d, int words) { return splits(words, d, T, 1536); }
size_t pipe_dh_bytes(int T, int d, int words) { return acc_bytes(T, d, pipe_dh_splits(T, d, words)); }
size_t pipe_dw_bytes(int T, int d, int words) {
  const int ks = pipe_dw_splits(T, d, words);
  return ks > 1 ? acc_bytes(words, d, ks) : 0;
}

// K of a product, and K per split of it.
static int pipe_k(int mode, const VocabArgs& p) { return mode == VL_DH ? p.vn : mode == VL_DW ? p.T : p.d; }
static int pipe_chunk(int mode, const VocabArgs& p) {
  if (mode == VL_DH) return split_chunk(p.ldp, pipe_dh_splits(p.T, p.d, p.ldp));
  return mode == VL_DW ? split_chunk(p.T, pipe_dw_splits(p.T, p.d, p.vn)) : p.d;
}
int pipe_ks(int mode, const VocabArgs& p) { return ceil_div(pipe_k(mode, p), pipe_chunk(mode, p)); }

hipError_t launch_pipe(int mode, const VocabArgs& p, hipStream_t s) {
  const int kchunk = pipe_chunk(mode, p), ks = pipe_ks(mode, p);
  switch (mode) {
    case VL_STATS: return launch<VL_STATS>(p, p.T, p.vn, p.d, kchunk, s);
    case VL_GRAD: return launch<VL_GRAD>(p, p.T, p.vn, p.d, kchunk, s);
    case VL_DH: return launch<VL_DH>(p, p.T, p.d, p.vn, kchunk, s);
    case VL_DW: {
      if (ks == 1) return launch<VL_DW>(p, p.vn, p.d, p.T, kchunk, s);
      const hipError_t e = launch<VL_DW_SPLIT>(p, p.vn, p.d, p.T, kchunk, s);
      if (e != hipSuccess) return e;
      return launch_join(p.dw_acc, reinterpret_cast<bf16_t*>(p.dw) + (size_t)p.v0 * p.d, p.vn, p.d, ks, p.scale, s);
    }
  }
  return hipErrorInvalidValue;
}

hipError_t launch_pipe_join(const VocabArgs& p, hipStream_t s) {
  VocabArgs first = p;   // the first piece, the widest, used every split
  first.vn = std::min(p.V, p.ldp);
  return launch_join(p.dh_acc, reinterpret_cast<bf16_t*>(p.dh), p.T, p.d, pipe_ks(VL_DH, first), p.scale, s);
}

}  // namespace vocab
}  // namespace moe
