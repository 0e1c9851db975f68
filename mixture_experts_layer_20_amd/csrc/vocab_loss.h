// Shared by the two kernels of the vocabulary loss.
#pragma once

#include "block_step.h"

namespace moe {
namespace vocab {

struct VocabArgs {
  const void* h;
  const void* w;
  const int32_t* target;
  const float* lse;
  const float* dloss;
  int T, d, V;
  int v0, vn;         // the piece: words v0 .. v0 + vn - 1
  int ldp;            // row length of P, a multiple of 256
  const float* scale; // [1] the largest |dloss|: P is kept relative to it
  float* scale_out;   // the same place where VL_GRAD's tiles are to find it (at most SCALE_ROWS rows), or NULL
  void* p;            // [T, ldp]; columns vn.. of a piece are zero as far as its last tile reaches
  float2* part;       // [parts][T] maximum and sum of exponentials of PIPE_PART or TILE_PART words
  float* dh_acc;      // dh of the pieces so far, fp32
  float* dw_acc;      // partial products of a piece's dw, fp32
  void* dh;
  void* dw;
  bool first, last;   // the piece is the first / the last one
  bool large;         // launch_tile, launch_tile_pair, launch_tile_join: 128x128 tiles
};

enum VocabMode { VL_STATS = 0, VL_GRAD = 1, VL_DH = 2, VL_DW = 3 };

constexpr int PIPE_PART = 64, TILE_PART = 32;   // words of a row's part, by the kernel that writes it
constexpr int NUM_CUS = 256;
constexpr int SCALE_ROWS = 1024;

// |dloss| of row t for the scale: 0 where the row has no loss or its gradient is not finite.
__device__ __forceinline__ float dloss_size(const VocabArgs& p, int t) {
  const int v = p.target[t];
  const float a = fabsf(p.dloss[t]);
  return v >= 0 && v < p.V && a <= 3.4028234664e38f ? a : 0.0f;
}

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// The pipelined bf16 kernel (256x256 tiles).  dh_acc and dw_acc hold the accumulator tiles of the
// splits' partial products in the kernel's own order; VL_DW joins its own, launch_pipe_join dh's.
int pipe_dh_splits(int T, int d, int words);
int pipe_dw_splits(int T, int d, int words);
size_t pipe_dh_bytes(int T, int d, int words);
size_t pipe_dw_bytes(int T, int d, int words);
int pipe_ks(int mode, const VocabArgs& p);   // partial products that a launch sums K in
hipError_t launch_pipe(int mode, const VocabArgs& p, hipStream_t s);
hipError_t launch_pipe_join(const VocabArgs& p, hipStream_t s);

// 64x64 or (p.large) 128x128 tiles, both types.  dh_acc and dw_acc hold tile_splits() partial products
// of all outputs.
long long tile_count(int M, int N, bool large);
int tile_splits(int M, int N, int K, bool large);
size_t tile_acc_bytes(int M, int N, int K, bool large);
int tile_ks(int mode, const VocabArgs& p, bool bf16);
hipError_t launch_tile(int mode, const VocabArgs& p, bool bf16, hipStream_t s);   // VL_DH, VL_DW: bf16
// VL_DH and VL_DW in one launch, and the joins that they need (dh's after the last piece).
hipError_t launch_tile_pair(const VocabArgs& p, bool bf16, hipStream_t s);
hipError_t launch_tile_join(const VocabArgs& p, hipStream_t s);   // dh's, of a bf16 VL_DH launched alone

}  // namespace vocab
}  // namespace moe
