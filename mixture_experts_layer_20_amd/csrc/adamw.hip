// AdamW over a list of tensors, with the gradients' clipping in the same pass.
//
//   g = c grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = (1 - lr wd) p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// (Loshchilov and Hutter's decoupled weight decay), c the clipping coefficient of moe_grad_scale, all of it
// fp32.  The states m and v are fp32, or 8 bits: E4M3 codes of m and of sqrt(v) with one float scale for 128
// elements, the block's largest magnitude / 448.  The root brings v's range into E4M3's: half the exponents.
// A state that moves by a fraction of a code's step (beta2 = 0.999 moves v by a thousandth, a step is up to
// an eighth) would stay where it is if it were rounded to nearest; so the rounding is random, up with the
// probability of the rest.  A positive v keeps at least the smallest code: m over a v that was rounded to
// zero would be a step of m / eps.  A bf16 parameter without a master copy is rounded in the same way.  The
// random bits are a hash of the element's run of 8 and the tensor's seed, and a linear congruential sequence
// (Knuth's and Lewis's) inside the run: the same call gives the same bits.  What keeps its mean in each rounding is
// the root; v's is then larger by the rounding's variance, which over many steps comes to 3 to 6% of it (a quarter
// to a third of spread, beta2 0.95 to 0.999): it stays there, since a root that hardly moves is near its code.
//
// Bound by memory: one pass, nothing read or written twice, parameters that have a master copy not read.
// 409 M bf16 parameters out of place: fp32 states and master copies, 28 bytes each, 2069 to 2117 us (11.5 GB, 5.4 to
// 5.5 TB/s), 8-bit states 713 to 733 us (4.1 GB, 5.6 to 5.8 TB/s), against 5.2 TB/s of a device copy; what the 8-bit
// form computes, about 430 vector instructions for 8 elements of a wave, would take 0.6 ms by itself.  128
// elements (a block) lie in 16 lanes, whose largest value is found with row rotations in registers.
#include "train_step.h"

#include "lanes.h"

#include <algorithm>
#include <memory>
#include <new>
#include <type_traits>

#pragma clang fp contract(off)

namespace moe {
namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int NT = 256;
constexpr int RUN = 8;              // elements that share a hash
constexpr int BLOCK = 128;          // elements that share a scale: 16 lanes
constexpr float TOP = 448.0f;       // the largest E4M3 value
constexpr float LEAST = 0x1p-9f;    // the smallest positive one
constexpr float TINY = 0x1p-100f;   // a block whose largest magnitude is below is stored as zeros

__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h ^= h >> 16;
  h *= 0x9D2B4F35u;
  h ^= h >> 15;
  h *= 0xC5A1E6B7u;
  return h ^ (h >> 16);
}

// sqrt(v), v >= 0, from the reciprocal root with one correction, nearly always rounded to nearest; the
// hardware's own, which is within a unit in the last place, would decide four times as many of the stored
// roots' roundings differently from the exact value.  (Of 200 M stored codes 131 of v and 250 of m differ from those
// of the formulas in 64 bits, the same ones with a root rounded to nearest, which takes 790 us for 733; in plain fp32
// operations it is 158 and 319.)  NaN for infinity.  Below 2^-126, the squares of gradients below 2^-63, the root comes
// out small.
__device__ __forceinline__ float root_of(float v) {
  const float q = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-126f));
  const float r = v * q;
  return __builtin_fmaf(__builtin_fmaf(-r, r, v), 0.5f * q, r);
}

// Loads of N elements (4 or 8) from element `at` of a chunk on.  FULL: all of them exist, 16-byte pieces (8 for 4
// bf16); otherwise `last` is the chunk's last element, which stands in for those behind it: every load is
// in range and none is under a condition, so that all of them are in flight together.
template <bool FULL, int N>
__device__ __forceinline__ void load_n(const float* p, uint32_t at, uint32_t last, float (&x)[N]) {
  if (FULL) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const u32x4_t a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + at) + q);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * q + e] = __uint_as_float(a[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = p[min(at + e, last)];
  }
}
template <bool FULL, int N>
__device__ __forceinline__ void load_n(const bf16_t* p, uint32_t at, uint32_t last, float (&x)[N]) {
  typedef uint32_t piece_t __attribute__((ext_vector_type(N / 2)));
  if (FULL) {
    const piece_t a = __builtin_nontemporal_load(reinterpret_cast<const piece_t*>(p + at));
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      x[2 * e] = __uint_as_float(a[e] << 16);
      x[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = bf16_to_f32(p[min(at + e, last)]);
  }
}
template <bool FULL>
__device__ __forceinline__ u32x2_t load8_codes(const uint8_t* p, uint32_t at, uint32_t last) {
  if (FULL) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p + at));
  uint32_t x[RUN];
#pragma unroll
  for (int e = 0; e < RUN; ++e) x[e] = p[min(at + e, last)];
  u32x2_t a;
#pragma unroll
  for (int q = 0; q < 2; ++q) a[q] = x[4 * q] | (x[4 * q + 1] << 8) | (x[4 * q + 2] << 16) | (x[4 * q + 3] << 24);
  return a;
}
__device__ __forceinline__ void decode8(const u32x2_t& a, float (&x)[RUN]) {   // E4M3
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[q], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[q], true);
    x[4 * q] = lo[0];
    x[4 * q + 1] = lo[1];
    x[4 * q + 2] = hi[0];
    x[4 * q + 3] = hi[1];
  }
}

template <bool FULL, int N>
__device__ __forceinline__ void store_n(float* p, uint32_t at, uint32_t last, const float (&x)[N]) {
  if (FULL) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      u32x4_t a;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(x[4 * q + e]);
      __builtin_nontemporal_store(a, reinterpret_cast<u32x4_t*>(p + at) + q);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (at + e <= last) p[at + e] = x[e];
  }
}
// bf16 pairs.
template <bool FULL, int H>
__device__ __forceinline__ void store_pairs(bf16_t* p, uint32_t at, uint32_t last, const uint32_t (&x)[H]) {
  typedef uint32_t piece_t __attribute__((ext_vector_type(H)));
  if (FULL) {
    piece_t a;
#pragma unroll
    for (int e = 0; e < H; ++e) a[e] = x[e];
    __builtin_nontemporal_store(a, reinterpret_cast<piece_t*>(p + at));
  } else {
#pragma unroll
    for (int e = 0; e < 2 * H; ++e)
      if (at + e <= last) p[at + e] = (bf16_t)(x[e >> 1] >> (16 * (e & 1)));
  }
}
template <bool FULL>
__device__ __forceinline__ void store8_codes(uint8_t* p, uint32_t at, uint32_t last, const u32x2_t& a) {
  if (FULL) {
    __builtin_nontemporal_store(a, reinterpret_cast<u32x2_t*>(p + at));
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e)
      if (at + e <= last) p[at + e] = (uint8_t)(a[e >> 2] >> (8 * (e & 3)));
  }
}

// Codes of 8 values of a block and its scale.  b: the bits of the lane's largest magnitude.  The
// instruction adds the upper 20 of the random bits below the code's last place and cuts off; 16 of them are
// random, the values' probabilities are in steps of 2^-16.  POSITIVE: x >= 0, and a value above zero gets a
// code above zero.  A block with an infinity or a NaN gets a scale of NaN, and stays so.
template <bool POSITIVE>
__device__ __forceinline__ float encode8(const float (&x)[RUN], uint32_t b, const uint32_t (&bits)[RUN], u32x2_t& codes) {
  b = row16_max(b);
  const bool lost = b >= 0x7f800000u;
  const float top = __uint_as_float(b);
  const bool fine = top >= TINY && !lost;
  const float inv = fine ? TOP / top : 0.0f;
  float y[RUN];
  uint32_t r[RUN];
#pragma unroll
  for (int e = 0; e < RUN; ++e) {
    y[e] = x[e] * inv;
    y[e] = __builtin_amdgcn_fmed3f(y[e], POSITIVE ? (y[e] > 0.0f ? LEAST : 0.0f) : -TOP, TOP);
    r[e] = POSITIVE ? bits[e] << 16 : bits[e] & 0xffff0000u;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    int c = 0;
    c = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * q], (int)r[4 * q], c, 0);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * q + 1], (int)r[4 * q + 1], c, 1);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * q + 2], (int)r[4 * q + 2], c, 2);
    c = __builtin_amdgcn_cvt_sr_fp8_f32(y[4 * q + 3], (int)r[4 * q + 3], c, 3);
    codes[q] = (uint32_t)c;
  }
  return fine ? top / TOP : (lost ? __uint_as_float(0x7fc00000u) : 0.0f);
}

// The tensors of one launch, in its kernel arguments: a call copies nothing to the device and can be
// captured.  36 tensors stay within 4 KiB; a longer list takes the large table, whose 28 KiB cost the host a
// microsecond and save the ends of launches (300 tensors, 20 M parameters, 8-bit states: 95 us in tables of 36,
// 75 of 72, 56 of 280).
constexpr int SMALL = 36, LARGE = 280;
template <int CAP>
struct Table {
  AdamWStep step;
  const void* param[CAP];
  const void* grad[CAP];
  const void* m[CAP];
  const void* v[CAP];
  const float* scale[CAP];
  const float* master[CAP];
  void* param_out[CAP];
  void* m_out[CAP];
  void* v_out[CAP];
  float* scale_out[CAP];
  float* master_out[CAP];
  int first[CAP + 1];      // first chunk of each tensor, among this launch's chunks
  uint32_t tail[CAP];      // elements of its last chunk; bit 31: bf16 gradient, bit 30: bf16 parameter
  float decay[CAP];
  uint32_t seed[CAP];
  int count;
  uint32_t chunk;
};
static_assert(sizeof(Table<SMALL>) <= 4096, "kernel arguments");

enum ParamKind { P_F32 = 0, P_BF16 = 1, P_MASTER = 2 };   // P_MASTER: bf16, rounded from an fp32 copy

// What a workgroup works on, out of the table: `n` elements of a tensor, whose pointers stand at the
// chunk's first element (32-bit offsets from there on, that loads and stores take beside a scalar base).
struct Chunk {
  const void* param;
  const void* grad;
  const void* m;
  const void* v;
  const float* scale_m;
  const float* scale_v;
  const float* master;
  void* param_out;
  void* m_out;
  void* v_out;
  float* scale_m_out;
  float* scale_v_out;
  float* master_out;
  float decay, c, beta1, one_minus_beta1, beta2, one_minus_beta2, inv_sqrt_bc2, step_size, eps;
  uint32_t n, seed;   // seed: with the chunk's first run of 8 in it
};

// Elements of a lane.  Blocks of 8-bit states take 8, so that their codes move in 8 bytes and bf16 in 16;
// fp32 states move in 16-byte pieces that follow each other from lane to lane: 4.  (With 8, in two pieces 32
// bytes apart, 409 M bf16 parameters with master copies took 2994 us instead of 2472.)
template <bool BITS8>
constexpr int lane_elements() { return BITS8 ? 8 : 4; }

// The elements from `at` on.
template <bool BITS8, int P, typename G, bool FULL>
__device__ __forceinline__ void update(const Chunk& k, uint32_t at) {
  constexpr int N = lane_elements<BITS8>();
  const uint32_t last = k.n - 1;
  float g[N], m[N], v[N], w[N];
  const uint32_t block = (FULL ? at : min(at, last)) / BLOCK;
  u32x2_t cm, cv;
  float sm = 1.0f, sv = 1.0f;
  load_n<FULL>(reinterpret_cast<const G*>(k.grad), at, last, g);
  if (P == P_MASTER) load_n<FULL>(k.master, at, last, w);
  else if (P == P_BF16) load_n<FULL>(reinterpret_cast<const bf16_t*>(k.param), at, last, w);
  else load_n<FULL>(reinterpret_cast<const float*>(k.param), at, last, w);
  if constexpr (BITS8) {
    cm = load8_codes<FULL>(reinterpret_cast<const uint8_t*>(k.m), at, last);
    cv = load8_codes<FULL>(reinterpret_cast<const uint8_t*>(k.v), at, last);
    sm = k.scale_m[block];
    sv = k.scale_v[block];
    decode8(cm, m);
    decode8(cv, v);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = v[e] * v[e];   // exact: codes have 4 bits
  } else {
    load_n<FULL>(reinterpret_cast<const float*>(k.m), at, last, m);
    load_n<FULL>(reinterpret_cast<const float*>(k.v), at, last, v);
  }
  // The scales of codes go into the factors.  With 32-bit states the root and the division are rounded to nearest,
  // which costs nothing beside the memory's time (2069 us, 2108 with the hardware's approximate ones, 409 M
  // parameters).  With 8-bit states the root is root_of's and the division a product with the hardware's reciprocal, a
  // unit in the last place of a step, which lr makes a small part of the parameter: rounded to nearest the root alone
  // would be 790 us for 733, both 864.
  const float b1 = k.beta1 * sm, b2 = k.beta2 * (sv * sv);
  float root[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float ge = g[e] * k.c;
    m[e] = __builtin_fmaf(b1, m[e], k.one_minus_beta1 * ge);
    v[e] = __builtin_fmaf(b2, v[e], k.one_minus_beta2 * (ge * ge));
    root[e] = BITS8 ? root_of(v[e]) : __builtin_sqrtf(v[e]);
    const float den = __builtin_fmaf(root[e], k.inv_sqrt_bc2, k.eps);
    const float step = BITS8 ? m[e] * __builtin_amdgcn_rcpf(den) : m[e] / den;
    w[e] = __builtin_fmaf(-k.step_size, step, k.decay * w[e]);
  }
  uint32_t bits[N];   // random
  if (BITS8 || P == P_BF16) {
    uint32_t h = mix(k.seed + at / RUN * 0x9E3779B1u);
    if (N < RUN) h = at % RUN ? h * 158984081u + 2868466484u : h;   // 4 steps of the sequence below
#pragma unroll
    for (int e = 0; e < N; ++e) bits[e] = h = h * 1664525u + 1013904223u;
  }
  uint32_t width[N];   // of the random bits added to a bf16 parameter: to a NaN, whose bits may all be set, none
#pragma unroll
  for (int e = 0; e < N; ++e) width[e] = w[e] == w[e] ? 16 : 0;
  if constexpr (BITS8) {
    if (!FULL) {   // what stood in for the elements behind the last is no part of their block
#pragma unroll
      for (int e = 0; e < N; ++e) {
        m[e] = at + e <= last ? m[e] : 0.0f;
        root[e] = at + e <= last ? root[e] : 0.0f;
      }
    }
    // The largest magnitudes, a NaN above all (`maximum` hands it on).  Where the root is lost, so is m; m can be by
    // itself, from a state that holds a NaN or an infinity.
    float top = 0.0f;
    uint32_t most = 0;   // root's bits: not negative
#pragma unroll
    for (int e = 0; e < N; ++e) {
      top = __builtin_elementwise_maximum(top, __builtin_fabsf(m[e]));
      most = max(most, __float_as_uint(root[e]));
    }
    const uint32_t lost = most >= 0x7f800000u ? most : __float_as_uint(top) & 0x7fffffffu;
    // One comparison for the lane's 8: a NaN of a state or a gradient is among them, and one of the parameter itself
    // has a lower half of zeros.  The other seven are cut off; their block is lost.
#pragma unroll
    for (int e = 0; e < N; ++e) width[e] = lost >= 0x7f800000u ? 0 : 16;
    sm = encode8<false>(m, lost, bits, cm);
    sv = encode8<true>(root, most, bits, cv);
    store8_codes<FULL>(reinterpret_cast<uint8_t*>(k.m_out), at, last, cm);
    store8_codes<FULL>(reinterpret_cast<uint8_t*>(k.v_out), at, last, cv);
    if ((threadIdx.x & 15) == 0 && (FULL || at <= last)) {
      k.scale_m_out[block] = sm;
      k.scale_v_out[block] = sv;
    }
  } else {
    store_n<FULL>(reinterpret_cast<float*>(k.m_out), at, last, m);
    store_n<FULL>(reinterpret_cast<float*>(k.v_out), at, last, v);
  }
  if (P == P_F32) {
    store_n<FULL>(reinterpret_cast<float*>(k.param_out), at, last, w);
    return;
  }
  uint32_t p[N / 2];
  if (P == P_MASTER) {
    store_n<FULL>(k.master_out, at, last, w);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const f32x2_t pair = {w[2 * e], w[2 * e + 1]};
      p[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, bf16x2_t));
    }
  } else {
    // Infinities stay: their lower bits are zero.  So do NaNs: with bits added, 0x7fffffff would carry into a zero.
    // (A result of arithmetic, a NaN has its upper half's quiet bit.)
    auto up = [&](int e) { return __float_as_uint(w[e]) + __builtin_amdgcn_ubfe(bits[e], 8, width[e]); };
#pragma unroll
    for (int e = 0; e < N / 2; ++e) p[e] = __builtin_amdgcn_perm(up(2 * e + 1), up(2 * e), 0x07060302u);   // the upper halves
  }
  store_pairs<FULL>(reinterpret_cast<bf16_t*>(k.param_out), at, last, p);
}

template <bool BITS8, int P, typename G>
__device__ __forceinline__ void update_chunk(const Chunk& k) {
  // a wave's elements at a time; the last ones of a tensor need not fill it
  constexpr uint32_t N = lane_elements<BITS8>();
  uint32_t at = __builtin_amdgcn_readfirstlane((threadIdx.x & ~63u) * N);
  const uint32_t lane = (threadIdx.x & 63u) * N;
  for (; at + 64 * N <= k.n; at += NT * N) update<BITS8, P, G, true>(k, at + lane);
  if (at < k.n) update<BITS8, P, G, false>(k, at + lane);
}

// n elements of `bytes` each, as they are.
__device__ __forceinline__ void copy_chunk(const void* from, void* to, uint32_t n, uint32_t bytes) {
  if (from == to) return;
  const uint8_t* f = reinterpret_cast<const uint8_t*>(from);
  uint8_t* o = reinterpret_cast<uint8_t*>(to);
  for (uint32_t i = threadIdx.x; i < n * bytes; i += NT) o[i] = f[i];
}

template <typename T>
__device__ __forceinline__ T* forward(T* p, long long bytes) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte_t;
  return p ? reinterpret_cast<T*>(reinterpret_cast<byte_t*>(p) + bytes) : p;
}

template <bool BITS8, int CAP>
__global__ __launch_bounds__(NT, BITS8 ? 5 : 8) void adamw_kernel(Table<CAP> t) {
  const int b = blockIdx.x;
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= b) lo = mid; else hi = mid;
  }
  const int i = lo;
  // Everything out of the table by value: a reference to it past this point would have the compiler keep a
  // copy of the whole table in scratch memory.
  const uint32_t tail = t.tail[i];
  const int first = t.first[i], chunks = t.first[i + 1] - first;
  const bool bf16 = tail >> 30 & 1, grad_bf16 = tail >> 31;
  const long long begin = (long long)(b - first) * t.chunk;
  const long long total = (long long)(chunks - 1) * t.chunk + (tail & 0x3fffffffu);
  const long long blocks = (total + BLOCK - 1) / BLOCK;
  Chunk k;
  k.n = b + 1 == first + chunks ? tail & 0x3fffffffu : t.chunk;
  k.param = forward(t.param[i], begin * (bf16 ? 2 : 4));
  k.grad = forward(t.grad[i], begin * (grad_bf16 ? 2 : 4));
  k.m = forward(t.m[i], begin * (BITS8 ? 1 : 4));
  k.v = forward(t.v[i], begin * (BITS8 ? 1 : 4));
  k.scale_m = forward(t.scale[i], begin / BLOCK * 4);
  k.scale_v = forward(t.scale[i], (blocks + begin / BLOCK) * 4);
  k.master = forward(t.master[i], begin * 4);
  k.param_out = forward(t.param_out[i], begin * (bf16 ? 2 : 4));
  k.m_out = forward(t.m_out[i], begin * (BITS8 ? 1 : 4));
  k.v_out = forward(t.v_out[i], begin * (BITS8 ? 1 : 4));
  k.scale_m_out = forward(t.scale_out[i], begin / BLOCK * 4);
  k.scale_v_out = forward(t.scale_out[i], (blocks + begin / BLOCK) * 4);
  k.master_out = forward(t.master_out[i], begin * 4);
  k.seed = t.seed[i] + (uint32_t)(begin / RUN) * 0x9E3779B1u;
  k.decay = t.decay[i];
  k.beta1 = t.step.beta1;
  k.one_minus_beta1 = t.step.one_minus_beta1;
  k.beta2 = t.step.beta2;
  k.one_minus_beta2 = t.step.one_minus_beta2;
  k.inv_sqrt_bc2 = t.step.inv_sqrt_bc2;
  k.step_size = t.step.step_size;
  k.eps = t.step.eps;
  k.c = 1.0f;
  if (t.step.sumsq) {
    const double norm = sqrt(*t.step.sumsq);
    if (!((float)norm <= 3.4028234664e38f)) {   // no step: the outputs are the inputs
      if (k.param) {
        copy_chunk(k.param, k.param_out, k.n, bf16 ? 2 : 4);
      } else {   // a master copy stands for it
        for (uint32_t e = threadIdx.x; e < k.n; e += NT)
          reinterpret_cast<bf16_t*>(k.param_out)[e] = f32_to_bf16(reinterpret_cast<const float*>(k.master)[e]);
      }
      copy_chunk(k.m, k.m_out, k.n, BITS8 ? 1 : 4);
      copy_chunk(k.v, k.v_out, k.n, BITS8 ? 1 : 4);
      if (k.master) copy_chunk(k.master, k.master_out, k.n, 4);
      if (BITS8) {
        copy_chunk(k.scale_m, k.scale_m_out, (k.n + BLOCK - 1) / BLOCK, 4);
        copy_chunk(k.scale_v, k.scale_v_out, (k.n + BLOCK - 1) / BLOCK, 4);
      }
      return;
    }
    const double q = t.step.max_norm / (norm + 1e-6);
    k.c = q < 1.0 ? (float)q : 1.0f;
  }
  if (grad_bf16) {
    if (k.master) update_chunk<BITS8, P_MASTER, bf16_t>(k);
    else if (bf16) update_chunk<BITS8, P_BF16, bf16_t>(k);
    else update_chunk<BITS8, P_F32, bf16_t>(k);
  } else {
    if (k.master) update_chunk<BITS8, P_MASTER, float>(k);
    else if (bf16) update_chunk<BITS8, P_BF16, float>(k);
    else update_chunk<BITS8, P_F32, float>(k);
  }
}

// Elements per chunk: one step of a workgroup, so that workgroups that run together work on neighbouring
// memory (409 M parameters with 8-bit states: 720 us, against 880 us with 64 Ki chunks over the list and 1010 us
// with 8 Ki; with fp32 states and master copies 2109 us, 2205 in chunks of two steps); more only where the grid
// of a launch would pass 2^30 threads, for lists of more than 2^32 elements.
long long chunk_size(long long total, bool bits8) {
  const long long step = NT * (bits8 ? lane_elements<true>() : lane_elements<false>());
  const long long c = (total + (1 << 22) - 1) >> 22;
  return (std::max<long long>(c, 1) + step - 1) / step * step;
}

template <int CAP>
hipError_t launch_tables(const AdamWItem* items, int count, const AdamWStep& step, bool bits8, hipStream_t s) {
  std::unique_ptr<Table<CAP>> table(new (std::nothrow) Table<CAP>());
  if (!table) return hipErrorOutOfMemory;
  Table<CAP>& t = *table;
  long long total = 0;
  for (int i = 0; i < count; ++i) total += items[i].n;
  const long long chunk = chunk_size(total, bits8);
  t.step = step;
  t.chunk = (uint32_t)chunk;
  for (int i = 0; i <= count; ++i) {
    if (i < count && items[i].n > 0) {
      const AdamWItem& a = items[i];
      const int k = t.count++;
      t.param[k] = a.param;
      t.grad[k] = a.grad;
      t.m[k] = a.m;
      t.v[k] = a.v;
      t.scale[k] = a.scale;
      t.master[k] = a.master;
      t.param_out[k] = a.param_out;
      t.m_out[k] = a.m_out;
      t.v_out[k] = a.v_out;
      t.scale_out[k] = a.scale_out;
      t.master_out[k] = a.master_out;
      t.decay[k] = a.decay;
      t.seed[k] = a.seed;
      const long long chunks = (a.n + chunk - 1) / chunk;
      t.tail[k] = (uint32_t)(a.n - (chunks - 1) * chunk) | (a.grad_bf16 ? 0x80000000u : 0u) | (a.bf16 ? 0x40000000u : 0u);
      t.first[k + 1] = t.first[k] + (int)chunks;
    }
    if (t.count == CAP || (i == count && t.count > 0)) {
      if (bits8) adamw_kernel<true, CAP><<<dim3(t.first[t.count]), dim3(NT), 0, s>>>(t);
      else adamw_kernel<false, CAP><<<dim3(t.first[t.count]), dim3(NT), 0, s>>>(t);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      t.count = 0;
    }
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_adamw(const AdamWItem* items, int count, const AdamWStep& step, bool bits8, hipStream_t s) {
  return count <= SMALL ? launch_tables<SMALL>(items, count, step, bits8, s) : launch_tables<LARGE>(items, count, step, bits8, s);
}

}  // namespace moe
