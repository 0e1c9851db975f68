// AdamW over a list of tensors, with the gradients' clipping in the same pass.
//
//   g = c grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
//   p = (1 - lr wd) p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// (Loshchilov and Hutter's decoupled weight decay), c the clipping coefficient of moe_grad_scale, all of
// it fp32, each operation rounded by itself.  The states m and v are fp32, or 8 bits: E4M3 codes of m and
// of sqrt(v) with one float scale for 128 elements, the block's largest magnitude / 448.  The root keeps
// v's range in E4M3's, twice the exponent.  A state that moves by a fraction of a code's step (b2 = 0.999
// moves v by a thousandth, a step is up to an eighth) would stay where it is if it were rounded to
// nearest; so the rounding is random, up with the probability of the rest.  A positive v keeps at least
// the smallest code: m over a v that was rounded to zero would be a step of m / eps.  A bf16 parameter
// without a master copy is rounded in the same way.  The random bits are a hash of the element's run of 8
// and the tensor's seed, and a linear congruential sequence inside the run: the same call gives the same
// bits.
//
// Bound by memory: one pass, nothing read or written twice.  8 elements a lane: a bf16 tensor moves in
// 16-byte pieces, 128 elements (a block of the 8-bit states) lie in 16 lanes, whose largest value is
// found with row rotations in registers.
#include "train_step.h"

#include <algorithm>

#pragma clang fp contract(off)

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr int NT = 256;
constexpr int RUN = 8;              // elements a lane
constexpr int STEP = NT * RUN;      // elements of a workgroup's step
constexpr int BLOCK = 128;          // elements that share a scale: 16 lanes
constexpr float TOP = 448.0f;       // the largest E4M3 value
constexpr float LOW = 0x1p-6f;      // the smallest normal one
constexpr float TINY = 0x1p-100f;   // a block whose largest magnitude is below is stored as zeros

__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h ^= h >> 16;
  h *= 0x9D2B4F35u;
  h ^= h >> 15;
  h *= 0xC5A1E6B7u;
  return h ^ (h >> 16);
}

// The largest of the 16 lanes of a row, in every one of them: bits of magnitudes, which order as the
// values do, a NaN above all.
__device__ __forceinline__ uint32_t row_max(uint32_t b) {
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0xB1, 0xf, 0xf, false));    // quad_perm 1,0,3,2
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x4E, 0xf, 0xf, false));    // quad_perm 2,3,0,1
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x124, 0xf, 0xf, false));   // row_ror 4
  b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, 0x128, 0xf, 0xf, false));   // row_ror 8
  return b;
}

// The E4M3 code of y in [0, 448], rounded up with the probability of the rest, in steps of 2^-16 (20
// bits are dropped, the random ones are the upper 16 of them).  Below the normal range 2^-6 is added, so
// that the dropped bits are those below the subnormals' step.
__device__ __forceinline__ uint32_t stochastic_e4m3(float y, uint32_t dither) {
  const bool low = y < LOW;
  const uint32_t b = __float_as_uint(low ? y + LOW : y) + (dither << 4);
  return (b >> 20) - (low ? 968u : 960u);
}

template <bool FULL>
__device__ __forceinline__ void load8(const float* p, int cnt, float (&x)[RUN]) {
  if (FULL) {
    const u32x4_t a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
    const u32x4_t b = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p) + 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = __uint_as_float(a[e]);
      x[4 + e] = __uint_as_float(b[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e) x[e] = e < cnt ? p[e] : 0.0f;
  }
}
template <bool FULL>
__device__ __forceinline__ void load8(const bf16_t* p, int cnt, float (&x)[RUN]) {
  if (FULL) {
    const u32x4_t a = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(a[e] << 16);
      x[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e) x[e] = e < cnt ? bf16_to_f32(p[e]) : 0.0f;
  }
}
template <bool FULL>
__device__ __forceinline__ void load8(const uint8_t* p, int cnt, float (&x)[RUN]) {   // E4M3
  u32x2_t a = {0u, 0u};
  if (FULL) {
    a = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e)
      if (e < cnt) a[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[q], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)a[q], true);
    x[4 * q] = lo[0];
    x[4 * q + 1] = lo[1];
    x[4 * q + 2] = hi[0];
    x[4 * q + 3] = hi[1];
  }
}

template <bool FULL>
__device__ __forceinline__ void store8(float* p, int cnt, const float (&x)[RUN]) {
  if (FULL) {
    u32x4_t a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = __float_as_uint(x[e]);
      b[e] = __float_as_uint(x[4 + e]);
    }
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4_t*>(p));
    __builtin_nontemporal_store(b, reinterpret_cast<u32x4_t*>(p) + 1);
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e)
      if (e < cnt) p[e] = x[e];
  }
}
// bf16 bit patterns, one in each word.
template <bool FULL>
__device__ __forceinline__ void store8(bf16_t* p, int cnt, const uint32_t (&x)[RUN]) {
  if (FULL) {
    u32x4_t a;
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = x[2 * e] | (x[2 * e + 1] << 16);
    __builtin_nontemporal_store(a, reinterpret_cast<u32x4_t*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e)
      if (e < cnt) p[e] = (bf16_t)x[e];
  }
}
template <bool FULL>
__device__ __forceinline__ void store8(uint8_t* p, int cnt, const uint32_t (&code)[RUN]) {
  if (FULL) {
    u32x2_t a;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      a[q] = code[4 * q] | (code[4 * q + 1] << 8) | (code[4 * q + 2] << 16) | (code[4 * q + 3] << 24);
    __builtin_nontemporal_store(a, reinterpret_cast<u32x2_t*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e)
      if (e < cnt) p[e] = (uint8_t)code[e];
  }
}

enum ParamKind { P_F32 = 0, P_BF16 = 1, P_MASTER = 2 };   // P_MASTER: bf16, rounded from an fp32 copy

// Codes and scale of 8 values of a block (x not negative where POSITIVE).  A block with an infinity or a
// NaN gets a scale of NaN, and stays so.
template <bool POSITIVE>
__device__ __forceinline__ float encode8(const float (&x)[RUN], const uint32_t (&dither)[RUN], uint32_t (&code)[RUN]) {
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < RUN; ++e) bits = max(bits, __float_as_uint(x[e]) & 0x7fffffffu);
  bits = row_max(bits);
  const bool lost = bits >= 0x7f800000u;
  const float top = __uint_as_float(bits);
  const bool fine = top >= TINY && !lost;
  const float inv = fine ? TOP / top : 0.0f;
#pragma unroll
  for (int e = 0; e < RUN; ++e) {
    const float y = fminf(fabsf(x[e]) * inv, TOP);
    uint32_t c = stochastic_e4m3(y, dither[e]);
    if (POSITIVE) c = y > 0.0f ? max(c, 1u) : c;
    else c |= x[e] < 0.0f ? 0x80u : 0u;
    code[e] = c;
  }
  return fine ? top / TOP : (lost ? __uint_as_float(0x7fc00000u) : 0.0f);
}

// The 8 elements from `at` on (cnt of them exist) of tensor i.
template <bool BITS8, int P, typename G, bool FULL>
__device__ __forceinline__ void update8(const AdamWTable& t, int i, long long at, int cnt, long long blocks, float c,
                                        uint32_t seed) {
  float g[RUN], m[RUN], v[RUN], w[RUN];
  load8<FULL>(reinterpret_cast<const G*>(t.grad[i]) + at, cnt, g);
  if (P == P_MASTER) load8<FULL>(t.master[i] + at, cnt, w);
  else if (P == P_BF16) load8<FULL>(reinterpret_cast<const bf16_t*>(t.param[i]) + at, cnt, w);
  else load8<FULL>(reinterpret_cast<const float*>(t.param[i]) + at, cnt, w);
  const long long block = at / BLOCK;
  if constexpr (BITS8) {
    const float sm = cnt > 0 ? t.scale[i][block] : 0.0f, sv = cnt > 0 ? t.scale[i][blocks + block] : 0.0f;
    load8<FULL>(reinterpret_cast<const uint8_t*>(t.m[i]) + at, cnt, m);
    load8<FULL>(reinterpret_cast<const uint8_t*>(t.v[i]) + at, cnt, v);
#pragma unroll
    for (int e = 0; e < RUN; ++e) {
      m[e] = m[e] * sm;
      v[e] = v[e] * sv;
      v[e] = v[e] * v[e];
    }
  } else {
    load8<FULL>(reinterpret_cast<const float*>(t.m[i]) + at, cnt, m);
    load8<FULL>(reinterpret_cast<const float*>(t.v[i]) + at, cnt, v);
  }
  const float decay = t.decay[i];
  float root[RUN];
#pragma unroll
  for (int e = 0; e < RUN; ++e) {
    const float ge = g[e] * c;
    m[e] = t.step.beta1 * m[e] + t.step.one_minus_beta1 * ge;
    v[e] = t.step.beta2 * v[e] + t.step.one_minus_beta2 * (ge * ge);
    root[e] = sqrtf(v[e]);
    w[e] = decay * w[e] - t.step.step_size * (m[e] / (root[e] * t.step.inv_sqrt_bc2 + t.step.eps));
  }
  uint32_t bits[RUN];   // random
  if (BITS8 || P == P_BF16) {
    uint32_t h = mix(seed + (uint32_t)(at / RUN) * 0x9E3779B1u);
#pragma unroll
    for (int e = 0; e < RUN; ++e) bits[e] = h = h * 1664525u + 1013904223u;
  }
  if constexpr (BITS8) {
    uint32_t dither[RUN], code[RUN];
#pragma unroll
    for (int e = 0; e < RUN; ++e) dither[e] = bits[e] >> 16;
    const float sm = encode8<false>(m, dither, code);
    store8<FULL>(reinterpret_cast<uint8_t*>(t.m_out[i]) + at, cnt, code);
#pragma unroll
    for (int e = 0; e < RUN; ++e) dither[e] = bits[e] & 0xffffu;
    const float sv = encode8<true>(root, dither, code);
    store8<FULL>(reinterpret_cast<uint8_t*>(t.v_out[i]) + at, cnt, code);
    if ((threadIdx.x & 15) == 0 && cnt > 0) {
      t.scale_out[i][block] = sm;
      t.scale_out[i][blocks + block] = sv;
    }
  } else {
    store8<FULL>(reinterpret_cast<float*>(t.m_out[i]) + at, cnt, m);
    store8<FULL>(reinterpret_cast<float*>(t.v_out[i]) + at, cnt, v);
  }
  if (P == P_F32) {
    store8<FULL>(reinterpret_cast<float*>(t.param_out[i]) + at, cnt, w);
    return;
  }
  uint32_t p[RUN];
  if (P == P_MASTER) {
    store8<FULL>(t.master_out[i] + at, cnt, w);
#pragma unroll
    for (int e = 0; e < RUN; ++e) p[e] = f32_to_bf16(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e) {   // infinities and NaN stay as they are
      const uint32_t b = __float_as_uint(w[e]);
      p[e] = (b & 0x7f800000u) == 0x7f800000u ? (uint32_t)f32_to_bf16(w[e]) : (b + ((bits[e] >> 8) & 0xffffu)) >> 16;
    }
  }
  store8<FULL>(reinterpret_cast<bf16_t*>(t.param_out[i]) + at, cnt, p);
}

template <bool BITS8, int P, typename G>
__device__ __forceinline__ void update_chunk(const AdamWTable& t, int i, long long begin, int n, long long blocks, float c) {
  const uint32_t seed = t.seed[i];
  int at = threadIdx.x * RUN;
  for (; at - (int)threadIdx.x * RUN + STEP <= n; at += STEP)
    update8<BITS8, P, G, true>(t, i, begin + at, RUN, blocks, c, seed);
  if (at - (int)threadIdx.x * RUN < n)
    update8<BITS8, P, G, false>(t, i, begin + at, max(0, min(RUN, n - at)), blocks, c, seed);
}

// Elements [begin, begin + n) of `bytes` each, as they are.
__device__ __forceinline__ void copy_chunk(const void* from, void* to, long long begin, int n, int bytes) {
  if (from == to) return;
  const uint8_t* f = reinterpret_cast<const uint8_t*>(from) + begin * bytes;
  uint8_t* o = reinterpret_cast<uint8_t*>(to) + begin * bytes;
  for (int i = threadIdx.x; i < n * bytes; i += NT) o[i] = f[i];
}

template <bool BITS8>
__global__ __launch_bounds__(NT) void adamw_kernel(AdamWTable t) {
  const int b = blockIdx.x;
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= b) lo = mid; else hi = mid;
  }
  const int i = lo;
  const uint32_t tail = t.tail[i];
  const long long begin = (long long)(b - t.first[i]) * t.chunk;
  const int last = (int)(tail & 0x3fffffffu);
  const int n = b + 1 == t.first[i + 1] ? last : (int)t.chunk;
  const long long total = (long long)(t.first[i + 1] - t.first[i] - 1) * t.chunk + last;
  const long long blocks = (total + BLOCK - 1) / BLOCK;
  float c = 1.0f;
  if (t.step.sumsq) {
    const double norm = sqrt(*t.step.sumsq);
    if (!((float)norm <= 3.4028234664e38f)) {   // no step: the outputs are the inputs
      copy_chunk(t.param[i], t.param_out[i], begin, n, tail >> 30 & 1 ? 2 : 4);
      copy_chunk(t.m[i], t.m_out[i], begin, n, BITS8 ? 1 : 4);
      copy_chunk(t.v[i], t.v_out[i], begin, n, BITS8 ? 1 : 4);
      if (t.master[i]) copy_chunk(t.master[i], t.master_out[i], begin, n, 4);
      if (BITS8) {
        copy_chunk(t.scale[i], t.scale_out[i], begin / BLOCK, (n + BLOCK - 1) / BLOCK, 4);
        copy_chunk(t.scale[i], t.scale_out[i], blocks + begin / BLOCK, (n + BLOCK - 1) / BLOCK, 4);
      }
      return;
    }
    const double q = t.step.max_norm / (norm + 1e-6);
    c = q < 1.0 ? (float)q : 1.0f;
  }
  if (tail >> 31) {
    if (t.master[i]) update_chunk<BITS8, P_MASTER, bf16_t>(t, i, begin, n, blocks, c);
    else if (tail >> 30 & 1) update_chunk<BITS8, P_BF16, bf16_t>(t, i, begin, n, blocks, c);
    else update_chunk<BITS8, P_F32, bf16_t>(t, i, begin, n, blocks, c);
  } else {
    if (t.master[i]) update_chunk<BITS8, P_MASTER, float>(t, i, begin, n, blocks, c);
    else if (tail >> 30 & 1) update_chunk<BITS8, P_BF16, float>(t, i, begin, n, blocks, c);
    else update_chunk<BITS8, P_F32, float>(t, i, begin, n, blocks, c);
  }
}

// Elements per chunk: about 8192 chunks over the list, at least one step of a workgroup.
long long chunk_size(long long total) {
  const long long c = (total + 8191) / 8192;
  return std::max<long long>(STEP, (c + STEP - 1) / STEP * STEP);
}

}  // namespace

hipError_t launch_adamw(const AdamWItem* items, int count, const AdamWStep& step, bool bits8, hipStream_t s) {
  static_assert(sizeof(AdamWTable) <= 4096, "kernel arguments");
  long long total = 0;
  for (int i = 0; i < count; ++i) total += items[i].n;
  const long long chunk = chunk_size(total);
  AdamWTable t{};
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
    if (t.count == kAdamWTable || (i == count && t.count > 0)) {
      if (bits8) adamw_kernel<true><<<dim3(t.first[t.count]), dim3(NT), 0, s>>>(t);
      else adamw_kernel<false><<<dim3(t.first[t.count]), dim3(NT), 0, s>>>(t);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      t.count = 0;
    }
  }
  return hipSuccess;
}

}  // namespace moe
