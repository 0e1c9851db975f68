// Global norm of a list of gradient tensors, and clipping.
//
//   norm = sqrt(sum_i sum_j g_i[j]^2),  out_i = c g_i,  c = min(1, max_norm / (norm + 1e-6))
//
// The list is cut into chunks of at most `chunk` elements of one tensor, one workgroup each; a
// chunk's sum of squares goes to its own place in the workspace and the sums are added in chunk
// order, so the norm does not depend on the order in which workgroups run.  Squares and sums are
// double: a gradient of 1e9 values loses nothing to the order of its additions, and a square of any
// fp32 value is in range.
//
// The tensor list travels in the kernel arguments (kGradTable tensors per launch), so a call needs no
// copy to the device and can be captured.
//
// Bound by memory: the sum reads the list once, the scaling reads it again and writes it.  409 M bf16
// values (818 MB): the sum 140 us (5.8 TB/s), the scaling 312 us (5.2 TB/s), against 5.1 TB/s of a
// device copy.  The scaling starts where the sum ended, whose last quarter of a GB is still in the
// last-level cache, and its own loads and stores are nontemporal so that they do not displace it:
// 365 us in the order of the sum with ordinary loads.
#include "block_step.h"

#include <algorithm>

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int NT = 256;
constexpr int IN_FLIGHT = 8;   // 16-byte loads of a thread ahead of their use

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
  return s;
}

// Sum over the workgroup, the same value in every thread.
__device__ __forceinline__ double block_sum(double s, double* red) {
  s = wave_sum(s);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// The chunk c of a launch: its tensor (the last one whose first chunk is <= c) and its elements.
struct Chunk {
  int tensor;
  bool bf16;
  long long begin, n;
};
__device__ __forceinline__ Chunk find_chunk(const GradTable& t, int c, long long chunk) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= c) lo = mid; else hi = mid;
  }
  Chunk k;
  k.tensor = lo;
  k.bf16 = t.tail[lo] >> 31;
  k.begin = (long long)(c - t.first[lo]) * chunk;
  k.n = c + 1 == t.first[lo + 1] ? (long long)(t.tail[lo] & 0x7fffffffu) : chunk;
  return k;
}

__global__ __launch_bounds__(NT) void grad_sumsq_kernel(GradTable t, long long chunk, double* partial) {
  __shared__ double red[NT / 64];
  const Chunk k = find_chunk(t, blockIdx.x, chunk);
  const long long n = k.n;
  double s = 0.0;
  if (k.bf16) {
    const bf16_t* g = reinterpret_cast<const bf16_t*>(t.grad[k.tensor]) + k.begin;
    const u32x4_t* v = reinterpret_cast<const u32x4_t*>(g);
    long long j = threadIdx.x;
    double s1 = 0.0;
    auto add = [&](const u32x4_t& w) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const double a = __uint_as_float(w[q] << 16), b = __uint_as_float(w[q] & 0xffff0000u);
        s += a * a;
        s1 += b * b;
      }
    };
    for (; j + (IN_FLIGHT - 1) * NT < n / 8; j += IN_FLIGHT * NT) {
      u32x4_t w[IN_FLIGHT];
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) w[u] = v[j + u * NT];
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) add(w[u]);
    }
    for (; j < n / 8; j += NT) add(v[j]);
    s += s1;
    for (long long j = n / 8 * 8 + threadIdx.x; j < n; j += NT) {
      const double a = bf16_to_f32(g[j]);
      s += a * a;
    }
  } else {
    const float* g = reinterpret_cast<const float*>(t.grad[k.tensor]) + k.begin;
    const float4* v = reinterpret_cast<const float4*>(g);
    long long j = threadIdx.x;
    double s1 = 0.0;
    auto add = [&](const float4& w) {
      s += (double)w.x * w.x;
      s1 += (double)w.y * w.y;
      s += (double)w.z * w.z;
      s1 += (double)w.w * w.w;
    };
    for (; j + (IN_FLIGHT - 1) * NT < n / 4; j += IN_FLIGHT * NT) {
      float4 w[IN_FLIGHT];
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) w[u] = v[j + u * NT];
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) add(w[u]);
    }
    for (; j < n / 4; j += NT) add(v[j]);
    s += s1;
    for (long long j = n / 4 * 4 + threadIdx.x; j < n; j += NT) s += (double)g[j] * g[j];
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[t.base + blockIdx.x] = s;
}

// The sum of `count` partials, in a fixed order: thread i adds every NT-th, then the tree of
// block_sum.  Every workgroup that calls it gets the same bits.
__device__ __forceinline__ double sum_partials(const double* partial, int count, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += NT) s += partial[i];
  return block_sum(s, red);
}

__global__ __launch_bounds__(NT) void grad_total_kernel(const double* partial, int count, double* sumsq, float* norm) {
  __shared__ double red[NT / 64];
  const double s = sum_partials(partial, count, red);
  if (threadIdx.x == 0) {
    if (sumsq) *sumsq = s;
    if (norm) *norm = (float)sqrt(s);
  }
}

// out = c g for every chunk of the launch, the last parts of the chunks first (blockIdx.y: one of
// gridDim.y equal parts).  sums[0..count) add up to the sum of squares.
__global__ __launch_bounds__(NT) void grad_scale_kernel(GradTable t, long long chunk, const double* sums, int count,
                                                        float max_norm, float* norm_out) {
  __shared__ double red[NT / 64];
  const double norm = sqrt(sum_partials(sums, count, red));
  if (norm_out && t.base == 0 && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double q = (double)max_norm / (norm + 1e-6);
  // A norm that is infinite or NaN as it is reported, in fp32, scales nothing: 3.4e38 < norm < 1e308 too
  const float c = q < 1.0 && (float)norm <= 3.4028234664e38f ? (float)q : 1.0f;
  const Chunk k = find_chunk(t, blockIdx.x, chunk);
  if (c == 1.0f && t.out[k.tensor] == t.grad[k.tensor]) return;
  const long long part = chunk / gridDim.y, at = (long long)(gridDim.y - 1 - blockIdx.y) * part;
  const long long n = min(part, k.n - at);
  if (n <= 0) return;
  if (k.bf16) {
    const bf16_t* g = reinterpret_cast<const bf16_t*>(t.grad[k.tensor]) + k.begin + at;
    bf16_t* o = reinterpret_cast<bf16_t*>(t.out[k.tensor]) + k.begin + at;
    const u32x4_t* v = reinterpret_cast<const u32x4_t*>(g);
    u32x4_t* to = reinterpret_cast<u32x4_t*>(o);
    auto scaled = [&](u32x4_t w) {
      if (c != 1.0f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = c * __uint_as_float(w[e] << 16), hi = c * __uint_as_float(w[e] & 0xffff0000u);
          w[e] = (uint32_t)f32_to_bf16(lo) | ((uint32_t)f32_to_bf16(hi) << 16);
        }
      }
      return w;
    };
    long long j = threadIdx.x;
    for (; j + (IN_FLIGHT - 1) * NT < n / 8; j += IN_FLIGHT * NT) {
      u32x4_t w[IN_FLIGHT];
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) w[u] = __builtin_nontemporal_load(v + j + u * NT);
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) __builtin_nontemporal_store(scaled(w[u]), to + j + u * NT);
    }
    for (; j < n / 8; j += NT) __builtin_nontemporal_store(scaled(v[j]), to + j);
    for (long long i = n / 8 * 8 + threadIdx.x; i < n; i += NT) o[i] = c == 1.0f ? g[i] : f32_to_bf16(c * bf16_to_f32(g[i]));
  } else {
    const float* g = reinterpret_cast<const float*>(t.grad[k.tensor]) + k.begin + at;
    float* o = reinterpret_cast<float*>(t.out[k.tensor]) + k.begin + at;
    const f32x4_t* v = reinterpret_cast<const f32x4_t*>(g);
    f32x4_t* to = reinterpret_cast<f32x4_t*>(o);
    long long j = threadIdx.x;
    for (; j + (IN_FLIGHT - 1) * NT < n / 4; j += IN_FLIGHT * NT) {
      f32x4_t w[IN_FLIGHT];
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) w[u] = __builtin_nontemporal_load(v + j + u * NT);
#pragma unroll
      for (int u = 0; u < IN_FLIGHT; ++u) __builtin_nontemporal_store(w[u] * c, to + j + u * NT);
    }
    for (; j < n / 4; j += NT) __builtin_nontemporal_store(v[j] * c, to + j);
    for (long long i = n / 4 * 4 + threadIdx.x; i < n; i += NT) o[i] = c * g[i];
  }
}

// Elements per chunk: about 2048 chunks over the list (eight workgroups per CU), at least 4096.
long long chunk_size(long long total) {
  const long long c = (total + 2047) / 2048;
  return std::max<long long>(4096, (c + 2047) / 2048 * 2048);
}

// A list whose chunks are this long (64 M elements) is scaled in eighths of chunks.
constexpr long long LONG_CHUNK = 32768;
// The partial sums of such a list, or more than this many (a tensor has one at least), are added by a
// launch of their own; otherwise every scaling workgroup adds them itself, at most 18 KB from the L2
// cache.  Whole calls with and without that launch (us): 300 tensors of 1500 values 21 and 20, 1500 of
// 4000 99 and 101, 2500 of 1500 110 and 125, 10000 of 1500 579 and 814, 40000 of 1500 3280 and 6617:
// what the workgroups read grows with the square of the number of tensors.
constexpr int MOST_SUMS = 2304;
constexpr int PARTS = 8;   // a chunk is a multiple of 2048 elements: a part starts at 16 bytes

}  // namespace

long long grad_chunks(const GradItem* g, int count) {
  long long total = 0, chunks = 0;
  for (int i = 0; i < count; ++i) total += g[i].n;
  const long long c = chunk_size(total);
  for (int i = 0; i < count; ++i) chunks += (g[i].n + c - 1) / c;
  return chunks;
}

namespace {

// Calls f(table) for each run of at most kTable tensors; tensors without elements are left out.
template <typename F>
hipError_t for_tables(const GradItem* g, int count, long long chunk, F&& f) {
  GradTable t{};
  int base = 0;
  for (int i = 0; i <= count; ++i) {
    if (i < count && g[i].n > 0) {
      const int k = t.count++;
      t.grad[k] = g[i].grad;
      t.out[k] = g[i].out;
      const long long chunks = (g[i].n + chunk - 1) / chunk;
      t.tail[k] = (uint32_t)(g[i].n - (chunks - 1) * chunk) | (g[i].bf16 ? 0x80000000u : 0u);
      t.first[k + 1] = t.first[k] + (int)chunks;
    }
    if (t.count == kGradTable || (i == count && t.count > 0)) {
      t.base = base;
      const hipError_t e = f(t);
      if (e != hipSuccess) return e;
      base += t.first[t.count];
      t.count = 0;
    }
  }
  return hipSuccess;
}

long long total_elements(const GradItem* g, int count) {
  long long total = 0;
  for (int i = 0; i < count; ++i) total += g[i].n;
  return total;
}

}  // namespace

hipError_t launch_grad_sumsq(const GradItem* g, int count, double* partial, hipStream_t s) {
  const long long chunk = chunk_size(total_elements(g, count));
  return for_tables(g, count, chunk, [&](const GradTable& t) {
    grad_sumsq_kernel<<<dim3(t.first[t.count]), dim3(NT), 0, s>>>(t, chunk, partial);
    return hipGetLastError();
  });
}

hipError_t launch_grad_total(const double* partial, int count, double* sumsq, float* norm, hipStream_t s) {
  grad_total_kernel<<<dim3(1), dim3(NT), 0, s>>>(partial, count, sumsq, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradItem* g, int count, double* sums, int nsums, float max_norm, float* norm,
                             hipStream_t s) {
  const long long chunk = chunk_size(total_elements(g, count));
  const bool parts = chunk >= LONG_CHUNK;
  if (nsums > 1 && (parts || nsums > MOST_SUMS)) {
    const hipError_t e = launch_grad_total(sums, nsums, sums + nsums, nullptr, s);
    if (e != hipSuccess) return e;
    sums += nsums;
    nsums = 1;
  }
  return for_tables(g, count, chunk, [&](const GradTable& t) {
    grad_scale_kernel<<<dim3(t.first[t.count], parts ? PARTS : 1), dim3(NT), 0, s>>>(t, chunk, sums, nsums, max_norm, norm);
    return hipGetLastError();
  });
}

}  // namespace moe
