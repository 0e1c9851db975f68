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
// The tensor list travels in the kernel arguments (kTable tensors per launch), so a call needs no
// copy to the device and can be captured.
#include "block_step.h"

#include <algorithm>

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int NT = 256;

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

// Tensor of chunk `c` of this launch: the last one whose first chunk is <= c.
__device__ __forceinline__ int find_tensor(const GradTable& t, int c) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= c) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(NT) void grad_sumsq_kernel(GradTable t, long long chunk, double* partial) {
  __shared__ double red[NT / 64];
  const int i = find_tensor(t, blockIdx.x);
  const long long e0 = (long long)(blockIdx.x - t.first[i]) * chunk;
  const long long n = min(chunk, (long long)t.n[i] - e0);
  double s = 0.0;
  if (t.bf16[i]) {
    const bf16_t* g = reinterpret_cast<const bf16_t*>(t.grad[i]) + e0;
    for (long long j = threadIdx.x; j < n / 8; j += NT) {
      const u32x4_t w = reinterpret_cast<const u32x4_t*>(g)[j];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const double a = __uint_as_float(w[q] << 16), b = __uint_as_float(w[q] & 0xffff0000u);
        s += a * a;
        s += b * b;
      }
    }
    for (long long j = n / 8 * 8 + threadIdx.x; j < n; j += NT) {
      const double a = bf16_to_f32(g[j]);
      s += a * a;
    }
  } else {
    const float* g = reinterpret_cast<const float*>(t.grad[i]) + e0;
    for (long long j = threadIdx.x; j < n / 4; j += NT) {
      const float4 w = reinterpret_cast<const float4*>(g)[j];
      s += (double)w.x * w.x;
      s += (double)w.y * w.y;
      s += (double)w.z * w.z;
      s += (double)w.w * w.w;
    }
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

// out = c g for every chunk of the launch; sums[0..count) add up to the sum of squares.
__global__ __launch_bounds__(NT) void grad_scale_kernel(GradTable t, long long chunk, const double* sums, int count,
                                                        float max_norm, float* norm_out) {
  __shared__ double red[NT / 64];
  const double norm = sqrt(sum_partials(sums, count, red));
  if (norm_out && t.base == 0 && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const double q = (double)max_norm / (norm + 1e-6);
  // a norm that is infinite or NaN scales nothing
  const float c = q < 1.0 && norm <= 1.7976931348623157e308 ? (float)q : 1.0f;
  const int i = find_tensor(t, blockIdx.x);
  if (c == 1.0f && t.out[i] == t.grad[i]) return;
  const long long e0 = (long long)(blockIdx.x - t.first[i]) * chunk;
  const long long n = min(chunk, (long long)t.n[i] - e0);
  if (t.bf16[i]) {
    const bf16_t* g = reinterpret_cast<const bf16_t*>(t.grad[i]) + e0;
    bf16_t* o = reinterpret_cast<bf16_t*>(t.out[i]) + e0;
    for (long long j = threadIdx.x; j < n / 8; j += NT) {
      u32x4_t w = reinterpret_cast<const u32x4_t*>(g)[j];
      if (c != 1.0f) {
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const float a = c * __uint_as_float(w[q4] << 16), b = c * __uint_as_float(w[q4] & 0xffff0000u);
          w[q4] = (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
        }
      }
      reinterpret_cast<u32x4_t*>(o)[j] = w;
    }
    for (long long j = n / 8 * 8 + threadIdx.x; j < n; j += NT) o[j] = c == 1.0f ? g[j] : f32_to_bf16(c * bf16_to_f32(g[j]));
  } else {
    const float* g = reinterpret_cast<const float*>(t.grad[i]) + e0;
    float* o = reinterpret_cast<float*>(t.out[i]) + e0;
    for (long long j = threadIdx.x; j < n / 4; j += NT) {
      float4 w = reinterpret_cast<const float4*>(g)[j];
      w.x *= c; w.y *= c; w.z *= c; w.w *= c;
      reinterpret_cast<float4*>(o)[j] = w;
    }
    for (long long j = n / 4 * 4 + threadIdx.x; j < n; j += NT) o[j] = c * g[j];
  }
}

// Elements per chunk: about 2048 chunks over the list (eight workgroups per CU), at least 4096.
long long chunk_size(long long total) {
  const long long c = (total + 2047) / 2048;
  return std::max<long long>(4096, (c + 2047) / 2048 * 2048);
}

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
      t.n[k] = g[i].n;
      t.bf16[k] = g[i].bf16;
      t.first[k + 1] = t.first[k] + (int)((g[i].n + chunk - 1) / chunk);
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

hipError_t launch_grad_scale(const GradItem* g, int count, const double* sums, int nsums, float max_norm, float* norm,
                             hipStream_t s) {
  const long long chunk = chunk_size(total_elements(g, count));
  return for_tables(g, count, chunk, [&](const GradTable& t) {
    grad_scale_kernel<<<dim3(t.first[t.count]), dim3(NT), 0, s>>>(t, chunk, sums, nsums, max_norm, norm);
    return hipGetLastError();
  });
}

}  // namespace moe
