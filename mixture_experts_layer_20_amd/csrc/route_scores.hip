// Routing by scores: softmax or sigmoid scores of the router's logits, a bias that takes part in the
// choice alone (it balances the experts' loads without touching the gates), expert groups of which each
// token may use some, top-k, renormalised and scaled gates; and the gradient of the gates.
//
//   s = sigmoid(l) or softmax(l);  c = s + bias
//   a group's score: the sum of its two largest c; the topk_groups best groups are open
//   chosen: the k largest c of the open groups;  gate = s (/ sum of the chosen s) * scale
//
// The choice turns floats into integers, so it is made on the exact values: without a bias the order of c
// is the order of the logits; with one c is formed in fp32, and a token whose order has two neighbours
// closer than the fp32 scores' error (2^-18 relative to 1 and to c, several times what exp, the sum and
// the division can be off) is decided again in double.  That is one token in a hundred or so; all of them
// in double would cost an fp64 exponential and division for each of T E scores.
//
// Gates of sigmoid scores are formed from exp(min(l, 0) - m) / (1 + exp(-|l|)), m the largest min(l, 0)
// of the chosen, so that they have a sum to divide by when every chosen score underflows.  Where all of a
// token's chosen scores are zero (logits of -inf), its gates are zero.
#include "train_step.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr float NEAR = 0x1p-18f;

// Values as unsigned codes in their order, NaN below every number, -0 equal to +0.
__device__ __forceinline__ uint32_t order_code(float v) {
  uint32_t b = __float_as_uint(v);
  b = b == 0x80000000u ? 0u : b;
  const uint32_t flip = (uint32_t)((int32_t)b >> 31) | 0x80000000u;
  return (b & 0x7fffffffu) > 0x7f800000u ? 0u : b ^ flip;
}
__device__ __forceinline__ uint64_t order_code(double v) {
  uint64_t b = (uint64_t)__double_as_longlong(v);
  b = b == 0x8000000000000000ull ? 0ull : b;
  const uint64_t flip = (uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull;
  return (b & 0x7fffffffffffffffull) > 0x7ff0000000000000ull ? 0ull : b ^ flip;
}
__device__ __forceinline__ float code_value(uint32_t code) {
  if (code == 0u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(code & 0x80000000u ? code & 0x7fffffffu : ~code);
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// The lanes of a token exchange values through LDS; they are lanes of one wave.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int CTRL>
__device__ __forceinline__ uint64_t max_dpp(uint64_t key) {
  const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)key, CTRL, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(key >> 32), CTRL, 0xf, 0xf, false);
  const uint64_t o = ((uint64_t)hi << 32) | lo;
  return o > key ? o : key;
}
// The largest key of the token's L lanes, in every one of them.
template <int L>
__device__ __forceinline__ uint64_t token_max(uint64_t best) {
  best = max_dpp<0xB1>(best);    // quad_perm 1,0,3,2
  best = max_dpp<0x4E>(best);    // quad_perm 2,3,0,1
  best = max_dpp<0x124>(best);   // row_ror 4
  best = max_dpp<0x128>(best);   // row_ror 8
  if constexpr (L == 32) {
    const uint32_t lo = __shfl_xor((int)(uint32_t)best, 16, 64);
    const uint32_t hi = __shfl_xor((int)(uint32_t)(best >> 32), 16, 64);
    const uint64_t o = ((uint64_t)hi << 32) | lo;
    best = o > best ? o : best;
  }
  return best;
}
template <int L, typename R>
__device__ __forceinline__ R token_sum(R v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
template <int L>
__device__ __forceinline__ float token_maxf(float v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}

// Lane j of a token holds experts j, j + L, ...
template <int L, int S, typename R>
__device__ __forceinline__ void token_scores(const RouteScores& r, int j, const float (&l)[S], R (&sc)[S]) {
  if (r.sigmoid) {
#pragma unroll
    for (int s = 0; s < S; ++s) sc[s] = R(1) / (R(1) + exp_of(-(R)l[s]));
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (j + s * L < r.E) top = fmaxf(top, l[s]);
  top = token_maxf<L>(top);
  if (top == -INFINITY) top = 0.0f;   // every logit is: all scores are zero
  R sum = 0;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    sc[s] = j + s * L < r.E ? exp_of((R)l[s] - (R)top) : R(0);
    sum += sc[s];
  }
  sum = token_sum<L>(sum);
  const R inv = sum > R(0) ? R(1) / sum : (sum == R(0) ? R(0) : sum);
#pragma unroll
  for (int s = 0; s < S; ++s) sc[s] = sc[s] * inv;
}

// The open groups of a token, as a flag for each in `open`, from the selection scores c in `cs`.  Returns
// whether the border between open and shut groups is nearer than fp32 scores tell.  q lanes walk a group
// (a power of two, at most L / groups); gsc holds the groups' scores.
template <int L, typename R>
__device__ __forceinline__ bool open_groups(const RouteScores& r, int j, const R* cs, R* gsc, uint8_t* open) {
  const int size = r.E / r.groups;
  int q = 1;
  while (q * 2 * r.groups <= L) q *= 2;
  const int sub = j % q;
  for (int g0 = 0; g0 < r.groups; g0 += L / q) {
    const int g = g0 + j / q;
    R a = -INFINITY, b = -INFINITY;   // the two largest; a NaN is none
    if (g < r.groups) {
      for (int i = sub; i < size; i += q) {
        const R c = cs[g * size + i];
        if (c > a) {
          b = a;
          a = c;
        } else if (c > b) {
          b = c;
        }
      }
    }
    for (int off = 1; off < q; off *= 2) {
      const R oa = __shfl_xor(a, off, 64), ob = __shfl_xor(b, off, 64);
      const R lo = a > oa ? oa : a;
      a = a > oa ? a : oa;
      b = b > ob ? b : ob;
      b = b > lo ? b : lo;
    }
    if (sub == 0 && g < r.groups) gsc[g] = size > 1 ? a + b : a;
  }
  wave_fence();
  R least = INFINITY, most = -INFINITY;   // of the open groups, of the shut ones
  for (int g = j; g < r.groups; g += L) {
    const auto mine = order_code(gsc[g]);
    int rank = 0;
    for (int o = 0; o < r.groups; ++o) {
      const auto other = order_code(gsc[o]);
      rank += other > mine || (other == mine && o < g) ? 1 : 0;
    }
    open[g] = rank < r.topk_groups;
    if (rank < r.topk_groups) least = gsc[g] < least ? gsc[g] : least;
    else most = gsc[g] > most ? gsc[g] : most;
  }
  wave_fence();
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) {
    const R a = __shfl_xor(least, off, 64), b = __shfl_xor(most, off, 64);
    least = a < least ? a : least;
    most = b > most ? b : most;
  }
  if (r.topk_groups == r.groups) return false;
  return !(least - most > R(2) * NEAR * (R(2) + (least < 0 ? -least : least) + (most < 0 ? -most : most)));
}

// A selection key: the value's code above the complement of the expert, so that of equal values the lower
// expert is the larger key; 0 is below every one.
__device__ __forceinline__ uint64_t select_key(float v, int e) { return ((uint64_t)order_code(v) << 32) | (uint32_t)~e; }

// The k largest values of a token, one after the other; lane r of the token keeps the r-th expert.  `near`
// (wanted where `check`): whether two neighbours of the order, the last chosen and the first left among
// them, are nearer than fp32 scores tell.
template <int L, int S>
__device__ __forceinline__ int choose(int k, int j, const float (&v)[S], uint32_t shut, int E, bool check, bool& near) {
  uint64_t key[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = j + s * L;
    key[s] = e < E && !(shut >> s & 1u) ? select_key(v[s], e) : 0ull;
  }
  uint64_t mine = 0;
  float before = 0.0f;
  const int rounds = check ? k + 1 : k;
  for (int r = 0; r < rounds; ++r) {
    uint64_t best = key[0];
#pragma unroll
    for (int s = 1; s < S; ++s) best = key[s] > best ? key[s] : best;
    best = token_max<L>(best);
    if (check && best != 0ull) {
      const float now = code_value((uint32_t)(best >> 32));
      if (r > 0 && !(before - now > NEAR * (2.0f + fabsf(before) + fabsf(now)))) near = true;
      before = now;
    }
#pragma unroll
    for (int s = 0; s < S; ++s) key[s] = key[s] == best ? 0ull : key[s];
    if (j == r) mine = best;
  }
  return (int)~(uint32_t)mine;
}

// The same in double.
template <int L, int S>
__device__ __forceinline__ int choose(int k, int j, const double (&v)[S], uint32_t shut, int E) {
  uint64_t code[S];
  uint32_t taken = shut;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    code[s] = order_code(v[s]);
    if (j + s * L >= E) taken |= 1u << s;
  }
  int mine = 0;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    int at = 0x7fffffff;   // no expert
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (!(taken >> s & 1u) && (at == 0x7fffffff || code[s] > best)) {
        best = code[s];
        at = j + s * L;
      }
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) {
      const uint64_t ob = (uint64_t)__shfl_xor((long long)best, off, 64);
      const int oa = __shfl_xor(at, off, 64);
      if (oa != 0x7fffffff && (at == 0x7fffffff || ob > best || (ob == best && oa < at))) {
        best = ob;
        at = oa;
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (j + s * L == at) taken |= 1u << s;
    if (j == r) mine = at;
  }
  return mine;
}

// Gates of the chosen experts: lane j < k of the token has the logit l of the j-th; lanes j >= k have none.
// top, sum: the largest of all the token's logits and the sum of exp(l - top) (softmax, not renormalised).
__device__ __forceinline__ float chosen_gate(const RouteScores& r, bool has, float l, float top, float sum) {
  if (r.sigmoid) {
    const float under = fminf(l, 0.0f), over = 1.0f + expf(-fabsf(l));
    if (!r.renormalize) return r.scale * (expf(under) / over);
    float m = has ? under : -INFINITY;
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    if (m == -INFINITY) m = 0.0f;
    const float w = has ? expf(under - m) / over : 0.0f;
    float total = w;
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) total += __shfl_xor(total, off, 64);
    return total == 0.0f ? 0.0f : r.scale * (w / total);
  }
  if (r.renormalize) {
    float m = has ? l : -INFINITY;
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    if (m == -INFINITY) m = 0.0f;
    const float w = has ? expf(l - m) : 0.0f;
    float total = w;
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) total += __shfl_xor(total, off, 64);
    return total == 0.0f ? 0.0f : r.scale * (w / total);
  }
  return sum == 0.0f ? 0.0f : r.scale * (expf(l - top) / sum);
}

template <int L, int S>
__global__ __launch_bounds__(256) void route_scores_kernel(RouteScores r, int32_t* topk_idx, float* topk_gate) {
  constexpr int TOK = 256 / L, EMAX = L * S;
  __shared__ float logit_s[TOK][EMAX];
  __shared__ double score_s[TOK][EMAX];   // the groups' walk: floats first, doubles where they do not tell
  __shared__ double group_s[TOK][EMAX];
  __shared__ uint8_t open_s[TOK][EMAX];
  const long long gl = (long long)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(gl / L), j = (int)(gl % L), slot = threadIdx.x / L;
  if (__builtin_amdgcn_readfirstlane(t) >= r.T) return;   // the wave's first token is past T
  const int tc = min(t, r.T - 1);
  float l[S], b[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int e = min(j + s * L, r.E - 1);
    l[s] = r.logits[(size_t)tc * r.E + e];
    b[s] = r.bias ? r.bias[e] : 0.0f;
  }
#pragma unroll
  for (int s = 0; s < S; ++s) logit_s[slot][j + s * L] = l[s];
  const bool grouped = r.groups > 1, biased = r.bias != nullptr;
  float c[S];
  if (grouped || biased) {
    token_scores<L, S, float>(r, j, l, c);
#pragma unroll
    for (int s = 0; s < S; ++s) c[s] = c[s] + b[s];
  }
  uint32_t shut = 0;
  if (grouped) {
    float* cs = reinterpret_cast<float*>(score_s[slot]);
#pragma unroll
    for (int s = 0; s < S; ++s) cs[j + s * L] = c[s];
    wave_fence();
    const bool near = open_groups<L, float>(r, j, cs, reinterpret_cast<float*>(group_s[slot]), open_s[slot]);
    if (__any(near)) {
      double cd[S];
      token_scores<L, S, double>(r, j, l, cd);
      wave_fence();
      if (near) {
#pragma unroll
        for (int s = 0; s < S; ++s) score_s[slot][j + s * L] = cd[s] + (double)b[s];
      }
      wave_fence();
      if (near) open_groups<L, double>(r, j, score_s[slot], group_s[slot], open_s[slot]);
    }
    wave_fence();
    const int size = r.E / r.groups;
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (j + s * L < r.E && !open_s[slot][(j + s * L) / size]) shut |= 1u << s;
  }
  bool near = false;
  int mine;
  if (biased) {
    mine = choose<L, S>(r.k, j, c, shut, r.E, true, near);
    if (__any(near)) {
      double cd[S];
      token_scores<L, S, double>(r, j, l, cd);
#pragma unroll
      for (int s = 0; s < S; ++s) cd[s] = cd[s] + (double)b[s];
      const int again = choose<L, S>(r.k, j, cd, shut, r.E);
      mine = near ? again : mine;
    }
  } else {
    mine = choose<L, S>(r.k, j, l, shut, r.E, false, near);
  }
  float top = 0.0f, sum = 0.0f;
  if (!r.sigmoid && !r.renormalize) {
    top = -INFINITY;
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (j + s * L < r.E) top = fmaxf(top, l[s]);
    top = token_maxf<L>(top);
    if (top == -INFINITY) top = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (j + s * L < r.E) sum += expf(l[s] - top);
    sum = token_sum<L>(sum);
  }
  wave_fence();
  const bool has = j < r.k;
  const float lm = has ? logit_s[slot][mine] : 0.0f;
  const float gate = chosen_gate(r, has, lm, top, sum);
  if (t < r.T && has) {
    topk_idx[(size_t)t * r.k + j] = mine;
    topk_gate[(size_t)t * r.k + j] = gate;
  }
}

// bias + rate sign(mean count - count): counts are whole numbers, so their mean is compared exactly.
__global__ __launch_bounds__(256) void route_bias_kernel(const int32_t* counts, int E, float rate, const float* bias,
                                                         float* out) {
  __shared__ long long part[4];
  const int e = threadIdx.x;
  const long long n = e < E ? counts[e] : 0;
  long long sum = n;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if ((e & 63) == 0) part[e >> 6] = sum;
  __syncthreads();
  const long long total = part[0] + part[1] + part[2] + part[3];
  if (e < E) out[e] = bias[e] + (n * E < total ? rate : n * E > total ? -rate : 0.0f);
}


// ------------------------------------------------------------------------------------------
// Backward.  With g the gates without the scale, dg their gradient, h_j = scale g_j:
//   sigmoid, renormalised   dl_j = (1 - s_j) h_j (dg_j - sum_i g_i dg_i)
//   softmax, renormalised   dl_j =           h_j (dg_j - sum_i g_i dg_i)
//   sigmoid                 dl_j = (1 - s_j) h_j dg_j
//   softmax                 dl_e = [e chosen] h_e dg_e - p_e sum_i h_i dg_i, for every e
// The renormalised gates sum to one, so dg_j - sum_i g_i dg_i is formed as sum_i g_i (dg_j - dg_i), which
// has no cancellation of large terms.

// Logit gradients of the chosen experts [T, k], one thread for each token.
__global__ __launch_bounds__(256) void scores_grad_kernel(RouteScores r, const float* dgate, const int32_t* idx, float* dl) {
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t >= r.T) return;
  float l[8], dg[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {   // loads at a clamped index, never under a condition
    const size_t a = (size_t)t * r.k + min(i, r.k - 1);
    l[i] = r.logits[(size_t)t * r.E + min(max(idx[a], 0), r.E - 1)];
    dg[i] = dgate[a];
  }
  float w[8], rest[8], m = -INFINITY, total = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < r.k) m = fmaxf(m, r.sigmoid ? fminf(l[i], 0.0f) : l[i]);
  if (m == -INFINITY || !r.renormalize) m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r.sigmoid) {
      const float over = 1.0f + expf(-fabsf(l[i]));
      w[i] = expf(fminf(l[i], 0.0f) - m) / over;
      rest[i] = expf(-fmaxf(l[i], 0.0f)) / over;   // 1 - s
    } else {
      w[i] = expf(l[i] - m);
      rest[i] = 1.0f;
    }
    if (i >= r.k) w[i] = 0.0f;
    total += w[i];
  }
  const float inv = r.renormalize ? (total > 0.0f ? 1.0f / total : 0.0f) : 1.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= r.k) break;
    float d = dg[j];
    if (r.renormalize) {
      d = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) d += (w[i] * inv) * (dg[j] - dg[i]);
    }
    dl[(size_t)t * r.k + j] = r.scale * (w[j] * inv) * rest[j] * d;
  }
}

// Logit gradients of all experts [T, E] (softmax scores as they are), one wave for each token.
__global__ __launch_bounds__(256) void scores_grad_dense_kernel(RouteScores r, const float* dgate, const int32_t* idx,
                                                                float* dl) {
  const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= r.T) return;
  float l[4];
  float top = -INFINITY;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int e = lane + 64 * s;
    l[s] = r.logits[(size_t)t * r.E + min(e, r.E - 1)];
    if (e < r.E) top = fmaxf(top, l[s]);
  }
  top = token_maxf<64>(top);
  if (top == -INFINITY) top = 0.0f;
  float p[4], sum = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    p[s] = lane + 64 * s < r.E ? expf(l[s] - top) : 0.0f;
    sum += p[s];
  }
  sum = token_sum<64>(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  float all = 0.0f;   // sum_i h_i dg_i
  float own[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= r.k) break;
    const int e = idx[(size_t)t * r.k + i];
    const float dg = r.scale * dgate[(size_t)t * r.k + i];
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (e == lane + 64 * s) {
        own[s] = dg;
        all += p[s] * inv * dg;
      }
  }
  all = token_sum<64>(all);
#pragma unroll
  for (int s = 0; s < 4; ++s)
    if (lane + 64 * s < r.E) dl[(size_t)t * r.E + lane + 64 * s] = p[s] * inv * (own[s] - all);
}

inline size_t align256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

size_t route_scores_bwd_ws_bytes(long long T, long long d, int E, int k, bool dense) {
  return align256((size_t)T * (dense ? E : k) * sizeof(float)) +
         (dense ? router_dense_bwd_ws_bytes(T, d, E) : route_bwd_ws_bytes(T, d, E, k));
}

hipError_t launch_route_scores_bwd(const RouteScores& r, const float* dgate, const int32_t* topk_idx,
                                   const int32_t* offsets, const int32_t* src_row, const void* x, const void* w, int d,
                                   bool bf16, float* dw, void* dx, void* ws, hipStream_t s) {
  const bool dense = route_scores_dense(r.sigmoid, r.renormalize);
  float* dl = reinterpret_cast<float*>(ws);
  void* rest = reinterpret_cast<char*>(ws) + align256((size_t)r.T * (dense ? r.E : r.k) * sizeof(float));
  if (r.T > 0) {
    if (dense) scores_grad_dense_kernel<<<dim3(ceil_div(r.T, 4)), dim3(256), 0, s>>>(r, dgate, topk_idx, dl);
    else scores_grad_kernel<<<dim3(ceil_div(r.T, 256)), dim3(256), 0, s>>>(r, dgate, topk_idx, dl);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dense) return launch_router_dense_bwd(dl, x, w, r.T, d, r.E, bf16, dw, dx, rest, s);
  // the gates' place empty: what stands in dgate's are the logits' gradients
  return launch_route_bwd(dl, nullptr, topk_idx, offsets, src_row, x, w, r.T, d, r.E, r.k, bf16, dw, dx, rest, s);
}

hipError_t launch_route_scores(const RouteScores& r, int32_t* topk_idx, float* topk_gate, hipStream_t s) {
  if (r.T == 0) return hipSuccess;
  if (r.E <= 64) route_scores_kernel<16, 4><<<dim3(ceil_div(r.T, 16)), dim3(256), 0, s>>>(r, topk_idx, topk_gate);
  else if (r.E <= 128) route_scores_kernel<16, 8><<<dim3(ceil_div(r.T, 16)), dim3(256), 0, s>>>(r, topk_idx, topk_gate);
  else route_scores_kernel<32, 8><<<dim3(ceil_div(r.T, 8)), dim3(256), 0, s>>>(r, topk_idx, topk_gate);
  return hipGetLastError();
}

hipError_t launch_route_bias(const int32_t* counts, int E, float rate, const float* bias, float* out, hipStream_t s) {
  route_bias_kernel<<<dim3(1), dim3(256), 0, s>>>(counts, E, rate, bias, out);
  return hipGetLastError();
}

}  // namespace moe
