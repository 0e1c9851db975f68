// Routing by scores: softmax or sigmoid scores of the router's logits, a bias that takes part in the
// choice alone (it balances the experts' loads without touching the gates), expert groups of which each
// token may use some, top-k, renormalised and scaled gates; and the gradient of the gates.
//
//   s = sigmoid(l) or softmax(l);  c = s + bias
//   a group's score: the sum of its two largest c; the topk_groups best groups are open
//   chosen: the k largest c of the open groups;  gate = s (/ sum of the chosen s) * scale
//
// The choice turns floats into integers, so it is made on the exact values: without a bias the order of c
// is the order of the logits; with one c is formed in fp32, and a wave with a token whose order has two
// neighbours closer than that tells is decided again in double; all of them in double would cost an fp64 exponential
// and division for each of T E scores.  With biases that differ it is one token in 200 (128 experts, k 8, logits of
// spread 1 to 6, biases of 0.1 or 0.01), one wave in 50.  Where scores are flat beside the tolerance, which is
// absolute, it is more, and their tokens have no gap behind the k-th that would end the candidates: with biases of
// zero and softmax logits of spread 4 6% of the waves, of spread 6 a third, and sigmoids of spread 6 all of them,
// 26, 33 and 35 us for 8192 tokens where 8.5 is usual.
//
// L lanes a token, S experts a lane in registers, in runs of 4 so that logits are read 16 bytes at a time;
// where the groups are a power of two, a group's experts are those of neighbouring lanes, so its two largest
// and the open groups are found by moves between lanes.  The choice works on 32-bit keys, three bits of which
// are the expert's place in its lane (so that they carry 20 bits of mantissa): every lane sorts its keys once,
// and a round is then a maximum over the lanes' first keys and a step of the winner's queue.
// 8192 tokens of 256 experts in 8 groups with k = 8: 13 us (9 MB, 2 us at the rate of a copy; one token 5.6 us, a
// launch), 2 of them for the waves that are decided again, whose time the launch waits for, 4 the launch; the 700
// instructions of a wave are 5 us where four waves share a SIMD.  The rest is latency, of the k + 2 rounds that
// follow from each other first.  Walking the groups in LDS and taking the k largest of 64-bit keys one after the other
// was 25.
//
// Gates of sigmoid scores are formed from exp(min(l, 0) - m) / (1 + exp(-|l|)), m the largest min(l, 0)
// of the chosen, so that they have a sum to divide by when every chosen score underflows.  Where all of a
// token's chosen scores are zero (logits of -inf), its gates are zero.
#include "train_step.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

// How near two scores a, b may be before fp32 does not tell their order: NEAR (2 + |a| + |b|).  A sigmoid is
// off by 2^-22 (s (1 - s) |l| 2^-23.4 + s (1 - s) 2^-23 of the exponential, 1.5 s 2^-23 of the sum and the
// reciprocal), a softmax by 2^-19 of itself (of its exponential and the sum, whose terms' distances from the
// top weigh ln 256 at most), the sum with the bias by 2^-24 |c|, a key by 2^-20 |c|: for two of them
// 2^-19 + 1.1 2^-20 (|a| + |b|) or less.
constexpr float NEAR = 0x1p-19f;

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
// A key of `choose` to its value, rounded down.
__device__ __forceinline__ float key_value(uint32_t key) {
  const uint32_t code = key & ~7u;
  return code < 0x00800000u ? -INFINITY : __uint_as_float(code & 0x80000000u ? code & 0x7fffffffu : ~code);
}

// The lanes of a token exchange values through LDS; they are lanes of one wave.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The value of the lane with the bits of D other: D = 1, 2 in a quad, 4, 8 by mirrors (the quads, or eights,
// then hold one value), 16 by a swap of rows.
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // rows 0 0 2 2 and 1 1 3 3
    return (threadIdx.x & 16) ? r[0] : r[1];
  } else {
    constexpr int CTRL = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, false);
  }
}
template <int D>
__device__ __forceinline__ float across(float v) { return __uint_as_float(across<D>(__float_as_uint(v))); }
template <int D>
__device__ __forceinline__ uint64_t across(uint64_t v) {
  return ((uint64_t)across<D>((uint32_t)(v >> 32)) << 32) | across<D>((uint32_t)v);
}
template <int D>
__device__ __forceinline__ double across(double v) {
  return __longlong_as_double((long long)across<D>((uint64_t)__double_as_longlong(v)));
}
// op over `lanes` lanes (a power of two up to 32), in every one of them.
template <typename V, typename Op>
__device__ __forceinline__ V over_lanes(int lanes, V v, Op op) {
  if (lanes >= 2) v = op(v, across<1>(v));
  if (lanes >= 4) v = op(v, across<2>(v));
  if (lanes >= 8) v = op(v, across<4>(v));
  if (lanes >= 16) v = op(v, across<8>(v));
  if (lanes >= 32) v = op(v, across<16>(v));
  return v;
}
// Of floats one instruction, which takes the number where the other is a NaN.
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return fmin(a, b); }
struct Max {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a > b ? a : b; }
  __device__ float operator()(float a, float b) const { return larger(a, b); }
  __device__ double operator()(double a, double b) const { return larger(a, b); }
};
struct Min {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a < b ? a : b; }
  __device__ float operator()(float a, float b) const { return smaller(a, b); }
  __device__ double operator()(double a, double b) const { return smaller(a, b); }
};
struct Sum {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a + b; }
};

// Place of a lane's experts: q lanes walk one run of `size` experts (a group; all E where the lanes are not
// dealt to groups), each 4 of them, then the 4 that are 4 q on.
struct Place {
  int q, size, first, sub;   // first: of the lane's run
  __device__ __forceinline__ int in_run(int s) const { return 4 * (sub + q * (s >> 2)) + (s & 3); }
  __device__ __forceinline__ bool has(int s) const { return in_run(s) < size; }
  __device__ __forceinline__ int expert(int s) const { return first + in_run(s); }
};

__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896340736f); }

template <int L, int S>
__device__ __forceinline__ float token_top(const Place& at, const float (&l)[S]) {
  float top = -INFINITY;
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (at.has(s)) top = fmaxf(top, l[s]);
  top = over_lanes(L, top, Max());
  return top == -INFINITY ? 0.0f : top;   // every logit is: all scores are zero
}
template <int L, int S>
__device__ __forceinline__ void token_scores(const RouteScores& r, const Place& at, const float (&l)[S], float (&sc)[S]) {
  if (r.sigmoid) {
#pragma unroll
    for (int s = 0; s < S; ++s) sc[s] = __builtin_amdgcn_rcpf(1.0f + exp_of(-l[s]));
    return;
  }
  const float top = token_top<L>(at, l);
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    sc[s] = at.has(s) ? exp_of(l[s] - top) : 0.0f;
    sum += sc[s];
  }
  sum = over_lanes(L, sum, Sum());
  const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
  for (int s = 0; s < S; ++s) sc[s] = sc[s] * inv;
}

__device__ __forceinline__ float finite(float v) { return fminf(fabsf(v), 3.4028234663852886e38f); }
__device__ __forceinline__ double finite(double v) { return fmin(fabs(v), 1.7976931348623157e308); }
// Whether the order of high >= low is not told (two values of -inf are equal, -inf is far from a number).
template <typename R>
__device__ __forceinline__ bool nearby(R high, R low, R tolerance) {
  return !(high - low > tolerance * (R(2) + finite(high) + finite(low)));
}
// How far a group's score may be off, from its two largest: what they lose goes by their own sizes, however small
// their sum is.  Two sigmoids 2^-21, or softmax scores, which sum to 1 at most, 2^-19; the sums with the bias and
// the group's 2^-23 (|a| + |b|).  Twice that.
template <typename R>
__device__ __forceinline__ R group_error(R a, R b) { return R(2 * NEAR) + R(0x1p-22f) * (finite(a) + finite(b)); }

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) { return (uint32_t)__shfl((int)v, lane, 64); }
__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) { return (uint64_t)__shfl((long long)v, lane, 64); }

// The two largest of a lane's values; a NaN is none.
template <typename R>
struct TopTwo {
  R a = -INFINITY, b = -INFINITY;
  __device__ __forceinline__ void take(R c) {
    const R v = larger(c, R(-INFINITY));
    b = larger(b, smaller(a, v));
    a = larger(a, v);
  }
};
// Whether this lane's group is open, from the two largest selection scores of its experts here; at.q lanes a
// group.
template <int L, typename R>
__device__ __forceinline__ bool group_open(const RouteScores& r, const Place& at, int j, TopTwo<R>& top, bool& near) {
  R &a = top.a, &b = top.b;   // of the lane, then of its group
  auto join = [&](R oa, R ob) {
    b = Max()(Max()(b, ob), Min()(a, oa));
    a = Max()(a, oa);
  };
  if (at.q >= 2) join(across<1>(a), across<1>(b));
  if (at.q >= 4) join(across<2>(a), across<2>(b));
  if (at.q >= 8) join(across<4>(a), across<4>(b));
  if (at.q >= 16) join(across<8>(a), across<8>(b));
  const R score = at.size > 1 ? a + b : a;
  const auto mine = order_code(score);
  const int g = j / at.q, lane0 = ((int)threadIdx.x & 63) - j;
  int rank = 0;
  for (int o = 0; o < r.groups; ++o) {
    const auto other = lane_value(mine, lane0 + o * at.q);
    rank += other > mine || (other == mine && o < g) ? 1 : 0;
  }
  const bool open = rank < r.topk_groups;
  if (r.topk_groups < r.groups) {
    const bool number = score == score;
    const R off = group_error<R>(a, at.size > 1 ? b : a);
    const R least = over_lanes(L, open && number ? score - off : R(INFINITY), Min());
    const R most = over_lanes(L, !open && number ? score + off : R(-INFINITY), Max());
    near = !(least > most);
  }
  return open;
}

// The same for any number of groups: cs holds the token's selection scores, gsc the groups' scores, goff how far
// these may be off and open their flags, in LDS.  q lanes walk a group (a power of two, at most L / groups).
template <int L, typename R>
__device__ __forceinline__ void walk_groups(const RouteScores& r, int j, const R* cs, R* gsc, float* goff, uint8_t* open, bool& near) {
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
      b = Max()(Max()(b, ob), Min()(a, oa));
      a = Max()(a, oa);
    }
    if (sub == 0 && g < r.groups) {
      gsc[g] = size > 1 ? a + b : a;
      goff[g] = group_error<float>((float)a, (float)(size > 1 ? b : a));
    }
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
    const R low = gsc[g] - goff[g], high = gsc[g] + goff[g];
    if (rank < r.topk_groups) least = low < least ? low : least;
    else most = high > most ? high : most;
  }
  wave_fence();
  least = over_lanes(L, least, Min());
  most = over_lanes(L, most, Max());
  near = r.topk_groups < r.groups && !(least > most);
}

// Selection scores in double, one at a time from a token's logits in LDS: the code of one exponential, which
// few waves come to, is loaded faster than that of eight.
template <int L>
struct Exact {
  const RouteScores& r;
  const float* logits;
  double top = 0.0, inv = 1.0;
  __device__ __forceinline__ Exact(const RouteScores& r_, const float* logits_, int j) : r(r_), logits(logits_) {
    if (r.sigmoid) return;
    float most = -INFINITY;
    for (int e = j; e < r.E; e += L) most = fmaxf(most, logits[e]);
    most = over_lanes(L, most, Max());
    top = most == -INFINITY ? 0.0 : (double)most;
    double sum = 0.0;
#pragma unroll 1
    for (int e = j; e < r.E; e += L) sum += exp((double)logits[e] - top);
    sum = over_lanes(L, sum, Sum());
    inv = sum == 0.0 ? 0.0 : 1.0 / sum;
  }
  __device__ __forceinline__ double operator()(int e) const {
    const double v = exp(r.sigmoid ? -(double)logits[e] : (double)logits[e] - top);
    return (r.sigmoid ? 1.0 / (1.0 + v) : v * inv) + (r.bias ? (double)r.bias[e] : 0.0);
  }
};

template <int S>
__device__ __forceinline__ void sort_down(uint32_t (&key)[S]) {
  auto pair = [&](int a, int b) {
    const uint32_t high = max(key[a], key[b]);
    key[b] = min(key[a], key[b]);
    key[a] = high;
  };
  auto four = [&](int o) {
    pair(o, o + 1), pair(o + 2, o + 3), pair(o, o + 2), pair(o + 1, o + 3), pair(o + 1, o + 2);
  };
  four(0);
  if constexpr (S == 8) {   // two sorted fours joined
    four(4);
    pair(0, 4), pair(1, 5), pair(2, 6), pair(3, 7), pair(2, 4), pair(3, 5), pair(1, 2), pair(3, 4), pair(5, 6);
  }
}

// A lane's values as keys in descending order, 0 where there is none.
template <int S>
__device__ __forceinline__ void sorted_keys(const float (&v)[S], uint32_t shut, uint32_t (&key)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s) {   // order_code's order, but a NaN is -inf
    const uint32_t b = __float_as_uint(fmaxf(v[s], -INFINITY) + 0.0f);
    const uint32_t code = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    key[s] = (shut >> s & 1u) ? 0u : (code & ~7u) | (7 - s);
  }
  sort_down<S>(key);
}
template <int S>
__device__ __forceinline__ void take_first(const Place& at, uint32_t (&key)[S], uint8_t* chosen) {
  *chosen = (uint8_t)at.expert(7 - (int)(key[0] & 7u));
#pragma unroll
  for (int s = 0; s + 1 < S; ++s) key[s] = key[s + 1];
  key[S - 1] = 0u;
}
// The n largest values of a token, largest first: their experts to LDS, and their keys, lane i that of the i-th
// (0: none).  Of equal keys the lower lane's comes first.
template <int L, int S>
__device__ __forceinline__ uint32_t choose(int n, int j, const Place& at, const float (&v)[S], uint32_t shut,
                                           uint8_t* chosen) {
  uint32_t key[S];
  sorted_keys<S>(v, shut, key);
  uint32_t mine = 0;
  const int lane0 = ((int)threadIdx.x & 63) - j;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const uint32_t top = over_lanes(L, key[0], Max());
    const unsigned long long same = __ballot(key[0] == top);
    const uint32_t here = (lane0 & 32 ? (uint32_t)(same >> 32) : (uint32_t)same) >> (lane0 & 31);
    if (j == __ffs((int)here) - 1 && top != 0u) take_first<S>(at, key, chosen + i);
    mine = j == i ? top : mine;
  }
  wave_fence();
  return mine;
}

// The order of n candidates (the largest by their keys, which may not tell their order) from exact values; lane i
// returns the i-th expert.
template <int L, typename Value>
__device__ __forceinline__ int order_exactly(int n, int most, int j, uint8_t* chosen, const Value& value) {
  const bool has = j < n;
  const int own = has ? chosen[j] : 0;
  const uint64_t code = has ? value(own) : 0ull;
  int rank = 0;
  const int lane0 = ((int)threadIdx.x & 63) - j;
#pragma unroll 4
  for (int o = 0; o < most; ++o) {
    const uint64_t other = (uint64_t)__shfl((long long)code, lane0 + o, 64);
    const int at_o = __shfl(own, lane0 + o, 64);
    rank += o < n && (other > code || (other == code && at_o < own)) ? 1 : 0;
  }
  wave_fence();
  if (has) chosen[rank] = (uint8_t)own;
  wave_fence();
  return chosen[j & 15];
}

// The k experts of the largest exact values, whatever is near; of equal values the lower expert first.
template <int L, int S, typename Value>
__device__ __forceinline__ int choose_exactly(int k, int j, const Place& at, uint32_t shut, const Value& value) {
  int mine = 0;
#pragma unroll 1
  for (int i = 0; i < k; ++i) {
    uint64_t best = 0;
    uint32_t expert = ~0u, place = 0;
#pragma unroll 1
    for (uint32_t left = ~shut & ((1u << S) - 1u); left != 0u; left &= left - 1u) {
      const int s = __ffs((int)left) - 1;
      const uint64_t code = value(at.expert(s));
      if (expert == ~0u || code > best) {
        best = code;
        expert = (uint32_t)at.expert(s);
        place = (uint32_t)s;
      }
    }
    const uint64_t top = over_lanes(L, best, Max());
    const uint32_t first = over_lanes(L, best == top ? expert : ~0u, Min());
    if (expert == first) shut |= 1u << place;
    if (j == i) mine = (int)first;
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

// 4 floats at p + i, whose index may be past the run: those of the last ones that are not.
__device__ __forceinline__ void load4(const float* p, int i, int size, bool whole, float* out) {
  if (whole) {   // runs of whole fours at 16 bytes
    const float4 v = *reinterpret_cast<const float4*>(p + min(i, size - 4));
    out[0] = v.x;
    out[1] = v.y;
    out[2] = v.z;
    out[3] = v.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = p[min(i + e, size - 1)];
  }
}

// WALK: the groups are not a power of two that L lanes can be dealt to.
template <int L, int S, bool WALK>
__global__ __launch_bounds__(256) void route_scores_kernel(RouteScores r, int32_t* topk_idx, float* topk_gate) {
  constexpr int TOK = 256 / L, EMAX = L * S, WTOK = WALK ? TOK : 1, WMAX = WALK ? EMAX : 1;
  __shared__ __attribute__((aligned(16))) float logit_s[TOK][EMAX];
  __shared__ uint8_t chosen_s[TOK][16];
  __shared__ double score_s[WTOK][WMAX];   // the groups' walk: floats first, doubles where they do not tell
  __shared__ double group_s[WTOK][WMAX];
  __shared__ float off_s[WTOK][WMAX];
  __shared__ uint8_t open_s[WTOK][WMAX];
  const long long gl = (long long)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(gl / L), j = (int)(gl % L), slot = threadIdx.x / L;
  if (__builtin_amdgcn_readfirstlane(t) >= r.T) return;   // the wave's first token is past T
  const int tc = min(t, r.T - 1);
  Place at;
  const int runs = WALK ? 1 : r.groups;
  at.q = L / runs;
  at.size = r.E / runs;
  at.first = (j / at.q) * at.size;
  at.sub = j % at.q;
  const bool grouped = r.groups > 1, biased = r.bias != nullptr;
  float l[S], b[S];
  uint32_t shut = 0;
#pragma unroll
  for (int s = 0; s < S; s += 4) {
    load4(r.logits + (size_t)tc * r.E + at.first, at.in_run(s), at.size, r.whole, l + s);
    if (biased) load4(r.bias + at.first, at.in_run(s), at.size, r.whole, b + s);
  }
  if (r.whole) {
#pragma unroll
    for (int s = 0; s < S; s += 4)
      if (at.has(s)) *reinterpret_cast<float4*>(&logit_s[slot][at.expert(s)]) = make_float4(l[s], l[s + 1], l[s + 2], l[s + 3]);
  } else {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (at.has(s)) logit_s[slot][at.expert(s)] = l[s];
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (!at.has(s)) shut |= 1u << s;
    if (!biased) b[s] = 0.0f;
  }
  float c[S];
  if (grouped || biased) {
    token_scores<L, S>(r, at, l, c);
#pragma unroll
    for (int s = 0; s < S; ++s) c[s] = c[s] + b[s];
  }
  if (grouped) {
    bool near = false;
    if constexpr (WALK) {
      float* cs = reinterpret_cast<float*>(score_s[slot]);
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (at.has(s)) cs[at.expert(s)] = c[s];
      wave_fence();
      walk_groups<L, float>(r, j, cs, reinterpret_cast<float*>(group_s[slot]), off_s[slot], open_s[slot], near);
      if (__any(near)) {
        const Exact<L> exact(r, logit_s[slot], j);
        wave_fence();
        for (int e = j; e < r.E; e += L) score_s[slot][e] = exact(e);
        wave_fence();
        walk_groups<L, double>(r, j, score_s[slot], group_s[slot], off_s[slot], open_s[slot], near);
      }
      const int size = r.E / r.groups;
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (at.has(s) && !open_s[slot][at.expert(s) / size]) shut |= 1u << s;
    } else {
      TopTwo<float> two;
#pragma unroll
      for (int s = 0; s < S; ++s) two.take(at.has(s) ? c[s] : -INFINITY);
      bool open = group_open<L, float>(r, at, j, two, near);
      if (__any(near)) {
        wave_fence();
        const Exact<L> exact(r, logit_s[slot], j);
        // exactly, of those that may be among the group's two largest: the fp32 scores' second, joined over
        // its lanes, is off by less than the margin
        uint32_t left = 0;
#pragma unroll
        for (int s = 0; s < S; ++s)
          if (at.has(s) && !(c[s] < two.b - 2 * NEAR * (2.0f + finite(two.b)))) left |= 1u << s;
        TopTwo<double> both;
#pragma unroll 1
        for (; left != 0u; left &= left - 1u) both.take(exact(at.expert(__ffs((int)left) - 1)));
        open = group_open<L, double>(r, at, j, both, near);
      }
      if (!open) shut = ~0u;
    }
  }
  float v[S];   // what is ordered
#pragma unroll
  for (int s = 0; s < S; ++s) v[s] = biased ? c[s] : l[s];
  uint8_t* chosen = chosen_s[slot];
  const uint32_t key = choose<L, S>(r.k + 2, j, at, v, shut, chosen);
  int mine = chosen[j & 15];
  const uint32_t next = (uint32_t)__shfl_down((int)key, 1, 64);
  const bool gap = next == 0u || (biased ? !nearby<float>(key_value(key), key_value(next), NEAR) : key >> 3 != next >> 3);
  if (__any(j < r.k && !gap)) {   // the keys do not tell some token's order
    const Exact<L> exact(r, logit_s[slot], j);
    auto value = [&](int e) { return biased ? order_code(exact(e)) : (uint64_t)order_code(logit_s[slot][e]) << 32; };
    // the candidates end at a gap behind the k-th, or behind one more
    const int n = (int)over_lanes(L, gap && j >= r.k - 1 && j <= r.k ? (uint32_t)j : 64u, Min()) + 1;
    if (__all(n <= r.k + 1)) mine = order_exactly<L>(n, r.k + 1, j, chosen, value);
    else mine = choose_exactly<L, S>(r.k, j, at, shut, value);
  }
  float top = 0.0f, sum = 0.0f;
  if (!r.sigmoid && !r.renormalize) {
    top = token_top<L>(at, l);
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (at.has(s)) sum += expf(l[s] - top);
    sum = over_lanes(L, sum, Sum());
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
__global__ __launch_bounds__(64) void scores_grad_kernel(RouteScores r, const float* dgate, const int32_t* idx, float* dl) {
  const int t = blockIdx.x * 64 + threadIdx.x;
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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
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
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  if (top == -INFINITY) top = 0.0f;
  float p[4], sum = 0.0f;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    p[s] = lane + 64 * s < r.E ? expf(l[s] - top) : 0.0f;
    sum += p[s];
  }
  sum = wave_sum(sum);
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
        own[s] += dg;
        all += p[s] * inv * dg;
      }
  }
  all = wave_sum(all);
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

bool route_scores_fits(long long T, int E) { return T * (E <= 128 ? 16 : 32) <= (1LL << 32) - 256; }

bool route_scores_bwd_fits(long long T, long long d, int E, int k, bool dense, bool bf16) {
  if (dense) return T <= (1LL << 26) - 4 && router_dense_bwd_fits(T, d, E);   // a wave of the gates' gradient a token
  return route_bwd_fits(T, d, E, k, bf16);
}

hipError_t launch_route_scores_bwd(const RouteScores& r, const float* dgate, const int32_t* topk_idx,
                                   const int32_t* offsets, const int32_t* src_row, const void* x, const void* w, int d,
                                   bool bf16, float* dw, void* dx, void* ws, hipStream_t s) {
  const bool dense = route_scores_dense(r.sigmoid, r.renormalize);
  float* dl = reinterpret_cast<float*>(ws);
  void* rest = reinterpret_cast<char*>(ws) + align256((size_t)r.T * (dense ? r.E : r.k) * sizeof(float));
  if (r.T > 0) {
    if (dense) scores_grad_dense_kernel<<<dim3(ceil_div(r.T, 4)), dim3(256), 0, s>>>(r, dgate, topk_idx, dl);
    else scores_grad_kernel<<<dim3(ceil_div(r.T, 64)), dim3(64), 0, s>>>(r, dgate, topk_idx, dl);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dense) return launch_router_dense_bwd(dl, x, w, r.T, d, r.E, bf16, dw, dx, rest, s);
  // the gates' place empty: what stands in dgate's are the logits' gradients
  return launch_route_bwd(dl, nullptr, topk_idx, offsets, src_row, x, w, r.T, d, r.E, r.k, bf16, dw, dx, rest, s);
}

template <int L, int S>
static void launch_scores(const RouteScores& r, int32_t* topk_idx, float* topk_gate, hipStream_t s) {
  const dim3 grid(ceil_div(r.T, 256 / L));
  if ((r.groups & (r.groups - 1)) == 0 && r.groups <= L) route_scores_kernel<L, S, false><<<grid, dim3(256), 0, s>>>(r, topk_idx, topk_gate);
  else route_scores_kernel<L, S, true><<<grid, dim3(256), 0, s>>>(r, topk_idx, topk_gate);
}

hipError_t launch_route_scores(const RouteScores& r0, int32_t* topk_idx, float* topk_gate, hipStream_t s) {
  if (r0.T == 0) return hipSuccess;
  RouteScores r = r0;
  const bool dealt = (r.groups & (r.groups - 1)) == 0;
  r.whole = (r.E / (dealt ? r.groups : 1)) % 4 == 0;   // with E: runs of whole fours, at 16 bytes
  if (r.E <= 64) launch_scores<16, 4>(r, topk_idx, topk_gate, s);
  else if (r.E <= 128) launch_scores<16, 8>(r, topk_idx, topk_gate, s);
  else launch_scores<32, 8>(r, topk_idx, topk_gate, s);
  return hipGetLastError();
}

hipError_t launch_route_bias(const int32_t* counts, int E, float rate, const float* bias, float* out, hipStream_t s) {
  route_bias_kernel<<<dim3(1), dim3(256), 0, s>>>(counts, E, rate, bias, out);
  return hipGetLastError();
}

}  // namespace moe
