// The sums of a row of logits, and their gradient, as the kernels on stored rows
// (logprob.cu) and the epilogues of the LM head's product (gemm.cu) compute them.
#pragma once
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "ptx.cuh"
#include "sf_internal.h"

namespace sf {

constexpr float kLog2e = 1.4426950408889634f;
// What a difference of logits is cut to where it multiplies a weight: its
// weight is exp(scale * kFar) = 0 for every scale allowed, and 0 * kFar is 0.
constexpr float kFar = -1e30f;
// What a log probability is cut to where it multiplies its p in a gradient: p is 0
// from -88 on (fp32 without denormals), and the product with the entropy's
// gradient stays finite however large that is (kFar would not: a loss scaled by 2^20
// and a scale of 2^10 already gave 0 times infinity at masked logits).
constexpr float kNoWeight = -128.f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The maximum, the sum and the weighted sum of a set of logits; the sum's
// rounding errors are kept beside it, because log S of a peaked row (S near 1)
// shows them.
struct Sums {
  float m, s, low, t;
};
__device__ __forceinline__ void raise(Sums& a, float m, float c) {
  const float dm = fmaxf(a.m - m, kFar), f = exp2_fast(dm * c);
  a.t = f * fmaf(a.s, dm, a.t);
  a.s *= f;
  a.low *= f;
  a.m = m;
}
__device__ __forceinline__ void add_sum(Sums& a, float s) {
  const float sum = a.s + s, b = sum - a.s;
  a.low += (a.s - (sum - b)) + (s - b);
  a.s = sum;
}
__device__ __forceinline__ Sums merge(Sums a, Sums b, float c) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m, c);
  raise(b, m, c);
  add_sum(a, b.s);
  a.low += b.low;
  a.t += b.t;
  return a;
}
// The sum of N terms.
template <int N>
__device__ __forceinline__ float tree(float (&e)[N]) {
#pragma unroll
  for (int w = N / 2; w > 0; w /= 2)
#pragma unroll
    for (int j = 0; j < w; ++j) e[j] += e[j + w];
  return e[0];
}
// Where a maximum stands alone (its exponential is 1), the tree of its group has
// rounded the group's others beside it, and others are all that log S has.  a.low gets
// the difference, from the logits z of that group, where S is below kAlone; from there
// on the trees lose at most log2(N) 2^-16 of the others.
constexpr float kAlone = 1.f + 1.f / 256;
template <int N>
__device__ __forceinline__ void keep_others(Sums& a, const float (&z)[N], float c) {
  float e[N], others = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    e[j] = exp2_fast((z[j] - a.m) * c);
    others += e[j] == 1.f ? 0.f : e[j];
  }
  a.low += others - (tree(e) - 1.f);
}
// N logits at once: one look at the maximum, and a tree of their exponentials.
// Returns their maximum.  Groups of more than eight are the head's product's, which
// has them but once: they are looked at for keep_others here.  (Octets of a stored row
// are looked at when the row is done; in here their logits take registers that spill,
// 4096 x 128256 bf16 233 us, 204 so.)
template <bool ENT, int N>
__device__ __forceinline__ float add(Sums& a, const float (&z)[N], float c) {
  float m = z[0];
#pragma unroll
  for (int j = 1; j < N; ++j) m = fmaxf(m, z[j]);
  if (m > a.m) raise(a, m, c);
  float e[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float x = z[j] - a.m;
    e[j] = exp2_fast(x * c);
    if (ENT) a.t = fmaf(e[j], fmaxf(x, kFar), a.t);
  }
  add_sum(a, tree(e));
  if constexpr (N > 8) {
    if (m == a.m && a.s < kAlone) keep_others(a, z, c);
  }
  return m;
}

// What a row's sums give.
struct RowStats {
  float m, scale, log_s, lse, entropy;
  bool none;  // nothing above -inf
  // log probability of a logit
  __device__ __forceinline__ float value(float v) const {
    return none ? -__uint_as_float(0x7f800000u) : fmaf(v - m, scale, -log_s);
  }
};
__device__ __forceinline__ RowStats row_stats(const Sums& a, float scale) {
  RowStats r;
  r.m = a.m;
  r.scale = scale;
  r.none = a.s == 0.f;  // it is at least 1 otherwise
  r.log_s = logf(a.s) + a.low / a.s;
  r.lse = r.none ? -__uint_as_float(0x7f800000u) : fmaf(a.m, scale, r.log_s);
  r.entropy = r.none ? 0.f : r.log_s - scale * (a.t / a.s);
  return r;
}

// The sums of the whole warp, in every lane.
__device__ __forceinline__ Sums warp_merge(Sums a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = merge(a, {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                  __shfl_xor_sync(0xffffffffu, a.low, o), __shfl_xor_sync(0xffffffffu, a.t, o)}, c);
  return a;
}

// The gradient of a logit f of a row, scale (dlogp [hot] - p (dlogp + dentropy
// (log p + entropy))), with everything but p and log p taken together:
// p (slope log p + base) [+ hot].
struct RowGrad {
  float lse, scale, slope, base, hot;
  int token;
  bool zero;  // both gradients are 0, or the row holds nothing but -inf
};
__device__ __forceinline__ RowGrad row_grad(const LogprobEpi& a, int64_t row, int vocab, int* err) {
  RowGrad g;
  g.token = a.tokens[row];
  if (g.token >= vocab) {  // outside the vocabulary: reported, and the row ignored
    record_error(err, kDevCeBadLabel);
    g.token = -1;
  }
  const float dl = g.token < 0 ? 0.f : a.dlogp[row], de = a.dentropy ? a.dentropy[row] : 0.f;
  g.lse = a.lse[row];
  g.scale = a.scale;
  g.slope = -a.scale * de;
  g.base = -a.scale * (a.dentropy ? fmaf(de, a.entropy[row], dl) : dl);
  g.hot = a.scale * dl;
  g.zero = (dl == 0.f && de == 0.f) || g.lse == -__uint_as_float(0x7f800000u);
  return g;
}
// N logits from column `at` on, in place.
template <int N>
__device__ __forceinline__ void logit_grads(const RowGrad& g, float (&f)[N], int at) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float lp = fmaf(f[j], g.scale, -g.lse), p = exp2_fast(lp * kLog2e);
    f[j] = p * fmaf(g.slope, fmaxf(lp, kNoWeight), g.base);
  }
  const int hot = g.token - at;
  if (hot >= 0 && hot < N) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j == hot) f[j] += g.hot;
  }
  if (g.zero) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = 0.f;
  }
}

}  // namespace sf
