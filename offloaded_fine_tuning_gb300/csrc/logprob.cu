// Log probabilities of given tokens from rows of logits, with the entropy of
// each row and its most likely alternatives, and their gradient.
//
// With t = scale * z, m = max t and S = sum exp(t - m):
//   lse = m + log S,  logp = t[token] - lse,
//   entropy = -sum p log p = log S - (sum exp(t - m) (t - m)) / S.
// Both terms of the last line are at least 0, so a peaked row loses nothing to
// cancellation.  m and S, and the weighted sum T with them, are carried online:
// a larger maximum M turns (m, S, T) into (M, f S, f (T + S (m - M))), f =
// exp(m - M).  Differences are taken before the scale is applied, so that large
// logits lose no more than their own rounding.
//
// A logit of -inf has probability 0 (p log p = 0).  A row of nothing else has
// lse, logp and every top value -inf and entropy 0.  A NaN or +inf makes the
// sums of its row NaN and its top ids -1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cstdint>

#include "launch.cuh"
#include "ptx.cuh"
#include "sf.h"
#include "sf_internal.h"

namespace sf {

namespace {

typedef __nv_bfloat16 bf16;

constexpr float kLog2e = 1.4426950408889634f;
// What a difference of logits is cut to where it multiplies a weight: its
// weight is exp(scale * kFar) = 0 for every scale allowed, and 0 * kFar is 0.
constexpr float kFar = -1e30f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct alignas(16) Eight {
  T v[8];
};
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&f)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }

// The maximum, the sum and the weighted sum of a set of logits.
struct Sums {
  float m, s, t;
};
__device__ __forceinline__ void raise(Sums& a, float m, float c) {
  const float dm = fmaxf(a.m - m, kFar), f = exp2_fast(dm * c);
  a.t = f * fmaf(a.s, dm, a.t);
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ void add(Sums& a, float z, float c) {
  const float x = z - a.m, e = exp2_fast(x * c);
  a.s += e;
  a.t = fmaf(e, fmaxf(x, kFar), a.t);
}
__device__ __forceinline__ Sums merge(Sums a, Sums b, float c) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m, c);
  raise(b, m, c);
  return {m, a.s + b.s, a.t + b.t};
}

// The order of the alternatives: larger values first, then lower ids.
__device__ __forceinline__ bool before(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

constexpr int kThreads = 256;

// Forward: a CTA takes a row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    logprob_rows_kernel(const T* __restrict__ z, int64_t ld, const int32_t* __restrict__ tokens, int vocab,
                        float scale, float* __restrict__ logp, float* __restrict__ lse_out,
                        float* __restrict__ entropy, int top, int32_t* __restrict__ ids,
                        float* __restrict__ top_logp, int* err) {
  __shared__ Sums part[kThreads / 32];
  __shared__ float best_v[kThreads / 32];
  __shared__ int best_i[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const T* zr = z + row * ld;
  const float c = scale * kLog2e;
  const int n8 = vocab >> 3;
  Sums a = {-FLT_MAX, 0.f, 0.f};
  for (int i = threadIdx.x; i < n8; i += kThreads) {
    float f[8];
    load8(zr + 8 * i, f);
    float m = f[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, f[j]);
    if (m > a.m) raise(a, m, c);
#pragma unroll
    for (int j = 0; j < 8; ++j) add(a, f[j], c);
  }
  if (8 * n8 + threadIdx.x < vocab) {
    const float f = to_float(zr[8 * n8 + threadIdx.x]);
    if (f > a.m) raise(a, f, c);
    add(a, f, c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = merge(a, {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                  __shfl_xor_sync(0xffffffffu, a.t, o)}, c);
  if (lane == 0) part[warp] = a;
  __syncthreads();
  a = part[0];
  for (int w = 1; w < kThreads / 32; ++w) a = merge(a, part[w], c);
  // s is at least 1 where any logit is above -inf
  const bool none = a.s == 0.f;
  const float log_s = logf(a.s);
  const float minus_inf = -__uint_as_float(0x7f800000u);
  auto value = [&](float v) { return none ? minus_inf : fmaf(v - a.m, scale, -log_s); };
  if (threadIdx.x == 0) {
    int token = tokens[row];
    if (token >= vocab) {  // outside the vocabulary: reported, and the row ignored
      record_error(err, kDevCeBadLabel);
      token = -1;
    }
    logp[row] = token < 0 ? 0.f : value(to_float(zr[token]));
    lse_out[row] = none ? minus_inf : fmaf(a.m, scale, log_s);
    if (entropy) entropy[row] = none ? 0.f : log_s - scale * (a.t / a.s);
  }
  // the alternatives, one after another: the first in order behind the last one
  float last_v = __uint_as_float(0x7f800000u);
  int last_i = -1;
  for (int r = 0; r < top; ++r) {
    float v = minus_inf;
    int at = INT_MAX;
    auto look = [&](float w, int j) {
      if (before(last_v, last_i, w, j) && before(w, j, v, at)) {
        v = w;
        at = j;
      }
    };
    if (a.s == a.s) {
      for (int i = threadIdx.x; i < n8; i += kThreads) {
        float f[8];
        load8(zr + 8 * i, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) look(f[j], 8 * i + j);
      }
      if (8 * n8 + threadIdx.x < vocab) look(to_float(zr[8 * n8 + threadIdx.x]), 8 * n8 + threadIdx.x);
    }
    auto join = [&](float w, int j) {
      if (before(w, j, v, at)) {
        v = w;
        at = j;
      }
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) join(__shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, at, o));
    if (lane == 0) {
      best_v[warp] = v;
      best_i[warp] = at;
    }
    __syncthreads();
    v = best_v[0];
    at = best_i[0];
    for (int w = 1; w < kThreads / 32; ++w) join(best_v[w], best_i[w]);
    __syncthreads();
    last_v = v;
    last_i = at;
    if (threadIdx.x == 0) {
      const bool bad = !(a.s == a.s);
      ids[row * top + r] = bad ? -1 : at;
      top_logp[row * top + r] = bad ? a.s : value(v);
    }
  }
}

// Backward, element by element from the row's lse and entropy:
//   dz = scale (dlogp (1[token] - p) - dentropy p (log p + entropy)).
// A CTA takes kPiece logits of a row.  Rows whose two upstream gradients are
// both 0 (padding) get zeros without being read, rows of -inf too.
constexpr int kPiece = kThreads * 8 * 4;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    logprob_rows_bwd_kernel(const T* z, int64_t ld, const int32_t* __restrict__ tokens, int64_t rows, int vocab,
                            float scale, const float* __restrict__ lse_in, const float* __restrict__ entropy,
                            const float* __restrict__ dlogp, const float* __restrict__ dentropy, bf16* dz,
                            int64_t lddz, int* err) {
  const int pieces = (vocab + kPiece - 1) / kPiece;
  for (int64_t item = blockIdx.x; item < rows * pieces; item += gridDim.x) {
    const int64_t row = item / pieces;
    const int first = (int)(item - row * pieces) * kPiece;
    int token = tokens[row];
    if (token >= vocab) {
      if (threadIdx.x == 0) record_error(err, kDevCeBadLabel);
      token = -1;
    }
    const float lse = lse_in[row];
    const float dl = token < 0 ? 0.f : dlogp[row], de = dentropy ? dentropy[row] : 0.f;
    const float hh = dentropy ? entropy[row] : 0.f;
    const bool zero = (dl == 0.f && de == 0.f) || lse == -__uint_as_float(0x7f800000u);
    const T* zr = z + row * ld;
    bf16* dr = dz + row * lddz;
    auto grad = [&](float f, int at) {
      const float lp = fmaf(f, scale, -lse), p = exp2_fast(lp * kLog2e);
      const float g = fmaf(de, fmaxf(lp, kFar) + hh, dl);
      return scale * fmaf(-p, g, at == token ? dl : 0.f);
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = first + (u * kThreads + threadIdx.x) * 8;
      if (at + 8 <= vocab) {
        float f[8];
        Eight<bf16> o;
        if (zero) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o.v[j] = __float2bfloat16_rn(0.f);
        } else {
          load8(zr + at, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) o.v[j] = __float2bfloat16_rn(grad(f[j], at + j));
        }
        *reinterpret_cast<Eight<bf16>*>(dr + at) = o;
      } else {
        for (int j = at; j < vocab; ++j) dr[j] = __float2bfloat16_rn(zero ? 0.f : grad(to_float(zr[j]), j));
      }
    }
  }
}

}  // namespace

void logprob_rows(const void* z, bool f32, int64_t ld, const int32_t* tokens, int64_t rows, int vocab, float scale,
                  float* logp, float* lse, float* entropy, int top, int32_t* ids, float* top_logp, int* err,
                  cudaStream_t st) {
  if (f32)
    logprob_rows_kernel<<<(unsigned)rows, kThreads, 0, st>>>(static_cast<const float*>(z), ld, tokens, vocab, scale,
                                                             logp, lse, entropy, top, ids, top_logp, err);
  else
    logprob_rows_kernel<<<(unsigned)rows, kThreads, 0, st>>>(static_cast<const bf16*>(z), ld, tokens, vocab, scale,
                                                             logp, lse, entropy, top, ids, top_logp, err);
}

void logprob_rows_bwd(const void* z, bool f32, int64_t ld, const int32_t* tokens, int64_t rows, int vocab,
                      float scale, const float* lse, const float* entropy, const float* dlogp, const float* dentropy,
                      bf16* dz, int64_t lddz, int* err, cudaStream_t st) {
  const int64_t items = rows * ((vocab + kPiece - 1) / kPiece);
  const unsigned grid = (unsigned)(items < INT32_MAX ? items : INT32_MAX);
  if (f32)
    logprob_rows_bwd_kernel<<<grid, kThreads, 0, st>>>(static_cast<const float*>(z), ld, tokens, rows, vocab, scale,
                                                       lse, entropy, dlogp, dentropy, dz, lddz, err);
  else
    logprob_rows_bwd_kernel<<<grid, kThreads, 0, st>>>(static_cast<const bf16*>(z), ld, tokens, rows, vocab, scale,
                                                       lse, entropy, dlogp, dentropy, dz, lddz, err);
}

}  // namespace sf
