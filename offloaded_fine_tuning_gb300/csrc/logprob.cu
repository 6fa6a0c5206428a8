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
#include "logprob.cuh"
#include "ptx.cuh"
#include "sf.h"
#include "sf_internal.h"

namespace sf {

namespace {

typedef __nv_bfloat16 bf16;

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

// The order of the alternatives: larger values first, then lower ids.
struct Logit {
  float v;
  int i;
};
__device__ __forceinline__ bool before(Logit a, Logit b) { return a.v > b.v || (a.v == b.v && a.i < b.i); }

constexpr int kThreads = 256;
constexpr int kList = 512;    // candidates that a CTA holds
constexpr int kGroups = 64;   // sets of threads whose maxima bound the alternatives
constexpr int kMaxCluster = 8;

// keep_others for the sums of a warp of which lane l has added octets first + l,
// first + l + STEP, ... below end, with `mine` the largest logit of a lane (perhaps
// one that belongs to no octet).  The lanes look for the octet among those of the lane
// that holds the maximum: remembered with each new maximum it costs every row
// (16384 x 4096 fp32 90 us, 81 so; 4096 x 128256 bf16 210 and 204).
template <int STEP, typename T>
__device__ __forceinline__ void keep_others_of_warp(Sums& a, float mine, const T* zr, int first, int end, float c) {
  const uint32_t owner = __ballot_sync(0xffffffffu, mine == a.m);  // one lane, or S would be 2
  if (!__any_sync(0xffffffffu, a.s < kAlone) || owner == 0) return;
  Sums alone = {a.m, 0.f, 0.f, 0.f};
  for (int i = first + __ffs(owner) - 1 + (threadIdx.x & 31) * STEP; i < end; i += 32 * STEP) {
    float f[8];
    load8(zr + 8 * i, f);
    float m = f[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, f[j]);
    if (m == a.m) keep_others(alone, f, c);
  }
  a.low += warp_sum(alone.low);
}

// The places that the entries of a list would have were it in order: four
// neighbouring threads count for an entry, and what() gets it with its place.
template <int NT, class F>
__device__ __forceinline__ void places(const Logit* list, int n, F what) {
  const int part = threadIdx.x & 3;
  for (int k = threadIdx.x >> 2; (k & ~7) < n; k += NT / 4) {  // a warp's eight entries together
    const Logit a = k < n ? list[k] : Logit{0.f, 0};
    int r = 0;
    for (int j = part; j < n; j += 4) r += before(list[j], a);
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    r += __shfl_xor_sync(0xffffffffu, r, 2);
    if (part == 0 && k < n) what(a, r);
  }
}

// Forward: a cluster of CTAs (one, or several where there are few rows) of NT
// threads takes a row, each CTA a range of it, and reads it once.
//
// The alternatives come from the threads' own maxima, which the sums need
// anyway: of the maxima of 64 sets of threads the top-th largest, v, is a bound
// that at least `top` logits reach (about 64 log(64 / (64 - top)) of them, 24
// for 20), and only threads whose maximum reaches it can hold such a logit.  A
// thread keeps the maxima of up to SPANS spans of its logits, so that only the
// spans that reach the bound are read again, and what reaches it is put in
// order by counting (4096 x 128256 fp32, 20 alternatives: 383 us with the
// threads' whole ranges read again, which L2 no longer holds, 314 us so).  Where
// more reach it than the list holds (equal logits, masked rows), the top-th of
// those that it does hold is the next bound.  Each such round leaves out at
// least kList - top of them; which ones the list held follows from the order of the
// atomics, what is left in the end does not.  A round reads what still reaches the
// bound again: 4096 x 128256 fp32 with one value, or with 5 logits above a mask, take
// 1,545 us (random ones 312).
template <typename T, bool ENT, int NT>
__global__ void __launch_bounds__(NT, NT == 256 || NT == 512 ? 1536 / NT : 1)
    logprob_rows_kernel(const T* __restrict__ z, int64_t ld, const int32_t* __restrict__ tokens, int vocab,
                        float scale, float* __restrict__ logp, float* __restrict__ lse_out,
                        float* __restrict__ entropy, int top, int32_t* __restrict__ ids,
                        float* __restrict__ top_logp, int* err) {
  constexpr int U = sizeof(T) == 4 ? 2 : 4;  // octets in flight: 64 bytes
  constexpr int SHARE = NT / kGroups;        // threads of a set
  constexpr int SPANS = NT == 256 || NT == 512 ? 8 : 1;
  __shared__ Sums part[NT / 32];
  __shared__ __align__(16) Sums total;         // read by the cluster
  __shared__ Logit best[SF_LOGPROB_TOP_MAX];   // read by the cluster
  __shared__ __align__(16) float maxima[kGroups];
  __shared__ float span_max[SPANS > 1 ? SPANS * NT : 1];
  __shared__ uint16_t hot[SPANS * NT];  // span * NT + thread
  __shared__ Logit list[kList];
  __shared__ Logit bound;
  __shared__ int hot_n, list_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t ncl;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ncl));
  const uint32_t rank = cluster_ctarank();
  const int64_t row = blockIdx.x / ncl;
  const T* zr = z + row * ld;
  const float c = scale * kLog2e;
  const float minus_inf = -__uint_as_float(0x7f800000u);
  const int n8 = vocab >> 3, each = (n8 + (int)ncl - 1) / (int)ncl;
  const int lo = min((int)rank * each, n8), hi = min(lo + each, n8);
  const int tail = rank == ncl - 1 && tid < (vocab & 7) ? 8 * n8 + tid : -1;  // the last logits, one a thread
  if (tid == 0) hot_n = list_n = 0;
  const int octets = (hi - lo + NT - 1) / NT;                        // of a thread
  const int length = ((octets + SPANS - 1) / SPANS + U - 1) / U * U;  // of a span
  const Sums empty = {-FLT_MAX, 0.f, 0.f, 0.f};
  Sums a = empty;
#pragma unroll 1
  for (int s = 0; s < SPANS; ++s) {
    float m = minus_inf;
    int i = lo + tid + s * length * NT;
    const int end = SPANS == 1 ? hi : min(i + length * NT, hi);
    for (; i + (U - 1) * NT < end; i += U * NT) {
      float f[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) load8(zr + 8 * (i + u * NT), f[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) m = fmaxf(m, add<ENT>(a, f[u], c));
    }
    for (; i < end; i += NT) {
      float f[8];
      load8(zr + 8 * i, f);
      m = fmaxf(m, add<ENT>(a, f, c));
    }
    if (SPANS > 1 && top > 0) span_max[s * NT + tid] = m;
  }
  if (tail >= 0) {
    const float f[1] = {to_float(zr[tail])};
    add<ENT>(a, f, c);
  }
  const float mine = a.s == 0.f ? minus_inf : a.m;  // s is at least 1 with any logit above -inf
  a = warp_merge(a, c);
  keep_others_of_warp<NT>(a, mine, zr, lo + warp * 32, hi, c);
  if (lane == 0) part[warp] = a;
  if (top > 0) {
    float group = mine;
#pragma unroll
    for (int o = 1; o < SHARE; o *= 2) group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, o));
    if (tid % SHARE == 0) maxima[tid / SHARE] = group;
    __syncthreads();
    // the SHARE threads of a set count the larger ones of the others, a part each
    int r = 0;
#pragma unroll
    for (int j = 0; j < kGroups / SHARE / 4; ++j) {
      const int at = tid % SHARE * (kGroups / SHARE) + 4 * j;
      const float4 q = *reinterpret_cast<const float4*>(maxima + at);
      const int me = tid / SHARE;
      r += (q.x > group || (q.x == group && at < me)) + (q.y > group || (q.y == group && at + 1 < me)) +
           (q.z > group || (q.z == group && at + 2 < me)) + (q.w > group || (q.w == group && at + 3 < me));
    }
#pragma unroll
    for (int o = 1; o < SHARE; o *= 2) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (r == top - 1) bound = {group, INT_MAX};  // each thread of one set
  }
  __syncthreads();
  if (warp == 0) {
    a = warp_merge(lane < NT / 32 ? part[lane] : empty, c);
    if (lane == 0) total = a;
  }
  if (top > 0) {
    Logit least = bound;
    if (mine >= least.v) {
      for (int s = 0; s < SPANS; ++s)
        if (SPANS == 1 || span_max[s * NT + tid] >= least.v) hot[atomicAdd(&hot_n, 1)] = (uint16_t)(s * NT + tid);
    }
    __syncthreads();
    const int nh = hot_n, items = nh * min(length, octets);
    auto look = [&](float v, int at) {
      if (v > least.v || (v == least.v && at <= least.i)) {  // never a NaN: the list has one order
        const int k = atomicAdd(&list_n, 1);
        if (k < kList) list[k] = {v, at};
      }
    };
    int n;
    while (true) {
      for (int k = tid; k < items; k += NT) {
        const int unit = hot[k % nh], at = lo + (unit / NT * length + k / nh) * NT + unit % NT;
        if (at < hi) {
          float f[8];
          load8(zr + 8 * at, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) look(f[j], 8 * at + j);
        }
      }
      if (tail >= 0) look(to_float(zr[tail]), tail);
      __syncthreads();
      n = list_n;
      if (n <= kList) break;
      places<NT>(list, kList, [&](Logit b, int r) {
        if (r == top - 1) bound = b;
      });
      __syncthreads();
      least = bound;
      if (tid == 0) list_n = 0;
      __syncthreads();
    }
    if (tid >= n && tid < top) best[tid] = {minus_inf, INT_MAX};  // a range shorter than top
    places<NT>(list, n, [&](Logit b, int r) {
      if (r < top) best[r] = b;
    });
  }
  if (ncl > 1) cluster_sync_all();
  else __syncthreads();
  if (rank == 0) {
    if (ncl > 1) {  // the ranges' alternatives in one order
      const int n = (int)ncl * top;
      for (int k = tid; k < n; k += NT) {
        const float2 x = ld_shared_cluster_f32x2(mapa_shared(smem_u32(&best[k % top]), k / top));
        list[k] = {x.x, __float_as_int(x.y)};
      }
      __syncthreads();
      places<NT>(list, n, [&](Logit b, int r) {
        if (r < top) best[r] = b;
      });
      __syncthreads();
    }
    if (warp == 0) {  // lane q has CTA q's sums; then one of the alternatives (32 at most)
      Sums all = total;
      if (ncl > 1) {
        all = empty;
        if (lane < (int)ncl) {
          const uint32_t at = mapa_shared(smem_u32(&total), lane);
          const float2 x = ld_shared_cluster_f32x2(at), y = ld_shared_cluster_f32x2(at + 8);
          all = {x.x, x.y, y.x, y.y};
        }
        all = warp_merge(all, c);
      }
      const RowStats r = row_stats(all, scale);
      const bool bad = !(all.s == all.s);
      if (lane == 0) {
        int token = tokens[row];
        if (token >= vocab) {  // outside the vocabulary: reported, and the row ignored
          record_error(err, kDevCeBadLabel);
          token = -1;
        }
        logp[row] = token < 0 ? 0.f : r.value(to_float(zr[token]));
        lse_out[row] = r.lse;
        if (ENT) entropy[row] = r.entropy;
      }
      if (lane < top) {
        ids[row * top + lane] = bad ? -1 : best[lane].i;
        top_logp[row * top + lane] = bad ? all.s : r.value(best[lane].v);
      }
    }
  }
  if (ncl > 1) cluster_sync_all();  // the first CTA has read its peers' results
}

// Short rows: a warp takes a row, without barriers, and reads it twice where
// alternatives are wanted (the second time from L1 or L2).  Their bound is the top-th of
// 64 maxima, two a lane: sorted in two runs of 32 by bitonic exchanges, of which
// the larger of each pair in opposite order are the 32 largest.  16384 x 500 with
// 20 alternatives: 25 us; 73 us with 64 threads a row, whose barriers and CTA starts
// outlast the row.  Five CTAs an SM for fp32, six for bf16: left to itself the compiler
// has fewer of fp32's loads in flight, and six CTAs' rows do not stay in L2 for the
// second reading (16384 x 4096, 20 alternatives: 91 us so, 81 with five; bf16 69 with
// five, 67 with six).
constexpr int kShortList = 128;  // candidates that a warp holds

// The lanes' values in falling order.
__device__ __forceinline__ float warp_sort(float v, int from) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size *= 2) {
    if (size < from) continue;
#pragma unroll
    for (int o = size / 2; o > 0; o /= 2) {
      const float w = __shfl_xor_sync(0xffffffffu, v, o);
      const bool first = (lane & o) == 0, down = size == 32 || (lane & size) == 0;
      v = first == down ? fmaxf(v, w) : fminf(v, w);
    }
  }
  return v;
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 5 : 6)
    logprob_short_kernel(const T* __restrict__ z, int64_t ld, const int32_t* __restrict__ tokens, int64_t rows,
                         int vocab, float scale, float* __restrict__ logp, float* __restrict__ lse_out,
                         float* __restrict__ entropy, int top, int32_t* __restrict__ ids,
                         float* __restrict__ top_logp, int* err) {
  __shared__ Logit lists[kThreads / 32][kShortList];
  __shared__ int counts[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  if (row >= rows) return;
  const T* zr = z + row * ld;
  const float c = scale * kLog2e, minus_inf = -__uint_as_float(0x7f800000u);
  const int n8 = vocab >> 3, tail = lane < (vocab & 7) ? 8 * n8 + lane : -1;
  Sums a = {-FLT_MAX, 0.f, 0.f, 0.f};
  float max_a = minus_inf, max_b = minus_inf;  // of the first and the last four of each octet
  for (int i = lane; i < n8; i += 32) {
    float f[8];
    load8(zr + 8 * i, f);
    add<ENT>(a, f, c);
    max_a = fmaxf(max_a, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
    max_b = fmaxf(max_b, fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));
  }
  if (tail >= 0) {
    const float f[1] = {to_float(zr[tail])};
    add<ENT>(a, f, c);
    max_a = fmaxf(max_a, f[0]);
  }
  a = warp_merge(a, c);
  keep_others_of_warp<32>(a, fmaxf(max_a, max_b), zr, 0, n8, c);
  const RowStats r = row_stats(a, scale);
  if (lane == 0) {
    int token = tokens[row];
    if (token >= vocab) {  // outside the vocabulary: reported, and the row ignored
      record_error(err, kDevCeBadLabel);
      token = -1;
    }
    logp[row] = token < 0 ? 0.f : r.value(to_float(zr[token]));
    lse_out[row] = r.lse;
    if (ENT) entropy[row] = r.entropy;
  }
  if (top == 0) return;
  if (!(a.s == a.s)) {  // a NaN or +inf
    if (lane < top) {
      ids[row * top + lane] = -1;
      top_logp[row * top + lane] = a.s;
    }
    return;
  }
  max_b = warp_sort(max_b, 2);
  const float best = warp_sort(fmaxf(warp_sort(max_a, 2), __shfl_xor_sync(0xffffffffu, max_b, 31)), 32);
  Logit least = {__shfl_sync(0xffffffffu, best, top - 1), INT_MAX};
  Logit* list = lists[warp];
  // the entries' places, were they in order
  auto places = [&](int n, auto what) {
    for (int k = lane; k < n; k += 32) {
      const Logit b = list[k];
      int place = 0;
      for (int j = 0; j < n; ++j) place += before(list[j], b);
      what(b, place);
    }
  };
  while (true) {
    if (lane == 0) counts[warp] = 0;
    __syncwarp();
    auto look = [&](float v, int at) {
      if (v > least.v || (v == least.v && at <= least.i)) {
        const int k = atomicAdd(&counts[warp], 1);
        if (k < kShortList) list[k] = {v, at};
      }
    };
    for (int i = lane; i < n8; i += 32) {
      float f[8];
      load8(zr + 8 * i, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) look(f[j], 8 * i + j);
    }
    if (tail >= 0) look(to_float(zr[tail]), tail);
    __syncwarp();
    const int n = counts[warp];
    if (n <= kShortList) {
      places(n, [&](Logit b, int place) {
        if (place < top) {
          ids[row * top + place] = b.i;
          top_logp[row * top + place] = r.value(b.v);
        }
      });
      return;
    }
    // more reach the bound than the list holds: the top-th of those that it does is the next one
    Logit next = {0.f, -1};
    places(kShortList, [&](Logit b, int place) {
      if (place == top - 1) next = b;
    });
    const int from = __ffs(__ballot_sync(0xffffffffu, next.i >= 0)) - 1;
    least = {__shfl_sync(0xffffffffu, next.v, from), __shfl_sync(0xffffffffu, next.i, from)};
    __syncwarp();
  }
}

// Backward, element by element from the row's lse and entropy:
//   dz = scale (dlogp (1[token] - p) - dentropy p (log p + entropy)).
// A CTA takes kPiece logits of a row.  Rows whose two upstream gradients are
// both 0 (padding) get zeros without being read, rows of -inf too.
constexpr int kPiece = kThreads * 8 * 4;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    logprob_rows_bwd_kernel(const T* z, int64_t ld, LogprobEpi a, int64_t rows, int vocab, bf16* dz, int64_t lddz,
                            int* err) {
  const int pieces = (vocab + kPiece - 1) / kPiece;
  for (int64_t item = blockIdx.x; item < rows * pieces; item += gridDim.x) {
    const int64_t row = item / pieces;
    const int first = (int)(item - row * pieces) * kPiece;
    const RowGrad g = row_grad(a, row, vocab, err);
    const T* zr = z + row * ld;
    bf16* dr = dz + row * lddz;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int at = first + (u * kThreads + threadIdx.x) * 8;
      if (at + 8 <= vocab) {
        float f[8] = {};
        Eight<bf16> o;
        if (!g.zero) load8(zr + at, f);
        logit_grads(g, f, at);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = __float2bfloat16_rn(f[j]);
        *reinterpret_cast<Eight<bf16>*>(dr + at) = o;
      } else {
        for (int j = at; j < vocab; ++j) {
          float f[1] = {g.zero ? 0.f : to_float(zr[j])};
          logit_grads(g, f, j);
          dr[j] = __float2bfloat16_rn(f[0]);
        }
      }
    }
  }
}

// The sums of rows from those of their tiles of columns (the LM head's product
// leaves them, [tiles][rows]) and the logits of the rows' tokens: a CTA takes 32
// rows with 32 warps, warp w merges the tiles w, w + 32, ... of its lane's row,
// then the warps' sums are merged in warp order.
__global__ void __launch_bounds__(1024)
    logprob_tiles_kernel(LogprobEpi a, int64_t rows, int tiles, int vocab, float* __restrict__ logp,
                         float* __restrict__ lse_out, float* __restrict__ entropy, int* err) {
  __shared__ float4 sh[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * 32 + lane;
  const float c = a.scale * kLog2e;
  wait_primary();
  Sums s = {-FLT_MAX, 0.f, 0.f, 0.f};
  if (row < rows) {
    for (int t = w; t < tiles; t += 32) {
      const float4 p = __ldcg(a.parts + (int64_t)t * rows + row);
      s = merge(s, {p.x, p.y, p.z, p.w}, c);
    }
  }
  sh[w][lane] = make_float4(s.m, s.s, s.low, s.t);
  __syncthreads();
  if (w != 0 || row >= rows) return;
  for (int k = 1; k < 32; ++k) {
    const float4 p = sh[k][lane];
    s = merge(s, {p.x, p.y, p.z, p.w}, c);
  }
  const RowStats r = row_stats(s, a.scale);
  int token = a.tokens[row];
  if (token >= vocab) {  // outside the vocabulary: reported, and the row ignored
    record_error(err, kDevCeBadLabel);
    token = -1;
  }
  logp[row] = token < 0 ? 0.f : r.value(__ldcg(a.token_logit + row));
  lse_out[row] = r.lse;
  if (entropy) entropy[row] = r.entropy;
}

}  // namespace

// Threads of a row.  Many rows: as few as still give each a dozen octets, so
// that one row's reductions hide behind the loads of others; short rows a warp.
// Few rows: more of them, up to eight CTAs of 1024.  Measured with 20 alternatives,
// a warp and 128 threads: 16384 x 2048 47 and 81 us, 16384 x 4096 81 and 96, 16384 x
// 8192 180 and 133, 1200 x 4096 23 and 22; 256 and 512 threads: 160 x 128256 33 and
// 25, 304 x 128256 37 and 32, 608 x 128256 54 and 66; 152 x 128256 38 us with four
// CTAs of 256, 20 with one of 1024.
struct RowShape {
  int threads, ctas;
};
static RowShape row_shape(int64_t rows, int vocab) {
  if (vocab <= 1024 || (vocab <= 4096 && rows > 16 * num_sms())) return {32, 1};
  if (vocab <= 16384) return {128, 1};
  if (rows > 2 * num_sms()) return {256, 1};
  if (rows > num_sms()) return {512, 1};
  int n = 1;
  // clusters of eight leave SMs without one: 16 of them take two turns
  while (n < kMaxCluster && rows * n * 2 <= num_sms() && vocab >= 2 * n * 1024 * 8 &&
         (n < 4 || rows * 12 <= num_sms()))
    n *= 2;
  return {1024, n};
}

__global__ void __launch_bounds__(kThreads)
    add_halves_kernel(const float* __restrict__ x, bf16* __restrict__ y, int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8;
  if (i >= n) return;
  float a[8], b[8];
  load8(x + i, a);
  load8(x + n + i, b);
  Eight<bf16> o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o.v[j] = __float2bfloat16_rn(a[j] + b[j]);
  *reinterpret_cast<Eight<bf16>*>(y + i) = o;
}

void add_halves_bf16(const float* x, bf16* y, int64_t n, cudaStream_t st) {
  add_halves_kernel<<<(unsigned)((n + 8 * kThreads - 1) / (8 * kThreads)), kThreads, 0, st>>>(x, y, n);
}

template <typename T, bool ENT, int NT>
static bool logprob_rows_as(const T* z, int64_t ld, const int32_t* tokens, int64_t rows, int vocab, float scale,
                            float* logp, float* lse, float* entropy, int top, int32_t* ids, float* top_logp, int* err,
                            int ctas, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * (unsigned)ctas);
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprob_rows_kernel<T, ENT, NT>, z, ld, tokens, vocab, scale, logp, lse, entropy,
                            top, ids, top_logp, err) == cudaSuccess;
}

template <typename T, bool ENT>
static bool logprob_rows_of(const T* z, int64_t ld, const int32_t* tokens, int64_t rows, int vocab, float scale,
                            float* logp, float* lse, float* entropy, int top, int32_t* ids, float* top_logp, int* err,
                            cudaStream_t st) {
  const RowShape s = row_shape(rows, vocab);
#define SF_LOGPROB(NT)                                                                                              \
  logprob_rows_as<T, ENT, NT>(z, ld, tokens, rows, vocab, scale, logp, lse, entropy, top, ids, top_logp, err, s.ctas, \
                              st)
  switch (s.threads) {
    case 32:
      logprob_short_kernel<T, ENT><<<(unsigned)((rows + 7) / 8), kThreads, 0, st>>>(z, ld, tokens, rows, vocab, scale,
                                                                                   logp, lse, entropy, top, ids,
                                                                                   top_logp, err);
      return true;
    case 128: return SF_LOGPROB(128);
    case 256: return SF_LOGPROB(256);
    case 512: return SF_LOGPROB(512);
    default: return SF_LOGPROB(1024);
  }
#undef SF_LOGPROB
}

bool logprob_rows(const void* z, bool f32, int64_t ld, const int32_t* tokens, int64_t rows, int vocab, float scale,
                  float* logp, float* lse, float* entropy, int top, int32_t* ids, float* top_logp, int* err,
                  cudaStream_t st) {
#define SF_LOGPROB(T, ENT)                                                                                        \
  logprob_rows_of<T, ENT>(static_cast<const T*>(z), ld, tokens, rows, vocab, scale, logp, lse, entropy, top, ids, \
                          top_logp, err, st)
  if (f32) return entropy ? SF_LOGPROB(float, true) : SF_LOGPROB(float, false);
  return entropy ? SF_LOGPROB(bf16, true) : SF_LOGPROB(bf16, false);
#undef SF_LOGPROB
}

void logprob_rows_bwd(const void* z, bool f32, int64_t ld, const LogprobEpi& a, int64_t rows, int vocab, bf16* dz,
                      int64_t lddz, int* err, cudaStream_t st) {
  const int64_t items = rows * ((vocab + kPiece - 1) / kPiece);
  const unsigned grid = (unsigned)(items < INT32_MAX ? items : INT32_MAX);
  if (f32)
    logprob_rows_bwd_kernel<<<grid, kThreads, 0, st>>>(static_cast<const float*>(z), ld, a, rows, vocab, dz, lddz, err);
  else
    logprob_rows_bwd_kernel<<<grid, kThreads, 0, st>>>(static_cast<const bf16*>(z), ld, a, rows, vocab, dz, lddz, err);
}

bool logprob_tiles(const LogprobEpi& a, int64_t rows, int tiles, int vocab, float* logp, float* lse, float* entropy,
                   int* err, cudaStream_t st) {
  return launch_dependent(logprob_tiles_kernel, dim3((unsigned)((rows + 31) / 32)), 1024, 0, st, a, rows, tiles, vocab,
                          logp, lse, entropy, err);
}

}  // namespace sf
