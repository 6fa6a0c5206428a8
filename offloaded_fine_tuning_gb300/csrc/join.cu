// Dropout, and the join of a block's output with the residual stream.
//
// Dropout keeps no mask: whether an element is kept follows from the seed, the
// offset and the element's place, so the backward asks again.  The bits come
// from Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", 2011): the counter is (octet, offset), 64 bits each, the
// key the seed; the four words of octet i give elements 8i .. 8i + 7 sixteen
// bits each, low half first.  An element is kept when its bits are at least
// T = round(65536 p), and scaled by 65536 / (65536 - T): p is rounded to
// 2^-16, so that one generator call serves eight elements (with 32 bits each
// it would cost as much time as the elements' traffic).
//
// The join, for a row x of the residual stream and h of the block's output:
//   u = h [/ rms(h) * g_post] [* gate],  v = dropout(u),
//   x' = alpha x + beta v,  y = g_next x' / rms(x').
// (The backward is in join_bwd.cu.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "join.cuh"
#include "ptx.cuh"
#include "sf.h"
#include "sf_internal.h"

namespace sf {

namespace {

// ------------------------------------------------------------------ dropout
constexpr int kDropThreads = 256;

// An octet of elements as it is stored, and its kept elements times scale.
template <bool F32>
struct Octet;
template <>
struct Octet<true> {
  float4 a, b;
  __device__ __forceinline__ void drop(const Words& w, const DropArgs& d) {
    a = pick(mul(a, d.scale), make_uint2(w.a, w.b), d.top);
    b = pick(mul(b, d.scale), make_uint2(w.c, w.d), d.top);
  }
};
template <>
struct Octet<false> {
  uint2 a, b;
  __device__ __forceinline__ void drop(const Words& w, const DropArgs& d) {
    const float4 x = pick(mul(unpack4(a), d.scale), make_uint2(w.a, w.b), d.top);
    const float4 y = pick(mul(unpack4(b), d.scale), make_uint2(w.c, w.d), d.top);
    a = pack4(x.x, x.y, x.z, x.w);
    b = pack4(y.x, y.y, y.z, y.w);
  }
};

// Two octets of elements a thread, loaded before their bits are drawn.
// Instructions bound it as much as memory: 16384 x 4096 bf16 takes 45.9 us (5,850
// GB/s, 0.86 of a copy's rate), about 18 instructions an element, 5 of them the
// generator's multiplications and logic.
// DROP false: bf16 with p = 0, a copy without the generator (42.8 us; fp32 with
// p = 0 gains nothing without it).
template <bool F32, bool DROP>
__global__ void __launch_bounds__(kDropThreads)
    dropout_kernel(const void* x, void* y, int64_t n, DropArgs a) {
  constexpr int SIZE = F32 ? 4 : 2;
  struct alignas(16) Stored { Octet<F32> v; };
  const int64_t first = (int64_t)blockIdx.x * (2 * kDropThreads) + threadIdx.x;
  Stored o[2] = {};
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t at = (first + u * kDropThreads) * 8;
    if (at + 8 <= n) o[u] = *reinterpret_cast<const Stored*>(static_cast<const char*>(x) + at * SIZE);
  }
  const uint64_t offset = launch_offset(a);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t octet = first + u * kDropThreads, at = octet * 8;
    if (at >= n) return;
    const Words w = DROP ? philox((uint64_t)octet, offset, a.seed) : Words{};
    if (at + 8 <= n) {
      o[u].v.drop(w, a);
      *reinterpret_cast<Stored*>(static_cast<char*>(y) + at * SIZE) = o[u];
    } else {  // the last few elements, one by one
      const uint32_t words[4] = {w.a, w.b, w.c, w.d};
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        if (at + i >= n) continue;
        const bool keep = i & 1 ? keep_hi(words[i / 2], a.top) : keep_lo(words[i / 2], a.top);
        if (F32) {
          static_cast<float*>(y)[at + i] = keep ? static_cast<const float*>(x)[at + i] * a.scale : 0.f;
        } else {
          const float v = __bfloat162float(static_cast<const bf16*>(x)[at + i]);
          static_cast<bf16*>(y)[at + i] = __float2bfloat16_rn(keep ? v * a.scale : 0.f);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ the join, forward
// Sum over the LANES threads of a row; sh holds a float for each warp.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* sh) {
  v = warp_sum(v);
  if (LANES > 32) {
    const int lane = threadIdx.x & 31, n = LANES / 32, first = threadIdx.x / LANES * n;
    if (lane == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum(lane < n ? sh[first + lane] : 0.f);
  }
  return v;
}

// Forward: LANES threads take a row and hold it (CH quads each; h as it is stored
// where there are more than four) in registers from the loads to the stores.  1024
// threads an SM: up to 12288 columns two rows or more, so that one's loads run
// beside the other's sums and stores.
// Up to four quads the generator runs while the loads are in flight; for more its
// words would cost the second row's registers.  16384 x 4096 with both norms, gate
// and dropout: 121 us (6,650 GB/s, 0.98 of a copy's rate); 144 us with a generator
// call for each quad, 128 us with the calls behind the first sum.
template <bool WIDE>
struct HQuad {
  typedef uint2 type;
};
template <>
struct HQuad<true> {
  typedef float4 type;
};
__device__ __forceinline__ float4 values(float4 v) { return v; }
__device__ __forceinline__ float4 values(uint2 v) { return unpack4(v); }

template <int LANES, int CH, bool H32>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256, 1024 / (LANES > 256 ? LANES : 256))
    join_fwd_kernel(JoinArgs a, const float* x, const void* h, float* xout, bf16* __restrict__ y,
                    float* __restrict__ rstd_post, float* __restrict__ rstd_next, float eps) {
  constexpr bool EARLY = CH <= 4;  // the generator runs while the loads are in flight
  typedef typename HQuad<EARLY || H32>::type Quad;
  constexpr int THREADS = LANES > 256 ? LANES : 256;
  __shared__ float sh[2][THREADS / 32];
  const int t = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const int n4 = row < a.rows ? a.d >> 2 : 0;
  const int64_t at = row * a.d;
  float4 xv[CH];
  Quad hv[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = t + k * LANES;
    xv[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    hv[k] = Quad{};
    if (i < n4) {
      xv[k] = *reinterpret_cast<const float4*>(x + at + 4 * i);
      typedef typename HQuad<H32>::type Stored;
      const Stored v = *reinterpret_cast<const Stored*>(static_cast<const char*>(h) + (at + 4 * i) * (H32 ? 4 : 2));
      if constexpr (EARLY) hv[k] = values(v);
      else hv[k] = v;
    }
  }
  uint2 words[EARLY ? CH : 2];
  auto draw = [&](int k, uint64_t offset) {
    pair_words((at >> 2) + t + k * LANES, LANES, t & 1, offset, a.drop.seed, words[EARLY ? k : 0],
               words[EARLY ? k + 1 : 1]);
  };
  if (EARLY && a.drop.top) {
    const uint64_t offset = launch_offset(a.drop);
#pragma unroll
    for (int k = 0; k < CH; k += 2) draw(k, offset);
  }
  const float inv_d = 1.f / a.d;
  float r1 = 1.f;
  if (a.g_post) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) ss += dot(values(hv[k]), values(hv[k]));
    r1 = rsqrtf(row_sum<LANES>(ss, sh[0]) * inv_d + eps);
    if (n4 > 0 && t == 0) rstd_post[row] = r1;
  }
  const float factor = a.beta * a.drop.scale;
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = t + k * LANES;
    if (!EARLY && k % 2 == 0 && a.drop.top) draw(k, launch_offset(a.drop));
    if (i < n4) {
      float4 u = values(hv[k]);
      if (a.g_post) u = mul(mul(u, r1), gain(a.g_post, i));
      if (a.gate) u = mul(u, gain(a.gate, i));
      if (a.drop.top) u = pick(u, words[EARLY ? k : k % 2], a.drop.top);
      float4& o = xv[k];
      o = make_float4(fmaf(factor, u.x, a.alpha * o.x), fmaf(factor, u.y, a.alpha * o.y),
                      fmaf(factor, u.z, a.alpha * o.z), fmaf(factor, u.w, a.alpha * o.w));
      *reinterpret_cast<float4*>(xout + at + 4 * i) = o;
      ss += dot(o, o);
    }
  }
  if (!a.g_next) return;
  const float r2 = rsqrtf(row_sum<LANES>(ss, sh[1]) * inv_d + eps);
  if (n4 > 0 && t == 0) rstd_next[row] = r2;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = t + k * LANES;
    if (i < n4) {
      const float4 o = mul(mul(xv[k], r2), gain(a.g_next, i));
      reinterpret_cast<uint2*>(y + at)[i] = pack4(o.x, o.y, o.z, o.w);
    }
  }
}

template <int LANES, int CH>
void join_fwd_as(const JoinArgs& a, const float* x, const void* h, bool h32, float* xout, bf16* y,
                 float* rstd_post, float* rstd_next, float eps, cudaStream_t st) {
  constexpr int THREADS = LANES > 256 ? LANES : 256, PER = THREADS / LANES;
  const unsigned grid = (unsigned)((a.rows + PER - 1) / PER);
  if (h32)
    join_fwd_kernel<LANES, CH, true><<<grid, THREADS, 0, st>>>(a, x, h, xout, y, rstd_post, rstd_next, eps);
  else
    join_fwd_kernel<LANES, CH, false><<<grid, THREADS, 0, st>>>(a, x, h, xout, y, rstd_post, rstd_next, eps);
}

}  // namespace

void dropout(const void* x, void* y, bool f32, int64_t n, const DropArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((n + 16 * kDropThreads - 1) / (16 * kDropThreads));
  auto* kernel = f32 ? dropout_kernel<true, true> : a.top ? dropout_kernel<false, true> : dropout_kernel<false, false>;
  kernel<<<grid, kDropThreads, 0, st>>>(x, y, n, a);
}

void join_fwd(const JoinArgs& a, const float* x, const void* h, bool h32, float* xout, bf16* y,
              float* rstd_post, float* rstd_next, float eps, cudaStream_t st) {
  const int d = a.d;
  if (d <= 256) join_fwd_as<32, 2>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 512) join_fwd_as<32, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 1024) join_fwd_as<64, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 2048) join_fwd_as<128, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 4096) join_fwd_as<256, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 8192) join_fwd_as<512, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 12288) join_fwd_as<512, 6>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else join_fwd_as<1024, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);  // d <= 16384
}

}  // namespace sf
