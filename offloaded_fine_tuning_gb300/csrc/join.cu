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
// Backward, with D = dres + (the gradient through the second norm) at x':
//   dx = alpha D,  dv = beta dropout(D),  A = sum over rows of dv hh
//   (hh = h / rms(h), or h),  dgate = g_post A,  dg_post = gate A,
//   dh = (the gradient of the first norm for w dv, w = g_post gate).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.cuh"
#include "ptx.cuh"
#include "sf.h"
#include "sf_internal.h"

namespace sf {

namespace {

typedef __nv_bfloat16 bf16;

struct Words {
  uint32_t a, b, c, d;
};

__device__ __forceinline__ Words philox(uint64_t octet, uint64_t offset, uint64_t seed) {
  Words w = {(uint32_t)octet, (uint32_t)(octet >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)0xD2511F53u * w.a, q = (uint64_t)0xCD9E8D57u * w.c;
    w = {(uint32_t)(q >> 32) ^ w.b ^ k0, (uint32_t)q, (uint32_t)(p >> 32) ^ w.d ^ k1, (uint32_t)p};
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return w;
}

// The offset of this launch: the caller's, plus the counter that a captured
// graph's owner advances between replays.
__device__ __forceinline__ uint64_t launch_offset(const DropArgs& a) { return a.offset + (a.step ? *a.step : 0); }

// Whether the elements of the low and the high half of a word are kept.
__device__ __forceinline__ bool keep_lo(uint32_t w, uint32_t top) { return (w << 16) >= top; }
__device__ __forceinline__ bool keep_hi(uint32_t w, uint32_t top) { return w >= top; }
// Four bits, one for each element of two words.
__device__ __forceinline__ uint32_t keep4(uint32_t v, uint32_t w, uint32_t top) {
  return (keep_lo(v, top) ? 1u : 0u) | (keep_hi(v, top) ? 2u : 0u) | (keep_lo(w, top) ? 4u : 0u) |
         (keep_hi(w, top) ? 8u : 0u);
}

__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
__device__ __forceinline__ float4 unpack4(uint2 u) {
  const float2 a = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// ------------------------------------------------------------------ dropout
constexpr int kDropThreads = 256;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_float(float& o, float v) { o = v; }
__device__ __forceinline__ void from_float(bf16& o, float v) { o = __float2bfloat16_rn(v); }

// One octet of elements a thread.
template <typename T>
__global__ void __launch_bounds__(kDropThreads)
    dropout_kernel(const T* x, T* y, int64_t n, DropArgs a) {
  struct alignas(16) Octet { T v[8]; };
  const int64_t octet = (int64_t)blockIdx.x * kDropThreads + threadIdx.x;
  if (octet * 8 >= n) return;
  const Words w = philox((uint64_t)octet, launch_offset(a), a.seed);
  const uint32_t bits = keep4(w.a, w.b, a.top) | (keep4(w.c, w.d, a.top) << 4);
  if (octet * 8 + 8 <= n) {
    Octet o = *reinterpret_cast<const Octet*>(x + octet * 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) from_float(o.v[i], (bits >> i) & 1 ? to_float(o.v[i]) * a.scale : 0.f);
    *reinterpret_cast<Octet*>(y + octet * 8) = o;
  } else {
    for (int i = 0; octet * 8 + i < n; ++i)
      from_float(y[octet * 8 + i], (bits >> i) & 1 ? to_float(x[octet * 8 + i]) * a.scale : 0.f);
  }
}

// ------------------------------------------------------------------ the join
// A thread's quads of four columns; h is bf16 or fp32.
template <bool H32>
__device__ __forceinline__ float4 load_h(const void* h, int64_t at) {
  if (H32) return *reinterpret_cast<const float4*>(static_cast<const float*>(h) + at);
  return unpack4(*reinterpret_cast<const uint2*>(static_cast<const bf16*>(h) + at));
}
template <bool H32>
__device__ __forceinline__ void store_h(void* h, int64_t at, const float4& v) {
  if (H32) *reinterpret_cast<float4*>(static_cast<float*>(h) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<bf16*>(h) + at) = pack4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ float4 gain(const bf16* g, int quad) {
  return unpack4(reinterpret_cast<const uint2*>(g)[quad]);
}
__device__ __forceinline__ float4 mul(const float4& a, const float4& b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 mul(const float4& a, float b) {
  return make_float4(a.x * b, a.y * b, a.z * b, a.w * b);
}
__device__ __forceinline__ float dot(const float4& a, const float4& b) {
  return (a.x * b.x + a.y * b.y) + (a.z * b.z + a.w * b.w);
}
__device__ __forceinline__ float4 pick(const float4& a, uint32_t bits) {
  return make_float4(bits & 1 ? a.x : 0.f, bits & 2 ? a.y : 0.f, bits & 4 ? a.z : 0.f, bits & 8 ? a.w : 0.f);
}

// The kept bits of the quad that starts at element 4 * quad of the tensor.
__device__ __forceinline__ uint32_t quad_bits(int64_t quad, uint64_t offset, const DropArgs& a) {
  const Words w = philox((uint64_t)(quad >> 1), offset, a.seed);
  return quad & 1 ? keep4(w.c, w.d, a.top) : keep4(w.a, w.b, a.top);
}

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

// Forward: LANES threads take a row and hold it (CH quads each) in registers
// from the loads to the stores.
template <int LANES, int CH, bool H32>
__global__ void __launch_bounds__(LANES > 256 ? LANES : 256)
    join_fwd_kernel(JoinArgs a, const float* x, const void* h, float* xout, bf16* __restrict__ y,
                    float* __restrict__ rstd_post, float* __restrict__ rstd_next, float eps) {
  constexpr int THREADS = LANES > 256 ? LANES : 256;
  __shared__ float sh[2][THREADS / 32];
  const int t = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * (THREADS / LANES) + threadIdx.x / LANES;
  const int n4 = row < a.rows ? a.d >> 2 : 0;
  const int64_t at = row * a.d;
  float4 xv[CH], hv[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = t + k * LANES;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    xv[k] = i < n4 ? *reinterpret_cast<const float4*>(x + at + 4 * i) : zero;
    hv[k] = i < n4 ? load_h<H32>(h, at + 4 * i) : zero;
  }
  const float inv_d = 1.f / a.d;
  float r1 = 1.f;
  if (a.g_post) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) ss += dot(hv[k], hv[k]);
    r1 = rsqrtf(row_sum<LANES>(ss, sh[0]) * inv_d + eps);
    if (n4 > 0 && t == 0) rstd_post[row] = r1;
  }
  const uint64_t offset = a.drop.top ? launch_offset(a.drop) : 0;
  const float factor = a.beta * a.drop.scale;
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = t + k * LANES;
    if (i < n4) {
      float4 u = hv[k];
      if (a.g_post) u = mul(mul(u, r1), gain(a.g_post, i));
      if (a.gate) u = mul(u, gain(a.gate, i));
      if (a.drop.top) u = pick(u, quad_bits((at >> 2) + i, offset, a.drop));
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

// Backward: one CTA of 512 threads per SM, in groups of `lanes` threads (a power
// of two, 32 to 512) that take a row each, so that a thread holds at most four
// quads; rows beyond 8192 columns are shared by a pair of CTAs, each with half
// of the columns.  A thread copies its quads of the row after next (xout, dy,
// dres and h, 56 bytes a quad) into its own places of a ring of two stages in
// shared memory with cp.async and reads them back itself, each array as soon
// as the row before has been read from there; with h in fp32 two stages do not
// fit, so dres is only brought into L2 ahead.  dx may be dres or dy: a thread has
// read its quads of a row before it writes them, and no other touches them.  No
// barrier but the two sums of a row stands between rows, and the gains' sums
// of a thread's columns stay in its registers over all of them.
constexpr int kBwdThreads = 512, kBwdWarps = kBwdThreads / 32;
constexpr int kQuads = 4;

template <bool H32>
struct BwdRing {
  static constexpr bool RES = !H32;  // dres is in the ring
  static constexpr int STAGES = 2;
  static constexpr int PER = kQuads * kBwdThreads;
  static constexpr int X = 0, DY = PER * 16, H = DY + PER * 16;
  static constexpr int DRES = H + PER * (H32 ? 16 : 8);
  static constexpr int STATS = DRES + (RES ? PER * 16 : 0);  // [warps]: the row's two rstd
  static constexpr int STAGE = STATS + kBwdWarps * 8;
};
static_assert(BwdRing<false>::STAGES * BwdRing<false>::STAGE <= 231000, "ring of bf16 h");
static_assert(BwdRing<true>::STAGES * BwdRing<true>::STAGE <= 231000, "ring of fp32 h");

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// A load that may be moved ahead of the kernel's stores to dx: with dx over the
// array that it reads, only the same thread writes the place, after this load.
__device__ __forceinline__ float4 load_early(const float* p) {
  float4 v;
  asm("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void st_shared_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The kept bits of a thread's quads i = t + k * lanes of a row that starts at
// quad `at` of the tensor (both even), quad k in the bits 4k to 4k + 3.  Two
// neighbouring lanes hold the two halves of each octet: the even one asks the
// generator for the octets of even k, the odd one for those of odd k.
__device__ __forceinline__ uint32_t row_bits(int64_t at, int t, int lanes, uint64_t offset, const DropArgs& a) {
  const int odd = t & 1;
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < kQuads; k += 2) {
    const Words w = philox((uint64_t)((at + t + (k + odd) * lanes) >> 1), offset, a.seed);
    const uint32_t lo = keep4(w.a, w.b, a.top), hi = keep4(w.c, w.d, a.top);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
    bits |= (odd ? other | (hi << 4) : lo | (other << 4)) << (4 * k);
  }
  return bits;
}

template <bool H32, bool PAIR>
__global__ void __launch_bounds__(kBwdThreads, 1)
    join_bwd_kernel(JoinArgs a, const float* __restrict__ xout, const void* __restrict__ h,
                    const float* __restrict__ rstd_post, const float* __restrict__ rstd_next,
                    const float* dy, const float* dres, float* dx, void* __restrict__ dh,
                    float* __restrict__ part, int lanes) {
  using R = BwdRing<H32>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sums[4][2 * kBwdWarps];  // the warps' sums, of four sums in turn; with the pair's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / lanes, t = threadIdx.x % lanes, groups = kBwdThreads / lanes;
  const int rank = PAIR ? (int)cluster_ctarank() : 0;
  const int n4 = a.d >> 2, half = PAIR ? (n4 / 2 + 1) & ~1 : 0;  // whole octets
  const int q0 = rank * half, q1 = PAIR && rank == 0 ? half : n4;  // this CTA's quads of a row
  const int first = q0 + t;
  const float inv_d = 1.f / a.d;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  uint2 gn[kQuads];
  float4 w[kQuads];  // g_post * gate
  float4 next_sum[kQuads], branch_sum[kQuads];
  const uint2 one = make_uint2(0x3f803f80u, 0x3f803f80u);
#pragma unroll
  for (int k = 0; k < kQuads; ++k) {
    const int i = first + k * lanes;
    next_sum[k] = branch_sum[k] = zero;
    gn[k] = a.g_next && i < q1 ? reinterpret_cast<const uint2*>(a.g_next)[i] : one;
    w[k] = unpack4(one);
    if (a.g_post && i < q1) w[k] = gain(a.g_post, i);
    if (a.gate && i < q1) w[k] = mul(w[k], gain(a.gate, i));
  }
  const uint64_t offset = a.drop.top ? launch_offset(a.drop) : 0;
  const float factor = a.beta * a.drop.scale;
  const bool post = a.g_post != nullptr, next = a.g_next != nullptr;
  const bool gains = post || a.gate != nullptr;  // h is read
  const uint32_t base = smem_u32(ring);
  int par = 0;
  auto sum = [&](float v) {
    v = warp_sum(v);
    if (PAIR) {
      const uint32_t at = smem_u32(&sums[par][rank * kBwdWarps + warp]);
      if (lane < 2) st_shared_cluster(mapa_shared(at, lane), v);
      cluster_sync_all();
      v = warp_sum(sums[par][lane]);
    } else if (lanes > 32) {
      if (lane == 0) sums[par][warp] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
      const int n = lanes >> 5;
      v = warp_sum(lane < n ? sums[par][group * n + lane] : 0.f);
    }
    par = (par + 1) & 3;
    return v;
  };
  // the copies of a row into a stage, in two parts: what the second sum needs
  // no more, and the rest
  auto issue_x = [&](int64_t row, int stage) {
    if (row >= a.rows) return;
    const uint32_t st = base + (uint32_t)stage * R::STAGE;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int i = first + k * lanes;
      if (i < q1) {
        const uint32_t at = (uint32_t)(k * kBwdThreads + threadIdx.x);
        const int64_t from = row * a.d + 4 * i;
        if (next) {
          cp_async16(st + R::X + at * 16, xout + from);
          cp_async16(st + R::DY + at * 16, dy + from);
        }
        if (dres) {
          if (R::RES) cp_async16(st + R::DRES + at * 16, dres + from);
          else asm volatile("prefetch.global.L2 [%0];" ::"l"(dres + from));
        }
      }
    }
  };
  auto issue_h = [&](int64_t row, int stage) {
    if (row < a.rows) {
      const uint32_t st = base + (uint32_t)stage * R::STAGE;
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        const int i = first + k * lanes;
        if (gains && i < q1) {
          const uint32_t at = (uint32_t)(k * kBwdThreads + threadIdx.x);
          const int64_t from = row * a.d + 4 * i;
          if (H32) cp_async16(st + R::H + at * 16, static_cast<const float*>(h) + from);
          else cp_async8(st + R::H + at * 8, static_cast<const bf16*>(h) + from);
        }
      }
      if (lane == 0 && next) cp_async4(st + R::STATS + warp * 8, rstd_next + row);
      if (lane == 1 && post) cp_async4(st + R::STATS + warp * 8 + 4, rstd_post + row);
    }
    cp_async_commit();
  };
  const int64_t stride = (int64_t)(PAIR ? gridDim.x / 2 : gridDim.x) * groups;
  const int64_t row0 = (int64_t)(PAIR ? blockIdx.x / 2 : blockIdx.x) * groups + group;
  for (int k = 0; k < R::STAGES; ++k) {
    issue_x(row0 + k * stride, k);
    issue_h(row0 + k * stride, k);
  }
  if (PAIR) cluster_sync_all();  // the peer has started: its shared memory may be written
  int stage = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.rows; row += stride, stage ^= 1) {
    const int64_t at = row * a.d;
    uint32_t bits = 0xffffu;
    if (a.drop.top) bits = row_bits((at >> 2) + q0, t, lanes, offset, a.drop);
    cp_async_wait<R::STAGES - 1>();
    __syncwarp();
    const uint8_t* st = ring + stage * R::STAGE;
    const float4* sx = reinterpret_cast<const float4*>(st + R::X) + threadIdx.x;
    const float4* sdy = reinterpret_cast<const float4*>(st + R::DY) + threadIdx.x;
    const float4* sdr = reinterpret_cast<const float4*>(st + R::DRES) + threadIdx.x;
    const float* stats = reinterpret_cast<const float*>(st + R::STATS) + warp * 2;
    auto load_hh = [&](int k) {
      if (H32) return reinterpret_cast<const float4*>(st + R::H)[k * kBwdThreads + threadIdx.x];
      return unpack4(reinterpret_cast<const uint2*>(st + R::H)[k * kBwdThreads + threadIdx.x]);
    };
    const float r2 = next ? stats[0] : 0.f, r1 = post ? stats[1] : 1.f;
    float c1 = 0.f;
    if (next) {
#pragma unroll
      for (int k = 0; k < kQuads; ++k) {
        if (first + k * lanes < q1) {
          const float4 p = mul(mul(sx[k * kBwdThreads], r2), sdy[k * kBwdThreads]);
          next_sum[k].x += p.x; next_sum[k].y += p.y; next_sum[k].z += p.z; next_sum[k].w += p.w;
          c1 += dot(p, unpack4(gn[k]));
        }
      }
      c1 = sum(c1) * inv_d;
    }
    float4 dv[kQuads];
    float c2 = 0.f;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int i = first + k * lanes;
      if (i < q1) {
        float4 o = zero;
        if (dres) o = R::RES ? sdr[k * kBwdThreads] : load_early(dres + at + 4 * i);
        if (next) {
          const float4 xh = mul(sx[k * kBwdThreads], r2), gd = mul(unpack4(gn[k]), sdy[k * kBwdThreads]);
          o.x += r2 * (gd.x - xh.x * c1);
          o.y += r2 * (gd.y - xh.y * c1);
          o.z += r2 * (gd.z - xh.z * c1);
          o.w += r2 * (gd.w - xh.w * c1);
        }
        *reinterpret_cast<float4*>(dx + at + 4 * i) = mul(o, a.alpha);
        o = pick(mul(o, factor), bits >> (4 * k));
        dv[k] = mul(o, w[k]);
        if (gains) {
          const float4 p = mul(mul(load_hh(k), r1), o);
          branch_sum[k].x += p.x; branch_sum[k].y += p.y; branch_sum[k].z += p.z; branch_sum[k].w += p.w;
          c2 += dot(p, w[k]);
        }
      }
    }
    issue_x(row + 2 * stride, stage);
    if (post) c2 = sum(c2) * inv_d;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      const int i = first + k * lanes;
      if (i < q1) {
        float4 o = dv[k];
        if (post) {
          const float4 hh = mul(load_hh(k), r1);
          o = make_float4(r1 * (o.x - hh.x * c2), r1 * (o.y - hh.y * c2), r1 * (o.z - hh.z * c2),
                          r1 * (o.w - hh.w * c2));
        }
        store_h<H32>(dh, at + 4 * i, o);
      }
    }
    __syncwarp();  // the warp's statistics have been read: the next copies may replace them
    issue_h(row + 2 * stride, stage);
  }
  cp_async_wait<0>();
  allow_dependents();
  if (!part) return;
  // the groups hold the same columns: joined in their order
  float4* join = reinterpret_cast<float4*>(ring);  // [groups][kQuads * lanes]
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float4* out = reinterpret_cast<float4*>(part + ((int64_t)(PAIR ? blockIdx.x / 2 : blockIdx.x) * 2 + s) * a.d);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kQuads; ++k) join[(group * kQuads + k) * lanes + t] = s ? branch_sum[k] : next_sum[k];
    __syncthreads();
    for (int i = threadIdx.x; i < q1 - q0; i += kBwdThreads) {
      float4 v = join[i];
      for (int u = 1; u < groups; ++u) {
        const float4 w = join[u * kQuads * lanes + i];
        v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
      }
      out[q0 + i] = v;
    }
  }
}

// The gains' gradients from the partials [parts, 2, d], in a fixed order: a CTA
// takes 32 columns with 32 warps, warp w adds the partials w, w + 32, ...
__global__ void __launch_bounds__(1024)
    join_sums_kernel(JoinArgs a, const float* __restrict__ part, int parts, bf16* __restrict__ dg_post,
                     bf16* __restrict__ dgate, bf16* __restrict__ dg_next) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int s = blockIdx.y, j = blockIdx.x * 32 + lane;
  wait_primary();
  float v = 0.f;
  if (j < a.d) {
#pragma unroll 8
    for (int p = w; p < parts; p += 32) v += __ldcg(part + ((int64_t)p * 2 + s) * a.d + j);
  }
  sh[w][lane] = v;
  __syncthreads();
  // warp w joins column w: one value per lane, added pairwise in a fixed tree
  const float sum = warp_sum(sh[lane][w]);
  const int c = blockIdx.x * 32 + w;
  if (lane != 0 || c >= a.d) return;
  if (s == 0) {
    if (dg_next) dg_next[c] = __float2bfloat16_rn(sum);
  } else {
    if (dg_post) dg_post[c] = __float2bfloat16_rn(a.gate ? sum * __bfloat162float(a.gate[c]) : sum);
    if (dgate) dgate[c] = __float2bfloat16_rn(a.g_post ? sum * __bfloat162float(a.g_post[c]) : sum);
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

// Threads of a row (or of a pair's half): enough for kQuads quads each, 32 to 512.
int bwd_lanes(int d) {
  int n = 32;
  while (n < kBwdThreads && n * 4 * kQuads < d) n *= 2;
  return n;
}
bool bwd_pair(int d) { return d > kBwdThreads * 4 * kQuads; }

template <bool H32, bool PAIR>
bool join_bwd_as(const JoinArgs& a, const float* xout, const void* h, const float* rstd_post,
                 const float* rstd_next, const float* dy, const float* dres, float* dx, void* dh,
                 float* part, int parts, cudaStream_t st) {
  constexpr int smem = BwdRing<H32>::STAGES * BwdRing<H32>::STAGE;
  if (!reserve_smem<join_bwd_kernel<H32, PAIR>>(smem)) return false;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR ? 2 : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(PAIR ? 2 * parts : parts));
  cfg.blockDim = dim3(kBwdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_bwd_kernel<H32, PAIR>, a, xout, h, rstd_post, rstd_next, dy, dres, dx, dh,
                            part, bwd_lanes(a.d)) == cudaSuccess;
}

}  // namespace

void dropout(const void* x, void* y, bool f32, int64_t n, const DropArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((n + 8 * kDropThreads - 1) / (8 * kDropThreads));
  if (f32)
    dropout_kernel<float><<<grid, kDropThreads, 0, st>>>(static_cast<const float*>(x), static_cast<float*>(y), n, a);
  else
    dropout_kernel<bf16><<<grid, kDropThreads, 0, st>>>(static_cast<const bf16*>(x), static_cast<bf16*>(y), n, a);
}

void join_fwd(const JoinArgs& a, const float* x, const void* h, bool h32, float* xout, bf16* y,
              float* rstd_post, float* rstd_next, float eps, cudaStream_t st) {
  const int d = a.d;
  if (d <= 512) join_fwd_as<32, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 1024) join_fwd_as<64, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 2048) join_fwd_as<128, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 4096) join_fwd_as<256, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 8192) join_fwd_as<512, 4>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else if (d <= 12288) join_fwd_as<512, 6>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);
  else join_fwd_as<512, 8>(a, x, h, h32, xout, y, rstd_post, rstd_next, eps, st);  // d <= 16384
}

int join_bwd_parts(int64_t rows, int d) {
  const int groups = kBwdThreads / bwd_lanes(d), most = bwd_pair(d) ? num_sms() / 2 : num_sms();
  const int64_t need = (rows + groups - 1) / groups;
  return need < most ? (int)(need > 0 ? need : 1) : most;
}

bool join_bwd(const JoinArgs& a, const float* xout, const void* h, bool h32, const float* rstd_post,
              const float* rstd_next, const float* dy, const float* dres, float* dx, void* dh,
              bf16* dg_post, bf16* dgate, bf16* dg_next, float* part, cudaStream_t st) {
  const int parts = join_bwd_parts(a.rows, a.d);
  if (!dg_post && !dgate && !dg_next) part = nullptr;
#define SF_JOIN_BWD(H32, PAIR) \
  join_bwd_as<H32, PAIR>(a, xout, h, rstd_post, rstd_next, dy, dres, dx, dh, part, parts, st)
  const bool ok = bwd_pair(a.d) ? (h32 ? SF_JOIN_BWD(true, true) : SF_JOIN_BWD(false, true))
                                : (h32 ? SF_JOIN_BWD(true, false) : SF_JOIN_BWD(false, false));
#undef SF_JOIN_BWD
  if (ok && part)
    launch_dependent(join_sums_kernel, dim3((unsigned)((a.d + 31) / 32), 2), 1024, 0, st, a, part, parts, dg_post,
                     dgate, dg_next);
  return ok;
}

}  // namespace sf
