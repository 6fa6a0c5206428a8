// 8-bit activation checkpoints: a layer's input (fp32 [rows, d]) kept as one
// byte an element with one fp32 scale for each block of 128 columns of a row,
// and RMSNorm computed on the way in (forward, saving) and on the way out
// (recompute and backward, from the codes).
//
// With a the largest magnitude of a block and T = 127 (int8) or 448 (e4m3):
//   scale = a / T,  code = round(x * (T / a)),  value = code * scale,
// all in fp32, round to nearest even.  int8 keeps 1/254 of the block's largest
// magnitude at worst; e4m3 keeps every value to 2^-4 of itself above a 2^-6
// of 448ths.  A block whose a is below 2^-100 (T / a would overflow) is stored
// as zeros; a block that holds an infinity or a NaN has a NaN scale, so it
// comes back as NaN and a step that diverged is not hidden.
//
// Every kernel here streams its rows once and is bound by memory traffic: 16384
// x 4096, forward saving int8 70 us (6,740 GB/s), forward from the codes 70 us,
// together 0.96 of a measured copy's rate; 4095 x 12288 e4m3, backward 133.7 us
// with its gain sums (757 MB, 5,660 GB/s, 0.84; the sums' launch is 6 us).  Alone,
// at 16384 x 4096 (337 MB): save 72 us (int8; e4m3 70), load 76 us (e4m3 56).  A
// lane holds four columns (a float4, or four codes), so a warp holds a block:
// its largest magnitude is one integer warp reduction of |x|'s bits, which
// order like the values, with infinities and NaNs on top.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.cuh"
#include "ptx.cuh"
#include "sf.h"
#include "sf_internal.h"

namespace sf {

namespace {

typedef __nv_bfloat16 bf16;

constexpr int kBlock = 128;   // columns that share a scale
constexpr int kThreads = 256;

template <int FMT>
constexpr float kTop = FMT == SF_CKPT_INT8 ? 127.f : 448.f;

// The block's scale and the factor to its codes (0: every code is 0), from the
// bits of its largest magnitude.
template <int FMT>
__device__ __forceinline__ void block_scale(uint32_t bits, float& scale, float& inv) {
  const float a = __uint_as_float(bits);
  inv = scale = 0.f;
  if (bits >= 0x7f800000u) {
    scale = __uint_as_float(0x7fc00000u);
  } else if (a >= 7.888609052210118e-31f) {  // 2^-100
    inv = __fdiv_rn(kTop<FMT>, a);
    scale = __fdiv_rn(a, kTop<FMT>);
  }
}

__device__ __forceinline__ uint32_t max_bits(const float4& v) {
  const uint32_t m = 0x7fffffffu;
  return max(max(__float_as_uint(v.x) & m, __float_as_uint(v.y) & m),
             max(__float_as_uint(v.z) & m, __float_as_uint(v.w) & m));
}

// Four codes, the lowest column in the lowest byte.
template <int FMT>
__device__ __forceinline__ uint32_t encode(const float4& v, float inv) {
  if (inv == 0.f) return 0u;  // a zero or a non-finite block
  if (FMT == SF_CKPT_INT8) {
    const uint32_t a = (uint32_t)__float2int_rn(v.x * inv), b = (uint32_t)__float2int_rn(v.y * inv);
    const uint32_t c = (uint32_t)__float2int_rn(v.z * inv), d = (uint32_t)__float2int_rn(v.w * inv);
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v.x * inv, v.y * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v.z * inv, v.w * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <int FMT>
__device__ __forceinline__ float4 decode(uint32_t q, float scale) {
  float4 v;
  if (FMT == SF_CKPT_INT8) {
    // code + 128 in the low mantissa byte of 2^23: exact, and no conversions
    const uint32_t u = q ^ 0x80808080u;
    v.x = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440)) - 8388736.f;
    v.y = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7441)) - 8388736.f;
    v.z = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7442)) - 8388736.f;
    v.w = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7443)) - 8388736.f;
  } else {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(q >> 16), __NV_E4M3);
    const float2 f = __half22float2(__half2(a)), g = __half22float2(__half2(b));
    v = make_float4(f.x, f.y, g.x, g.y);
  }
  return make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
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

// ------------------------------------------------------------------ save and load alone
constexpr int kCopyBlocks = 4;  // blocks a warp has in flight

template <int FMT>
__global__ void __launch_bounds__(kThreads)
    save_kernel(const float* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ scale,
                int64_t blocks, int nb, int d) {
  const int lane = threadIdx.x & 31;
  const int64_t first = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kCopyBlocks;
  float4 v[kCopyBlocks];
  int64_t at[kCopyBlocks];
#pragma unroll
  for (int u = 0; u < kCopyBlocks; ++u) {
    const int64_t b = first + u, row = b / nb;
    const int col = (int)(b - row * nb) * kBlock + 4 * lane;
    at[u] = b < blocks && col < d ? row * d + col : -1;
    v[u] = at[u] >= 0 ? *reinterpret_cast<const float4*>(x + at[u]) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int u = 0; u < kCopyBlocks; ++u) {
    float s, inv;
    block_scale<FMT>(__reduce_max_sync(0xffffffffu, max_bits(v[u])), s, inv);
    if (at[u] >= 0) *reinterpret_cast<uint32_t*>(q + at[u]) = encode<FMT>(v[u], inv);
    if (lane == 0 && first + u < blocks) scale[first + u] = s;
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads)
    load_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scale,
                float* __restrict__ x, int64_t blocks, int nb, int d) {
  const int lane = threadIdx.x & 31;
  const int64_t first = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kCopyBlocks;
  uint32_t c[kCopyBlocks];
  float s[kCopyBlocks];
  int64_t at[kCopyBlocks];
#pragma unroll
  for (int u = 0; u < kCopyBlocks; ++u) {
    const int64_t b = first + u, row = b / nb;
    const int col = (int)(b - row * nb) * kBlock + 4 * lane;
    at[u] = b < blocks && col < d ? row * d + col : -1;
    c[u] = at[u] >= 0 ? *reinterpret_cast<const uint32_t*>(q + at[u]) : 0u;
    s[u] = at[u] >= 0 ? scale[b] : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kCopyBlocks; ++u)
    if (at[u] >= 0) *reinterpret_cast<float4*>(x + at[u]) = decode<FMT>(c[u], s[u]);
}

// ------------------------------------------------------------------ RMSNorm forward
// Groups of LANES threads (a power of two, 32 to 256) take a row each, so
// that narrow rows fill a CTA too (65536 x 512: save 88.7 us with a CTA per
// row, 43.7 us so); thread t of a group holds the quads t, t + LANES, ... (CH of them), so
// each warp holds whole blocks.  LOAD: the row comes from the codes (and is
// written to xout unless that is null); else from x, and is saved.
// When saving, the squares are added in rmsnorm_fwd's order, so that saving
// changes no bit of y and rstd: there thread t of 256 has the quads t, t + 256,
// ..., and its eight warps' sums meet in a tree (w with w ^ 4, w ^ 2, w ^ 1).  A
// thread of a narrower group stands for SUMS threads of those, whose sums it
// keeps apart until their warps' sums are joined in that tree (65536 x 1024:
// 82.6 us, 80.5 us with one sum; no difference at 512 and 2048).
template <int LANES, int CH, int FMT, bool LOAD>
__global__ void __launch_bounds__(kThreads)
    norm_fwd8_kernel(const float* __restrict__ x, const bf16* __restrict__ g,
                     bf16* __restrict__ y, float* __restrict__ rstd_out, uint8_t* q, float* scale,
                     float* __restrict__ xout, int64_t rows, int nb, int d, float eps) {
  constexpr int SUMS = LOAD ? 1 : kThreads / LANES < CH ? kThreads / LANES : CH;
  static_assert(SUMS == 1 || CH == 4, "the joins below");
  __shared__ float sh[kThreads / 32];
  const int group = threadIdx.x / LANES, t = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / LANES) + group;
  const int n4 = LANES == kThreads || row < rows ? d >> 2 : 0, lane = threadIdx.x & 31;
  uint32_t* qr = reinterpret_cast<uint32_t*>(q + row * d);
  float* sr = scale + row * nb;
  float4 v[CH];
  float part[SUMS] = {};
  if (LOAD) {
    uint32_t c[CH];
    float s[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int i = t + k * LANES;
      c[k] = i < n4 ? qr[i] : 0u;
      s[k] = i < n4 ? sr[i >> 5] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) v[k] = decode<FMT>(c[k], s[k]);
  } else {
    const float4* xr = reinterpret_cast<const float4*>(x + row * d);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int i = t + k * LANES;
      v[k] = i < n4 ? xr[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
#pragma unroll
  for (int k = 0; k < CH; ++k)
    part[k % SUMS] += v[k].x * v[k].x + v[k].y * v[k].y + v[k].z * v[k].z + v[k].w * v[k].w;
  if (!LOAD) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int i = t + k * LANES;
      float s, inv;
      block_scale<FMT>(__reduce_max_sync(0xffffffffu, max_bits(v[k])), s, inv);
      if (i < n4) {
        qr[i] = encode<FMT>(v[k], inv);
        if (lane == 0) sr[i >> 5] = s;
      }
    }
  } else if (xout) {
    float4* xo = reinterpret_cast<float4*>(xout + row * d);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int i = t + k * LANES;
      if (i < n4) xo[i] = v[k];
    }
  }
#pragma unroll
  for (int k = 0; k < SUMS; ++k) part[k] = warp_sum(part[k]);
  float ss = SUMS == 4 ? (part[0] + part[2 % SUMS]) + (part[1 % SUMS] + part[3 % SUMS])
             : SUMS == 2 ? part[0] + part[1 % SUMS] : part[0];
  if (LANES > 32) {
    if (lane == 0) sh[threadIdx.x >> 5] = ss;
    __syncthreads();
    const int n = LANES >> 5;
    ss = warp_sum(lane < n ? sh[group * n + lane] : 0.f);
  }
  if (n4 == 0) return;
  const float rstd = rsqrtf(ss / d + eps);
  if (t == 0) rstd_out[row] = rstd;
  const uint2* gr = reinterpret_cast<const uint2*>(g);
  uint2* yr = reinterpret_cast<uint2*>(y + row * d);
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = t + k * LANES;
    if (i < n4) {
      const float4 gg = unpack4(gr[i]);
      yr[i] = pack4(v[k].x * rstd * gg.x, v[k].y * rstd * gg.y, v[k].z * rstd * gg.z, v[k].w * rstd * gg.w);
    }
  }
}

template <int FMT, bool LOAD>
void norm_fwd8(const float* x, const bf16* g, bf16* y, float* rstd, uint8_t* q, float* scale,
               float* xout, int64_t rows, int d, float eps, cudaStream_t st) {
  const int nb = (d + kBlock - 1) / kBlock;
#define SF_NORM8(LANES, CH)                                                                           \
  do {                                                                                                \
    const int per = kThreads / LANES;                                                                 \
    norm_fwd8_kernel<LANES, CH, FMT, LOAD><<<(unsigned)((rows + per - 1) / per), kThreads, 0, st>>>(  \
        x, g, y, rstd, q, scale, xout, rows, nb, d, eps);                                             \
  } while (0)
  if (d <= 512) SF_NORM8(32, 4);
  else if (d <= 1024) SF_NORM8(64, 4);
  else if (d <= 2048) SF_NORM8(128, 4);
  else if (d <= 4096) SF_NORM8(256, 4);
  else if (d <= 8192) SF_NORM8(256, 8);
  else if (d <= 12288) SF_NORM8(256, 12);
  else SF_NORM8(256, 16);  // d <= 16384
#undef SF_NORM8
}

// ------------------------------------------------------------------ RMSNorm backward
// One CTA of 512 threads per SM, in groups of `lanes` threads (a power of two,
// 32 to 512) that take a row each, so a thread holds at most CH quads of four
// columns: 4 up to d = 8192 (narrower rows run several at a time), then 6 and
// 8.  A thread copies its quads of the rows ahead (dy, dres and the codes, 36
// bytes a quad; a warp's scales and the row's rstd with them) into its own
// places of a ring in shared memory with cp.async and reads them back itself.
// While a row is computed the others of the ring are in flight, whatever the
// registers hold: 147 KB per SM at CH 4 (three rows of 74 KB), 110 KB at CH 6
// (two rows), and at CH 8 82 KB (two rows, where the ring holds dy and the codes,
// and dres is only brought into L2 ahead).  No barrier but the row's sum stands
// between rows, and d % 16 == 8 needs no special case, as a bulk copy would.
// The gain gradient of a thread's columns stays in registers over all rows.
// dx may be dres or dy: a thread reads its quads of a row before it writes them,
// and no other thread touches them.
// 4095 x 12288: 245 us with a row's loads held by registers, 133 us with the
// ring; 16384 x 4096: 168 us, where the fp32 checkpoint's backward takes 190;
// 4096 x 16384 (CH 8): 216 us, 4,680 GB/s, bound by dres's late loads.
constexpr int kBwdThreads = 512;

template <int CH>
struct BwdRing {
  static constexpr bool RES = CH <= 6;  // dres is in the ring
  static constexpr int STAGES = CH <= 4 ? 3 : 2;
  static constexpr int DY = 0, DRES = CH * kBwdThreads * 16;
  static constexpr int CODES = DRES + (RES ? CH * kBwdThreads * 16 : 0);
  static constexpr int SCALES = CODES + CH * kBwdThreads * 4;  // [16 warps][12]: CH scales, rstd at 8
  static constexpr int STAGE = SCALES + kBwdThreads / 32 * 48;
};
static_assert(BwdRing<4>::STAGES * BwdRing<4>::STAGE <= 230000, "ring of 4 quads");
static_assert(BwdRing<6>::STAGES * BwdRing<6>::STAGE <= 230000, "ring of 6 quads");
static_assert(BwdRing<8>::STAGES * BwdRing<8>::STAGE <= 230000, "ring of 8 quads");

// A load that may be moved ahead of the kernel's stores to dx: with dx over the
// array that it reads, only the same thread writes the place, after this load.
__device__ __forceinline__ float4 load_early(const float* p) {
  float4 v;
  asm("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

template <int CH, int FMT>
__global__ void __launch_bounds__(kBwdThreads, 1)
    norm_bwd8_kernel(const uint8_t* __restrict__ q, const float* __restrict__ scale,
                     const bf16* __restrict__ g, const float* __restrict__ rstd,
                     const float* dy, const float* dres, float* dx, bf16* __restrict__ dxb,
                     float* __restrict__ dg_part, int64_t rows, int nb, int d, int lanes) {
  using R = BwdRing<CH>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sums[2][kBwdThreads / 32];  // the warps' sums of a row, of two rows in turn
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = threadIdx.x / lanes, t = threadIdx.x % lanes, groups = kBwdThreads / lanes;
  const int n4 = d >> 2;
  const float inv_d = 1.f / d;
  const int64_t stride = (int64_t)gridDim.x * groups;
  uint2 gg[CH];
  float4 gacc[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int i = t + k * lanes;
    gacc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    gg[k] = i < n4 ? reinterpret_cast<const uint2*>(g)[i] : make_uint2(0u, 0u);
  }
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  int put = 0;
  auto issue = [&](int64_t row) {
    if (row < rows) {
      const uint32_t st = base + (uint32_t)put * R::STAGE;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int i = t + k * lanes;
        if (i < n4) {
          const uint32_t at = (uint32_t)(k * kBwdThreads + threadIdx.x);
          cp_async16(st + R::DY + at * 16, dy + row * d + 4 * i);
          if (dres) {
            if (R::RES) cp_async16(st + R::DRES + at * 16, dres + row * d + 4 * i);
            else asm volatile("prefetch.global.L2 [%0];" ::"l"(dres + row * d + 4 * i));
          }
          cp_async4(st + R::CODES + at * 4, q + row * d + 4 * i);
        }
      }
      // lane k < CH copies the scale of the warp's k-th block
      const int i0 = (t & ~31) + lane * lanes;
      if (lane < CH && i0 < n4)
        cp_async4(st + R::SCALES + (uint32_t)(warp * 12 + lane) * 4, scale + row * nb + (i0 >> 5));
      if (lane == 8) cp_async4(st + R::SCALES + (uint32_t)(warp * 12 + 8) * 4, rstd + row);
    }
    cp_async_commit();
    put = put + 1 == R::STAGES ? 0 : put + 1;
  };
  const int64_t row0 = (int64_t)blockIdx.x * groups + group;
  for (int k = 0; k < R::STAGES - 1; ++k) issue(row0 + k * stride);
  int get = 0, par = 0;
#pragma unroll 1
  for (int64_t row = row0; row < rows; row += stride) {
    issue(row + (R::STAGES - 1) * stride);
    cp_async_wait<R::STAGES - 1>();
    __syncwarp();
    const uint8_t* st = ring + get * R::STAGE;
    const float4* sdy = reinterpret_cast<const float4*>(st + R::DY);
    const float4* sdr = reinterpret_cast<const float4*>(st + R::DRES);
    const uint32_t* sq = reinterpret_cast<const uint32_t*>(st + R::CODES);
    const float* ss = reinterpret_cast<const float*>(st + R::SCALES) + warp * 12;
    const float r = ss[8];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int at = k * kBwdThreads + threadIdx.x;
      if (t + k * lanes < n4) {
        const float4 dv = sdy[at], w = unpack4(gg[k]);
        float4 xh = decode<FMT>(sq[at], ss[k]);
        xh = make_float4(xh.x * r, xh.y * r, xh.z * r, xh.w * r);
        const float4 p = make_float4(dv.x * xh.x, dv.y * xh.y, dv.z * xh.z, dv.w * xh.w);
        gacc[k].x += p.x; gacc[k].y += p.y; gacc[k].z += p.z; gacc[k].w += p.w;
        dot += w.x * p.x + w.y * p.y + w.z * p.z + w.w * p.w;
      }
    }
    dot = warp_sum(dot);
    if (lanes > 32) {
      if (lane == 0) sums[par][warp] = dot;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
      const int first = group * (lanes >> 5), n = lanes >> 5;
      dot = warp_sum(lane < n ? sums[par][first + lane] : 0.f);
      par ^= 1;
    }
    dot *= inv_d;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int at = k * kBwdThreads + threadIdx.x, i = t + k * lanes;
      if (i < n4) {
        const float4 dv = sdy[at], w = unpack4(gg[k]);
        float4 xh = decode<FMT>(sq[at], ss[k]);
        xh = make_float4(xh.x * r, xh.y * r, xh.z * r, xh.w * r);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        if (dres) o = R::RES ? sdr[at] : load_early(dres + row * d + 4 * i);
        o.x += r * (w.x * dv.x - xh.x * dot);
        o.y += r * (w.y * dv.y - xh.y * dot);
        o.z += r * (w.z * dv.z - xh.z * dot);
        o.w += r * (w.w * dv.w - xh.w * dot);
        reinterpret_cast<float4*>(dx + row * d)[i] = o;
        reinterpret_cast<uint2*>(dxb + row * d)[i] = pack4(o.x, o.y, o.z, o.w);
      }
    }
    __syncwarp();  // the warp's scales have been read: the next copies may replace them
    get = get + 1 == R::STAGES ? 0 : get + 1;
  }
  cp_async_wait<0>();
  allow_dependents();
  float4* part = reinterpret_cast<float4*>(dg_part + (int64_t)blockIdx.x * d);
  if (groups == 1) {
#pragma unroll
    for (int k = 0; k < CH; ++k)
      if (t + k * lanes < n4) part[t + k * lanes] = gacc[k];
    return;
  }
  // the groups hold the same columns: joined in their order
  __syncthreads();
  float4* join = reinterpret_cast<float4*>(ring);  // [groups][CH * lanes]
#pragma unroll
  for (int k = 0; k < CH; ++k) join[(group * CH + k) * lanes + t] = gacc[k];
  __syncthreads();
  for (int i = threadIdx.x; i < n4; i += kBwdThreads) {
    float4 s = join[i];
    for (int u = 1; u < groups; ++u) {
      const float4 v = join[u * CH * lanes + i];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    part[i] = s;
  }
}

// Threads of a row: enough for four quads each, 32 to 512.
int bwd_lanes(int d) {
  int n = 32;
  while (n < kBwdThreads && n * 16 < d) n *= 2;
  return n;
}

template <int CH, int FMT>
bool norm_bwd8(const uint8_t* q, const float* scale, const bf16* g, const float* rstd,
               const float* dy, const float* dres, float* dx, bf16* dxb, float* dg_part, int parts,
               int64_t rows, int d, cudaStream_t st) {
  using R = BwdRing<CH>;
  if (!reserve_smem<norm_bwd8_kernel<CH, FMT>>(R::STAGES * R::STAGE)) return false;
  const int lanes = bwd_lanes(d);
  const int64_t per = (rows + (int64_t)parts * (kBwdThreads / lanes) - 1) / ((int64_t)parts * (kBwdThreads / lanes));
  // few rows a group: no more of the ring than they use
  const int smem = (int)(per < R::STAGES ? per : R::STAGES) * R::STAGE;
  norm_bwd8_kernel<CH, FMT><<<parts, kBwdThreads, smem, st>>>(q, scale, g, rstd, dy, dres, dx, dxb, dg_part, rows,
                                                              (d + kBlock - 1) / kBlock, d, lanes);
  return true;
}

template <int FMT>
bool norm_bwd8_any(const uint8_t* q, const float* scale, const bf16* g, const float* rstd,
                   const float* dy, const float* dres, float* dx, bf16* dxb, float* dg_part,
                   int parts, int64_t rows, int d, cudaStream_t st) {
  if (d <= 4 * 4 * kBwdThreads)
    return norm_bwd8<4, FMT>(q, scale, g, rstd, dy, dres, dx, dxb, dg_part, parts, rows, d, st);
  if (d <= 6 * 4 * kBwdThreads)
    return norm_bwd8<6, FMT>(q, scale, g, rstd, dy, dres, dx, dxb, dg_part, parts, rows, d, st);
  return norm_bwd8<8, FMT>(q, scale, g, rstd, dy, dres, dx, dxb, dg_part, parts, rows, d, st);
}

}  // namespace

void ckpt8_save(const float* x, uint8_t* q, float* scale, int fmt, int64_t rows, int d,
                cudaStream_t st) {
  const int nb = (d + kBlock - 1) / kBlock, per = kThreads / 32 * kCopyBlocks;
  const int64_t blocks = rows * nb;
  const unsigned grid = (unsigned)((blocks + per - 1) / per);
  if (fmt == SF_CKPT_INT8)
    save_kernel<SF_CKPT_INT8><<<grid, kThreads, 0, st>>>(x, q, scale, blocks, nb, d);
  else
    save_kernel<SF_CKPT_E4M3><<<grid, kThreads, 0, st>>>(x, q, scale, blocks, nb, d);
}

void ckpt8_load(const uint8_t* q, const float* scale, float* x, int fmt, int64_t rows, int d,
                cudaStream_t st) {
  const int nb = (d + kBlock - 1) / kBlock, per = kThreads / 32 * kCopyBlocks;
  const int64_t blocks = rows * nb;
  const unsigned grid = (unsigned)((blocks + per - 1) / per);
  if (fmt == SF_CKPT_INT8)
    load_kernel<SF_CKPT_INT8><<<grid, kThreads, 0, st>>>(q, scale, x, blocks, nb, d);
  else
    load_kernel<SF_CKPT_E4M3><<<grid, kThreads, 0, st>>>(q, scale, x, blocks, nb, d);
}

void rmsnorm_fwd_save8(const float* x, const bf16* g, bf16* y, float* rstd, uint8_t* q,
                       float* scale, int fmt, int64_t rows, int d, float eps, cudaStream_t st) {
  if (fmt == SF_CKPT_INT8)
    norm_fwd8<SF_CKPT_INT8, false>(x, g, y, rstd, q, scale, nullptr, rows, d, eps, st);
  else
    norm_fwd8<SF_CKPT_E4M3, false>(x, g, y, rstd, q, scale, nullptr, rows, d, eps, st);
}

void rmsnorm_fwd_load8(const uint8_t* q, const float* scale, const bf16* g, bf16* y, float* rstd,
                       float* xout, int fmt, int64_t rows, int d, float eps, cudaStream_t st) {
  uint8_t* qq = const_cast<uint8_t*>(q);
  float* ss = const_cast<float*>(scale);
  if (fmt == SF_CKPT_INT8)
    norm_fwd8<SF_CKPT_INT8, true>(nullptr, g, y, rstd, qq, ss, xout, rows, d, eps, st);
  else
    norm_fwd8<SF_CKPT_E4M3, true>(nullptr, g, y, rstd, qq, ss, xout, rows, d, eps, st);
}

int rmsnorm_bwd_load8_parts(int64_t rows, int d) {
  const int groups = kBwdThreads / bwd_lanes(d), sms = num_sms();
  const int64_t need = (rows + groups - 1) / groups;
  return need < sms ? (int)(need > 0 ? need : 1) : sms;
}

bool rmsnorm_bwd_load8(const uint8_t* q, const float* scale, const bf16* g, const float* rstd,
                       const float* dy, const float* dres, float* dx, bf16* dxb, float* dg_part,
                       int parts, int fmt, int64_t rows, int d, cudaStream_t st) {
  return fmt == SF_CKPT_INT8 ? norm_bwd8_any<SF_CKPT_INT8>(q, scale, g, rstd, dy, dres, dx, dxb, dg_part,
                                                           parts, rows, d, st)
                             : norm_bwd8_any<SF_CKPT_E4M3>(q, scale, g, rstd, dy, dres, dx, dxb, dg_part,
                                                           parts, rows, d, st);
}

}  // namespace sf
