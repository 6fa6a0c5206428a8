// Norms of queries and keys for each head, with the rotary embedding in the
// same pass, forward and backward.
//
// A head x of hd columns (bf16) becomes z = g * x * r, r = 1 / sqrt(mean(x^2)
// + eps), and then y = z rotated: pair (j, j + hd/2) by the angle of its
// token's position.  Backward: dz is dy rotated back, and with xh = x * r
//   dg += dz * xh,   dx = r * (g dz - xh * mean(g dz xh)).
// r comes from x again in the backward (a sum over one head), so the forward
// stores nothing but y.
//
// Both directions only stream rows, so both are bound by memory traffic.  A
// head is held by TPH lanes (hd / 16, rounded up to a power of two); a lane
// has eight columns of each half, i.e. eight whole pairs, so the rotation
// needs no exchange and the sums take log2(TPH) shuffles.  Every load and
// store is 16 bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "sf_internal.h"

namespace sf {

namespace {

typedef __nv_bfloat16 bf16;

constexpr int kQkThreads = 256;
constexpr int kQkWarps = kQkThreads / 32;
constexpr int kQkFwdSteps = 4;  // head groups a warp has in flight, forward
constexpr int kQkBwdSteps = 2;  // and backward (x and dy)

__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 pack(const float* f) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}

template <int TPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = TPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// (cos, sin) of the lane's eight pairs at token t; a position outside the
// table is recorded and not rotated.
__device__ __forceinline__ void rotation(const QkNormArgs& a, int64_t t, int sub, float (&co)[8],
                                         float (&si)[8], int* err) {
  const int p = a.pos ? a.pos[t] : (int)(t % a.seq);
  if (p < 0 || p >= a.seq) {
    record_error(err, kDevBadPosition);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      co[i] = 1.f;
      si[i] = 0.f;
    }
    return;
  }
  const float4* row = reinterpret_cast<const float4*>(a.cs + (int64_t)p * (a.hd / 2) + 8 * sub);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = row[i];
    co[2 * i] = v.x;
    si[2 * i] = v.y;
    co[2 * i + 1] = v.z;
    si[2 * i + 1] = v.w;
  }
}

// One warp per token and chunk of kQkFwdSteps groups of 32 / TPH heads; the
// heads from Hq + Hkv on (the values) are copied.
template <int TPH>
__global__ void __launch_bounds__(kQkThreads)
    qknorm_fwd_kernel(const QkNormArgs a, const bf16* x, int64_t ldx, bf16* y,
                      int64_t ldy, int heads, int chunks, int* err) {
  constexpr int G = 32 / TPH;
  const int lane = threadIdx.x & 31, sub = lane % TPH, slot = lane / TPH;
  const int64_t unit = (int64_t)blockIdx.x * kQkWarps + (threadIdx.x >> 5);
  const int64_t t = unit / chunks;
  const int h0 = (int)(unit - t * chunks) * (kQkFwdSteps * G) + slot;
  if (t >= a.tokens) return;
  const int half = a.hd / 2;
  const bool in = 8 * sub < half;
  uint4 lo[kQkFwdSteps], hi[kQkFwdSteps];
#pragma unroll
  for (int u = 0; u < kQkFwdSteps; ++u) {
    const int h = h0 + u * G;
    lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
    if (in && h < heads) {
      const bf16* p = x + t * ldx + (int64_t)h * a.hd + 8 * sub;
      lo[u] = *reinterpret_cast<const uint4*>(p);
      hi[u] = *reinterpret_cast<const uint4*>(p + half);
    }
  }
  float co[8], si[8];
  uint4 g[2][2] = {};
  if (in) {
    rotation(a, t, sub, co, si, err);
    g[0][0] = *reinterpret_cast<const uint4*>(a.gq + 8 * sub);
    g[0][1] = *reinterpret_cast<const uint4*>(a.gq + half + 8 * sub);
    g[1][0] = *reinterpret_cast<const uint4*>(a.gk + 8 * sub);
    g[1][1] = *reinterpret_cast<const uint4*>(a.gk + half + 8 * sub);
  }
#pragma unroll
  for (int u = 0; u < kQkFwdSteps; ++u) {
    const int h = h0 + u * G;
    float x1[8], x2[8], ss = 0.f;
    unpack(lo[u], x1);
    unpack(hi[u], x2);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x1[i] * x1[i] + x2[i] * x2[i];
    ss = head_sum<TPH>(ss);
    if (!in || h >= heads) continue;
    if (h < a.Hq + a.Hkv) {
      const float r = rsqrtf(ss / a.hd + a.eps);
      float g1[8], g2[8], y1[8], y2[8];
      unpack(h < a.Hq ? g[0][0] : g[1][0], g1);
      unpack(h < a.Hq ? g[0][1] : g[1][1], g2);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z1 = x1[i] * r * g1[i], z2 = x2[i] * r * g2[i];
        y1[i] = z1 * co[i] - z2 * si[i];
        y2[i] = z2 * co[i] + z1 * si[i];
      }
      lo[u] = pack(y1);
      hi[u] = pack(y2);
    }
    bf16* p = y + t * ldy + (int64_t)h * a.hd + 8 * sub;
    *reinterpret_cast<uint4*>(p) = lo[u];
    *reinterpret_cast<uint4*>(p + half) = hi[u];
  }
}

// The heads [first, first + count) of every token with gain g: writes dx and
// adds dz * xh of the lane's columns into acc (eight of each half).
template <int TPH>
__device__ __forceinline__ void bwd_heads(const QkNormArgs& a, const bf16* __restrict__ x,
                                          int64_t ldx, const bf16* dy, int64_t lddy, bf16* dx,
                                          int64_t lddx, int first, int count, const bf16* g,
                                          float (&acc)[16], int* err) {
  constexpr int G = 32 / TPH;
  const int lane = threadIdx.x & 31, sub = lane % TPH, slot = lane / TPH;
  const int half = a.hd / 2;
  const bool in = 8 * sub < half;
  const int chunks = (count + kQkBwdSteps * G - 1) / (kQkBwdSteps * G);
  const int64_t units = a.tokens * chunks;
  const float inv_hd = 1.f / a.hd;
  float g1[8], g2[8];
  {
    uint4 a1 = make_uint4(0, 0, 0, 0), a2 = a1;
    if (in) {
      a1 = *reinterpret_cast<const uint4*>(g + 8 * sub);
      a2 = *reinterpret_cast<const uint4*>(g + half + 8 * sub);
    }
    unpack(a1, g1);
    unpack(a2, g2);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int64_t unit = (int64_t)blockIdx.x * kQkWarps + (threadIdx.x >> 5); unit < units;
       unit += (int64_t)gridDim.x * kQkWarps) {
    const int64_t t = unit / chunks;
    const int h0 = (int)(unit - t * chunks) * (kQkBwdSteps * G) + slot;
    uint4 xl[kQkBwdSteps], xh[kQkBwdSteps], dl[kQkBwdSteps], dh[kQkBwdSteps];
#pragma unroll
    for (int u = 0; u < kQkBwdSteps; ++u) {
      const int h = h0 + u * G;
      xl[u] = xh[u] = dl[u] = dh[u] = make_uint4(0, 0, 0, 0);
      if (in && h < count) {
        const int64_t c = (int64_t)(first + h) * a.hd + 8 * sub;
        xl[u] = *reinterpret_cast<const uint4*>(x + t * ldx + c);
        xh[u] = *reinterpret_cast<const uint4*>(x + t * ldx + c + half);
        dl[u] = *reinterpret_cast<const uint4*>(dy + t * lddy + c);
        dh[u] = *reinterpret_cast<const uint4*>(dy + t * lddy + c + half);
      }
    }
    float co[8], si[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) co[i] = si[i] = 0.f;
    if (in) rotation(a, t, sub, co, si, err);
#pragma unroll
    for (int u = 0; u < kQkBwdSteps; ++u) {
      const int h = h0 + u * G;
      float x1[8], x2[8], d1[8], d2[8], ss = 0.f, dot = 0.f;
      unpack(xl[u], x1);
      unpack(xh[u], x2);
      unpack(dl[u], d1);
      unpack(dh[u], d2);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += x1[i] * x1[i] + x2[i] * x2[i];
        const float z1 = d1[i] * co[i] + d2[i] * si[i], z2 = d2[i] * co[i] - d1[i] * si[i];
        d1[i] = z1;
        d2[i] = z2;
        dot += g1[i] * z1 * x1[i] + g2[i] * z2 * x2[i];
      }
      ss = head_sum<TPH>(ss);
      dot = head_sum<TPH>(dot);
      const float r = rsqrtf(ss * inv_hd + a.eps);
      const float m = r * dot * inv_hd * r;  // mean(g dz xh) * r, to multiply x by
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i] += d1[i] * (x1[i] * r);
        acc[8 + i] += d2[i] * (x2[i] * r);
        d1[i] = r * (g1[i] * d1[i] - m * x1[i]);
        d2[i] = r * (g2[i] * d2[i] - m * x2[i]);
      }
      if (in && h < count) {
        bf16* p = dx + t * lddx + (int64_t)(first + h) * a.hd + 8 * sub;
        *reinterpret_cast<uint4*>(p) = pack(d1);
        *reinterpret_cast<uint4*>(p + half) = pack(d2);
      }
    }
  }
  // the head groups of the warp hold the same columns
#pragma unroll
  for (int o = 16; o >= TPH; o >>= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
}

// Persistent CTAs: all query heads, then all key heads (so one gain and one
// set of sums is in registers at a time), then the value columns are copied.
// Every CTA writes the sums of its heads to its row of part [gridDim, 2 hd].
template <int TPH>
__global__ void __launch_bounds__(kQkThreads, 2)
    qknorm_bwd_kernel(const QkNormArgs a, const bf16* __restrict__ x, int64_t ldx, const bf16* dy,
                      int64_t lddy, bf16* dx, int64_t lddx, float* __restrict__ part, int* err) {
  __shared__ float sums[kQkWarps][2][16 * TPH];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = a.hd / 2;
  float acc[16];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    bwd_heads<TPH>(a, x, ldx, dy, lddy, dx, lddx, k ? a.Hq : 0, k ? a.Hkv : a.Hq, k ? a.gk : a.gq,
                   acc, err);
    if (lane < TPH) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[warp][k][8 * lane + i] = acc[i];
        sums[warp][k][8 * TPH + 8 * lane + i] = acc[8 + i];
      }
    }
  }
  if (dx != dy) {
    const int n = a.Hkv * a.hd / 8;  // 16-byte pieces of a token's values
    const int64_t c0 = (int64_t)(a.Hq + a.Hkv) * a.hd;
    for (int64_t i = (int64_t)blockIdx.x * kQkThreads + threadIdx.x; i < a.tokens * n;
         i += (int64_t)gridDim.x * kQkThreads) {
      const int64_t t = i / n, c = c0 + (i - t * n) * 8;
      *reinterpret_cast<uint4*>(dx + t * lddx + c) = *reinterpret_cast<const uint4*>(dy + t * lddy + c);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.hd; i += kQkThreads) {
    const int k = i / a.hd, j = i - k * a.hd;
    const int at = j < half ? j : 8 * TPH + j - half;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kQkWarps; ++w) s += sums[w][k][at];
    part[(int64_t)blockIdx.x * 2 * a.hd + i] = s;
  }
}

// dgq[j] and dgk[j]: column sums of the partials, in a fixed order.  A CTA
// takes 32 columns; warp w adds the partials w, w + 32, ... of its lane's
// column, then the 32 sums are added in warp order.
__global__ void __launch_bounds__(1024)
    qknorm_gain_kernel(const float* __restrict__ part, int parts, int hd, bf16* __restrict__ dgq,
                       bf16* __restrict__ dgk) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (j < 2 * hd) {
#pragma unroll 8
    for (int p = w; p < parts; p += 32) s += part[(int64_t)p * 2 * hd + j];
  }
  sh[w][lane] = s;
  __syncthreads();
  if (w == 0 && j < 2 * hd) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sh[i][lane];
    if (j < hd) dgq[j] = __float2bfloat16_rn(t);
    else dgk[j - hd] = __float2bfloat16_rn(t);
  }
}

int lanes_per_head(int hd) {
  int n = 1;
  while (n * 16 < hd) n *= 2;
  return n;
}

template <int TPH>
void fwd(const QkNormArgs& a, const bf16* x, int64_t ldx, bf16* y, int64_t ldy, int* err,
         cudaStream_t st) {
  const int heads = a.Hq + (x == y ? 1 : 2) * a.Hkv;
  const int per = kQkFwdSteps * (32 / TPH);
  const int chunks = (heads + per - 1) / per;
  const int64_t grid = (a.tokens * chunks + kQkWarps - 1) / kQkWarps;
  qknorm_fwd_kernel<TPH><<<(unsigned)grid, kQkThreads, 0, st>>>(a, x, ldx, y, ldy, heads, chunks, err);
}

}  // namespace

int qknorm_parts(int64_t tokens, int Hq, int Hkv, int hd) {
  // as many CTAs as the query heads fill, at most what the SMs hold at once
  const int per = kQkBwdSteps * (32 / lanes_per_head(hd));
  const int64_t need = (tokens * ((Hq + per - 1) / per) + kQkWarps - 1) / kQkWarps;
  const int most = 2 * num_sms();
  (void)Hkv;
  return need < most ? (int)(need > 0 ? need : 1) : most;
}

void qknorm_rope_fwd(const QkNormArgs& a, const bf16* x, int64_t ldx, bf16* y, int64_t ldy,
                     int* err, cudaStream_t st) {
  switch (lanes_per_head(a.hd)) {
    case 1: return fwd<1>(a, x, ldx, y, ldy, err, st);
    case 2: return fwd<2>(a, x, ldx, y, ldy, err, st);
    case 4: return fwd<4>(a, x, ldx, y, ldy, err, st);
    case 8: return fwd<8>(a, x, ldx, y, ldy, err, st);
    default: return fwd<16>(a, x, ldx, y, ldy, err, st);
  }
}

void qknorm_rope_bwd(const QkNormArgs& a, const bf16* x, int64_t ldx, const bf16* dy, int64_t lddy,
                     bf16* dx, int64_t lddx, float* part, bf16* dgq, bf16* dgk, int* err,
                     cudaStream_t st) {
  const int parts = qknorm_parts(a.tokens, a.Hq, a.Hkv, a.hd);
#define SF_QK_BWD(T) \
  qknorm_bwd_kernel<T><<<parts, kQkThreads, 0, st>>>(a, x, ldx, dy, lddy, dx, lddx, part, err)
  switch (lanes_per_head(a.hd)) {
    case 1: SF_QK_BWD(1); break;
    case 2: SF_QK_BWD(2); break;
    case 4: SF_QK_BWD(4); break;
    case 8: SF_QK_BWD(8); break;
    default: SF_QK_BWD(16);
  }
#undef SF_QK_BWD
  qknorm_gain_kernel<<<(2 * a.hd + 31) / 32, 1024, 0, st>>>(part, parts, a.hd, dgq, dgk);
}

}  // namespace sf
