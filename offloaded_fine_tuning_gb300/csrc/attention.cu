// Causal grouped-query attention: the small memory-bound kernels around the
// tcgen05 forward and backward (attention_tc.cu).
//
// Inputs come straight from the QKV projection's output row [T, (Hq+2Hkv)*hd]
// (token t = b*S + s): query head h at column h*hd, kv head g at (Hq+g)*hd
// (K) and (Hq+Hkv+g)*hd (V); query head h reads kv head h / (Hq/Hkv).
//
// attn_delta: D = rowsum(dO * O) per (token, head), the softmax-gradient term.
// attn_dq_finalize: dQ from the fp32 accumulation of the backward kernel
// (one buffer, or one slot per 128-key block summed in key order when the
// backward runs deterministically), scaled, inverse-rotated (RoPE) and
// written as bf16 into the query columns of dqkv.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.cuh"
#include "ptx.cuh"
#include "sf_internal.h"

namespace sf {

typedef __nv_bfloat16 bf16;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// ------------------------------------------------------------------ backward
// delta[b, h, s] = sum_j dO[t, h*hd + j] * O[t, h*hd + j]: TPR = hd / 8
// threads per (token, head) row, each reading 16 bytes of O and of dO, summed
// across the row's threads with shuffles.  Consecutive rows are consecutive
// heads of a token, so a warp reads contiguous memory.  The thread also zeroes
// the same eight columns of zero [T, Hq*hd] unless that is null (the buffer
// that the backward adds dQ into).
template <int TPR>
__global__ void attn_delta_kernel(const bf16* __restrict__ o, const bf16* __restrict__ dout,
                                  float* __restrict__ delta, float* __restrict__ zero, int64_t rows,
                                  int S, int Hq) {
  constexpr int HD = TPR * 8;
  const int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t w = g / TPR;
  const int sub = (int)(g % TPR);
  float acc = 0.f;
  if (w < rows) {  // no early return: every lane takes part in the shuffles
    const int64_t off = w * HD + sub * 8;  // row w = t * Hq + h starts at t*Hq*hd + h*hd
    const uint4 a = *reinterpret_cast<const uint4*>(o + off);
    const uint4 c = *reinterpret_cast<const uint4*>(dout + off);
    if (zero) {
      float4* z = reinterpret_cast<float4*>(zero + off);
      z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a);
    const __nv_bfloat162* c2 = reinterpret_cast<const __nv_bfloat162*>(&c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __bfloat1622float2(a2[i]), y = __bfloat1622float2(c2[i]);
      acc += x.x * y.x + x.y * y.y;
    }
  }
#pragma unroll
  for (int k = TPR / 2; k > 0; k >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, k);
  if (sub == 0 && w < rows) {
    const int64_t t = w / Hq;
    const int h = (int)(w % Hq);
    const int64_t b = t / S, s = t % S;
    delta[(b * Hq + h) * S + s] = acc;
  }
}

// dQ = scale * (sum of the fp32 partials), inverse RoPE, into the query
// columns of dqkv (8 pairs per thread).  slots == 0: one accumulated buffer
// [T, Hq*hd]; else slot j [T, Hq*hd] holds key block j's part, written for
// positions s >= 128 j, and the parts are added in the order j = 0, 1, ...
// With a window (> 0) only the sinks' key blocks and those from the start of
// the window of s's query block (128 queries) have parts, the latter in slots that blocks take in turn.
__global__ void attn_dq_kernel(const float* __restrict__ dq_acc, bf16* __restrict__ dqkv,
                               int64_t tokens, int S, int Hq, int Hkv, int hd, float scale,
                               const float2* __restrict__ cs, int slots, int window, int sinks) {
  wait_primary();
  const int half = hd / 2, groups = half / 8;
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= tokens * Hq * groups) return;
  const int gr = (int)(idx % groups);
  const int64_t th = idx / groups;
  const int h = (int)(th % Hq);
  const int64_t t = th / Hq;
  const int s = (int)(t % S);
  const int64_t ld = (int64_t)Hq * hd;
  const int ns = window > 0 ? (sinks + 127) / 128 : 0;
  const int wb = window > 0 ? max(0, s / 128 * 128 - window + 1) / 128 : 0;
  auto slot_of = [&](int j) -> int64_t {
    return window > 0 && j >= ns ? ns + (j - ns) % attn_window_slots(window) : j;
  };
  const int first = slots > 0 && ns == 0 ? wb : 0;
  const float* base = dq_acc + t * ld + (int64_t)h * hd + gr * 8;
  const float* src = base + (slots > 0 ? slot_of(first) : 0) * tokens * ld;
  bf16* dst = dqkv + t * (int64_t)(Hq + 2 * Hkv) * hd + (int64_t)h * hd + gr * 8;
  float x1[8], x2[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    float4 a = *reinterpret_cast<const float4*>(src + i);
    float4 c = *reinterpret_cast<const float4*>(src + half + i);
    x1[i] = a.x; x1[i + 1] = a.y; x1[i + 2] = a.z; x1[i + 3] = a.w;
    x2[i] = c.x; x2[i + 1] = c.y; x2[i + 2] = c.z; x2[i + 3] = c.w;
  }
  const int last = slots > 0 ? s / 128 : 0;
  for (int j = first + 1; j <= last; ++j) {
    if (j >= ns && j < wb) continue;
    const float* p = base + slot_of(j) * tokens * ld;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      float4 a = *reinterpret_cast<const float4*>(p + i);
      float4 c = *reinterpret_cast<const float4*>(p + half + i);
      x1[i] += a.x; x1[i + 1] += a.y; x1[i + 2] += a.z; x1[i + 3] += a.w;
      x2[i] += c.x; x2[i + 1] += c.y; x2[i + 2] += c.z; x2[i + 3] += c.w;
    }
  }
  uint32_t o1[4], o2[4];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float a1 = x1[i] * scale, b1 = x1[i + 1] * scale, a2 = x2[i] * scale, b2 = x2[i + 1] * scale;
    if (cs) {
      const float2 ca = cs[(int64_t)s * half + gr * 8 + i], cb = cs[(int64_t)s * half + gr * 8 + i + 1];
      const float y1a = a1 * ca.x + a2 * ca.y, y2a = a2 * ca.x - a1 * ca.y;
      const float y1b = b1 * cb.x + b2 * cb.y, y2b = b2 * cb.x - b1 * cb.y;
      a1 = y1a; a2 = y2a; b1 = y1b; b2 = y2b;
    }
    o1[i / 2] = pack2(a1, b1);
    o2[i / 2] = pack2(a2, b2);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
  *reinterpret_cast<uint4*>(dst + half) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
}

// dK and dV of the first blocks * 128 keys from the backward's partial sums
// [B, Hkv, blocks, splits + 1, dK | dV, 128, hd]: part 0 has every key, the
// others the sinks alone; they are added in their order.  dK is scaled and
// rotated back as dQ is.  A thread takes 8 pairs of dK and the same of dV.
__global__ void attn_sink_join_kernel(const float* __restrict__ part, bf16* __restrict__ dqkv,
                                      int64_t rows, int S, int Hq, int Hkv, int hd, float scale,
                                      const float2* __restrict__ cs, int blocks, int splits,
                                      int sinks) {
  wait_primary();
  const int half = hd / 2, groups = half / 8;
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t row = idx / groups;  // (b, g, key)
  if (row >= rows) return;
  const int gr = (int)(idx - row * groups);
  const int64_t bg = row / (blocks * 128);
  const int key = (int)(row - bg * (blocks * 128)), j = key / 128;
  if (key >= S) return;
  const int64_t step = (int64_t)256 * hd;  // floats of a part
  const float* src = part + ((bg * blocks + j) * (splits + 1) * 256 + (key & 127)) * hd + gr * 8;
  const int n = key < sinks ? splits + 1 : 1;
  float x[4][8] = {};  // dK at gr * 8 and half + gr * 8, dV there
  for (int c = 0; c < n; ++c, src += step)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4* v = reinterpret_cast<const float4*>(src + (u >> 1) * 128 * hd + (u & 1) * half);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[u][4 * i] += v[i].x;
        x[u][4 * i + 1] += v[i].y;
        x[u][4 * i + 2] += v[i].z;
        x[u][4 * i + 3] += v[i].w;
      }
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = x[0][i] * scale, b = x[1][i] * scale;
    const float2 c = cs ? cs[(int64_t)key * half + gr * 8 + i] : make_float2(1.f, 0.f);
    x[0][i] = a * c.x + b * c.y;
    x[1][i] = b * c.x - a * c.y;
  }
  const int64_t b = bg / Hkv;
  const int g = (int)(bg - b * Hkv);
  bf16* dst = dqkv + (b * S + key) * (int64_t)(Hq + 2 * Hkv) * hd + (int64_t)(Hq + g) * hd + gr * 8;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *reinterpret_cast<uint4*>(dst + (u >> 1) * (int64_t)Hkv * hd + (u & 1) * half) =
        make_uint4(pack2(x[u][0], x[u][1]), pack2(x[u][2], x[u][3]), pack2(x[u][4], x[u][5]),
                   pack2(x[u][6], x[u][7]));
}

// CTAs of 256 threads for that many threads
static dim3 grid256(int64_t threads) { return dim3((unsigned)((threads + 255) / 256)); }

void attn_delta(const bf16* o, const bf16* dout, float* delta, float* zero, int B, int S, int Hq,
                int hd, cudaStream_t st) {
  const int64_t rows = (int64_t)B * S * Hq;
  const dim3 grid = grid256(rows * (hd / 8));
  if (hd == 128)
    attn_delta_kernel<16><<<grid, 256, 0, st>>>(o, dout, delta, zero, rows, S, Hq);
  else
    attn_delta_kernel<8><<<grid, 256, 0, st>>>(o, dout, delta, zero, rows, S, Hq);
}

void attn_dq_finalize(const float* dq_acc, bf16* dqkv, int B, int S, int Hq, int Hkv, int hd,
                      float scale, const float2* cs, int slots, int window, int sinks,
                      cudaStream_t st) {
  const int64_t T = (int64_t)B * S;
  const int64_t n = T * Hq * (hd / 16);
  launch_dependent(attn_dq_kernel, grid256(n), 256, 0, st, dq_acc, dqkv, T, S, Hq, Hkv, hd, scale, cs, slots, window, sinks);
}

void attn_sink_join(const float* part, bf16* dqkv, int B, int S, int Hq, int Hkv, int hd,
                    float scale, const float2* cs, int splits, int sinks, cudaStream_t st) {
  const int blocks = (sinks + 127) / 128;
  const int64_t rows = (int64_t)B * Hkv * blocks * 128;
  launch_dependent(attn_sink_join_kernel, grid256(rows * (hd / 16)), 256, 0, st, part, dqkv, rows, S, Hq, Hkv,
                   hd, scale, cs, blocks, splits, sinks);
}

}  // namespace sf
