// What the kernels of dropout and of the residual join share (join.cu, join_bwd.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sf_internal.h"

namespace sf {

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

__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
__device__ __forceinline__ float4 unpack4(uint2 u) {
  const float2 a = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}

// ------------------------------------------------------------------ the join
// A thread's quads of four columns; h is bf16 or fp32.
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
  return fmaf(a.x, b.x, a.y * b.y) + fmaf(a.z, b.z, a.w * b.w);
}
// The elements of a quad that its two words keep, and 0 for the others.
__device__ __forceinline__ float4 pick(const float4& a, uint2 w, uint32_t top) {
  return make_float4(keep_lo(w.x, top) ? a.x : 0.f, keep_hi(w.x, top) ? a.y : 0.f, keep_lo(w.y, top) ? a.z : 0.f,
                     keep_hi(w.y, top) ? a.w : 0.f);
}

// The words of two of a thread's quads, `quad` and, `lanes` further, another, both
// counted from the start of the tensor.  Two neighbouring lanes hold the two
// halves of each octet: the even one asks the generator for the octet of both
// first quads, the odd one for that of the second.
__device__ __forceinline__ void pair_words(int64_t quad, int lanes, bool odd, uint64_t offset, uint64_t seed,
                                           uint2& first, uint2& second) {
  const Words w = philox((uint64_t)((quad + (odd ? lanes : 0)) >> 1), offset, seed);
  const uint2 mine = odd ? make_uint2(w.c, w.d) : make_uint2(w.a, w.b);
  const uint2 theirs = odd ? make_uint2(w.a, w.b) : make_uint2(w.c, w.d);
  const uint2 got = make_uint2(__shfl_xor_sync(0xffffffffu, theirs.x, 1), __shfl_xor_sync(0xffffffffu, theirs.y, 1));
  first = odd ? got : mine;
  second = odd ? mine : got;
}

}  // namespace sf
