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
//
// 16384 tokens, 32 + 8 + 8 heads of 128: forward 68.1 us (403 MB, 5,920 GB/s,
// 0.87 of a measured copy's rate), backward with its gain sums 97.9 us (571
// MB, 5,830 GB/s, 0.86; the sums' launch is 6 us of it); in place, where the
// value heads stay, 62 and 93 us.  With the rows in flight held by registers
// (256 threads a CTA) the first two took 79.8 and 140 us.
// 5003 packed tokens of 16 + 2 + 2 heads with positions, backward, the value
// heads copied: 25.7 us where the bytes take 11: the second phase has few steps
// to a warp, and its first rows, the rotations and the gain sums' launch are not
// hidden.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "sf_internal.h"

namespace sf {

namespace {

typedef __nv_bfloat16 bf16;

constexpr int kQkThreads = 128;
constexpr int kQkWarps = kQkThreads / 32;
// Resident CTAs an SM is given, as measured when they were chosen (the first size
// above): forward 4, 5, 6: 71.7, 68.6, 80 us; backward 3, 4, 5: 104.6, 100.3 and
// (too few registers) 166 us.
constexpr int kQkFwdCtas = 5;
constexpr int kQkBwdCtas = 4;
constexpr int kQkFwdStages = 5;  // steps a lane has in flight, forward (x)
constexpr int kQkBwdStages = 5;  // and backward (x and dy)

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

__device__ __forceinline__ uint4 lds16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}

// Head ranges that a token's steps go through: steps of 32 / TPH heads, of the
// query heads, the key heads and the value heads.
struct Steps {
  int q, k, v;
  __device__ __forceinline__ int all() const { return q + k + v; }
};

// The steps of all tokens in token order, of which each warp takes an equal
// contiguous range.  The forward (NS == 2) goes through a token's query, key and
// value steps in turn.  The backward (NS == 4) takes one kind of normed heads at a
// time; the value steps, as many as the key steps, follow these one by one, so
// that the heads that a warp sums a gain's gradient over are the same whether or
// not the value heads are copied.
// A lane copies its 16-byte pieces of the steps ahead (NS of them a step: both
// halves of x, and of dy) into its own places of a ring in shared memory, STAGES
// - 1 steps before it reads them back, so no barrier is needed and the bytes in
// flight do not depend on registers.
// body(t, kind, h, live, piece[NS]) gets the token, the kind of head (0 query,
// 1 key, 2 value), the lane's head and whether the lane holds a piece of it.
template <int TPH, int NS, int STAGES, class Body>
__device__ __forceinline__ void each_step(const QkNormArgs& a, const Steps& ss, uint32_t ring,
                                          const bf16* x, int64_t ldx, const bf16* dy, int64_t lddy,
                                          Body&& body) {
  constexpr int G = 32 / TPH;
  constexpr bool BWD = NS == 4;
  const int lane = threadIdx.x & 31, sub = lane % TPH, slot = lane / TPH;
  const int hd = a.hd, half = hd / 2;
  const bool in = 8 * sub < half;
  const int val = BWD && ss.v > 0 ? 1 : 0;  // every other step is of value heads
  const int all = ss.all(), per = all >> val;  // steps of a token, and what ranges count
  // kind and head of the lane at step i; false where it has none
  auto head = [&](int i, int& kind, int& h) -> bool {
    bool live;
    if (BWD) {
      h = (i >> val) * G + slot;
      live = in && h < (ss.q ? a.Hq : a.Hkv);
      kind = i & val ? 2 : ss.q ? 0 : 1;
    } else {
      kind = i < ss.q ? 0 : i < ss.q + ss.k ? 1 : 2;
      h = (i - (kind == 0 ? 0 : kind == 1 ? ss.q : ss.q + ss.k)) * G + slot;
      live = in && h < (kind == 0 ? a.Hq : a.Hkv);
    }
    h += kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + a.Hkv;
    return live;
  };
  const int64_t warps = (int64_t)gridDim.x * kQkWarps, n = a.tokens * per;
  const int64_t w = (int64_t)blockIdx.x * kQkWarps + (threadIdx.x >> 5);
  // warp w's range: n / warps steps, the first n % warps warps one more
  const int64_t each = n / warps, more = n - each * warps;
  const int64_t begin = w * each + (w < more ? w : more);
  const int left0 = (int)(each + (w < more ? 1 : 0)) << val;
  struct Cursor {
    int64_t t;
    int i, left;
  };
  Cursor pf{begin / per, (int)(begin % per) << val, left0}, cur = pf;
  auto advance = [&](Cursor& c) {
    --c.left;
    if (++c.i == all) {
      c.i = 0;
      ++c.t;
    }
  };
  int put = 0;
  auto issue = [&]() {
    if (pf.left > 0) {
      int kind, h;
      if (head(pf.i, kind, h)) {
        const int64_t c = (int64_t)h * hd + 8 * sub;
        const uint32_t at = ring + (uint32_t)(put * NS * kQkThreads) * 16u;
        if (NS == 2 || kind < 2) {  // of the values only the gradient is needed
          cp_async16(at, x + pf.t * ldx + c);
          cp_async16(at + kQkThreads * 16, x + pf.t * ldx + c + half);
        }
        if (NS == 4) {
          cp_async16(at + 2 * kQkThreads * 16, dy + pf.t * lddy + c);
          cp_async16(at + 3 * kQkThreads * 16, dy + pf.t * lddy + c + half);
        }
      }
      advance(pf);
    }
    cp_async_commit();
    put = put + 1 == STAGES ? 0 : put + 1;
  };
#pragma unroll 1
  for (int k = 0; k < STAGES - 1; ++k) issue();
  int get = 0;
#pragma unroll 1
  while (cur.left > 0) {
    cp_async_wait<STAGES - 2>();
    int kind, h;
    const bool live = head(cur.i, kind, h);
    uint4 piece[NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      piece[k] = make_uint4(0, 0, 0, 0);
      if (live) piece[k] = lds16(ring + (uint32_t)((get * NS + k) * kQkThreads) * 16u);
    }
    body(cur.t, kind, h, live, piece);
    // into the place that the step before this one was read from
    issue();
    advance(cur);
    get = get + 1 == STAGES ? 0 : get + 1;
  }
  cp_async_wait<0>();
}

template <int TPH>
__device__ __forceinline__ Steps steps_of(const QkNormArgs& a, bool q, bool k, bool v) {
  constexpr int G = 32 / TPH;
  const int kv = (a.Hkv + G - 1) / G;
  return {q ? (a.Hq + G - 1) / G : 0, k ? kv : 0, v ? kv : 0};
}

// Persistent CTAs; the value heads are copied unless the call is in place.
template <int TPH>
__global__ void __launch_bounds__(kQkThreads, kQkFwdCtas)
    qknorm_fwd_kernel(const QkNormArgs a, const bf16* x, int64_t ldx, bf16* y, int64_t ldy, int* err) {
  __shared__ __align__(16) uint8_t buf[2 * kQkFwdStages * kQkThreads * 16];
  const uint32_t ring = smem_u32(buf) + threadIdx.x * 16;
  const int sub = (threadIdx.x & 31) % TPH, half = a.hd / 2;
  const bool in = 8 * sub < half;
  uint4 gq1 = {}, gq2 = {}, gk1 = {}, gk2 = {};
  if (in) {
    gq1 = *reinterpret_cast<const uint4*>(a.gq + 8 * sub);
    gq2 = *reinterpret_cast<const uint4*>(a.gq + half + 8 * sub);
    gk1 = *reinterpret_cast<const uint4*>(a.gk + 8 * sub);
    gk2 = *reinterpret_cast<const uint4*>(a.gk + half + 8 * sub);
  }
  float co[8], si[8];
  int64_t at = -1;  // the token whose rotation is in co, si
  each_step<TPH, 2, kQkFwdStages>(
      a, steps_of<TPH>(a, true, true, x != y), ring, x, ldx, nullptr, 0,
      [&](int64_t t, int kind, int h, bool live, uint4 (&piece)[2]) {
        if (kind < 2) {
          if (t != at) {
            if (in) rotation(a, t, sub, co, si, err);
            at = t;
          }
          float x1[8], x2[8], g1[8], g2[8], ss = 0.f;
          unpack(piece[0], x1);
          unpack(piece[1], x2);
          unpack(kind ? gk1 : gq1, g1);
          unpack(kind ? gk2 : gq2, g2);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += x1[i] * x1[i] + x2[i] * x2[i];
          ss = head_sum<TPH>(ss);
          const float r = rsqrtf(ss / a.hd + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float z1 = x1[i] * r * g1[i], z2 = x2[i] * r * g2[i];
            x1[i] = z1 * co[i] - z2 * si[i];
            x2[i] = z2 * co[i] + z1 * si[i];
          }
          piece[0] = pack(x1);
          piece[1] = pack(x2);
        }
        if (!live) return;
        bf16* p = y + t * ldy + (int64_t)h * a.hd + 8 * sub;
        *reinterpret_cast<uint4*>(p) = piece[0];
        *reinterpret_cast<uint4*>(p + half) = piece[1];
      });
}

// Persistent CTAs: all query heads, then all key heads (so one gain and one
// set of sums is in registers at a time) with the value heads, which are copied
// unless the call is in place.
// Every CTA writes the sums of its heads to its row of part [gridDim, 2 hd].
template <int TPH>
__global__ void __launch_bounds__(kQkThreads, kQkBwdCtas)
    qknorm_bwd_kernel(const QkNormArgs a, const bf16* __restrict__ x, int64_t ldx, const bf16* dy,
                      int64_t lddy, bf16* dx, int64_t lddx, float* __restrict__ part, int* err) {
  __shared__ __align__(16) uint8_t buf[4 * kQkBwdStages * kQkThreads * 16];
  const uint32_t ring = smem_u32(buf) + threadIdx.x * 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % TPH, half = a.hd / 2;
  const bool in = 8 * sub < half;
  const float inv_hd = 1.f / a.hd;
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    float g1[8] = {}, g2[8] = {}, co[8] = {}, si[8] = {}, acc[16] = {};
    if (in) {
      const bf16* g = (k ? a.gk : a.gq) + 8 * sub;
      unpack(*reinterpret_cast<const uint4*>(g), g1);
      unpack(*reinterpret_cast<const uint4*>(g + half), g2);
    }
    int64_t at = -1;  // the token whose rotation is in co, si
    each_step<TPH, 4, kQkBwdStages>(
        a, steps_of<TPH>(a, k == 0, k == 1, k == 1 && dx != dy), ring, x, ldx, dy, lddy,
        [&](int64_t t, int kind, int h, bool live, const uint4 (&piece)[4]) {
          bf16* p = dx + t * lddx + (int64_t)h * a.hd + 8 * sub;
          if (kind == 2) {
            if (live) {
              *reinterpret_cast<uint4*>(p) = piece[2];
              *reinterpret_cast<uint4*>(p + half) = piece[3];
            }
            return;
          }
          if (t != at) {
            if (in) rotation(a, t, sub, co, si, err);
            at = t;
          }
          float x1[8], x2[8], d1[8], d2[8], ss = 0.f, dot = 0.f;
          unpack(piece[0], x1);
          unpack(piece[1], x2);
          unpack(piece[2], d1);
          unpack(piece[3], d2);
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
          if (!live) return;
          *reinterpret_cast<uint4*>(p) = pack(d1);
          *reinterpret_cast<uint4*>(p + half) = pack(d2);
        });
    // the head groups of the warp hold the same columns
#pragma unroll
    for (int o = 16; o >= TPH; o >>= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    // the warps' sums meet in the ring, which every lane has emptied
    float* sums = reinterpret_cast<float*>(buf);
    __syncthreads();
    if (lane < TPH) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[warp * 16 * TPH + 8 * lane + i] = acc[i];
        sums[warp * 16 * TPH + 8 * TPH + 8 * lane + i] = acc[8 + i];
      }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.hd; j += kQkThreads) {
      const int c = j < half ? j : 8 * TPH + j - half;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kQkWarps; ++w) s += sums[w * 16 * TPH + c];
      part[((int64_t)blockIdx.x * 2 + k) * a.hd + j] = s;
    }
    __syncthreads();
  }
  allow_dependents();
}

int lanes_per_head(int hd) {
  int n = 1;
  while (n * 16 < hd) n *= 2;
  return n;
}

// CTAs for n steps (each a group of 32 / TPH heads of a token): as many as the
// steps fill, at most per_sm for each SM.
int qk_ctas(int64_t n, int per_sm) {
  const int64_t need = (n + kQkWarps - 1) / kQkWarps;
  const int most = per_sm * num_sms();
  return need < most ? (int)(need > 0 ? need : 1) : most;
}

int64_t head_steps(int heads, int hd) {
  const int per = 32 / lanes_per_head(hd);
  return (heads + per - 1) / per;
}

}  // namespace

int qknorm_parts(int64_t tokens, int Hq, int hd) { return qk_ctas(tokens * head_steps(Hq, hd), kQkBwdCtas); }

void qknorm_rope_fwd(const QkNormArgs& a, const bf16* x, int64_t ldx, bf16* y, int64_t ldy,
                     int* err, cudaStream_t st) {
  const int grid = qk_ctas(a.tokens * (head_steps(a.Hq, a.hd) + (x == y ? 1 : 2) * head_steps(a.Hkv, a.hd)),
                           kQkFwdCtas);
#define SF_QK_FWD(T) qknorm_fwd_kernel<T><<<grid, kQkThreads, 0, st>>>(a, x, ldx, y, ldy, err)
  switch (lanes_per_head(a.hd)) {
    case 1: SF_QK_FWD(1); break;
    case 2: SF_QK_FWD(2); break;
    case 4: SF_QK_FWD(4); break;
    case 8: SF_QK_FWD(8); break;
    default: SF_QK_FWD(16);
  }
#undef SF_QK_FWD
}

void qknorm_rope_bwd(const QkNormArgs& a, const bf16* x, int64_t ldx, const bf16* dy, int64_t lddy,
                     bf16* dx, int64_t lddx, float* part, bf16* dgq, bf16* dgk, int* err,
                     cudaStream_t st) {
  const int parts = qknorm_parts(a.tokens, a.Hq, a.hd);
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
  gain_sums(part, parts, a.hd, dgq, a.hd, dgk, st);
}

}  // namespace sf
