// Backward of the join of a block's output h with the residual stream
// (join.cu): x' = alpha x + beta dropout(u), u = h [/ rms(h) * g_post] [* gate],
// y = g_next x' / rms(x').  With r1 and r2 the saved 1 / rms of h and x', dres the
// gradient of x' from elsewhere, w = g_post gate and means over a row's columns:
//   D = dres + r2 g_next dy - x' r2^3 mean(g_next dy x'),   dx = alpha D,
//   v = beta dropout(D),
//   dh = r1 w v - h r1^3 mean(w v h)    (without g_post: w v),
//   dg_next = sum over rows of dy x' r2,  A = sum over rows of v h r1,
//   dg_post = gate A,  dgate = g_post A.
//
// Both means come from one pass over a row, because v is linear in D:
//   sum(w v h) = beta (sum(m w h (dres + r2 g_next dy)) - k sum(m w h x')),
// with m the kept elements' factor and k = r2^3 mean(g_next dy x').  So a row's
// threads meet once, for three sums, and everything else is a second pass.
//
// It streams its arrays once and is bound by memory traffic: 20 bytes an element
// with h in bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "join.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "sf.h"
#include "sf_internal.h"

namespace sf {

namespace {

// One CTA of 512 threads per SM, in groups of LANES threads that take a row each,
// so that a thread holds Q quads of four columns: up to four, or three with h in
// fp32.  Wider rows are shared by a cluster of CL CTAs.  A thread copies its
// quads of the rows ahead (xout, dy, dres and h, 56 or 64 bytes a quad) into its
// own places of a ring in shared memory with cp.async and reads them back itself.
// The ring has as many stages as fit: two of 115 KB, more where rows are narrow or
// arrays are not there.  dx may be dres or dy: a thread has read its quads of a
// row before it writes them, and no other touches them.  No barrier but the one
// for a row's sums stands between rows, and the gains' sums of a thread's columns
// stay in its registers over all of them.
// The loops over a thread's quads have no branches, so that the quads' chains
// run beside one another: quads beyond the row are copied as zeros and not
// stored, and what an absent array would hold is read from another one and not
// used.
// With both norms, gate and dropout: 16384 x 4096 207 us (6,470 GB/s, 0.95 of a
// copy's rate; 543 us without the ring), 8192 x 8192 203 us (0.98; 230 us with a
// barrier for each norm), 16384 x 4096 with fp32 h 249 us (0.95; 272), 4095 x 12288
// without gate and dropout 170 us (0.87; 214 us with two cluster barriers a row).
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kRingBytes = 230000;

// Places of a stage's arrays, in bytes (0 for an absent one).
struct BwdRing {
  int stages = 0, stage = 0, last = 0;     // last: the place of the last stage
  int dy = 0, dres = 0, h = 0, stats = 0;  // xout at 0; stats: a row's two rstd for each warp
};

// Wait for the oldest of the stages' copies.
__device__ __forceinline__ void wait_stage(int stages) {
  if (stages == 1) cp_async_wait<0>();
  else if (stages == 2) cp_async_wait<1>();
  else if (stages == 3) cp_async_wait<2>();
  else if (stages == 4) cp_async_wait<3>();
  else cp_async_wait<7>();
}

// 16 or 8 bytes, or as many zeros where `there` is false (nothing is read then).
__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8_if(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
}
// A float into another CTA's shared memory, counted on that CTA's mbarrier
// (shared::cluster addresses).  It orders nothing else, so it does not wait for
// this thread's stores to global memory, as a release at cluster scope does.
__device__ __forceinline__ void st_async(uint32_t addr, float v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(addr), "f"(v),
               "r"(bar)
               : "memory");
}

__device__ __forceinline__ void add_mul(float4& s, const float4& a, float b) {
  s.x = fmaf(a.x, b, s.x);
  s.y = fmaf(a.y, b, s.y);
  s.z = fmaf(a.z, b, s.z);
  s.w = fmaf(a.w, b, s.w);
}

template <bool H32, int LANES, int Q, int CL>
__global__ void __launch_bounds__(kThreads, 1)
    join_bwd_kernel(JoinArgs a, const float* __restrict__ xout, const void* __restrict__ h,
                    const float* __restrict__ rstd_post, const float* __restrict__ rstd_next,
                    const float* dy, const float* dres, float* dx, void* __restrict__ dh,
                    float* __restrict__ part, BwdRing r, int* err) {
  static_assert(CL == 1 || LANES == kThreads, "a cluster's CTAs hold one row");
  constexpr int NT = kThreads, WARPS = kWarps, GROUPS = NT / LANES;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sums[2][3][CL * WARPS];  // the warps' sums, of two rows in turn; the cluster's
  __shared__ __align__(8) uint64_t bars[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = tid / LANES, t = tid % LANES;
  const int rank = CL > 1 ? (int)cluster_ctarank() : 0;
  const int n4 = a.d >> 2, each = ((n4 + CL - 1) / CL + 1) & ~1;  // whole octets
  const int q0 = rank * each, q1 = min(q0 + each, n4);            // this CTA's quads of a row
  const int first = q0 + t;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool post = a.g_post != nullptr, next = a.g_next != nullptr;
  const bool gains = post || a.gate != nullptr;  // h is read
  uint2 gn[Q];
  float4 w[Q], next_sum[Q], branch_sum[Q];  // w: g_post * gate
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    const int i = first + k * LANES;
    next_sum[k] = branch_sum[k] = zero;
    gn[k] = next && i < q1 ? reinterpret_cast<const uint2*>(a.g_next)[i] : make_uint2(0u, 0u);
    w[k] = make_float4(1.f, 1.f, 1.f, 1.f);
    if (post && i < q1) w[k] = gain(a.g_post, i);
    if (a.gate && i < q1) w[k] = mul(w[k], gain(a.gate, i));
  }
  const uint64_t offset = a.drop.top ? launch_offset(a.drop) : 0;
  const float factor = a.beta * a.drop.scale;
  const uint32_t base = smem_u32(ring) + tid * 16;
  int uses = 0;       // a warp comes to the next row but one only after all have read this row's sums
  bool dead = false;  // a wait ran out: no more waits
  auto row_sums = [&](float (&v)[3]) {
    const int par = uses & 1;
#pragma unroll
    for (int j = 0; j < 3; ++j) v[j] = warp_sum(v[j]);
    if (CL > 1) {
      const uint32_t bar = smem_u32(&bars[par]);
      if (tid == 0) mbar_arrive_expect_tx(bar, CL * WARPS * 12);
      if (lane < CL) {
#pragma unroll
        for (int j = 0; j < 3; ++j)
          st_async(mapa_shared(smem_u32(&sums[par][j][rank * WARPS + warp]), lane), v[j], mapa_shared(bar, lane));
      }
      if (!dead && !mbar_wait(bar, (uses >> 1) & 1, nullptr)) {
        record_error(err, kDevJoinTimeout);
        dead = true;
      }
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        v[j] = lane < CL * WARPS ? sums[par][j][lane] : 0.f;
        if (CL * WARPS > 32) v[j] += sums[par][j][32 + lane];
        v[j] = warp_sum(v[j]);
      }
    } else if (LANES > 32) {
      if (lane < 3) sums[par][lane][warp] = lane == 0 ? v[0] : lane == 1 ? v[1] : v[2];
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(LANES) : "memory");
      constexpr int n = LANES / 32;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        v[j] = lane < n ? sums[par][j][group * n + lane] : 0.f;
#pragma unroll
        for (int o = n / 2; o > 0; o /= 2) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
        v[j] = __shfl_sync(0xffffffffu, v[j], 0);
      }
    }
    ++uses;
  };
  const uint32_t rows = (uint32_t)a.rows;
  auto issue = [&](uint32_t row, uint32_t stage) {
    if (row < rows) {
      const uint32_t st = base + stage;
      const int64_t from = (int64_t)row * a.d + 4 * first;
      auto copy = [&](uint32_t to, const float* p) {
#pragma unroll
        for (int k = 0; k < Q; ++k) {
          const bool there = first + k * LANES < q1;
          cp_async16_if(to + k * NT * 16, there ? p + from + k * LANES * 4 : p, there);
        }
      };
      if (next) {
        copy(st, xout);
        copy(st + r.dy, dy);
      }
      if (dres) copy(st + r.dres, dres);
      if (gains && H32) copy(st + r.h, static_cast<const float*>(h));
      if (gains && !H32) {
#pragma unroll
        for (int k = 0; k < Q; ++k) {
          const bool there = first + k * LANES < q1;
          cp_async8_if(st + r.h - tid * 8 + k * NT * 8,
                       static_cast<const bf16*>(h) + (there ? from + k * LANES * 4 : 0), there);
        }
      }
      if (lane == 0 && next) cp_async4(st - tid * 16 + r.stats + warp * 8, rstd_next + row);
      if (lane == 1 && post) cp_async4(st - tid * 16 + r.stats + warp * 8 + 4, rstd_post + row);
    }
    cp_async_commit();
  };
  // rows below 2^31, and a few strides beyond: 32 bits without a sign
  const uint32_t stride = gridDim.x / CL * GROUPS;
  uint32_t row = blockIdx.x / CL * GROUPS + group;
  for (int k = 0; k < r.stages; ++k) issue(row + k * stride, k * r.stage);
  if (CL > 1) {
    if (tid == 0) {
      for (int k = 0; k < 2; ++k) mbar_init(smem_u32(&bars[k]), 1);
      fence_mbar_init();
    }
    cluster_sync_all();  // the peers' shared memory may be written
  }
  const uint32_t ahead = r.stages * stride;
  uint32_t stage = 0;  // its place in the ring
#pragma unroll 1
  for (; row < rows; row += stride) {
    const int64_t at = (int64_t)row * a.d + 4 * first;
    uint2 words[Q] = {};
    if (a.drop.top) {
      const int64_t quad = (int64_t)row * n4 + first;
#pragma unroll
      for (int k = 0; k + 1 < Q; k += 2)
        pair_words(quad + k * LANES, LANES, t & 1, offset, a.drop.seed, words[k], words[k + 1]);
      if constexpr (Q & 1) {
        const Words x = philox((uint64_t)((quad + (Q - 1) * LANES) >> 1), offset, a.drop.seed);
        words[Q - 1] = t & 1 ? make_uint2(x.c, x.d) : make_uint2(x.a, x.b);
      }
    }
    wait_stage(r.stages);
    __syncwarp();
    const uint8_t* st = ring + stage;
    const float4* sx = reinterpret_cast<const float4*>(st) + tid;
    const float4* sdy = reinterpret_cast<const float4*>(st + r.dy) + tid;
    const float4* sdr = reinterpret_cast<const float4*>(st + r.dres) + tid;
    const float* stats = reinterpret_cast<const float*>(st + r.stats) + warp * 2;
    auto load_hh = [&](int k) {
      if (H32) return reinterpret_cast<const float4*>(st + r.h)[k * NT + tid];
      return unpack4(reinterpret_cast<const uint2*>(st + r.h)[k * NT + tid]);
    };
    const float r2 = stats[0], r1 = post ? stats[1] : 1.f;
    // dres + r2 g_next dy of quad k; the kept elements of a quad (top 0 keeps all).
    // What comes back to a dropped element counts as 0 in the sums whatever it is
    // (0 times infinity would not), so it is masked itself
    auto known = [&](int k) {
      float4 o = sdr[k * NT];
      if (!dres) o = zero;
      add_mul(o, mul(unpack4(gn[k]), sdy[k * NT]), r2);
      return o;
    };
    auto keep = [&](int k, const float4& v) { return pick(v, words[k], a.drop.top); };
    float v[3] = {0.f, 0.f, 0.f};
    if (next) {
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        const float4 x = sx[k * NT], p = mul(x, sdy[k * NT]);
        add_mul(next_sum[k], p, r2);
        v[0] += dot(p, unpack4(gn[k]));
        if (post) {
          const float4 hw = keep(k, mul(load_hh(k), w[k]));
          v[1] += dot(hw, keep(k, known(k)));
          v[2] += dot(hw, x);
        }
      }
    } else if (post) {
#pragma unroll
      for (int k = 0; k < Q; ++k) v[1] += dot(mul(load_hh(k), w[k]), keep(k, sdr[k * NT]));
    }
    if (next || post) row_sums(v);
    const float c1 = next ? v[0] / a.d * r2 * r2 * r2 : 0.f;  // in this order: r2^3 alone may overflow
    const float c2 = post ? factor * (v[1] - c1 * v[2]) / a.d * r1 * r1 * r1 : 0.f;
    // the rest of a quad from D
    auto finish = [&](int k, float4 o) {
      const bool there = first + k * LANES < q1;
      if (there) *reinterpret_cast<float4*>(dx + at + k * LANES * 4) = mul(o, a.alpha);
      o = keep(k, mul(o, factor));
      const float4 hv = load_hh(k);
      add_mul(branch_sum[k], mul(hv, o), r1);
      o = mul(mul(o, w[k]), r1);
      if (post) add_mul(o, hv, -c2);
      if (there) store_h<H32>(dh, at + k * LANES * 4, o);
    };
    if (next) {
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        float4 o = known(k);
        add_mul(o, sx[k * NT], -c1);
        finish(k, o);
      }
    } else {
#pragma unroll
      for (int k = 0; k < Q; ++k) finish(k, sdr[k * NT]);
    }
    __syncwarp();  // the warp's statistics have been read: the next copies may replace them
    issue(row + ahead, stage);
    stage = stage == (uint32_t)r.last ? 0 : stage + r.stage;
  }
  cp_async_wait<0>();
  if (CL > 1) cluster_sync_all();  // no peer writes here any more
  allow_dependents();
  if (!part) return;
  // the groups hold the same columns: joined in their order
  float4* join = reinterpret_cast<float4*>(ring);  // [groups][Q * LANES]
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float4* out = reinterpret_cast<float4*>(part + ((int64_t)(blockIdx.x / CL) * 2 + s) * a.d);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < Q; ++k)
      join[(group * Q + k) * LANES + t] = s ? branch_sum[k] : next_sum[k];
    __syncthreads();
    for (int i = tid; i < q1 - q0; i += NT) {
      float4 v = join[i];
      for (int u = 1; u < GROUPS; ++u) {
        const float4 x = join[u * Q * LANES + i];
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      out[q0 + i] = v;
    }
  }
}

// The gains' gradients from the partials [parts, 2, d], in a fixed order: a CTA
// takes 64 columns of one sum, a quad for each of 16 lanes, and 32 half warps;
// half warp w adds the partials w, w + 32, ..., then their sums are added in that
// order.
constexpr int kSumGroups = 32;

__global__ void __launch_bounds__(16 * kSumGroups)
    join_sums_kernel(JoinArgs a, const float* __restrict__ part, int parts, bf16* __restrict__ dg_post,
                     bf16* __restrict__ dgate, bf16* __restrict__ dg_next) {
  __shared__ float4 sh[kSumGroups][16];
  const int t = threadIdx.x & 15, w = threadIdx.x >> 4;
  const int s = blockIdx.y, quad = blockIdx.x * 16 + t;
  wait_primary();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (quad < a.d / 4) {
#pragma unroll 5
    for (int p = w; p < parts; p += kSumGroups) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(part + ((int64_t)p * 2 + s) * a.d) + quad);
      v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
  }
  sh[w][t] = v;
  __syncthreads();
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x >= 64 || c >= a.d) return;
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kSumGroups; ++k) sum += reinterpret_cast<const float*>(sh[k])[threadIdx.x];
  if (s == 0) {
    if (dg_next) dg_next[c] = __float2bfloat16_rn(sum);
  } else {
    if (dg_post) dg_post[c] = __float2bfloat16_rn(a.gate ? sum * __bfloat162float(a.gate[c]) : sum);
    if (dgate) dgate[c] = __float2bfloat16_rn(a.g_post ? sum * __bfloat162float(a.g_post[c]) : sum);
  }
}

// How a row of d columns is shared out: threads of a CTA, of a row within it,
// quads of a thread and CTAs of a row.
struct BwdShape {
  int lanes, quads, ctas;
};
// Whether a row of 2,049 to 4,096 columns of bf16 h has a CTA to itself (two quads for
// each of 512 threads) rather than half of one (four for 256): where its traffic hides
// a row's chain, that is with a second norm (dy and xout to read), no dropout and few
// quads beyond the row.  16384 rows, us alone and in halves: with a norm after the
// block 2304 columns 186 and 158, 3584 199 and 193, 3648 200 and 197, 3712 200 and 204,
// 4096 207 and 225; without it 2304 158 and 125, 3200 166 and 165, 3264 167 and 169,
// 4096 190 and 207.  4096 columns with dropout 240 and 211 (without a norm after the
// block 215 and 224), without a second norm 190 and 159, 157 and 128 without dropout.
// Near the borders 3000 rows differ by 8% either way.
bool row_alone(const JoinArgs& a) { return a.g_next && !a.drop.top && a.d > (a.g_post ? 3648 : 3200); }

BwdShape bwd_shape(int d, bool h32, bool alone) {
  const int few = h32 ? 2 : 4, most = h32 ? 3 : 4;
  for (int q = 1; q < few; q *= 2)
    if (32 * q * 4 >= d) return {32, q, 1};
  int n = 32;
  while (n < kThreads && n * few * 4 < d) n *= 2;
  if (!h32 && alone && n == 256) return {512, 2, 1};
  for (int c = 1;; c *= 2)
    for (int q = c == 1 ? few : 2; q <= most; ++q)
      if (c * n * q * 4 >= d) return {n, q, c};
}
// CTAs (clusters, where ctas > 1) that all SMs hold at a time, at most.
int bwd_most(const BwdShape& s) { return num_sms() > s.ctas ? num_sms() / s.ctas : 1; }
int bwd_parts(int64_t rows, const BwdShape& s, int most) {
  const int groups = kThreads / s.lanes;
  const int64_t need = (rows + groups - 1) / groups;
  return need < most ? (int)(need > 0 ? need : 1) : most;
}

BwdRing bwd_ring(const JoinArgs& a, const BwdShape& s, bool h32, bool dres, int parts) {
  const int per = s.quads * kThreads;
  const bool next = a.g_next != nullptr, gains = a.g_post || a.gate;
  BwdRing r;
  int at = next ? per * 16 : 0;
  auto place = [&](bool there, int bytes) {
    const int p = at;
    at += there ? per * bytes : 0;
    return there ? p : 0;
  };
  r.dy = place(next, 16);
  r.dres = place(dres, 16);
  r.h = place(gains, h32 ? 16 : 8);
  r.stats = at;
  r.stage = at + kWarps * 8;
  const int64_t groups = (int64_t)parts * (kThreads / s.lanes), rows = (a.rows + groups - 1) / groups;
  for (int n : {1, 2, 3, 4, 8})
    if (n == 1 || (n * r.stage <= kRingBytes && n <= rows)) r.stages = n;
  r.last = (r.stages - 1) * r.stage;
  return r;
}

// What a launch takes besides its shape.
struct BwdCall {
  JoinArgs a;
  const float* xout;
  const void* h;
  const float *rstd_post, *rstd_next, *dy, *dres;
  float* dx;
  void* dh;
  float* part;
  int* err;
  cudaStream_t st;
};

// Returns the number of partial sums, or 0: no launch.
template <bool H32, int LANES, int Q, int CL>
int launch_bwd(const BwdCall& c) {
  constexpr auto kern = join_bwd_kernel<H32, LANES, Q, CL>;
  if (!reserve_smem<kern>(kRingBytes)) return 0;
  const BwdShape s = {LANES, Q, CL};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int most = bwd_most(s);
  if (CL > 1) {  // clusters that are resident at once: more would take a second turn
    static std::atomic<int> resident[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = resident[dev].load(std::memory_order_relaxed);
    if (n == 0) {  // threads that come here first find the same number
      cfg.gridDim = dim3((unsigned)(CL * most));
      cfg.dynamicSmemBytes = kRingBytes;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return 0;
      resident[dev].store(n, std::memory_order_relaxed);
    }
    if (n < most) most = n;
  }
  const int parts = bwd_parts(c.a.rows, s, most);
  const BwdRing r = bwd_ring(c.a, s, H32, c.dres != nullptr, parts);
  cfg.gridDim = dim3((unsigned)(CL * parts));
  cfg.dynamicSmemBytes = (size_t)(r.stages * r.stage);
  return cudaLaunchKernelEx(&cfg, kern, c.a, c.xout, c.h, c.rstd_post, c.rstd_next, c.dy, c.dres, c.dx, c.dh, c.part,
                            r, c.err) == cudaSuccess
             ? parts
             : 0;
}

template <bool H32>
int launch_bwd_for(const BwdShape& s, const BwdCall& c) {
  constexpr int Q = H32 ? 2 : 4;
  if (s.ctas == 1) {
    if (s.quads == 1) return launch_bwd<H32, 32, 1, 1>(c);
    if (!H32 && s.quads == 2) return s.lanes == 32 ? launch_bwd<H32, 32, 2, 1>(c) : launch_bwd<H32, 512, 2, 1>(c);
    if (H32 && s.quads == 3) return launch_bwd<H32, 512, H32 ? 3 : Q, 1>(c);
    switch (s.lanes) {
      case 32: return launch_bwd<H32, 32, Q, 1>(c);
      case 64: return launch_bwd<H32, 64, Q, 1>(c);
      case 128: return launch_bwd<H32, 128, Q, 1>(c);
      case 256: return launch_bwd<H32, 256, Q, 1>(c);
      default: return launch_bwd<H32, 512, Q, 1>(c);
    }
  }
  if (s.quads == 3) return launch_bwd<H32, 512, 3, 2>(c);
  if constexpr (H32) {
    if (s.ctas == 4) return launch_bwd<H32, 512, 2, 4>(c);
  }
  return launch_bwd<H32, 512, Q, 2>(c);
}

}  // namespace

int join_bwd_parts(int64_t rows, int d) {
  int most = 0;
  for (const BwdShape s : {bwd_shape(d, false, false), bwd_shape(d, false, true), bwd_shape(d, true, true)}) {
    const int p = bwd_parts(rows, s, bwd_most(s));
    most = p > most ? p : most;
  }
  return most;
}

bool join_bwd(const JoinArgs& a, const float* xout, const void* h, bool h32, const float* rstd_post,
              const float* rstd_next, const float* dy, const float* dres, float* dx, void* dh,
              bf16* dg_post, bf16* dgate, bf16* dg_next, float* part, int* err, cudaStream_t st) {
  if (!dg_post && !dgate && !dg_next) part = nullptr;
  const BwdShape s = bwd_shape(a.d, h32, row_alone(a));
  const BwdCall c = {a, xout, h, rstd_post, rstd_next, dy, dres, dx, dh, part, err, st};
  const int parts = h32 ? launch_bwd_for<true>(s, c) : launch_bwd_for<false>(s, c);
  if (parts && part)
    launch_dependent(join_sums_kernel, dim3((unsigned)((a.d + 63) / 64), 2), 16 * kSumGroups, 0, st, a, part, parts, dg_post,
                     dgate, dg_next);
  return parts > 0;
}

}  // namespace sf
