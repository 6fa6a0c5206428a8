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
// It streams its arrays once and is bound by memory traffic: 20 bytes an element
// with h in bf16.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "join.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "sf.h"
#include "sf_internal.h"

namespace sf {

namespace {

// CTAs of NT threads, as many as fit on the SMs, in groups of LANES threads that
// take a row each, so that a thread holds at most Q quads of four columns: four,
// or two with h in fp32.  Rows wider than 512 threads hold are shared by a
// cluster of CL CTAs of 256, two CTAs an SM.  A thread copies its quads of the
// rows ahead (xout, dy, dres and h, 56 or 64 bytes a quad) into its own places of
// a ring in shared memory with cp.async and reads them back itself, each array
// as soon as the row before has been read from there.  The ring has as many
// stages as fit: two of 115 KB for 512 threads, more where rows are narrow or
// arrays are not there.  dx may be dres or dy: a thread has read its quads of a row
// before it writes them, and no other touches them.  No barrier but the two
// sums of a row stands between rows, and the gains' sums of a thread's columns
// stay in its registers over all of them.
template <int NT>
constexpr int kRingBytes = NT == 512 ? 230000 : 114000;

// Places of a stage's arrays, in bytes, for the quads that a thread uses.
struct BwdRing {
  int quads = 0, stages = 0, stage = 0;
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

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
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

template <bool H32, int NT, int LANES, int CL>
__global__ void __launch_bounds__(NT, NT == 512 ? 1 : 2)
    join_bwd_kernel(JoinArgs a, const float* __restrict__ xout, const void* __restrict__ h,
                    const float* __restrict__ rstd_post, const float* __restrict__ rstd_next,
                    const float* dy, const float* dres, float* dx, void* __restrict__ dh,
                    float* __restrict__ part, BwdRing r, int* err) {
  static_assert(CL == 1 || LANES == NT, "a cluster's CTAs hold one row");
  constexpr int Q = H32 ? 2 : 4, WARPS = NT / 32, GROUPS = NT / LANES, HB = H32 ? 16 : 8;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sums[4][CL * WARPS];  // the warps' sums, of four sums in turn; the cluster's
  __shared__ __align__(8) uint64_t bars[4];
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
  int uses = 0;
  bool dead = false;  // a wait ran out: no more waits
  auto sum = [&](float v) {
    v = warp_sum(v);
    const int par = uses & 3;
    if (CL > 1) {
      const uint32_t bar = smem_u32(&bars[par]);
      if (tid == 0) mbar_arrive_expect_tx(bar, CL * WARPS * 4);
      if (lane < CL)
        st_async(mapa_shared(smem_u32(&sums[par][rank * WARPS + warp]), lane), v, mapa_shared(bar, lane));
      if (!dead && !mbar_wait(bar, (uses >> 2) & 1, nullptr)) {
        record_error(err, kDevJoinTimeout);
        dead = true;
      }
      v = lane < CL * WARPS ? sums[par][lane] : 0.f;
      if (CL * WARPS > 32) v += sums[par][32 + lane];
      v = warp_sum(v);
    } else if (LANES > 32) {
      if (lane == 0) sums[par][warp] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(LANES) : "memory");
      constexpr int n = LANES / 32;
      v = warp_sum(lane < n ? sums[par][group * n + lane] : 0.f);
    }
    ++uses;
    return v;
  };
  // the copies of a row into a stage, in two parts: what the second sum needs
  // no more, and the rest
  auto issue_x = [&](int64_t row, int stage) {
    if (row >= a.rows) return;
    const uint32_t st = base + (uint32_t)(stage * r.stage);
    const int64_t from = row * a.d + 4 * first;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      if (first + k * LANES < q1) {
        if (next) {
          cp_async16(st + k * NT * 16, xout + from + k * LANES * 4);
          cp_async16(st + r.dy + k * NT * 16, dy + from + k * LANES * 4);
        }
        if (dres) cp_async16(st + r.dres + k * NT * 16, dres + from + k * LANES * 4);
      }
    }
  };
  auto issue_h = [&](int64_t row, int stage) {
    if (row < a.rows) {
      const uint32_t st = base - tid * 16 + (uint32_t)(stage * r.stage);
      const int64_t from = row * a.d + 4 * first;
      if (gains) {
#pragma unroll
        for (int k = 0; k < Q; ++k) {
          if (first + k * LANES < q1) {
            const uint32_t to = st + r.h + (uint32_t)(tid * HB + k * NT * HB);
            if (H32) cp_async16(to, static_cast<const float*>(h) + from + k * LANES * 4);
            else cp_async8(to, static_cast<const bf16*>(h) + from + k * LANES * 4);
          }
        }
      }
      if (lane == 0 && next) cp_async4(st + r.stats + warp * 8, rstd_next + row);
      if (lane == 1 && post) cp_async4(st + r.stats + warp * 8 + 4, rstd_post + row);
    }
    cp_async_commit();
  };
  const int64_t stride = (int64_t)(gridDim.x / CL) * GROUPS;
  const int64_t row0 = (int64_t)(blockIdx.x / CL) * GROUPS + group;
  for (int k = 0; k < r.stages; ++k) {
    issue_x(row0 + k * stride, k);
    issue_h(row0 + k * stride, k);
  }
  if (CL > 1) {
    if (tid == 0) {
      for (int k = 0; k < 4; ++k) mbar_init(smem_u32(&bars[k]), 1);
      fence_mbar_init();
    }
    cluster_sync_all();  // the peers' shared memory may be written
  }
  int stage = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.rows; row += stride) {
    const int64_t at = row * a.d + 4 * first;
    uint2 words[Q];
    if (a.drop.top) row_words<Q>(row * n4 + q0, t, LANES, offset, a.drop.seed, words);
    wait_stage(r.stages);
    __syncwarp();
    const uint8_t* st = ring + stage * r.stage;
    const float4* sx = reinterpret_cast<const float4*>(st) + tid;
    const float4* sdy = reinterpret_cast<const float4*>(st + r.dy) + tid;
    const float4* sdr = reinterpret_cast<const float4*>(st + r.dres) + tid;
    const float* stats = reinterpret_cast<const float*>(st + r.stats) + warp * 2;
    auto load_hh = [&](int k) {
      if (H32) return reinterpret_cast<const float4*>(st + r.h)[k * NT + tid];
      return unpack4(reinterpret_cast<const uint2*>(st + r.h)[k * NT + tid]);
    };
    const float r2 = next ? stats[0] : 0.f, r1 = post ? stats[1] : 1.f;
    float c1 = 0.f;
    if (next) {
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        if (first + k * LANES < q1) {
          const float4 p = mul(sx[k * NT], sdy[k * NT]);
          add_mul(next_sum[k], p, r2);
          c1 += dot(p, unpack4(gn[k]));
        }
      }
      c1 = sum(c1) / a.d * r2 * r2 * r2;  // in this order: r2^3 alone may overflow
    }
    float4 dv[Q];
    float c2 = 0.f;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      if (first + k * LANES < q1) {
        float4 o = zero;
        if (dres) o = sdr[k * NT];
        if (next) {
          add_mul(o, mul(unpack4(gn[k]), sdy[k * NT]), r2);
          add_mul(o, sx[k * NT], -c1);
        }
        *reinterpret_cast<float4*>(dx + at + k * LANES * 4) = mul(o, a.alpha);
        o = mul(o, factor);
        if (a.drop.top) o = pick(o, words[k], a.drop.top);
        dv[k] = mul(o, w[k]);
        if (gains) {
          const float4 hv = load_hh(k);
          add_mul(branch_sum[k], mul(hv, o), r1);
          c2 += dot(hv, dv[k]);
        }
      }
    }
    issue_x(row + r.stages * stride, stage);
    if (post) c2 = sum(c2) / a.d * r1 * r1 * r1;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      if (first + k * LANES < q1) {
        float4 o = dv[k];
        if (post) {
          o = mul(o, r1);
          add_mul(o, load_hh(k), -c2);
        }
        store_h<H32>(dh, at + k * LANES * 4, o);
      }
    }
    __syncwarp();  // the warp's statistics have been read: the next copies may replace them
    issue_h(row + r.stages * stride, stage);
    stage = stage + 1 == r.stages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  if (CL > 1) cluster_sync_all();  // no peer writes here any more
  allow_dependents();
  if (!part) return;
  // the groups hold the same columns: joined in their order
  float4* join = reinterpret_cast<float4*>(ring);  // [groups][quads * LANES]
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float4* out = reinterpret_cast<float4*>(part + ((int64_t)(blockIdx.x / CL) * 2 + s) * a.d);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < Q; ++k)
      if (k < r.quads) join[(group * r.quads + k) * LANES + t] = s ? branch_sum[k] : next_sum[k];
    __syncthreads();
    for (int i = tid; i < q1 - q0; i += NT) {
      float4 v = join[i];
      for (int u = 1; u < GROUPS; ++u) {
        const float4 x = join[u * r.quads * LANES + i];
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
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

// How a row of d columns is shared out: threads of a CTA, of a row within it,
// and CTAs of a row.
struct BwdShape {
  int threads, lanes, ctas;
};
BwdShape bwd_shape(int d, bool h32) {
  const int cols = h32 ? 8 : 16;  // of a thread
  int n = 32;
  while (n < 512 && n * cols < d) n *= 2;
  if (n * cols >= d) return {512, n, 1};
  int c = 2;
  while (c * 256 * cols < d) c *= 2;
  return {256, 256, c};
}
// CTAs (clusters, where ctas > 1) that all SMs hold at a time, at most.
int bwd_most(const BwdShape& s) { return num_sms() * (512 / s.threads) / s.ctas; }
int bwd_parts(int64_t rows, const BwdShape& s, int most) {
  const int groups = s.threads / s.lanes;
  const int64_t need = (rows + groups - 1) / groups;
  return need < most ? (int)(need > 0 ? need : 1) : most;
}

BwdRing bwd_ring(const JoinArgs& a, const BwdShape& s, bool h32, bool dres, int parts) {
  const int n4 = a.d / 4, each = ((n4 + s.ctas - 1) / s.ctas + 1) & ~1;
  BwdRing r;
  r.quads = (each + s.lanes - 1) / s.lanes;
  const int per = r.quads * s.threads;
  const bool next = a.g_next != nullptr, gains = a.g_post || a.gate;
  int at = next ? per * 16 : 0;
  r.dy = at;
  at += next ? per * 16 : 0;
  r.dres = at;
  at += dres ? per * 16 : 0;
  r.h = at;
  at += gains ? per * (h32 ? 16 : 8) : 0;
  r.stats = at;
  r.stage = at + s.threads / 32 * 8;
  const int64_t groups = (int64_t)parts * (s.threads / s.lanes), rows = (a.rows + groups - 1) / groups;
  const int bytes = s.threads == 512 ? kRingBytes<512> : kRingBytes<256>;
  for (int n : {1, 2, 3, 4, 8})
    if (n == 1 || (n * r.stage <= bytes && n <= rows)) r.stages = n;
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
template <bool H32, int NT, int LANES, int CL>
int launch_bwd(const BwdCall& c) {
  constexpr auto kern = join_bwd_kernel<H32, NT, LANES, CL>;
  if (!reserve_smem<kern>(kRingBytes<NT>)) return 0;
  const BwdShape s = {NT, LANES, CL};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(NT);
  cfg.stream = c.st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int most = bwd_most(s);
  if (CL > 1) {  // clusters that are resident at once: more would take a second turn
    cfg.gridDim = dim3((unsigned)(CL * most));
    cfg.dynamicSmemBytes = kRingBytes<NT>;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return 0;
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
  switch (s.ctas * s.lanes) {
    case 32: return launch_bwd<H32, 512, 32, 1>(c);
    case 64: return launch_bwd<H32, 512, 64, 1>(c);
    case 128: return launch_bwd<H32, 512, 128, 1>(c);
    case 256: return launch_bwd<H32, 512, 256, 1>(c);
    case 512: return launch_bwd<H32, 512, 512, 1>(c);
    case 1024: return launch_bwd<H32, 256, 256, 4>(c);
    default: return launch_bwd<H32, 256, 256, H32 ? 8 : 4>(c);
  }
}

}  // namespace

int join_bwd_parts(int64_t rows, int d) {
  const BwdShape s = bwd_shape(d, false), t = bwd_shape(d, true);
  const int p = bwd_parts(rows, s, bwd_most(s)), q = bwd_parts(rows, t, bwd_most(t));
  return p > q ? p : q;
}

bool join_bwd(const JoinArgs& a, const float* xout, const void* h, bool h32, const float* rstd_post,
              const float* rstd_next, const float* dy, const float* dres, float* dx, void* dh,
              bf16* dg_post, bf16* dgate, bf16* dg_next, float* part, int* err, cudaStream_t st) {
  if (!dg_post && !dgate && !dg_next) part = nullptr;
  const BwdShape s = bwd_shape(a.d, h32);
  const BwdCall c = {a, xout, h, rstd_post, rstd_next, dy, dres, dx, dh, part, err, st};
  const int parts = h32 ? launch_bwd_for<true>(s, c) : launch_bwd_for<false>(s, c);
  if (parts && part)
    launch_dependent(join_sums_kernel, dim3((unsigned)((a.d + 31) / 32), 2), 1024, 0, st, a, part, parts, dg_post,
                     dgate, dg_next);
  return parts > 0;
}

}  // namespace sf
