// Causal grouped-query attention, forward and backward, on the tcgen05
// tensor cores.
//
// Forward: online softmax over key blocks (Milakov & Gimelshein 2018; the
// blocking of Dao et al., FlashAttention 2022), laid out for sm_103a.  The
// kernel is persistent: one CTA per SM walks items of two 128-query tiles in
// longest-first order.  Both tiles of an item read the same K and V blocks,
// and they take turns on the tensor core: while one tile's softmax warps turn
// S into P, the tensor core runs the other tile's O += P V and next S = Q K^T.
// Four softmax warps per tile give one thread per query row, so the row max
// and row sum need no shuffles.  P goes back into TMEM over its S columns, as
// the tensor-memory A operand of P V.
//
// Two measurements on GB300 set the shape of the softmax code.
//   - One thread issues every MMA, and each 128 x 128 x 16 MMA runs only
//     about 64 cycles.
//   - Scalar fp32 max instructions in the softmax warps slow that issuing
//     warp more than twice over.
// So the row max uses three-input maxima, the exponent arguments and row
// sums use paired fp32 instructions, and the causal mask is compiled only
// into the diagonal block's code.
//
// Operands: Q and K tiles are K-major [128 rows][hd] (128-byte swizzle, 64
// columns per box); V is the MN-major operand of P V ([128 keys][64 hd]
// boxes).  The qkv rows are read through a 3-D tensor map (column, position,
// batch), so rows past the sequence end arrive as zeros.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "launch.cuh"
#include "ptx.cuh"
#include "sf_internal.h"

namespace sf {

namespace {

// 2^x on the special-function unit (relative error ~2^-22, flushes denormals).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(a, b, c) in one instruction
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// (x, y) * c + (d, d) as one paired fp32 FMA (round to nearest)
__device__ __forceinline__ void fma2_scalar(float& x, float& y, float c, float d) {
  asm("{\n\t.reg .b64 t, u, w;\n\t"
      "mov.b64 t, {%0, %1};\n\t"
      "mov.b64 u, {%2, %2};\n\t"
      "mov.b64 w, {%3, %3};\n\t"
      "fma.rn.f32x2 t, t, u, w;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(c), "f"(d));
}

// (x, y) * c + (d0, d1) as one paired fp32 FMA (round to nearest)
__device__ __forceinline__ void fma2(float& x, float& y, float c, float d0, float d1) {
  asm("{\n\t.reg .b64 t, u, w;\n\t"
      "mov.b64 t, {%0, %1};\n\t"
      "mov.b64 u, {%2, %2};\n\t"
      "mov.b64 w, {%3, %4};\n\t"
      "fma.rn.f32x2 t, t, u, w;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(c), "f"(d0), "f"(d1));
}

// (x, y) *= (a, b) as one paired fp32 multiply
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 t, u;\n\t"
      "mov.b64 t, {%0, %1};\n\t"
      "mov.b64 u, {%2, %3};\n\t"
      "mul.rn.f32x2 t, t, u;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// (x, y) += (a, b) as one paired fp32 add
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n\t.reg .b64 t, u;\n\t"
      "mov.b64 t, {%0, %1};\n\t"
      "mov.b64 u, {%2, %3};\n\t"
      "add.rn.f32x2 t, t, u;\n\t"
      "mov.b64 {%0, %1}, t;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// The n lowest bits set (n < 0: none, n > 31: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// A sliding window with sinks (the kernels' WIN variants): query q sees key k
// when k <= q and (q - k < size or k < sinks).  The host clips both to S.
// splits: far parts of a sinks' key block in the backward (attn_window_splits).
struct AttWindow {
  int size, sinks, splits;
};

}  // namespace

// ------------------------------------------------------------------ forward, two query tiles per CTA
// The same online softmax with two 128-query tiles per CTA that share every
// K and V tile: two query heads of one kv group at the same query block when
// the group size is even, else query blocks 2p and 2p + 1 of one head (block
// 2p + 1 is then fully masked for the first tile).  Sharing halves the K/V
// bytes each tensor-core FLOP pulls from L2, and the two tiles ping-pong: the
// tensor core runs one tile's P V and next Q K^T while the other tile's
// softmax warps work, so each tile's TMEM holds one S (P written over it as
// bf16) and one O.
//
//   warp 0      TMA: one ring of K/V entries (2 at head dim 128, 4 at 64;
//               entry G + 1 carries V(G) and K(G + 1), what the MMA step of
//               block G reads), both Q tiles at an item's first block
//   warp 1      MMA issuer; TMEM owner (S0 | S1 | O0 | O1)
//   warp 2      TMA store of each staged O tile
//   warps 3-6   softmax of tile 0, one thread per query row
//   warps 7-10  softmax of tile 1
//
// Per block G the MMA thread waits once for its K/V entry, issues O0 += P0
// V, S0' = Q0 K'^T, O1 += P1 V, S1' = Q1 K'^T, and releases the entry once.
// S' overwrites the columns that held P: the tensor core
// executes one thread's MMAs in issue order, so P is read before it is
// overwritten.  A commit after S' also covers every earlier P V of the CTA,
// so once a softmax thread sees S' it may rescale its O row: no P V of its
// tile is in flight until it publishes the next P.
namespace {
constexpr int kAttFwd2Threads = 352;

template <int HD>
struct AttFwd2Cfg {
  static constexpr int TILE = HD / 64 * 16384;  // 128 rows x HD bf16
  static constexpr int NE = HD == 128 ? 2 : 4;  // stages of the K/V ring (K and V tiles each)
  static constexpr int OFF_Q = 0;  // Q of tile 0, then of tile 1
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + NE * TILE;
  static constexpr int OFF_O = OFF_V + NE * TILE;  // staging of an O tile for its TMA store
  static constexpr int OFF_BAR = OFF_O + TILE;
  static constexpr int NBAR = 13 + 2 * NE;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
};
static_assert(AttFwd2Cfg<128>::SMEM <= 232448, "forward shared memory");
}  // namespace

template <int HD, bool WIN>
__global__ void __launch_bounds__(kAttFwd2Threads, 1)
    attn_fwd_pp_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_o,
                       float* __restrict__ lse, int S, int Hq, int Hkv, int B, float scale_log2,
                       int pair_heads, AttWindow win, int* err) {
  using C = AttFwd2Cfg<HD>;
  constexpr int NB = HD / 64;  // 64-column boxes per tile
  constexpr uint32_t ID_S = umma_idesc_bf16(128, 128, false, false);
  constexpr uint32_t ID_O = umma_idesc_bf16(128, HD, false, true);
  constexpr uint32_t TMEM_COLS = 512;
  constexpr uint32_t O_COL = 256;  // O of tile t at O_COL + t * HD; S (and P) of tile t at t * 128

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem);
  const uint32_t sQ = s0 + C::OFF_Q, sK = s0 + C::OFF_K, sV = s0 + C::OFF_V, sO = s0 + C::OFF_O;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  const uint32_t b0 = smem_u32(bars);
  auto q_full = [&](int t) { return b0 + 8u * t; };
  auto q_empty = [&](int t) { return b0 + 8u * (2 + t); };
  auto s_full = [&](int t) { return b0 + 8u * (4 + t); };
  auto p_full = [&](int t) { return b0 + 8u * (6 + t); };
  auto o_done = [&](int t) { return b0 + 8u * (8 + t); };
  const uint32_t st_ready = b0 + 8u * 10;  // an O tile's rows are in the staging buffer
  const uint32_t st_free = b0 + 8u * 11;   // the staging buffer has been read by the TMA store
  const uint32_t drain = b0 + 8u * 12;
  // Entry e of the K/V ring holds K(e) in K stage e % NE and V(e - 1) in V
  // stage (e - 1) % NE, G counting key blocks over all items of the CTA: the
  // MMA step of block G reads V(G) and K(G + 1), i.e. entry G + 1, and frees
  // it at the step's end.
  auto kv_full = [&](int s) { return b0 + 8u * (13 + s); };
  auto kv_empty = [&](int s) { return b0 + 8u * (13 + C::NE + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nqb = (S + 127) / 128;
  const int grp = Hq / Hkv;
  // Items in longest-first order (every item of the most keys comes first);
  // CTA c takes items c, c + gridDim.x, ...
  const int npb = pair_heads ? nqb : (nqb + 1) / 2;  // query positions of an item
  const int per_rank = pair_heads ? (Hq / 2) * B : Hq * B;
  const int num_items = npb * per_rank;
  // The key blocks of an item: 0 .. nkv - 1, or, with a window, its first ns
  // (the sinks') and then those from ns + skip on (the window's).
  struct Item { int h0, h1, qb0, qb1, b, g, nkv, ns, skip; };
  auto item_of = [&](int t) -> Item {
    const int rank = t / per_rank, rem = t - rank * per_rank;
    Item x;
    if (pair_heads) {
      const int hp = rem % (Hq / 2);
      x.b = rem / (Hq / 2);
      x.h0 = 2 * hp;
      x.h1 = 2 * hp + 1;
      x.qb0 = x.qb1 = nqb - 1 - rank;
    } else {
      x.h0 = x.h1 = rem % Hq;
      x.b = rem / Hq;
      x.qb0 = 2 * (npb - 1 - rank);
      x.qb1 = x.qb0 + 1;
    }
    x.g = x.h0 / grp;
    x.nkv = x.qb1 + 1 < nqb ? x.qb1 + 1 : nqb;
    x.ns = x.skip = 0;
    if (WIN) {
      const int lo = x.qb0 * 128 - win.size + 1;  // the first tile's first key
      const int wb = lo > 0 ? lo / 128 : 0, sb = (win.sinks + 127) / 128;
      x.ns = sb < wb ? sb : wb;
      x.skip = wb - x.ns;
      x.nkv -= x.skip;
    }
    return x;
  };
  auto key_block = [&](const Item& x, int j) { return WIN && j >= x.ns ? j + x.skip : j; };
  // Keys of an item's j-th block that the tensor core takes: a block before the
  // window has only its sinks (rounded up to the MMAs' 16).
  auto block_keys = [&](const Item& x, int j) {
    const int n = (win.sinks - j * 128 + 15) & ~15;
    return WIN && j < x.ns && n < 128 ? n : 128;
  };

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(q_empty(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 128);
      mbar_init(o_done(t), 1);
    }
    for (int s = 0; s < C::NE; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    mbar_init(st_ready, 128);
    mbar_init(st_free, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm);
    tma_prefetch_desc(&tm_o);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    // Entries in order: entry e carries K(e) and V(e - 1); both Q tiles of an
    // item follow the entry with the item's first K (each once the previous
    // item's last S of that tile has read the buffer); a last entry carries
    // the last V alone.
    bool ok = true;
    long e = 0;  // entries issued
    int it = 0, q_issued[2] = {-1, -1};
    int pv_col = 0, pv_row = 0, pv_b = 0;  // where the previous block's V comes from
    auto entry = [&](bool with_k, int colK, int krow, int kb) -> bool {
      const int st = (int)(e % C::NE);
      if (!mbar_wait(kv_empty(st), (uint32_t)((e / C::NE) & 1) ^ 1u, abort_flag)) return false;
      mbar_arrive_expect_tx(kv_full(st), (uint32_t)((with_k ? C::TILE : 0) + (e > 0 ? C::TILE : 0)));
      if (with_k) {
#pragma unroll
        for (int c = 0; c < NB; ++c)
          tma_load_3d(sK + st * C::TILE + c * 16384, &tm, kv_full(st), colK + 64 * c, krow, kb);
      }
      if (e > 0) {
        const int vs = (int)((e - 1) % C::NE);
#pragma unroll
        for (int c = 0; c < NB; ++c)
          tma_load_3d(sV + vs * C::TILE + c * 16384, &tm, kv_full(st), pv_col + 64 * c, pv_row, pv_b);
      }
      ++e;
      return true;
    };
    for (int t = blockIdx.x; ok && t < num_items; t += gridDim.x, ++it) {
      const Item x = item_of(t);
      const int colK = (Hq + x.g) * HD, colV = (Hq + Hkv + x.g) * HD;
      for (int j = 0; j < x.nkv; ++j) {
        const int krow = key_block(x, j) * 128;
        if (!entry(true, colK, krow, x.b)) { ok = false; break; }
        pv_col = colV;
        pv_row = krow;
        pv_b = x.b;
        if (j == 0) {
          for (int tt = 0; tt < 2; ++tt) {
            if (it > 0 && !mbar_wait(q_empty(tt), (uint32_t)((it - 1) & 1), abort_flag)) { ok = false; break; }
            mbar_arrive_expect_tx(q_full(tt), C::TILE);
            const int h = tt ? x.h1 : x.h0, qb = tt ? x.qb1 : x.qb0;
#pragma unroll
            for (int c = 0; c < NB; ++c)
              tma_load_3d(sQ + tt * C::TILE + c * 16384, &tm, q_full(tt), h * HD + 64 * c, qb * 128, x.b);
            q_issued[tt] = it;
          }
          if (!ok) break;
        }
      }
    }
    if (ok && e > 0 && !entry(false, 0, 0, 0)) ok = false;  // the last V
    if (!ok) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
      // let the copies already issued land before the CTA's shared memory goes away
      for (int tt = 0; tt < 2; ++tt)
        if (q_issued[tt] >= 0) mbar_wait(q_full(tt), (uint32_t)(q_issued[tt] & 1), nullptr);
      for (long k = e - 1; k >= 0 && k >= e - C::NE; --k)
        mbar_wait(kv_full((int)(k % C::NE)), (uint32_t)((k / C::NE) & 1), nullptr);
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    bool ok = true;
    // Descriptors of the buffers' first rows; an operand at byte offset o
    // within a buffer is the base descriptor plus o / 16 (the address field
    // cannot carry: shared addresses stay below 2^18).
    const uint64_t dQ = smem_desc_sw128(sQ, 16, 1024), dK = smem_desc_sw128(sK, 16, 1024);
    const uint64_t dV = smem_desc_sw128(sV, 16384, 1024);
    // S_t = Q_t K(G)^T into the S columns of tile t
    auto issue_s = [&](int tt, long G, int keys) {
      const uint32_t id = WIN ? umma_idesc_bf16(128, keys, false, false) : ID_S;
      const uint32_t ks = (uint32_t)(G % C::NE);
      const uint64_t a0 = dQ + (uint32_t)(tt * C::TILE / 16), b0 = dK + ks * (uint32_t)(C::TILE / 16);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) / 16;
        umma_bf16(tmem_base + tt * 128, a0 + off, b0 + off, id, kk > 0 ? 1u : 0u);
      }
      umma_commit(s_full(tt));
    };
    long G = 0;  // global index of the current key block over the CTA's items
    int it = 0;
    int t = blockIdx.x;
    if (t < num_items) {  // the first item's S of both tiles
      const Item x = item_of(t);
      for (int tt = 0; ok && tt < 2; ++tt) {
        if ((tt == 0 && !mbar_wait(kv_full(0), 0, abort_flag)) || !mbar_wait(q_full(tt), 0, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        issue_s(tt, 0, block_keys(x, 0));
        if (x.nkv == 1) umma_commit(q_empty(tt));
      }
      if (ok) umma_commit(kv_empty(0));  // entry 0: K(0) alone
    }
    for (; ok && t < num_items; t += gridDim.x, ++it) {
      const Item x = item_of(t);
      const bool has_next_item = t + (int)gridDim.x < num_items;
      const Item nx = has_next_item ? item_of(t + gridDim.x) : x;
      const int nkv_next = has_next_item ? nx.nkv : 0;
      for (int j = 0; ok && j < x.nkv; ++j, ++G) {
        const bool last = j + 1 == x.nkv;
        const bool has_next = !last || has_next_item;
        const long Gn = G + 1;
        // the next block's S: the last of its item releases that item's Q tile
        const bool next_is_last = last ? nkv_next == 1 : j + 2 == x.nkv;
        const int keys = block_keys(x, j), keys_next = last ? block_keys(nx, 0) : block_keys(x, j + 1);
        const int vs = (int)(G % C::NE);
        const int es = (int)(Gn % C::NE);  // entry G + 1: V(G) and K(G + 1)
        if (!mbar_wait(kv_full(es), (uint32_t)((Gn / C::NE) & 1), abort_flag)) {
          ok = false;
          break;
        }
        for (int tt = 0; tt < 2; ++tt) {
          if (!mbar_wait(p_full(tt), (uint32_t)(G & 1), abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t bv = dV + (uint32_t)vs * (uint32_t)(C::TILE / 16);
          // O_t += P_t V: P as the tensor-memory A operand.  Two loops, as the
          // full one is on this thread's critical path: one loop that tests keys
          // before each MMA gives the same results and costs 2% (window 1024
          // at head dim 128: 283 and 289 us).
          if (WIN && keys < 128) {  // only the sinks
#pragma unroll 1
            for (int kk = 0; kk < keys / 16; ++kk)
              umma_bf16_ts(tmem_base + O_COL + tt * HD, tmem_base + tt * 128 + kk * 8, bv + kk * (2048 / 16),
                           ID_O, (j > 0 || kk > 0) ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_bf16_ts(tmem_base + O_COL + tt * HD, tmem_base + tt * 128 + kk * 8, bv + kk * (2048 / 16),
                           ID_O, (j > 0 || kk > 0) ? 1u : 0u);
          }
          if (last) umma_commit(o_done(tt));
          if (has_next) {
            if (last && !mbar_wait(q_full(tt), (uint32_t)((it + 1) & 1), abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            issue_s(tt, Gn, keys_next);
            if (next_is_last) umma_commit(q_empty(tt));
          }
        }
        if (!ok) break;
        umma_commit(kv_empty(es));  // V(G) and K(G + 1) have been read
      }
    }
    if (!ok) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
      umma_commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else if (warp == 2 && lane == 0) {
    // ---------------------------------------------------------------- O store
    bool ok = true;
    int c = 0;  // O tiles stored so far: tile 0 then tile 1 of each item
    for (int t = blockIdx.x; ok && t < num_items; t += gridDim.x) {
      const Item x = item_of(t);
      for (int tt = 0; tt < 2; ++tt, ++c) {
        if (!mbar_wait(st_ready, (uint32_t)(c & 1), abort_flag)) { ok = false; break; }
        const int h = tt ? x.h1 : x.h0, qb = tt ? x.qb1 : x.qb0;
        if (qb * 128 < S) {  // rows past the sequence end are outside the tensor map and not written
#pragma unroll
          for (int cc = 0; cc < NB; ++cc) tma_store_3d(&tm_o, sO + cc * 16384, h * HD + 64 * cc, qb * 128, x.b);
          bulk_commit_group();
          bulk_wait_group_read0();
        }
        mbar_arrive(st_free);
      }
    }
    bulk_wait_group0();
    if (!ok) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
    }
  } else if (warp >= 3) {
    // ---------------------------------------------------------------- softmax
    const int tt = (warp - 3) >> 2;
    const int quarter = warp & 3;  // TMEM lanes a warp may access: 32 x (warp % 4)
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = (uint32_t)tt * 128u, o_col = O_COL + (uint32_t)tt * HD;
    bool ok = true;
    long G = 0;
    int it = 0;
    for (int t = blockIdx.x; ok && t < num_items; t += gridDim.x, ++it) {
      const Item x = item_of(t);
      const int qb = tt ? x.qb1 : x.qb0, h = tt ? x.h1 : x.h0;
      const int q = qb * 128 + row;
      // m: the row max in log2 units that the exponentials are taken against;
      // it only moves when a block's max exceeds it by more than 8, so O in
      // TMEM is rarely rescaled (O / l does not depend on the choice of m).
      float m = -INFINITY, l = 0.f;
      // One key block (the item's j-th, block kb): S from TMEM, P back over it.
      // Compiled twice, with the mask (the diagonal block and any block past
      // it, and blocks that the window's start cuts) and without.  With a
      // window, up to a third of the blocks are cut, so the masked code works
      // by groups of 32 columns, read from TMEM once for the row max and once
      // for P: a group that none of the warp's rows sees is not read (its P is
      // 0), one that all see is not masked, and the others take one mask word
      // per row (2 x 8192 tokens, 32 / 8 heads of 128, window 1024, 4 sinks:
      // 390 us with the mask as comparisons on 128 columns, 281 us so: 920
      // TFLOP/s of visible pairs, 0.48 of the measured burst; with the cut
      // blocks 1.14 times as many pairs are multiplied).
      auto block = [&](int j, int kb, long G, auto diag) -> bool {
        constexpr bool DIAG = decltype(diag)::value;
        if (!__all_sync(0xffffffffu, mbar_wait(s_full(tt), (uint32_t)(G & 1), abort_flag))) return false;
        tc_fence_after();
        constexpr bool CUT = WIN && DIAG;
        float s[CUT ? 32 : 128];
        float mx = -INFINITY;
        // CUT: group c of 32 columns into s; false when no row of the warp sees it
        auto load_group = [&](int c) -> bool {
          const int q0 = qb * 128 + quarter * 32, kc = kb * 128 + 32 * c;
          if (kc > q0 + 31 || (kc >= win.sinks && q0 - (kc + 31) >= win.size)) return false;
          uint32_t r[32];
          tmem_ld_32x32b_x32(lane_base + s_col + 32 * c, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(r[i]);
          if (kc + 31 > q0 || (kc + 31 >= win.sinks && q0 + 31 - kc >= win.size)) {
            const uint32_t seen = low_bits(q - kc + 1) &
                                  (~low_bits(q - win.size + 1 - kc) | low_bits(win.sinks - kc));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen & (1u << i))) s[i] = -INFINITY;
          }
          return true;
        };
        if constexpr (CUT) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (!load_group(c)) continue;
            float mx4[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) mx4[a] = max3f(mx, s[a], s[4 + a]);
#pragma unroll
            for (int i = 8; i < 32; i += 8)
#pragma unroll
              for (int a = 0; a < 4; ++a) mx4[a] = max3f(mx4[a], s[i + a], s[i + 4 + a]);
            mx = fmaxf(max3f(mx4[0], mx4[1], mx4[2]), mx4[3]);
          }
        } else {
          uint32_t r[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(lane_base + s_col + 32 * c, r[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) s[32 * c + i] = __uint_as_float(r[c][i]);
          if (DIAG) {  // keys after the query are masked (every key of a block past the diagonal)
            const int lim = q - kb * 128;
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i > lim) s[i] = -INFINITY;
          }
          // row max: eight chains of three-input maxima over columns 16..127
          float mx8[8];
#pragma unroll
          for (int a = 0; a < 8; ++a) mx8[a] = fmaxf(s[a], s[a + 8]);
#pragma unroll
          for (int i = 16; i < 128; i += 16)
#pragma unroll
            for (int a = 0; a < 8; ++a) mx8[a] = max3f(mx8[a], s[i + a], s[i + 8 + a]);
          mx = max3f(max3f(mx8[0], mx8[1], mx8[2]), max3f(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        }
        mx *= scale_log2;  // the scale is positive: the max commutes with it
        const bool grow = mx > m + 8.f;
        float m_new = grow ? mx : m;
        // A window can start inside or after this block for some rows: until a
        // row has seen a key its m is -inf, and exponents are taken against 0
        // (-inf - -inf would be NaN); every p of such a row is 0.
        const bool none = CUT && m_new == -INFINITY;
        if (none) m_new = 0.f;
        const float corr = ex2_approx(m - m_new);  // 1 without growth, 0 on the first block
        // p = 2^(s * scale - m): the arguments and the partial row sums as
        // paired fp32 operations, the exponentials on the special-function unit
        float ps8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        auto exps = [&](float* v, int n) {
#pragma unroll
          for (int i = 0; i < n; i += 2) {
            fma2_scalar(v[i], v[i + 1], scale_log2, -m_new);
            v[i] = ex2_approx(v[i]);
            v[i + 1] = ex2_approx(v[i + 1]);
            add2(ps8[i & 7], ps8[(i & 7) + 1], v[i], v[i + 1]);
          }
        };
        if constexpr (CUT) {
          // P of group c takes columns 16 c to 16 c + 15, where the S of groups
          // up to c / 2 was, which has been read for the last time
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
            if (load_group(c)) {
              exps(s, 32);
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = pack2_bf16(s[2 * i], s[2 * i + 1]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = 0u;
            }
            tmem_st_32x32b_x16(lane_base + s_col + 16 * c, pk);
          }
        } else {
          exps(s, 128);
          // the row of P, bf16 pairs, over the first 64 columns of S
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = pack2_bf16(s[64 * hh + 2 * i], s[64 * hh + 2 * i + 1]);
            tmem_st_32x32b_x32(lane_base + s_col + 32 * hh, pk);
          }
        }
        const float ps = ((ps8[0] + ps8[1]) + (ps8[2] + ps8[3])) + ((ps8[4] + ps8[5]) + (ps8[6] + ps8[7]));
        l = l * corr + ps;
        m = none ? -INFINITY : m_new;
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          // every P V of this tile so far has completed (the S commit covers
          // them), and the next waits for this thread's P arrival below
#pragma unroll
          for (int c = 0; c < HD / 32; ++c) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(lane_base + o_col + 32 * c, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * corr);
            tmem_st_32x32b_x32(lane_base + o_col + 32 * c, r);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full(tt));
        return true;
      };
      for (int j = 0; j < x.nkv; ++j, ++G) {
        const int kb = key_block(x, j);
        bool masked = kb >= qb;
        if (WIN) masked = masked || (qb * 128 + 127 - kb * 128 >= win.size && kb * 128 + 127 >= win.sinks);
        ok = masked ? block(j, kb, G, std::true_type{}) : block(j, kb, G, std::false_type{});
        if (!ok) break;
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait(o_done(tt), (uint32_t)(it & 1), abort_flag));
      // the staging buffer is free once the previous O tile's store has read it
      const int c = 2 * it + tt;
      if (ok && c > 0) ok = __all_sync(0xffffffffu, mbar_wait(st_free, (uint32_t)((c - 1) & 1), abort_flag));
      if (!ok) break;
      tc_fence_after();
      const float inv = 1.f / l;
      // the O row, bf16, into the staging buffer in the tensor map's swizzled
      // layout: box c / 2 holds columns [64 (c / 2), 64 (c / 2) + 64)
      const uint32_t orow = sO + (uint32_t)row * 128u;
#pragma unroll
      for (int cc = 0; cc < HD / 32; ++cc) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(lane_base + o_col + 32 * cc, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int chunk = (cc & 1) * 4 + k;  // 16-byte chunk within the 128-byte row
          const uint32_t addr = orow + (cc >> 1) * 16384 + (uint32_t)((chunk ^ (row & 7)) * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                       "r"(pack2_bf16(__uint_as_float(r[8 * k + 0]) * inv, __uint_as_float(r[8 * k + 1]) * inv)),
                       "r"(pack2_bf16(__uint_as_float(r[8 * k + 2]) * inv, __uint_as_float(r[8 * k + 3]) * inv)),
                       "r"(pack2_bf16(__uint_as_float(r[8 * k + 4]) * inv, __uint_as_float(r[8 * k + 5]) * inv)),
                       "r"(pack2_bf16(__uint_as_float(r[8 * k + 6]) * inv, __uint_as_float(r[8 * k + 7]) * inv))
                       : "memory");
        }
      }
      // O has left TMEM: the next item's first P V of this tile (issued after
      // this thread's next P arrival) may overwrite it
      tc_fence_before();
      fence_proxy_async_smem();
      mbar_arrive(st_ready);
      if (q < S) lse[((int64_t)x.b * Hq + h) * S + q] = (m + log2f(l)) * 0.69314718055994531f;
    }
    if (!ok && lane == 0) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ backward
namespace {
// With a window: the last query that sees a key of the 128-key block at k0.
__device__ __forceinline__ int last_query(const AttWindow& win, int k0, int S) {
  const int q = k0 + 127 + win.size - 1;
  return k0 < win.sinks || q > S - 1 ? S - 1 : q;
}
// What one item of the backward works on: key block j against count query
// blocks from the first on.  slot: where the item's dK and dV go, -1 for the
// output itself, else fp32 partial sums that attn_sink_join adds.
struct KeyWork {
  int j, first, count, slot;
};
// The item of a rank, query blocks of 128.  A sinks' key block is seen by every
// later query, which would make it an item many times the others' length (2 x
// 8192 tokens, window 1024, 4 sinks: 256 steps against 36; longer than all the
// rest of the work where the sequence is long and the window short).  So the
// queries behind its window are split into win.splits items of their own, and
// its other item (slot 0) is like every key block's (1 x 16384, 16 heads in
// groups of 8, window 256, 4 sinks: head dim 128 2,479 us with one item, 303 us
// split; 64 1,987 and 223 us).  The parts come first, as they can be longer than
// the others (130 sinks there: 286 and 271 us; 364 and 356 us with them last).
//
// PART: the variants of the kernels for win.splits > 0; the decoding of items
// and the parts' epilogue are on the critical path of short items (8 x 1001, 16
// heads of 64, window 250: 85 us without, 93 us in one variant with them).
template <bool WIN, bool PART>
__device__ __forceinline__ KeyWork key_work(const AttWindow& win, int rank, int S) {
  const int nq = (S + 127) / 128;
  if (!WIN) return {rank, rank, nq - rank, -1};
  if (!PART) return {rank, rank, last_query(win, rank * 128, S) / 128 + 1 - rank, -1};
  const int ns = (win.sinks + 127) / 128, parts = ns * win.splits;
  const bool part = rank < parts;
  KeyWork w;
  w.slot = -1;
  w.j = rank - parts;
  int c = 0;
  if (part) {
    w.j = rank / win.splits;
    c = rank - w.j * win.splits;
  }
  const int seen = w.j * 128 + 127 + win.size - 1;  // the last query with a key in its window
  const int end = seen > S - 1 ? nq : seen / 128 + 1;
  w.first = w.j;
  w.count = end - w.first;
  if (part) {
    const int n = nq - end, b0 = n * c / win.splits, b1 = n * (c + 1) / win.splits;
    w.first = end + b0;
    w.count = b1 - b0;
    w.slot = c + 1;
  } else if (w.j < ns) {
    w.slot = 0;
  }
  return w;
}
// Keys of the item that have to be worked on: behind the window only the sinks
// (rounded up to the MMAs' 16 keys).
__device__ __forceinline__ int live_keys(const AttWindow& win, const KeyWork& w) {
  const int n = (win.sinks - w.j * 128 + 15) & ~15;
  return w.slot > 0 && n < 128 ? n : 128;
}
// Row r of the item's fp32 dK; its dV follows 128 rows later.
template <int HD>
__device__ __forceinline__ float* part_row(float* part, const AttWindow& win, const KeyWork& w, int g,
                                           int Hkv, int b, int r) {
  const int ns = (win.sinks + 127) / 128;
  const int64_t at = (((int64_t)b * Hkv + g) * ns + w.j) * (win.splits + 1) + w.slot;
  return part + (at * 256 + r) * HD;
}
// The deterministic variant's dQ slot of key block j: the sinks' blocks have
// their own, the others take attn_window_slots of them in turn (attn_dq_kernel
// sums the slots of a query's blocks in key order).
__device__ __forceinline__ int dq_slot(const AttWindow& win, int j) {
  const int ns = (win.sinks + 127) / 128;
  return j < ns ? j : ns + (j - ns) % attn_window_slots(win.size);
}
}  // namespace

// Backward for head_dim 64.  An item is one (128-key block j, kv head g, batch
// b): every query head of the group and every 128-query block that sees its
// keys (or a part of them, KeyWork).  The CTAs are persistent, one per SM, and take the items longest first,
// every other round in reverse order, so that long and short ones add up.  Per
// (head, block):
//   MMA:     S^T = K Q^T -> TMEM[0,128),  dP^T = V dO^T -> TMEM[128,256)
//   threads: one per key row and half of the queries: P^T = exp2(S^T*scale*
//            log2e - lse*log2e) (masked) -> TMEM[320,384) as bf16, dS^T = P^T *
//            (dP^T - D) to shared memory (bf16, swizzled)
//   MMA:     dV += P^T dO (P^T as the tensor-memory A), dK += dS^T Q
//            (TMEM[384,512), kept over the walk); dQ = dS K -> TMEM[256,320)
//   threads: one per query row and half of the columns: dQ through shared
//            memory into the fp32 dq_acc by TMA reduce-add (or, deterministic,
//            a TMA store into the key block's own slot)
// dS^T is stored once and read both as the K-major A of dK and as the MN-major
// A (dS) of dQ.  The threads release the S^T and dP^T columns once they hold
// them in registers, so the next block's are formed while they work, and dV,
// dK and dQ run behind.
//
// What bounds it: a block takes 3,900 clocks in a long walk (clock stamps).  One
// thread needs 2,550 to issue the 32 MMAs, which is shared memory's 128 bytes a
// clock: counted are 1,408 for their operands (S^T, dP^T 512, dV 128, dK 384, dQ
// 384), 256 for Q and dO coming in, 256 for dS^T and 512 for dQ through its
// staging tiles.  Another 630 it waits for P^T and dS^T, since the threads'
// chain is as long (1,450 for the exponentials and dS^T, 400 to store, 830 for
// dQ).  Four warps of their own for dQ, dK and dV leave the threads fewer
// registers, so that S^T and dP^T are released later: 268 us against 256 us (2 x
// 4096 tokens, 16 / 4 heads).  Blocks have 128 queries: 64-query blocks in two
// CTAs per SM (MMAs 64 wide read 6 KB in 32 clocks of work) lost where walks are
// long.  Whole backward, 8 x 1024 tokens, 16 heads, causal: 193 us with 64-query
// blocks, 97 us so (443 TFLOP/s).  With two Q / dO stages the
// loads of a block started only when the block two before it was done, 1,300
// cycles of waiting a block; P^T in TMEM makes room for three.  lse and D come
// from a warp of their own, two blocks ahead.  A CTA per item spent more time
// on setting up, the first loads and the last stores than on a short window's
// four blocks, so the barriers' phases count on over all items, K and V have
// two stages, and the first block of the next item is formed (S^T, P^T) before
// the previous item's dK and dV are read; those leave through that item's own
// K and V buffers.
namespace {
// TMA warp, MMA warp, 8 softmax-gradient warps, dK / dV store warp, lse / D warp
constexpr int kAttBwdThreads = 384;
struct AttBwdCfg {
  static constexpr int HD = 64;
  static constexpr int TILE = 16384;  // 128 rows x 64 hd
  static constexpr int NQ = 3;        // Q / dO stages
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = 2 * TILE;
  static constexpr int OFF_Q = 4 * TILE;  // K and V: two stages each
  static constexpr int OFF_DO = OFF_Q + NQ * TILE;
  static constexpr int OFF_DST = OFF_DO + NQ * TILE;  // 128 keys x 128 queries, two boxes of 64
  static constexpr int OFF_DQS = OFF_DST + 32768;    // dQ staging: 8 warps x [32 q][32 d] fp32
  static constexpr int OFF_LD = OFF_DQS + 8 * 4096;  // [2][lse 128 | D 128]
  static constexpr int OFF_BAR = OFF_LD + 2 * 256 * 4;
  static constexpr int NBAR = 26;
  // no room to align the base: it is 1024-byte aligned where a kernel has no
  // static shared memory, which the kernel checks
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
};
static_assert(AttBwdCfg::SMEM <= 232448, "backward shared memory");

// Division of 0 <= t < 2^31 by a fixed d: one high product and a correction (m
// = floor(2^32 / d), 2^32 - 1 for d = 1, so the estimate is the quotient or one
// less).  The roles decode items with single threads on their critical path.
struct FixedDiv {
  uint32_t d, m;
  FixedDiv(int d_) : d((uint32_t)d_), m(d_ == 1 ? 0xffffffffu : (uint32_t)((1ull << 32) / (uint32_t)d_)) {}
  __device__ __forceinline__ int operator()(int t, int& rem) const {
    uint32_t q = __umulhi((uint32_t)t, m), r = (uint32_t)t - q * d;
    if (r >= d) {
      ++q;
      r -= d;
    }
    rem = (int)r;
    return (int)q;
  }
};
}  // namespace

template <bool DET, bool WIN, bool PART>
__global__ void __launch_bounds__(kAttBwdThreads, 1)
    attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap tm_qkv,
                       const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ CUtensorMap tm_dq,
                       const __grid_constant__ CUtensorMap tm_dkv, const float* __restrict__ lse,
                       const float* __restrict__ delta, const float2* __restrict__ cs, int S,
                       int Hq, int Hkv, int B, FixedDiv per_block, FixedDiv per_batch, float scale,
                       float scale_log2, AttWindow win, float* __restrict__ part, int* err) {
  using C = AttBwdCfg;
  constexpr int HD = C::HD;
  constexpr uint32_t ID_SP = umma_idesc_bf16(128, 128, false, false);  // S^T, dP^T
  constexpr uint32_t ID_KV = umma_idesc_bf16(128, HD, false, true);    // dV, dK
  constexpr uint32_t ID_Q = umma_idesc_bf16(128, HD, true, true);      // dQ
  constexpr uint32_t TMEM_COLS = 512;
  constexpr uint32_t COL_DP = 128, COL_DQ = 256, COL_P = 320, COL_DV = 384,
                     COL_DK = 448;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t s0 = smem_u32(smem);
  if (s0 & 1023u) {
    if (threadIdx.x == 0) record_error(err, kDevSharedBase);
    return;
  }
  const uint32_t sK = s0 + C::OFF_K, sV = s0 + C::OFF_V, sQ = s0 + C::OFF_Q, sDO = s0 + C::OFF_DO;
  const uint32_t sDSt = s0 + C::OFF_DST, sDQS = s0 + C::OFF_DQS;
  float* sLD = reinterpret_cast<float*>(smem + C::OFF_LD);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  const uint32_t b0 = smem_u32(bars);
  const uint32_t sp_full = b0, s_free = b0 + 8, ps_full = b0 + 16, pds_free = b0 + 24,
                 acc_done = b0 + 32, drain = b0 + 40, acc_free = b0 + 48, dkv_full = b0 + 56,
                 dq_full = b0 + 64, dq_free = b0 + 72;
  auto kv_full = [&](int i) { return b0 + 80u + 8u * i; };
  auto kv_empty = [&](int i) { return b0 + 96u + 8u * i; };
  auto ld_full = [&](int i) { return b0 + 112u + 8u * i; };
  auto ld_empty = [&](int i) { return b0 + 128u + 8u * i; };
  auto qdo_full = [&](int i) { return b0 + 144u + 8u * i; };
  auto qdo_empty = [&](int i) { return b0 + 168u + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = Hq / Hkv, nkb = (S + 127) / 128;
  // without a window key block 0 sees the most query blocks
  const int num_items = (nkb + (PART ? (win.sinks + 127) / 128 * win.splits : 0)) * Hkv * B;
  struct Item { KeyWork w; int g, b, n_it; };
  // this CTA's n-th item (n_it = 0: none left)
  auto item_of = [&](int n) -> Item {
    const int c = n & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
    const int t = n * (int)gridDim.x + c;
    if (t >= num_items) return {{0, 0, 1, -1}, 0, 0, 0};
    Item x;
    int rem;
    x.w = key_work<WIN, PART>(win, per_block(t, rem), S);  // t by Hkv * B
    x.b = per_batch(rem, x.g);                             // by Hkv
    x.n_it = grp * x.w.count;  // (head, query block) pairs
    return x;
  };

  // Blocks in the order of the walk: a head's query blocks, then the next
  // head's, then the next item's (counted on, without a division per block).
  struct Walk { int n, left, h, qb, j, b, first, end; };  // left: blocks of the item, this one included
  auto start = [&](int n) -> Walk {
    const Item x = item_of(n);
    return {n, x.n_it, x.g * grp, x.w.first, x.w.j, x.b, x.w.first, x.w.first + x.w.count};
  };
  auto advance = [&](Walk& w) {
    if (--w.left == 0) {
      w = start(w.n + 1);
    } else if (++w.qb == w.end) {
      w.qb = w.first;
      ++w.h;
    }
  };

  if (threadIdx.x == 0) {
    mbar_init(sp_full, 1);
    mbar_init(s_free, 256);
    mbar_init(ps_full, 256);
    mbar_init(pds_free, 1);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    mbar_init(acc_free, 256);
    mbar_init(dkv_full, 256);
    mbar_init(dq_full, 1);
    mbar_init(dq_free, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(kv_empty(i), 1);
      mbar_init(ld_full(i), 32);
      mbar_init(ld_empty(i), 256);
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(qdo_full(i), 1);
      mbar_init(qdo_empty(i), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_qkv);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_dq);
    tma_prefetch_desc(&tm_dkv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    bool ok = true;
    int issued = 0, kv_issued = 0;  // Q / dO stages and K / V tiles asked for
    for (int n = 0; ok; ++n) {
      const Item x = item_of(n);
      if (x.n_it == 0) break;
      const int ks = n & 1;
      if (!mbar_wait(kv_empty(ks), ((n >> 1) & 1) ^ 1, abort_flag)) { ok = false; break; }
      mbar_arrive_expect_tx(kv_full(ks), 2 * C::TILE);
      tma_load_3d(sK + ks * C::TILE, &tm_qkv, kv_full(ks), (Hq + x.g) * HD, x.w.j * 128, x.b);
      tma_load_3d(sV + ks * C::TILE, &tm_qkv, kv_full(ks), (Hq + Hkv + x.g) * HD, x.w.j * 128, x.b);
      kv_issued = n + 1;
      for (int it = 0; it < x.n_it; ++it) {
        const int bq = issued % C::NQ;
        const int h = x.g * grp + it / x.w.count;
        const int q0 = (x.w.first + it % x.w.count) * 128;
        if (!mbar_wait(qdo_empty(bq), ((issued / C::NQ) & 1) ^ 1, abort_flag)) { ok = false; break; }
        mbar_arrive_expect_tx(qdo_full(bq), 2 * C::TILE);
        tma_load_3d(sQ + bq * C::TILE, &tm_qkv, qdo_full(bq), h * HD, q0, x.b);
        tma_load_3d(sDO + bq * C::TILE, &tm_do, qdo_full(bq), h * HD, q0, x.b);
        ++issued;
      }
    }
    if (!ok) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
      for (int n = kv_issued - 1; n >= 0 && n >= kv_issued - 2; --n)
        mbar_wait(kv_full(n & 1), (n >> 1) & 1, nullptr);
      for (int it = issued - 1; it >= 0 && it >= issued - C::NQ; --it)
        mbar_wait(qdo_full(it % C::NQ), (it / C::NQ) & 1, nullptr);
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    bool ok = true;
    // base descriptors; an operand at byte offset o is the base plus o / 16
    const uint64_t dK = smem_desc_sw128(sK, 16, 1024), dV = smem_desc_sw128(sV, 16, 1024);
    const uint64_t dQk = smem_desc_sw128(sQ, 16, 1024), dDOk = smem_desc_sw128(sDO, 16, 1024);
    const uint64_t dDSt = smem_desc_sw128(sDSt, 16, 1024);
    const uint64_t dQm = smem_desc_sw128(sQ, 16384, 1024), dDOm = smem_desc_sw128(sDO, 16384, 1024);
    const uint64_t dKm = smem_desc_sw128(sK, 16384, 1024), dDStm = smem_desc_sw128(sDSt, 16384, 1024);
    // S^T and dP^T of block G, the first of item n or a later one, G counting
    // the blocks of all items: once the threads hold block G - 1's
    auto issue_sp = [&](int G, int n, bool first) -> bool {
      const int bq = G % C::NQ, ks = n & 1;
      if (first && !mbar_wait(kv_full(ks), (n >> 1) & 1, abort_flag)) return false;
      if (!mbar_wait(qdo_full(bq), (G / C::NQ) & 1, abort_flag)) return false;
      if (G >= 1 && !mbar_wait(s_free, (G - 1) & 1, abort_flag)) return false;
      tc_fence_after();
      const uint32_t qo = (uint32_t)bq * (uint32_t)(C::TILE / 16), ko = (uint32_t)ks * (uint32_t)(C::TILE / 16);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        umma_bf16(tmem_base, dK + ko + kk * 2, dQk + qo + kk * 2, ID_SP, kk > 0 ? 1u : 0u);
        umma_bf16(tmem_base + COL_DP, dV + ko + kk * 2, dDOk + qo + kk * 2, ID_SP, kk > 0 ? 1u : 0u);
      }
      umma_commit(sp_full);
      return true;
    };
    Item x = item_of(0), next = item_of(1);
    int G = 0;
    if (x.n_it > 0) ok = issue_sp(0, 0, true);
    for (int n = 0; ok && x.n_it > 0; ++n) {
      const uint32_t ko = (uint32_t)(n & 1) * (uint32_t)(C::TILE / 16);
      for (int it = 0; ok && it < x.n_it; ++it, ++G) {
        // the next block first: the threads work on it while this one's other
        // products run
        const bool last = it + 1 == x.n_it;
        if (!last ? !issue_sp(G + 1, n, false) : next.n_it > 0 && !issue_sp(G + 1, n + 1, true)) {
          ok = false;
          break;
        }
        const int bq = G % C::NQ;
        // P^T and dS^T of this block are there, and the accumulators of the
        // previous item have been read
        if (!mbar_wait(ps_full, G & 1, abort_flag) ||
            (it == 0 && n > 0 && !mbar_wait(acc_free, (n - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t qo = (uint32_t)bq * (uint32_t)(C::TILE / 16);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {  // over the 128 queries
          const uint32_t acc = (it > 0 || kk > 0) ? 1u : 0u;
          const uint32_t ao = ((kk >> 2) * 16384 + (kk & 3) * 32) / 16;
          umma_bf16_ts(tmem_base + COL_DV, tmem_base + COL_P + kk * 8, dDOm + qo + kk * 128, ID_KV, acc);
          umma_bf16(tmem_base + COL_DK, dDSt + ao, dQm + qo + kk * 128, ID_KV, acc);
        }
        umma_commit(qdo_empty(bq));
        // dQ of the previous block has been read
        if (G >= 1 && !mbar_wait(dq_free, (G - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // over the 128 keys
          umma_bf16(tmem_base + COL_DQ, dDStm + kk * 128, dKm + ko + kk * 128, ID_Q, kk > 0 ? 1u : 0u);
        umma_commit(dq_full);
        umma_commit(pds_free);
      }
      if (ok) umma_commit(acc_done);
      x = next;
      next = item_of(n + 2);
    }
    if (!ok) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
      umma_commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else if (warp == 10 && lane == 0) {
    // ---------------------------------------------------------------- dK and dV store
    bool ok = true;
    for (int n = 0;; ++n) {
      const Item x = item_of(n);
      if (x.n_it == 0) break;
      ok = mbar_wait(dkv_full, n & 1, abort_flag);
      if (!ok) break;
      const uint32_t at = (uint32_t)(n & 1) * C::TILE;
      if (!PART || x.w.slot < 0) {  // key rows past the sequence end are outside the map
        tma_store_3d(&tm_dkv, sK + at, (Hq + x.g) * HD, x.w.j * 128, x.b);
        tma_store_3d(&tm_dkv, sV + at, (Hq + Hkv + x.g) * HD, x.w.j * 128, x.b);
        bulk_commit_group();
        bulk_wait_group_read0();
      }
      mbar_arrive(kv_empty(n & 1));
    }
    if (!ok) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
    }
    bulk_wait_group0();
  } else if (warp == 11) {
    // ---------------------------------------------------------------- lse and D
    // 128 of each (lse in log2 units; zeros behind the sequence's end) into one
    // of two buffers, as soon as the block two before has been computed
    wait_primary();  // D
    bool ok = true;
    Walk w = start(0);
    for (int G = 0; w.left > 0; ++G, advance(w)) {
      const int64_t row = ((int64_t)w.b * Hq + w.h) * S;
      float lv[4], dv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = w.qb * 128 + 32 * i + lane;
        lv[i] = q < S ? lse[row + q] * 1.4426950408889634f : 0.f;
        dv[i] = q < S ? delta[row + q] : 0.f;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(ld_empty(G & 1), ((G >> 1) & 1) ^ 1, abort_flag));
      if (!ok) break;
      float* bL = sLD + (G & 1) * 256 + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bL[32 * i] = lv[i];
        bL[128 + 32 * i] = dv[i];
      }
      mbar_arrive(ld_full(G & 1));
    }
    if (!ok && lane == 0) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
    }
  } else if (warp >= 2 && warp < 10) {
    // ---------------------------------------------------------------- threads
    // Two warps per TMEM lane quarter, each taking half of the block's queries
    // (of S^T and dP^T) and half of the head's columns (of dQ).
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int r = quarter * 32 + lane;  // key row of S^T / dP^T; query row of dQ
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    bool ok = true;
    // dQ of a block, the G-th of all (this warp's 32 queries and 32 columns) into the warp's
    // staging tile, in the tensor map's 128-byte swizzle, then one TMA
    // reduce-add (or store).  The tile is rewritten only after the previous
    // one has finished reading it.
    const uint32_t stage = sDQS + (uint32_t)(warp - 2) * 4096u;
    struct Done { int h, qb, b, j, n; };  // a block whose dQ is still to be stored
    auto emit_dq = [&](const Done& w, int G) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(dq_full, G & 1, abort_flag))) return false;
      tc_fence_after();
      uint32_t v[32];
      tmem_ld_32x32b_x32(lane_base + COL_DQ + 32 * half, v);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(dq_free);
      if (lane == 0) bulk_wait_group_read0();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         stage + (uint32_t)lane * 128u + (uint32_t)((k ^ (lane & 7)) * 16)),
                     "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]), "r"(v[4 * k + 3])
                     : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int qb_ = w.qb * 128 + 32 * quarter;
        if (qb_ < S) {  // rows past the sequence end are outside the map
          if (DET)  // this key block's own slot of the dQ buffer
            tma_store_3d(&tm_dq, stage, w.h * HD + 32 * half, qb_,
                         (WIN ? dq_slot(win, w.j) : w.j) * B + w.b);
          else
            tma_reduce_add_3d(&tm_dq, stage, w.h * HD + 32 * half, qb_, w.b);
        }
        bulk_commit_group();
      }
      return true;
    };
    // dK and dV of item n, once all its products are done: into its own K and V
    // buffers (no MMA reads them any more), in the tensor map's swizzled
    // layout, for the store warp.
    auto finish = [&](int j, int n) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(acc_done, n & 1, abort_flag))) return false;
      tc_fence_after();
      const int key = j * 128 + r;
      auto put = [&](uint32_t tile, int chunk, uint32_t a, uint32_t b_, uint32_t c_, uint32_t d_) {
        const uint32_t addr = tile + (uint32_t)(n & 1) * C::TILE + (uint32_t)r * 128u +
                              (uint32_t)((chunk ^ (r & 7)) * 16);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b_),
                     "r"(c_), "r"(d_)
                     : "memory");
      };
      if (PART && j < (win.sinks + 127) / 128) {  // a part: fp32, neither scaled nor rotated
        const Item x = item_of(n);
        float* dst = part_row<HD>(part, win, x.w, x.g, Hkv, x.b, r) + 32 * half;
        const bool live = r < live_keys(win, x.w);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(lane_base + (c ? COL_DV : COL_DK) + 32 * half, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 8 && live; ++k)
            *reinterpret_cast<uint4*>(dst + c * 128 * HD + 4 * k) =
                make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      } else {
        // dK: pairs (d, d + HD/2) get the inverse rotation of the key's position;
        // this warp takes d in [16 half, 16 half + 16) and their partners
        {
          uint32_t x1[16], x2[16];
          tmem_ld_32x32b_x16(lane_base + COL_DK + 16 * half, x1);
          tmem_ld_32x32b_x16(lane_base + COL_DK + HD / 2 + 16 * half, x2);
          tmem_ld_wait();
          const int kp = key < S ? key : S - 1;  // rows past the end are computed, not stored
          uint32_t o1[8], o2[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float a1 = __uint_as_float(x1[e]) * scale, b1 = __uint_as_float(x1[e + 1]) * scale;
            float a2 = __uint_as_float(x2[e]) * scale, b2 = __uint_as_float(x2[e + 1]) * scale;
            if (cs) {
              const float2 ca = cs[(int64_t)kp * (HD / 2) + 16 * half + e];
              const float2 cb = cs[(int64_t)kp * (HD / 2) + 16 * half + e + 1];
              const float y1a = a1 * ca.x + a2 * ca.y, y2a = a2 * ca.x - a1 * ca.y;
              const float y1b = b1 * cb.x + b2 * cb.y, y2b = b2 * cb.x - b1 * cb.y;
              a1 = y1a; a2 = y2a; b1 = y1b; b2 = y2b;
            }
            o1[e / 2] = pack2_bf16(a1, b1);
            o2[e / 2] = pack2_bf16(a2, b2);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            put(sK, 2 * half + k, o1[4 * k], o1[4 * k + 1], o1[4 * k + 2], o1[4 * k + 3]);
            put(sK, 4 + 2 * half + k, o2[4 * k], o2[4 * k + 1], o2[4 * k + 2], o2[4 * k + 3]);
          }
        }
        {
          uint32_t v[32];
          tmem_ld_32x32b_x32(lane_base + COL_DV + 32 * half, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            put(sV, 4 * half + k, pack2_bf16(__uint_as_float(v[8 * k + 0]), __uint_as_float(v[8 * k + 1])),
                pack2_bf16(__uint_as_float(v[8 * k + 2]), __uint_as_float(v[8 * k + 3])),
                pack2_bf16(__uint_as_float(v[8 * k + 4]), __uint_as_float(v[8 * k + 5])),
                pack2_bf16(__uint_as_float(v[8 * k + 6]), __uint_as_float(v[8 * k + 7])));
        }
      }
      tc_fence_before();
      mbar_arrive(acc_free);  // the next item's dV and dK may be formed
      fence_proxy_async_smem();
      // the store warp has taken the item before: its barrier cannot run ahead
      if (n > 0 && !__all_sync(0xffffffffu, mbar_wait(kv_empty((n - 1) & 1), ((n - 1) >> 1) & 1, abort_flag)))
        return false;
      mbar_arrive(dkv_full);
      return true;
    };
    wait_primary();  // the zeros in dq_acc
    const uint32_t rowoff = (uint32_t)r * 128u + (uint32_t)half * 16384u;
    Walk cur = start(0);
    Done prev{};
    int G = 0;
    for (; ok && cur.left > 0; ++G) {
      const int key = cur.j * 128 + r;
      // the last query that sees this thread's key (before the key: no one does)
      const int q_end = !WIN || key < win.sinks || key > S - win.size ? S - 1 : key + win.size - 1;
      const int qc = cur.qb * 128 + 64 * half;  // first query of this thread's columns
      float* bL = sLD + (G & 1) * 256;
      float* bD = bL + 128;
      ok = __all_sync(0xffffffffu, mbar_wait(ld_full(G & 1), (G >> 1) & 1, abort_flag));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(sp_full, G & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[2][32], dr[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tmem_ld_32x32b_x32(lane_base + 64 * half + 32 * c, sr[c]);
        tmem_ld_32x32b_x32(lane_base + COL_DP + 64 * half + 32 * c, dr[c]);
      }
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(s_free);  // S^T / dP^T are in registers: the next block may overwrite them
      // P^T over S^T's registers, dS^T over dP^T's, packed
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int q1 = qc + 32 * c;
        const uint32_t seen = low_bits(q_end - q1 + 1) & ~low_bits(key - q1);
        const float4* L4 = reinterpret_cast<const float4*>(bL + 64 * half + 32 * c);
        const float4* D4 = reinterpret_cast<const float4*>(bD + 64 * half + 32 * c);
        auto grad_tile = [&](auto mask_tag) {
          constexpr bool kMask = decltype(mask_tag)::value;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 l4 = L4[k], d4 = D4[k];
            const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
            const float dv[4] = {d4.x, d4.y, d4.z, d4.w};
            float pv[4], sv[4];
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const int e = 4 * k + i;
              float x0 = __uint_as_float(sr[c][e]), x1 = __uint_as_float(sr[c][e + 1]);
              fma2(x0, x1, scale_log2, -lv[i], -lv[i + 1]);
              x0 = ex2_approx(x0);
              x1 = ex2_approx(x1);
              if (kMask && !(seen & (1u << e))) x0 = 0.f;
              if (kMask && !(seen & (2u << e))) x1 = 0.f;
              float d0 = __uint_as_float(dr[c][e]), d1 = __uint_as_float(dr[c][e + 1]);
              add2(d0, d1, -dv[i], -dv[i + 1]);
              mul2(d0, d1, x0, x1);
              pv[i] = x0;
              pv[i + 1] = x1;
              sv[i] = d0;
              sv[i + 1] = d1;
            }
            sr[c][2 * k] = pack2_bf16(pv[0], pv[1]);
            sr[c][2 * k + 1] = pack2_bf16(pv[2], pv[3]);
            dr[c][2 * k] = pack2_bf16(sv[0], sv[1]);
            dr[c][2 * k + 1] = pack2_bf16(sv[2], sv[3]);
          }
        };
        if (__all_sync(0xffffffffu, seen == 0xffffffffu))
          grad_tile(std::false_type{});
        else
          grad_tile(std::true_type{});
      }
      mbar_arrive(ld_empty(G & 1));
      if (G >= 1) {  // P^T, dS^T of the previous block consumed
        ok = __all_sync(0xffffffffu, mbar_wait(pds_free, (G - 1) & 1, abort_flag));
        if (!ok) break;
      }
      {
        uint32_t pk[32];  // P^T of the thread's 64 queries
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          pk[i] = sr[0][i];
          pk[16 + i] = sr[1][i];
        }
        tmem_st_32x32b_x32(lane_base + COL_P + 32 * half, pk);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t off = rowoff + (uint32_t)(((4 * c + k) ^ (r & 7)) * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sDSt + off), "r"(dr[c][4 * k]),
                       "r"(dr[c][4 * k + 1]), "r"(dr[c][4 * k + 2]), "r"(dr[c][4 * k + 3])
                       : "memory");
        }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(ps_full);
      // while the tensor core works on this block's products: dQ of the one
      // before, and, at an item's first block, the previous item's dK and dV
      if (G > 0) ok = emit_dq(prev, G - 1) && (prev.n == cur.n || finish(prev.j, prev.n));
      prev = {cur.h, cur.qb, cur.b, cur.j, cur.n};
      advance(cur);
    }
    if (ok && G > 0) ok = emit_dq(prev, G - 1) && finish(prev.j, prev.n);
    if (!ok && lane == 0) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
    }
    if (lane == 0) bulk_wait_group0();  // this warp's stores are complete
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Backward for head_dim 128.  A CTA works on one item (as at head dim 64, in
// longest-first order), block by block of 128 keys x 128 queries:
//   MMA:     S^T = K Q^T -> TMEM[0,128)
//   threads: P^T = exp2(S^T*scale*log2e - lse*log2e) (masked), kept in fp32
//            registers, and as bf16 over the S^T columns that the warp has read
//   MMA:     dP^T = V dO^T -> TMEM[128,256);  dV += P^T dO (P^T as the
//            tensor-memory A; TMEM[256,384))
//   threads: dS^T = P^T * (dP^T - D) to shared memory (bf16, swizzled)
//   MMA:     dQ^T = K^T dS^T over the dP^T columns; dK += dS^T Q (TMEM[384,512))
//   4 warps: dQ^T through shared memory into the fp32 dq_acc by TMA reduce-add
//            (deterministic: by TMA store into the key block's own slot)
// The accumulators take all of TMEM, hence the shared columns.  The MMAs of
// block i are issued in the order dV(i), S^T(i+1), dQ^T(i), dK(i), dP^T(i+1):
// the threads form dS^T(i) under the first two and P^T(i+1) under the next
// two, and dQ^T is read under dK.  (P^T is overwritten by the next S^T, which
// is issued after dV and so executes after it.)
//
// What bounds it: shared memory's 128 bytes a clock.  An MMA with both
// operands in shared memory reads 4 + 4 KB in its 64 clocks, with P^T in TMEM
// half of that: 2,304 clocks a block for operands, and 1,792 for Q and dO
// coming in, dS^T, and dQ^T going through (its fp32 sums are 64 KB a block);
// a block takes 4,450 clocks.  Blocks of 64 queries (MMAs 64 wide, which read
// 6 KB in 32 clocks of work) took 2 x 2,450.  Whole backward, 8 x 2048 tokens,
// 32 / 8 heads: 897 us then, 790 us with 128 queries, 711 us (967 TFLOP/s) with
// the heads in chunks (head_chunks); 2 x 8192, window 1024, 4 sinks: 968 us
// then, now 793 us in repeated calls and up to 822 us on a box that does other
// work in between (deterministic 1,200 us).  Measured on the way to 790: the threads storing dQ themselves, as one
// reduction instruction per row, 862 us, and four warps of their own doing so
// 918 us (such instructions leave an SM at 32 bytes a clock and hold up the
// stores of dS^T behind them); dO's one buffer refilled after the next but one
// Q, 1,020 us.  Testing the barriers a step ahead gained nothing here.
//
// Every mbarrier below completes at most once before its waiter has seen the
// previous completion (each has a dependency chain through its waiter), so
// parity waits are unambiguous.
namespace {
// The order of the items of a grid (ranks, kv heads, batch); CTAs are dispatched
// roughly in linear block order.  Longest first over the whole grid (rank 0,
// which without a window sees the most query blocks, for every head before rank
// 1) balances the SMs, but each rank reads every head's Q and dO and adds to its
// dQ anew, from DRAM where the heads do not fit into L2 together.  So without a
// window the first `chunked` of the heads (of all batches) are taken `size` at a
// time, longest first in each chunk (head_chunks).
struct HeadChunks {
  int size, chunked;
  __device__ __forceinline__ void item(int& rank, int& g, int& b) const {
    int lin = (int)(blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z));
    const int ranks = (int)gridDim.x;
    int head0 = 0, n = size;
    if (lin < chunked * ranks) {
      const int c = lin / (size * ranks);
      head0 = c * size;
      lin -= c * size * ranks;
    } else {
      head0 = chunked;
      n = (int)(gridDim.y * gridDim.z) - chunked;
      lin -= chunked * ranks;
    }
    rank = lin / n;
    const int head = head0 + lin - rank * n;
    b = head / (int)gridDim.y;
    g = head - b * (int)gridDim.y;
  }
};
constexpr int kAttBwd2Threads = 448;  // TMA warp, MMA warp, 8 softmax-gradient warps, 4 dQ warps
struct AttBwd2Cfg {
  static constexpr int KV = 32768;  // 128 keys x 128 hd
  static constexpr int QT = 32768;  // 128 queries x 128 hd
  static constexpr int NQ = 2;      // Q stages (dO has one)
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = KV;
  static constexpr int OFF_Q = 2 * KV;
  static constexpr int OFF_DO = OFF_Q + NQ * QT;
  static constexpr int OFF_DST = OFF_DO + QT;      // 128 keys x 128 queries, two boxes of 64
  static constexpr int OFF_DQS = OFF_DST + 32768;  // dQ staging: 4 warps x 2 x [32 q][32 d] fp32
  static constexpr int OFF_LD = OFF_DQS + 32768;   // [2][lse 128 | D 128]
  static constexpr int OFF_BAR = OFF_LD + 2 * 256 * 4;
  static constexpr int NBAR = 19;
  // no room to align the base: it is 1024-byte aligned where a kernel has no
  // static shared memory, which the kernel checks
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
};
static_assert(AttBwd2Cfg::SMEM <= 232448, "backward shared memory");
}  // namespace

template <bool DET, bool WIN, bool PART>
__global__ void __launch_bounds__(kAttBwd2Threads, 1)
    attn_bwd_tc2_kernel(const __grid_constant__ CUtensorMap tm_kv,
                        const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ CUtensorMap tm_do,
                        const __grid_constant__ CUtensorMap tm_dq,
                        const __grid_constant__ CUtensorMap tm_dkv, const float* __restrict__ lse,
                        const float* __restrict__ delta, const float2* __restrict__ cs, int S,
                        int Hq, int Hkv, float scale, float scale_log2, AttWindow win,
                        HeadChunks chunks, float* __restrict__ part, int* err) {
  using C = AttBwd2Cfg;
  constexpr int HD = 128;
  constexpr uint32_t ID_SP = umma_idesc_bf16(128, 128, false, false);  // S^T, dP^T
  constexpr uint32_t ID_KV = umma_idesc_bf16(128, HD, false, true);    // dV, dK
  constexpr uint32_t ID_Q = umma_idesc_bf16(128, 128, true, true);     // dQ^T
  constexpr uint32_t TMEM_COLS = 512;
  constexpr uint32_t COL_DP = 128, COL_DV = 256, COL_DK = 384;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t s0 = smem_u32(smem);
  if (s0 & 1023u) {
    if (threadIdx.x == 0) record_error(err, kDevSharedBase);
    return;
  }
  const uint32_t sK = s0 + C::OFF_K, sV = s0 + C::OFF_V, sQ = s0 + C::OFF_Q, sDO = s0 + C::OFF_DO;
  const uint32_t sDSt = s0 + C::OFF_DST, sDQS = s0 + C::OFF_DQS;
  float* sLD = reinterpret_cast<float*>(smem + C::OFF_LD);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  const uint32_t b0 = smem_u32(bars);
  const uint32_t kv_full = b0;
  auto q_full = [&](int i) { return b0 + 8u * (1 + i); };
  auto q_empty = [&](int i) { return b0 + 8u * (4 + i); };
  const uint32_t do_full = b0 + 56, do_empty = b0 + 64;
  const uint32_t s_full = b0 + 72, p_full = b0 + 80, dp_full = b0 + 88, ds_full = b0 + 96;
  const uint32_t dq_full = b0 + 104, dq_free = b0 + 112, acc_done = b0 + 120, drain = b0 + 128;
  auto ld_full = [&](int i) { return b0 + 136u + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int rank, g, b;
  chunks.item(rank, g, b);
  const KeyWork work = key_work<WIN, PART>(win, rank, S);
  const int grp = Hq / Hkv;
  const int j = work.j, k0 = j * 128;
  const int first = work.first, per_head = work.count;  // query blocks that see these keys
  const int keys = PART ? live_keys(win, work) : 128;
  const int n_it = grp * per_head;

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
    }
    mbar_init(do_full, 1);
    mbar_init(do_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, 256);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 256);
    mbar_init(dq_full, 1);
    mbar_init(dq_free, 128);
    for (int i = 0; i < 2; ++i) mbar_init(ld_full(i), 128);
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_kv);
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_dq);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    mbar_arrive_expect_tx(kv_full, 2 * C::KV);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      tma_load_3d(sK + c * 16384, &tm_kv, kv_full, (Hq + g) * HD + 64 * c, k0, b);
      tma_load_3d(sV + c * 16384, &tm_kv, kv_full, (Hq + Hkv + g) * HD + 64 * c, k0, b);
    }
    bool ok = true;
    int q_issued = 0, do_issued = 0, bq = 0, bph = 0;
    int qh = g * grp, qq = first, wh = qh, wq = first;  // head and query block of the next Q, dO
    // in the order in which the buffers come free: dO of block it (after block
    // it - 1's dV), then Q of block it + 1 (after block it - 1's dK)
    for (int it = -1; it < n_it; ++it) {
      if (it >= 0) {
        if (!mbar_wait(do_empty, (it & 1) ^ 1, abort_flag)) { ok = false; break; }
        mbar_arrive_expect_tx(do_full, C::QT);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          tma_load_3d(sDO + c * 16384, &tm_do, do_full, wh * HD + 64 * c, wq * 128, b);
        ++do_issued;
        if (++wq == first + per_head) {
          wq = first;
          ++wh;
        }
      }
      if (it + 1 == n_it) break;
      if (!mbar_wait(q_empty(bq), bph ^ 1, abort_flag)) { ok = false; break; }
      mbar_arrive_expect_tx(q_full(bq), C::QT);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tma_load_3d(sQ + bq * C::QT + c * 16384, &tm_q, q_full(bq), qh * HD + 64 * c, qq * 128, b);
      ++q_issued;
      if (++bq == C::NQ) {
        bq = 0;
        bph ^= 1;
      }
      if (++qq == first + per_head) {
        qq = first;
        ++qh;
      }
    }
    if (!ok) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
      mbar_wait(kv_full, 0, nullptr);
      for (int it = q_issued - 1; it >= 0 && it >= q_issued - C::NQ; --it)
        mbar_wait(q_full(it % C::NQ), (it / C::NQ) & 1, nullptr);
      if (do_issued > 0) mbar_wait(do_full, (do_issued - 1) & 1, nullptr);
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    bool ok = mbar_wait(kv_full, 0, abort_flag);
    // Descriptors of each operand's first row (K-major views, then the
    // MN-major views of the P V-style products); an operand at byte offset o
    // is the base plus o / 16 (shared addresses stay below 2^18, so the
    // 14-bit address field cannot carry).
    const uint64_t dK = smem_desc_sw128(sK, 16, 1024), dV = smem_desc_sw128(sV, 16, 1024);
    const uint64_t dQk = smem_desc_sw128(sQ, 16, 1024), dDOk = smem_desc_sw128(sDO, 16, 1024);
    const uint64_t dQm = smem_desc_sw128(sQ, 16384, 1024), dDOm = smem_desc_sw128(sDO, 16384, 1024);
    const uint64_t dDSt = smem_desc_sw128(sDSt, 16, 1024);
    const uint64_t dKm = smem_desc_sw128(sK, 16384, 1024), dDStm = smem_desc_sw128(sDSt, 16384, 1024);
    auto issue_s = [&](int it) -> bool {
      const int bq = it % C::NQ;
      if (!mbar_wait(q_full(bq), (it / C::NQ) & 1, abort_flag)) return false;
      tc_fence_after();
      const uint32_t qo = (uint32_t)bq * (uint32_t)(C::QT / 16);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) / 16;
        umma_bf16(tmem_base, dK + o, dQk + qo + o, ID_SP, kk > 0 ? 1u : 0u);
      }
      umma_commit(s_full);
      return true;
    };
    auto issue_dp = [&](int it) -> bool {
      if (!mbar_wait(do_full, it & 1, abort_flag)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * 16384 + (kk & 3) * 32) / 16;
        umma_bf16(tmem_base + COL_DP, dV + o, dDOk + o, ID_SP, kk > 0 ? 1u : 0u);
      }
      umma_commit(dp_full);
      return true;
    };
    if (ok) ok = issue_s(0) && issue_dp(0);
    for (int it = 0; ok && it < n_it; ++it) {
      // P^T of the block is there (and S^T has been read)
      if (!mbar_wait(p_full, it & 1, abort_flag)) { ok = false; break; }
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)  // over the 128 queries
        umma_bf16_ts(tmem_base + COL_DV, tmem_base + (kk >> 2) * 64 + (kk & 3) * 8, dDOm + kk * 128, ID_KV,
                     (it > 0 || kk > 0) ? 1u : 0u);
      umma_commit(do_empty);
      // the next S^T, over P^T, which the tensor core has used by then
      if (it + 1 < n_it && !issue_s(it + 1)) { ok = false; break; }
      // dS^T is in shared memory, dP^T has been read: dQ^T takes its columns
      if (!mbar_wait(ds_full, it & 1, abort_flag)) { ok = false; break; }
      tc_fence_after();
      if (PART && keys < 128) {  // only the sinks (apart from the full loop: 1 to 2%, as in the forward)
#pragma unroll 1
        for (int kk = 0; kk < keys / 16; ++kk)
          umma_bf16(tmem_base + COL_DP, dKm + kk * 128, dDStm + kk * 128, ID_Q, kk > 0 ? 1u : 0u);
      } else {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // over the 128 keys
          umma_bf16(tmem_base + COL_DP, dKm + kk * 128, dDStm + kk * 128, ID_Q, kk > 0 ? 1u : 0u);
      }
      umma_commit(dq_full);
      const uint32_t qo = (uint32_t)(it % C::NQ) * (uint32_t)(C::QT / 16);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)  // over the 128 queries
        umma_bf16(tmem_base + COL_DK, dDSt + ((kk >> 2) * 16384 + (kk & 3) * 32) / 16, dQm + qo + kk * 128, ID_KV,
                  (it > 0 || kk > 0) ? 1u : 0u);
      umma_commit(q_empty(it % C::NQ));
      // the next dP^T, once dQ^T has been read
      if (it + 1 < n_it && (!mbar_wait(dq_free, it & 1, abort_flag) || !issue_dp(it + 1))) { ok = false; break; }
    }
    if (ok) {
      umma_commit(acc_done);
    } else {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
      umma_commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else if (warp >= 10) {
    // ---------------------------------------------------------------- dQ
    // dQ^T of each block, a thread per head-dim lane, by 32 queries: out of TMEM,
    // into one of the warp's two staging tiles, and from there the TMA unit
    // adds it into the fp32 dQ buffer (deterministic: stores it into the key
    // block's own slot).
    const int quarter = warp & 3;
    const uint32_t at = tmem_base + ((uint32_t)(quarter * 32) << 16) + COL_DP;
    const uint32_t stage = sDQS + (uint32_t)quarter * 8192u;
    wait_primary();  // the zeros in dq_acc
    bool ok = true;
    int h = g * grp, qb = first;
    auto emit = [&](int c, const uint32_t (&v)[32]) {
      const uint32_t tile = stage + (uint32_t)(c & 1) * 4096u;
      if (lane == 0) bulk_wait_group_read1();
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 32; ++e)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(tile + (uint32_t)e * 128u + (uint32_t)lane * 4u), "r"(v[e])
                     : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int col = h * HD + 32 * quarter, q = qb * 128 + 32 * c;
        if (DET)
          tma_store_3d(&tm_dq, tile, col, q, (WIN ? dq_slot(win, j) : j) * (int)gridDim.z + b);
        else
          tma_reduce_add_3d(&tm_dq, tile, col, q, b);
        bulk_commit_group();
      }
    };
    for (int it = 0; it < n_it; ++it) {
      ok = __all_sync(0xffffffffu, mbar_wait(dq_full, it & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t v0[32], v1[32], v2[32];
      tmem_ld_32x32b_x32(at, v0);
      tmem_ld_32x32b_x32(at + 32, v1);
      tmem_ld_32x32b_x32(at + 64, v2);
      tmem_ld_wait();
      emit(0, v0);
      tmem_ld_32x32b_x32(at + 96, v0);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(dq_free);
      emit(1, v1);
      emit(2, v2);
      emit(3, v0);
      if (++qb == first + per_head) {
        qb = first;
        ++h;
      }
    }
    if (lane == 0) bulk_wait_group0();  // this warp's copies are complete
    if (!ok && lane == 0) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
    }
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- threads
    // Eight warps: two per TMEM lane quarter, each taking one half (64) of the
    // block's queries.
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    const int r = quarter * 32 + lane;  // key row of S^T / dP^T; head-dim lane of dQ^T
    const int key = k0 + r;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const int tid = threadIdx.x - 64;
    // the last query that sees this thread's key (before the key: no one does)
    const int q_end = WIN ? (key < win.sinks || key > S - win.size ? S - 1 : key + win.size - 1) : 0;
    bool ok = true;
    auto fetch = [&](int it_, int h_, int qq_, float& lv, float& dv) {
      lv = 0.f;
      dv = 0.f;
      if (it_ >= n_it || tid >= 128) return;
      const int q_ = qq_ * 128 + tid;
      if (q_ < S) {
        const int64_t o = ((int64_t)b * Hq + h_) * S + q_;
        lv = lse[o];
        dv = delta[o];
      }
    };
    wait_primary();  // D, and the zeros in dq_acc
    float next_l, next_d;
    fetch(0, g * grp, first, next_l, next_d);
    const uint32_t rowoff = (uint32_t)r * 128u;
    // no key of this warp's lanes counts behind the window of a sinks' block
    const bool idle = PART && quarter * 32 >= keys;
    float p[64];  // P of the thread's key and 64 queries
    // P^T of block it_ from S^T, in bf16 over its columns
    auto form_p = [&](int it_, int h_, int q_, int nh, int nq) -> bool {
      float* bL = sLD + (it_ & 1) * 256;
      // The buffer written here was last read for dS^T of block it_ - 2; this
      // thread has since seen block it_ - 1's dP^T, which was formed after
      // every thread's dS^T of it_ - 2.
      if (tid < 128) {
        bL[tid] = next_l * 1.4426950408889634f;
        bL[128 + tid] = next_d;
        mbar_arrive(ld_full(it_ & 1));
      }
      fetch(it_ + 1, nh, nq, next_l, next_d);
      bool good = __all_sync(0xffffffffu, mbar_wait(ld_full(it_ & 1), (it_ >> 1) & 1, abort_flag));
      if (good) good = __all_sync(0xffffffffu, mbar_wait(s_full, it_ & 1, abort_flag));
      if (!good) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (idle) break;
        uint32_t sr[16];
        tmem_ld_32x32b_x16(lane_base + 64 * half + 16 * c, sr);
        tmem_ld_wait();
        const float4* L4 = reinterpret_cast<const float4*>(bL + 64 * half + 16 * c);
        const int qb = q_ * 128 + 64 * half + 16 * c;     // first query of these columns
        const int e_lo = key - qb, e_hi = q_end - qb;     // this thread's visible columns (WIN)
        uint32_t pp[8];
        auto tile = [&](auto mask_tag) {
          constexpr bool kMask = decltype(mask_tag)::value;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 l4 = L4[k];
            const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const int e = 4 * k + i;
              // (x0, x1) = s * scale_log2 - lse * log2(e), one paired FMA
              float x0 = __uint_as_float(sr[e]), x1 = __uint_as_float(sr[e + 1]);
              fma2(x0, x1, scale_log2, -lv[i], -lv[i + 1]);
              x0 = ex2_approx(x0);
              x1 = ex2_approx(x1);
              if (WIN) {
                if (kMask && (e < e_lo || e > e_hi)) x0 = 0.f;
                if (kMask && (e + 1 < e_lo || e + 1 > e_hi)) x1 = 0.f;
              } else {
                if (kMask && !(qb + e < S && key <= qb + e)) x0 = 0.f;
                if (kMask && !(qb + e + 1 < S && key <= qb + e + 1)) x1 = 0.f;
              }
              p[16 * c + e] = x0;
              p[16 * c + e + 1] = x1;
              pp[2 * k + i / 2] = pack2_bf16(x0, x1);
            }
          }
        };
        // Only blocks that touch the diagonal, the sequence end or the window's
        // start need the mask.
        const bool cut = WIN && qb + 15 - k0 >= win.size && k0 + 127 >= win.sinks;
        if (qb < k0 + 128 || qb + 16 > S || cut)
          tile(std::true_type{});
        else
          tile(std::false_type{});
        tmem_st_32x32b_x8(lane_base + 64 * half + 8 * c, pp);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_full);
      return true;
    };
    // dS^T = P^T (dP^T - D) of block it_ into shared memory (the tile's readers
    // of the block before were done before this dP^T)
    auto form_ds = [&](int it_) -> bool {
      const float* bD = sLD + (it_ & 1) * 256 + 128;
      if (!__all_sync(0xffffffffu, mbar_wait(dp_full, it_ & 1, abort_flag))) return false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (idle) break;
        uint32_t dr[16];
        tmem_ld_32x32b_x16(lane_base + COL_DP + 64 * half + 16 * c, dr);
        tmem_ld_wait();
        const float4* D4 = reinterpret_cast<const float4*>(bD + 64 * half + 16 * c);
        uint32_t dd[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 d4 = D4[k];
          const float dv[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const int e = 4 * k + i;
            float d0 = __uint_as_float(dr[e]), d1 = __uint_as_float(dr[e + 1]);
            add2(d0, d1, -dv[i], -dv[i + 1]);
            mul2(d0, d1, p[16 * c + e], p[16 * c + e + 1]);
            dd[2 * k + i / 2] = pack2_bf16(d0, d1);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int jj = c * 2 + k;  // 16-byte chunk of the 128-byte row
          const uint32_t off = (uint32_t)half * 16384u + rowoff + (uint32_t)((jj ^ (r & 7)) * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sDSt + off), "r"(dd[4 * k]),
                       "r"(dd[4 * k + 1]), "r"(dd[4 * k + 2]), "r"(dd[4 * k + 3])
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(ds_full);
      return true;
    };
    // head and query block of the block in hand, and of the next two
    int wh = g * grp, wq = first;
    auto step = [&](int& h_, int& q_) {
      if (++q_ == first + per_head) {
        q_ = first;
        ++h_;
      }
    };
    int nh = wh, nq = wq;
    step(nh, nq);
    ok = form_p(0, wh, wq, nh, nq);
    for (int it = 0; ok && it < n_it; ++it) {
      ok = form_ds(it);
      wh = nh;
      wq = nq;
      step(nh, nq);
      // the next block's P^T while the tensor core forms dQ^T
      if (ok && it + 1 < n_it) ok = form_p(it + 1, wh, wq, nh, nq);
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(acc_done, 0, abort_flag));
    if (ok) {
      tc_fence_after();
      if (PART && work.slot >= 0) {  // a part: fp32, neither scaled nor rotated
        float* dst = part_row<HD>(part, win, work, g, Hkv, b, r) + 64 * half;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(lane_base + (c >> 1 ? COL_DV : COL_DK) + 64 * half + 32 * (c & 1), v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 8 && r < keys; ++k)
            *reinterpret_cast<uint4*>(dst + (c >> 1) * 128 * HD + 32 * (c & 1) + 4 * k) =
                make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      } else {
        // dK and dV rows go into the K and V tiles' shared memory (every MMA
        // that read them has completed), in the tensor map's swizzled layout;
        // one thread then stores both tiles with the TMA unit.
        auto put = [&](uint32_t tile, int col, uint32_t a, uint32_t b_, uint32_t c_, uint32_t d_) {
          const int chunk = (col & 63) >> 3;  // 16-byte chunk of the 128-byte row
          const uint32_t addr = tile + (uint32_t)(col >> 6) * 16384u + (uint32_t)r * 128u +
                                (uint32_t)((chunk ^ (r & 7)) * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b_),
                       "r"(c_), "r"(d_)
                       : "memory");
        };
        // dK: pairs (d, d + HD/2) get the inverse rotation of the key's position;
        // this warp takes d in [32 half, 32 half + 32) and its partners
        {
          const int c = half;
          uint32_t x1[32], x2[32];
          tmem_ld_32x32b_x32(lane_base + COL_DK + 32 * c, x1);
          tmem_ld_32x32b_x32(lane_base + COL_DK + HD / 2 + 32 * c, x2);
          tmem_ld_wait();
          {
            const int kp = key < S ? key : S - 1;  // rows past the end are computed, not stored
            uint32_t o1[16], o2[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float a1 = __uint_as_float(x1[e]) * scale, b1 = __uint_as_float(x1[e + 1]) * scale;
              float a2 = __uint_as_float(x2[e]) * scale, b2 = __uint_as_float(x2[e + 1]) * scale;
              if (cs) {
                const float2 ca = cs[(int64_t)kp * (HD / 2) + 32 * c + e];
                const float2 cb = cs[(int64_t)kp * (HD / 2) + 32 * c + e + 1];
                const float y1a = a1 * ca.x + a2 * ca.y, y2a = a2 * ca.x - a1 * ca.y;
                const float y1b = b1 * cb.x + b2 * cb.y, y2b = b2 * cb.x - b1 * cb.y;
                a1 = y1a; a2 = y2a; b1 = y1b; b2 = y2b;
              }
              o1[e / 2] = pack2_bf16(a1, b1);
              o2[e / 2] = pack2_bf16(a2, b2);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              put(sK, 32 * c + 8 * k, o1[4 * k], o1[4 * k + 1], o1[4 * k + 2], o1[4 * k + 3]);
              put(sK, HD / 2 + 32 * c + 8 * k, o2[4 * k], o2[4 * k + 1], o2[4 * k + 2], o2[4 * k + 3]);
            }
          }
        }
        // dV: this warp takes columns [64 half, 64 half + 64)
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int c = 2 * half + cc;
          uint32_t v[32];
          tmem_ld_32x32b_x32(lane_base + COL_DV + 32 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            put(sV, 32 * c + 8 * k, pack2_bf16(__uint_as_float(v[8 * k + 0]), __uint_as_float(v[8 * k + 1])),
                pack2_bf16(__uint_as_float(v[8 * k + 2]), __uint_as_float(v[8 * k + 3])),
                pack2_bf16(__uint_as_float(v[8 * k + 4]), __uint_as_float(v[8 * k + 5])),
                pack2_bf16(__uint_as_float(v[8 * k + 6]), __uint_as_float(v[8 * k + 7])));
        }
      }
      fence_proxy_async_smem();
    } else if (lane == 0) {
      record_error(err, kDevAttnTimeout);
      *abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  } else if (threadIdx.x == 64 && !*abort_flag && (!PART || work.slot < 0)) {
    // dK and dV tiles; key rows past the sequence end are outside the map
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      tma_store_3d(&tm_dkv, sK + c * 16384, (Hq + g) * HD + 64 * c, k0, b);
      tma_store_3d(&tm_dkv, sV + c * 16384, (Hq + Hkv + g) * HD + 64 * c, k0, b);
    }
    bulk_commit_group();
    bulk_wait_group0();
  }
}

// ------------------------------------------------------------------ host side
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn_att() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

template <int HD, bool WIN>
int fwd_pp(const __nv_bfloat16* qkv, __nv_bfloat16* o, float* lse, int B, int S, int Hq, int Hkv,
           AttWindow win, int* err, cudaStream_t st) {
  using C = AttFwd2Cfg<HD>;
  auto fn = encode_fn_att();
  if (!fn) return -3;
  const int64_t W = (int64_t)(Hq + 2 * Hkv) * HD, WO = (int64_t)Hq * HD;
  CUtensorMap tm, tm_o;
  cuuint64_t dims[3] = {(cuuint64_t)W, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t strides[2] = {(cuuint64_t)(W * 2), (cuuint64_t)(S * W * 2)};
  cuuint64_t dims_o[3] = {(cuuint64_t)WO, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t strides_o[2] = {(cuuint64_t)(WO * 2), (cuuint64_t)(S * WO * 2)};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  if (fn(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(qkv), dims, strides,
         box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      fn(&tm_o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, o, dims_o, strides_o, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return -3;
  if (!reserve_smem<attn_fwd_pp_kernel<HD, WIN>>(C::SMEM)) return -3;
  // two query heads of a group per item when the group size is even, else
  // two consecutive query blocks of one head
  const int pair_heads = (Hq / Hkv) % 2 == 0 ? 1 : 0;
  const int nqb = (S + 127) / 128;
  const int items = pair_heads ? nqb * (Hq / 2) * B : ((nqb + 1) / 2) * Hq * B;
  const int grid = items < num_sms() ? items : num_sms();
  attn_fwd_pp_kernel<HD, WIN><<<grid, kAttFwd2Threads, C::SMEM, st>>>(
      tm, tm_o, lse, S, Hq, Hkv, B, 1.4426950408889634f / sqrtf((float)HD), pair_heads, win, err);
  return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

template <bool DET, bool WIN, bool PART>
int bwd_tc(const __nv_bfloat16* qkv, const __nv_bfloat16* o, const __nv_bfloat16* dout,
           const float* lse, float* delta, float* dq_acc, __nv_bfloat16* dqkv, int B, int S, int Hq,
           int Hkv, const float2* cs, AttWindow win, int* err, cudaStream_t st) {
  using C = AttBwdCfg;
  constexpr int HD = C::HD;
  auto fn = encode_fn_att();
  if (!fn) return -3;
  const int64_t W = (int64_t)(Hq + 2 * Hkv) * HD, WO = (int64_t)Hq * HD;
  CUtensorMap tq, td, tdq, tdkv;
  cuuint32_t box[3] = {64, 128, 1}, box_dq[3] = {32, 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  cuuint64_t dq[3] = {(cuuint64_t)W, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t sq[2] = {(cuuint64_t)(W * 2), (cuuint64_t)(S * W * 2)};
  cuuint64_t dd[3] = {(cuuint64_t)WO, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t sd[2] = {(cuuint64_t)(WO * 2), (cuuint64_t)(S * WO * 2)};
  const int slots = WIN ? attn_window_dq_slots(S, win.size, win.sinks) : (S + 127) / 128;
  cuuint64_t ddq[3] = {(cuuint64_t)WO, (cuuint64_t)S, (cuuint64_t)(DET ? (int64_t)B * slots : B)};
  cuuint64_t sdq[2] = {(cuuint64_t)(WO * 4), (cuuint64_t)(S * WO * 4)};
  auto enc = [&](CUtensorMap* m, CUtensorMapDataType type, const void* base, cuuint64_t* dims,
                 cuuint64_t* strides, cuuint32_t* bx, CUtensorMapL2promotion l2) {
    return fn(m, type, 3, const_cast<void*>(base), dims, strides, bx, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, l2,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  if (!enc(&tq, bf, qkv, dq, sq, box, l2) || !enc(&td, bf, dout, dd, sd, box, l2) ||
      !enc(&tdkv, bf, dqkv, dq, sq, box, l2) ||
      !enc(&tdq, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dq_acc, ddq, sdq, box_dq,
           CU_TENSOR_MAP_L2_PROMOTION_NONE))
    return -3;
  if (!reserve_smem<attn_bwd_tc_kernel<DET, WIN, PART>>(C::SMEM)) return -3;
  attn_delta(o, dout, delta, DET ? nullptr : dq_acc, B, S, Hq, HD, st);
  const float scale = 1.f / sqrtf((float)HD);
  const int ranks = (S + 127) / 128 + (PART ? (win.sinks + 127) / 128 * win.splits : 0);
  const int items = ranks * Hkv * B, sms = num_sms();
  // the sinks' partial dK and dV follow dQ in the scratch
  float* part = dq_acc + (DET ? (int64_t)slots : 1) * B * S * WO;
  if (!launch_dependent(attn_bwd_tc_kernel<DET, WIN, PART>, dim3(items < sms ? items : sms), kAttBwdThreads,
                        C::SMEM, st, tq, td, tdq, tdkv, lse, (const float*)delta, cs, S, Hq, Hkv, B,
                        FixedDiv(Hkv * B), FixedDiv(Hkv), scale, scale * 1.4426950408889634f, win, part, err)) {
    cudaGetLastError();
    return -3;
  }
  if (PART)
    attn_sink_join(part, dqkv, B, S, Hq, Hkv, HD, scale, cs, win.splits, win.sinks, st);
  attn_dq_finalize(dq_acc, dqkv, B, S, Hq, Hkv, HD, scale, cs, DET ? (S + 127) / 128 : 0,
                   WIN ? win.size : 0, win.sinks, st);
  return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

// A chunk has an item for every SM.  The heads left for the end, longest first
// together, are worth 1.2 times the longest item to each SM: with half of that
// the ends of the SMs' work lie further apart (8 x 2048 tokens, 32 / 8 heads:
// 790 us without chunks, 711 us so, 727 us with half; 8192 tokens, 8 heads: 296
// us, and 313 us with half; 8 x 1024, 32 heads: 378 and 303 us; chunks of twice
// the size 714 and 309 us).  With a window neighbouring ranks share most of what
// they read, so nothing is gained (2 x 8192, window 1024: 736 us, 742 with
// chunks).
HeadChunks head_chunks(const dim3& grid, bool window) {
  const int heads = (int)(grid.y * grid.z), sms = num_sms(), ranks = (int)grid.x;
  HeadChunks c{heads, 0};
  if (window) return c;
  // an item of rank r has ranks - r blocks (times the group's heads)
  const int tail = (12 * sms / 5 + ranks) / (ranks + 1), size = (sms + ranks - 1) / ranks;
  if (heads < tail + size) return c;
  c.size = size;
  c.chunked = (heads - tail) / size * size;
  return c;
}

template <bool DET, bool WIN, bool PART>
int bwd_tc2(const __nv_bfloat16* qkv, const __nv_bfloat16* o, const __nv_bfloat16* dout,
            const float* lse, float* delta, float* dq_acc, __nv_bfloat16* dqkv, int B, int S, int Hq,
            int Hkv, const float2* cs, AttWindow win, int* err, cudaStream_t st) {
  using C = AttBwd2Cfg;
  constexpr int HD = 128;
  auto fn = encode_fn_att();
  if (!fn) return -3;
  const int64_t W = (int64_t)(Hq + 2 * Hkv) * HD, WO = (int64_t)Hq * HD;
  CUtensorMap tkv, tq, td, tdq, tdkv;
  cuuint32_t box_kv[3] = {64, 128, 1}, box_q[3] = {64, 128, 1}, box_dq[3] = {32, 32, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  cuuint64_t dq[3] = {(cuuint64_t)W, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t sq[2] = {(cuuint64_t)(W * 2), (cuuint64_t)(S * W * 2)};
  cuuint64_t dd[3] = {(cuuint64_t)WO, (cuuint64_t)S, (cuuint64_t)B};
  cuuint64_t sd[2] = {(cuuint64_t)(WO * 2), (cuuint64_t)(S * WO * 2)};
  auto enc = [&](CUtensorMap* m, const void* base, cuuint64_t* dims, cuuint64_t* strides,
                 cuuint32_t* box) {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const int nkb = (S + 127) / 128;
  const int slots = WIN ? attn_window_dq_slots(S, win.size, win.sinks) : nkb;
  cuuint64_t sdq[2] = {(cuuint64_t)(WO * 4), (cuuint64_t)(S * WO * 4)};
  cuuint64_t ddq[3] = {(cuuint64_t)WO, (cuuint64_t)S, (cuuint64_t)(DET ? (int64_t)B * slots : B)};
  if (!enc(&tkv, qkv, dq, sq, box_kv) || !enc(&tq, qkv, dq, sq, box_q) ||
      !enc(&td, dout, dd, sd, box_q) || !enc(&tdkv, dqkv, dq, sq, box_kv) ||
      fn(&tdq, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, dq_acc, ddq, sdq, box_dq, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return -3;
  if (!reserve_smem<attn_bwd_tc2_kernel<DET, WIN, PART>>(C::SMEM)) return -3;
  attn_delta(o, dout, delta, DET ? nullptr : dq_acc, B, S, Hq, HD, st);
  const float scale = 1.f / sqrtf((float)HD);
  dim3 grid(nkb + (PART ? (win.sinks + 127) / 128 * win.splits : 0), Hkv, B);
  // the sinks' partial dK and dV follow dQ in the scratch
  float* part = dq_acc + (DET ? (int64_t)slots : 1) * B * S * WO;
  if (!launch_dependent(attn_bwd_tc2_kernel<DET, WIN, PART>, grid, kAttBwd2Threads, C::SMEM, st, tkv, tq, td,
                        tdq, tdkv, lse, (const float*)delta, cs, S, Hq, Hkv, scale,
                        scale * 1.4426950408889634f, win, head_chunks(grid, WIN), part, err)) {
    cudaGetLastError();
    return -3;
  }
  if (PART)
    attn_sink_join(part, dqkv, B, S, Hq, Hkv, HD, scale, cs, win.splits, win.sinks, st);
  attn_dq_finalize(dq_acc, dqkv, B, S, Hq, Hkv, HD, scale, cs, DET ? nkb : 0, WIN ? win.size : 0,
                   win.sinks, st);
  return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace

namespace {
template <bool DET, bool WIN, bool PART = false>
int bwd(const __nv_bfloat16* qkv, const __nv_bfloat16* o, const __nv_bfloat16* dout,
        const float* lse, float* delta, float* dq_acc, __nv_bfloat16* dqkv, int B, int S, int Hq,
        int Hkv, int hd, const float2* cs, AttWindow win, int* err, cudaStream_t st) {
  if (hd == 64)
    return bwd_tc<DET, WIN, PART>(qkv, o, dout, lse, delta, dq_acc, dqkv, B, S, Hq, Hkv, cs, win, err, st);
  if (hd == 128)
    return bwd_tc2<DET, WIN, PART>(qkv, o, dout, lse, delta, dq_acc, dqkv, B, S, Hq, Hkv, cs, win, err, st);
  return -1;
}
// The window as the kernels take it.  At head dim 128, where the hardware deals
// the items out, the sinks' queries are split only where one item with all of
// them would take longer than an even share of the work: else it runs beside
// the others from the start, its queries a little ahead of theirs (2 x 8192, 32
// / 8 heads of 128, window 1024, 4 sinks: 792 us in one item, 841 us split).
// At 64 the items are dealt out in advance and a long one delays those behind
// it (1 x 16384, 16 heads, window 1024, 64 sinks: 505 us and 372 us).
AttWindow clip(int window, int sinks, int S, int B, int Hq, int Hkv, int hd) {
  AttWindow win{window < S ? window : S, sinks < S ? sinks : S, attn_window_splits(S, window, sinks)};
  if (hd == 128 && win.splits > 0) {
    const int64_t nq = (S + 127) / 128, near = (126 + win.size) / 128 + 1, ns = (win.sinks + 127) / 128;
    const int64_t work = (int64_t)B * Hq * ((S + 127) / 128 * near + ns * (nq - near));
    if ((int64_t)(Hq / Hkv) * nq * num_sms() <= work) win.splits = 0;
  }
  return win;
}
}  // namespace

int attn_bwd(const __nv_bfloat16* qkv, const __nv_bfloat16* o, const __nv_bfloat16* dout,
             const float* lse, float* delta, float* dq_acc, __nv_bfloat16* dqkv, int B, int S,
             int Hq, int Hkv, int hd, const float2* cs, bool deterministic, int* err,
             cudaStream_t st) {
  if (B <= 0 || S <= 0) return 0;
  if (Hkv <= 0 || Hq % Hkv) return -1;
  const AttWindow all{S, 0, 0};
  return deterministic ? bwd<true, false>(qkv, o, dout, lse, delta, dq_acc, dqkv, B, S, Hq, Hkv,
                                          hd, cs, all, err, st)
                       : bwd<false, false>(qkv, o, dout, lse, delta, dq_acc, dqkv, B, S, Hq, Hkv,
                                           hd, cs, all, err, st);
}

int attn_window_bwd(const __nv_bfloat16* qkv, const __nv_bfloat16* o, const __nv_bfloat16* dout,
                    const float* lse, float* delta, float* dq_acc, __nv_bfloat16* dqkv, int B,
                    int S, int Hq, int Hkv, int hd, int window, int sinks, const float2* cs,
                    bool deterministic, int* err, cudaStream_t st) {
  if (B <= 0 || S <= 0) return 0;
  if (Hkv <= 0 || Hq % Hkv || window < 1 || sinks < 0) return -1;
  if (window >= S || sinks >= S)  // nothing but the causal mask (which has a slot per key block too)
    return attn_bwd(qkv, o, dout, lse, delta, dq_acc, dqkv, B, S, Hq, Hkv, hd, cs, deterministic, err, st);
  const AttWindow win = clip(window, sinks, S, B, Hq, Hkv, hd);
  const auto fn = win.splits > 0 ? (deterministic ? bwd<true, true, true> : bwd<false, true, true>)
                                 : (deterministic ? bwd<true, true> : bwd<false, true>);
  return fn(qkv, o, dout, lse, delta, dq_acc, dqkv, B, S, Hq, Hkv, hd, cs, win, err, st);
}

int attn_fwd(const __nv_bfloat16* qkv, __nv_bfloat16* o, float* lse, int B, int S, int Hq, int Hkv,
             int hd, int* err, cudaStream_t st) {
  if (B <= 0 || S <= 0) return 0;
  if (Hkv <= 0 || Hq % Hkv) return -1;
  if ((reinterpret_cast<uintptr_t>(qkv) & 15) != 0) return -1;
  const AttWindow all{S, 0, 0};
  if (hd == 64) return fwd_pp<64, false>(qkv, o, lse, B, S, Hq, Hkv, all, err, st);
  if (hd == 128) return fwd_pp<128, false>(qkv, o, lse, B, S, Hq, Hkv, all, err, st);
  return -1;
}

int attn_window_fwd(const __nv_bfloat16* qkv, __nv_bfloat16* o, float* lse, int B, int S, int Hq,
                    int Hkv, int hd, int window, int sinks, int* err, cudaStream_t st) {
  if (B <= 0 || S <= 0) return 0;
  if (Hkv <= 0 || Hq % Hkv || window < 1 || sinks < 0) return -1;
  if (window >= S || sinks >= S) return attn_fwd(qkv, o, lse, B, S, Hq, Hkv, hd, err, st);
  const AttWindow win = clip(window, sinks, S, B, Hq, Hkv, hd);
  if (hd == 64) return fwd_pp<64, true>(qkv, o, lse, B, S, Hq, Hkv, win, err, st);
  if (hd == 128) return fwd_pp<128, true>(qkv, o, lse, B, S, Hq, Hkv, win, err, st);
  return -1;
}

}  // namespace sf
