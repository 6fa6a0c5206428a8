// Kernel-level C ABI (sf.h, "kernel API"): single operations of the step on
// caller-owned device buffers.  Argument checks happen here, on the host,
// before any launch; the kernels themselves assume checked arguments.
#include <cuda_runtime.h>

#include <cmath>
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "sf.h"
#include "sf_internal.h"

namespace {

using bf16 = __nv_bfloat16;

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// an array that kernels read or write element by element
template <class T>
bool al1(const T* p) { return (reinterpret_cast<uintptr_t>(p) & (sizeof(T) - 1)) == 0; }

// One device error word per device, created on first use.
constexpr int kMaxDev = 64;
int* g_err[kMaxDev] = {nullptr};
std::mutex g_err_m;

int* dev_err_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return nullptr;
  std::lock_guard<std::mutex> l(g_err_m);
  if (!g_err[dev]) {
    int* p = nullptr;
    if (cudaMalloc(&p, sizeof(int)) != cudaSuccess) return nullptr;
    if (cudaMemset(p, 0, sizeof(int)) != cudaSuccess) return nullptr;
    g_err[dev] = p;
  }
  return g_err[dev];
}

cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }
int launched() { return cudaGetLastError() == cudaSuccess ? SF_OK : SF_ECUDA; }

// Kernels launched by the calling thread's last sf_op_lce call.
thread_local int64_t lce_launches = 0;

}  // namespace

extern "C" {

int sf_op_gemm(int32_t layout, int32_t epi, int64_t M, int64_t N, int64_t K, const void* A,
               int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc, const float* R,
               int64_t ldr, float alpha, void* stream) {
  if (epi < 0 || epi > 3 || layout < 0 || layout > 2) return SF_EINVAL;
  sf::GemmArgs g;
  g.layout = layout; g.epi = epi; g.M = M; g.N = N; g.K = K;
  g.A = A; g.lda = lda; g.B = B; g.ldb = ldb; g.C = C; g.ldc = ldc; g.R = R; g.ldr = ldr;
  g.alpha = alpha;
  char why[128];
  if (sf::gemm_check(g, why) != 0) return SF_EINVAL;
  if (M == 0 || N == 0) return SF_OK;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  const int st = sf::gemm(g, err, S(stream), why);
  if (st == -1) return SF_EINVAL;
  if (st != 0) return SF_ECUDA;
  return SF_OK;
}

int sf_op_gemm_bias(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                    int64_t ldb, void* C, int64_t ldc, const uint16_t* bias, float alpha,
                    void* stream) {
  sf::GemmArgs g;
  g.layout = sf::kNT; g.epi = sf::kEpiBF16Bias; g.M = M; g.N = N; g.K = K;
  g.A = A; g.lda = lda; g.B = B; g.ldb = ldb; g.C = C; g.ldc = ldc; g.alpha = alpha;
  g.bias = bias;
  char why[128];
  if (sf::gemm_check(g, why) != 0) return SF_EINVAL;
  if (M == 0 || N == 0) return SF_OK;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  const int st = sf::gemm(g, err, S(stream), why);
  if (st == -1) return SF_EINVAL;
  if (st != 0) return SF_ECUDA;
  return SF_OK;
}

int64_t sf_op_bias_grad_scratch(int64_t rows, int32_t cols) {
  if (rows < 0 || cols < 0) return -1;
  return (int64_t)sf::rmsnorm_bwd_parts(rows, cols) * cols;
}

int sf_op_bias_grad(const uint16_t* dy, int64_t ld, int64_t rows, int32_t cols, float* part,
                    uint16_t* db, void* stream) {
  if (rows < 0 || cols < 2 || cols % 2 || ld < cols || ld % 2) return SF_EINVAL;
  if (!dy || !part || !db || (reinterpret_cast<uintptr_t>(dy) & 3)) return SF_EINVAL;
  if (rows == 0) return SF_EINVAL;
  sf::bias_grad(reinterpret_cast<const bf16*>(dy), ld, rows, cols, part,
                sf::rmsnorm_bwd_parts(rows, cols), reinterpret_cast<bf16*>(db), S(stream));
  return cudaGetLastError() == cudaSuccess ? SF_OK : SF_ECUDA;
}

int sf_op_rmsnorm_fwd(const float* x, const uint16_t* g, uint16_t* y, float* rstd, int64_t rows,
                      int32_t d, float eps, void* stream) {
  if (rows < 0 || d < 8 || d % 8 || d > 16384 || !(eps > 0.f)) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!x || !g || !y || !rstd || !al16(x) || !al16(y) || (reinterpret_cast<uintptr_t>(g) & 7))
    return SF_EINVAL;
  sf::rmsnorm_fwd(x, reinterpret_cast<const bf16*>(g), reinterpret_cast<bf16*>(y), rstd, rows, d,
                  eps, S(stream));
  return launched();
}

int64_t sf_op_rmsnorm_bwd_scratch(int64_t rows, int32_t d) {
  return (int64_t)sf::rmsnorm_bwd_parts(rows, d) * d;
}

int sf_op_rmsnorm_bwd(const float* x, const uint16_t* g, const float* rstd, const float* dy,
                      const float* dres, float* dx, uint16_t* dxb, uint16_t* dg, float* scratch,
                      int64_t rows, int32_t d, void* stream) {
  if (rows < 1 || d < 8 || d % 8 || d > 16384) return SF_EINVAL;
  if (!x || !g || !rstd || !dy || !dx || !dxb || !dg || !scratch) return SF_EINVAL;
  if (!al16(x) || !al16(dy) || !al16(dx) || !al16(dxb) || !al16(scratch) ||
      (dres && !al16(dres)) || (reinterpret_cast<uintptr_t>(g) & 7))
    return SF_EINVAL;
  const int parts = sf::rmsnorm_bwd_parts(rows, d);
  sf::rmsnorm_bwd(x, reinterpret_cast<const bf16*>(g), rstd, dy, dres, dx,
                  reinterpret_cast<bf16*>(dxb), scratch, parts, rows, d, S(stream));
  sf::reduce_parts_bf16(scratch, parts, d, reinterpret_cast<bf16*>(dg), S(stream));
  return launched();
}

int sf_rope_table(int32_t seq, int32_t head_dim, float rope_base, float* out) {
  if (seq < 1 || head_dim < 2 || head_dim % 2 || !(rope_base > 1.f) || !out) return SF_EINVAL;
  const int half = head_dim / 2;
  for (int j = 0; j < half; ++j) {
    const double inv_freq = std::pow((double)rope_base, -2.0 * j / head_dim);
    for (int s = 0; s < seq; ++s) {
      const double ang = (double)s * inv_freq;
      out[((int64_t)s * half + j) * 2 + 0] = (float)std::cos(ang);
      out[((int64_t)s * half + j) * 2 + 1] = (float)std::sin(ang);
    }
  }
  return SF_OK;
}

int sf_op_rope(uint16_t* x, int64_t ld, int64_t tokens, int32_t seq, int32_t heads,
               int32_t head_dim, const float* table, int32_t inverse, void* stream) {
  if (tokens < 0 || seq < 1 || heads < 1 || head_dim < 16 || head_dim % 16 || ld % 8 ||
      ld < (int64_t)heads * head_dim)
    return SF_EINVAL;
  if (tokens == 0) return SF_OK;
  if (!x || !table || !al16(x) || (reinterpret_cast<uintptr_t>(table) & 7)) return SF_EINVAL;
  sf::rope_inplace(reinterpret_cast<bf16*>(x), ld, tokens, seq, heads, head_dim,
                   reinterpret_cast<const float2*>(table), inverse, S(stream));
  return launched();
}

int sf_op_attn_fwd(const uint16_t* qkv, uint16_t* o, float* lse, int32_t B, int32_t S_,
                   int32_t Hq, int32_t Hkv, int32_t hd, void* stream) {
  if (B < 0 || S_ < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || (hd != 64 && hd != 128)) return SF_EINVAL;
  if (B == 0 || S_ == 0) return SF_OK;
  if (!qkv || !o || !lse || !al16(qkv) || !al16(o)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  if (sf::attn_fwd(reinterpret_cast<const bf16*>(qkv), reinterpret_cast<bf16*>(o), lse, B, S_,
                   Hq, Hkv, hd, err, S(stream)) != 0)
    return SF_ECUDA;
  return SF_OK;
}

int sf_op_attn_bwd(const uint16_t* qkv, const uint16_t* o, const uint16_t* dout,
                   const float* lse, float* delta, float* dq_acc, uint16_t* dqkv, int32_t B,
                   int32_t S_, int32_t Hq, int32_t Hkv, int32_t hd, const float* table,
                   int32_t deterministic, void* stream) {
  if (B < 0 || S_ < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || (hd != 64 && hd != 128)) return SF_EINVAL;
  if (B == 0 || S_ == 0) return SF_OK;
  if (!qkv || !o || !dout || !lse || !delta || !dq_acc || !dqkv) return SF_EINVAL;
  if (!al16(qkv) || !al16(o) || !al16(dout) || !al16(dq_acc) || !al16(dqkv)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  if (sf::attn_bwd(reinterpret_cast<const bf16*>(qkv), reinterpret_cast<const bf16*>(o),
                   reinterpret_cast<const bf16*>(dout), lse, delta, dq_acc,
                   reinterpret_cast<bf16*>(dqkv), B, S_, Hq, Hkv, hd,
                   reinterpret_cast<const float2*>(table), deterministic != 0, err, S(stream)) != 0)
    return SF_ECUDA;
  return SF_OK;
}

// Sizes of the windowed attention; its backward's grid bounds B and Hkv.
static bool window_sizes(int32_t B, int32_t S_, int32_t Hq, int32_t Hkv, int32_t hd, int32_t window,
                         int32_t sinks) {
  if (!(B >= 0 && B <= 65535 && S_ >= 0 && S_ <= (1 << 30) && Hq >= 1 && Hkv >= 1 && Hkv <= 65535 &&
        Hq % Hkv == 0 && (int64_t)Hq + 2 * (int64_t)Hkv <= (1 << 22) && (hd == 64 || hd == 128) &&
        window >= 1 && sinks >= 0))
    return false;
  // no device holds more than 2^38 elements, and the scratch's size stays in 64 bits
  return (int64_t)B * S_ <= ((int64_t)1 << 38) / (((int64_t)Hq + 2 * (int64_t)Hkv) * hd);
}

int sf_op_attn_window_fwd(const uint16_t* qkv, uint16_t* o, float* lse, int32_t B, int32_t S_,
                          int32_t Hq, int32_t Hkv, int32_t hd, int32_t window, int32_t sinks,
                          void* stream) {
  if (!window_sizes(B, S_, Hq, Hkv, hd, window, sinks)) return SF_EINVAL;
  if (B == 0 || S_ == 0) return SF_OK;
  if (!qkv || !o || !lse || !al16(qkv) || !al16(o) || !al1(lse)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  if (sf::attn_window_fwd(reinterpret_cast<const bf16*>(qkv), reinterpret_cast<bf16*>(o), lse, B,
                          S_, Hq, Hkv, hd, window, sinks, err, S(stream)) != 0)
    return SF_ECUDA;
  return SF_OK;
}

int64_t sf_op_attn_window_dq_scratch(int32_t B, int32_t S_, int32_t Hq, int32_t hd, int32_t window,
                                     int32_t sinks, int32_t deterministic) {
  if (!window_sizes(B, S_, Hq, 1, hd, window, sinks)) return -1;
  const int64_t slots = deterministic ? sf::attn_window_dq_slots(S_, window, sinks) : 1;
  return slots * B * S_ * Hq * hd + sf::attn_window_part_floats(B, S_, Hq, hd, window, sinks);
}

int sf_op_attn_window_bwd(const uint16_t* qkv, const uint16_t* o, const uint16_t* dout,
                          const float* lse, float* delta, float* dq_acc, uint16_t* dqkv,
                          int32_t B, int32_t S_, int32_t Hq, int32_t Hkv, int32_t hd,
                          int32_t window, int32_t sinks, const float* table,
                          int32_t deterministic, void* stream) {
  if (!window_sizes(B, S_, Hq, Hkv, hd, window, sinks)) return SF_EINVAL;
  if (B == 0 || S_ == 0) return SF_OK;
  if (!qkv || !o || !dout || !lse || !delta || !dq_acc || !dqkv) return SF_EINVAL;
  if (!al16(qkv) || !al16(o) || !al16(dout) || !al16(dq_acc) || !al16(dqkv)) return SF_EINVAL;
  if ((reinterpret_cast<uintptr_t>(table) & 7) || !al1(lse) || !al1(delta)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  if (sf::attn_window_bwd(reinterpret_cast<const bf16*>(qkv), reinterpret_cast<const bf16*>(o),
                          reinterpret_cast<const bf16*>(dout), lse, delta, dq_acc,
                          reinterpret_cast<bf16*>(dqkv), B, S_, Hq, Hkv, hd, window, sinks,
                          reinterpret_cast<const float2*>(table), deterministic != 0, err,
                          S(stream)) != 0)
    return SF_ECUDA;
  return SF_OK;
}

// The sizes both directions of the query/key norm take.
static bool qknorm_sizes(int64_t tokens, int32_t Hq, int32_t Hkv, int32_t hd) {
  if (tokens < 0 || Hq < 1 || Hkv < 1 || hd < 16 || hd > 256 || hd % 16) return false;
  // bounds the launch grids (and no device holds such a tensor)
  const int64_t heads = (int64_t)Hq + 2 * (int64_t)Hkv;
  return heads <= 65536 && tokens <= ((int64_t)1 << 34) / heads;
}

static bool qknorm_check(int64_t tokens, int32_t seq, int32_t Hq, int32_t Hkv, int32_t hd,
                         const uint16_t* gq, const uint16_t* gk, float eps, const float* table,
                         const int32_t* pos, sf::QkNormArgs* a) {
  if (seq < 1 || !(eps > 0.f) || !gq || !gk || !table || !al16(gq) || !al16(gk) || !al16(table) ||
      !al1(pos))
    return false;
  a->tokens = tokens; a->seq = seq; a->Hq = Hq; a->Hkv = Hkv; a->hd = hd;
  a->gq = reinterpret_cast<const bf16*>(gq);
  a->gk = reinterpret_cast<const bf16*>(gk);
  a->eps = eps;
  a->cs = reinterpret_cast<const float2*>(table);
  a->pos = pos;
  return true;
}

int sf_op_qknorm_rope_fwd(const uint16_t* x, int64_t ldx, uint16_t* y, int64_t ldy,
                          int64_t tokens, int32_t seq, int32_t Hq, int32_t Hkv, int32_t head_dim,
                          const uint16_t* gq, const uint16_t* gk, float eps, const float* table,
                          const int32_t* pos, void* stream) {
  if (!qknorm_sizes(tokens, Hq, Hkv, head_dim)) return SF_EINVAL;
  const int64_t width = ((int64_t)Hq + 2 * (int64_t)Hkv) * head_dim;
  if (ldx % 8 || ldy % 8 || ldx < width || ldy < width || (x == y && ldx != ldy)) return SF_EINVAL;
  sf::QkNormArgs a;
  if (!qknorm_check(tokens, seq, Hq, Hkv, head_dim, gq, gk, eps, table, pos, &a)) return SF_EINVAL;
  if (tokens == 0) return SF_OK;
  if (!x || !y || !al16(x) || !al16(y)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  sf::qknorm_rope_fwd(a, reinterpret_cast<const bf16*>(x), ldx, reinterpret_cast<bf16*>(y), ldy,
                      err, S(stream));
  return launched();
}

int64_t sf_op_qknorm_rope_bwd_scratch(int64_t tokens, int32_t Hq, int32_t Hkv, int32_t head_dim) {
  if (!qknorm_sizes(tokens, Hq, Hkv, head_dim)) return -1;
  return (int64_t)sf::qknorm_parts(tokens, Hq, head_dim) * 2 * head_dim;
}

int sf_op_qknorm_rope_bwd(const uint16_t* x, int64_t ldx, const uint16_t* dy, int64_t lddy,
                          uint16_t* dx, int64_t lddx, int64_t tokens, int32_t seq, int32_t Hq,
                          int32_t Hkv, int32_t head_dim, const uint16_t* gq, const uint16_t* gk,
                          float eps, const float* table, const int32_t* pos, float* scratch,
                          uint16_t* dgq, uint16_t* dgk, void* stream) {
  if (tokens < 1 || !qknorm_sizes(tokens, Hq, Hkv, head_dim)) return SF_EINVAL;
  const int64_t width = ((int64_t)Hq + 2 * (int64_t)Hkv) * head_dim;
  if (ldx % 8 || lddy % 8 || lddx % 8 || ldx < width || lddy < width || lddx < width) return SF_EINVAL;
  if (x == dx || (dx == dy && lddx != lddy)) return SF_EINVAL;
  sf::QkNormArgs a;
  if (!qknorm_check(tokens, seq, Hq, Hkv, head_dim, gq, gk, eps, table, pos, &a)) return SF_EINVAL;
  if (!x || !dy || !dx || !scratch || !dgq || !dgk) return SF_EINVAL;
  if (!al16(x) || !al16(dy) || !al16(dx) || !al16(scratch) || !al1(dgq) || !al1(dgk)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  sf::qknorm_rope_bwd(a, reinterpret_cast<const bf16*>(x), ldx, reinterpret_cast<const bf16*>(dy),
                      lddy, reinterpret_cast<bf16*>(dx), lddx, scratch,
                      reinterpret_cast<bf16*>(dgq), reinterpret_cast<bf16*>(dgk), err, S(stream));
  return launched();
}

// Sizes and format of an 8-bit checkpoint.
static bool ckpt8_sizes(int32_t fmt, int64_t rows, int32_t d) {
  return (fmt == SF_CKPT_INT8 || fmt == SF_CKPT_E4M3) && rows >= 0 && rows <= INT32_MAX && d >= 8 &&
         d % 8 == 0 && d <= 16384;
}

int64_t sf_op_ckpt8_scales(int64_t rows, int32_t d) {
  if (!ckpt8_sizes(SF_CKPT_INT8, rows, d)) return -1;
  return rows * ((d + 127) / 128);
}

int sf_op_ckpt8_save(const float* x, uint8_t* q, float* scale, int32_t fmt, int64_t rows,
                     int32_t d, void* stream) {
  if (!ckpt8_sizes(fmt, rows, d)) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!x || !q || !scale || !al16(x) || !al16(q) || !al16(scale)) return SF_EINVAL;
  sf::ckpt8_save(x, q, scale, fmt, rows, d, S(stream));
  return launched();
}

int sf_op_ckpt8_load(const uint8_t* q, const float* scale, float* x, int32_t fmt, int64_t rows,
                     int32_t d, void* stream) {
  if (!ckpt8_sizes(fmt, rows, d)) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!x || !q || !scale || !al16(x) || !al16(q) || !al16(scale)) return SF_EINVAL;
  sf::ckpt8_load(q, scale, x, fmt, rows, d, S(stream));
  return launched();
}

int sf_op_rmsnorm_fwd_save8(const float* x, const uint16_t* g, uint16_t* y, float* rstd,
                            uint8_t* q, float* scale, int32_t fmt, int64_t rows, int32_t d,
                            float eps, void* stream) {
  if (!ckpt8_sizes(fmt, rows, d) || !(eps > 0.f)) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!x || !g || !y || !rstd || !q || !scale) return SF_EINVAL;
  if (!al16(x) || !al16(y) || !al16(q) || !al16(scale) || !al16(g) || !al1(rstd)) return SF_EINVAL;
  sf::rmsnorm_fwd_save8(x, reinterpret_cast<const bf16*>(g), reinterpret_cast<bf16*>(y), rstd, q,
                        scale, fmt, rows, d, eps, S(stream));
  return launched();
}

int sf_op_rmsnorm_fwd_load8(const uint8_t* q, const float* scale, const uint16_t* g, uint16_t* y,
                            float* rstd, float* x, int32_t fmt, int64_t rows, int32_t d, float eps,
                            void* stream) {
  if (!ckpt8_sizes(fmt, rows, d) || !(eps > 0.f)) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!q || !scale || !g || !y || !rstd) return SF_EINVAL;
  if (!al16(q) || !al16(scale) || !al16(g) || !al16(y) || !al16(x) || !al1(rstd)) return SF_EINVAL;
  sf::rmsnorm_fwd_load8(q, scale, reinterpret_cast<const bf16*>(g), reinterpret_cast<bf16*>(y),
                        rstd, x, fmt, rows, d, eps, S(stream));
  return launched();
}

int sf_op_rmsnorm_bwd_load8(const uint8_t* q, const float* scale, const uint16_t* g,
                            const float* rstd, const float* dy, const float* dres, float* dx,
                            uint16_t* dxb, uint16_t* dg, float* scratch, int32_t fmt, int64_t rows,
                            int32_t d, void* stream) {
  if (!ckpt8_sizes(fmt, rows, d) || rows < 1) return SF_EINVAL;
  if (!q || !scale || !g || !rstd || !dy || !dx || !dxb || !dg || !scratch) return SF_EINVAL;
  if (!al16(q) || !al16(scale) || !al16(g) || !al16(dy) || !al16(dres) || !al16(dx) ||
      !al16(dxb) || !al16(scratch) || !al1(rstd) || !al1(dg))
    return SF_EINVAL;
  const int parts = sf::rmsnorm_bwd_load8_parts(rows, d);
  if (!sf::rmsnorm_bwd_load8(q, scale, reinterpret_cast<const bf16*>(g), rstd, dy, dres, dx,
                             reinterpret_cast<bf16*>(dxb), scratch, parts, fmt, rows, d, S(stream))) {
    cudaGetLastError();
    return SF_ECUDA;
  }
  sf::gain_sums(scratch, parts, d, reinterpret_cast<bf16*>(dg), 0, nullptr, S(stream));
  return launched();
}

// The mask of sf_op_dropout; false for a p or step that is refused.
static bool drop_args(float p, uint64_t seed, uint64_t offset, const uint64_t* step, sf::DropArgs* a) {
  if (!(p >= 0.f && p <= 1.f) || !al1(step)) return false;
  const long t = std::lrint((double)p * 65536.0);
  if (t > 65535) return false;
  a->top = (uint32_t)t << 16;
  a->scale = (float)(65536.0 / (65536.0 - (double)t));
  a->seed = seed;
  a->offset = offset;
  a->step = step;
  return true;
}
static bool a_type(int32_t t) { return t == SF_BF16 || t == SF_F32; }

int sf_op_dropout(const void* x, void* y, int32_t type, int64_t n, float p, uint64_t seed,
                  uint64_t offset, const uint64_t* step, void* stream) {
  sf::DropArgs a;
  if (!a_type(type) || n < 0 || n > ((int64_t)1 << 40) || !drop_args(p, seed, offset, step, &a))
    return SF_EINVAL;
  if (n == 0) return SF_OK;
  if (!x || !y || !al16(x) || !al16(y)) return SF_EINVAL;
  sf::dropout(x, y, type == SF_F32, n, a, S(stream));
  return launched();
}

// What both directions of the join take.
static bool join_sizes(int64_t rows, int32_t d) {
  return rows >= 0 && rows <= INT32_MAX && d >= 8 && d % 8 == 0 && d <= 16384;
}
static bool join_args(int32_t h_type, const uint16_t* g_post, const uint16_t* gate,
                      const uint16_t* g_next, float alpha, float beta, float p, uint64_t seed,
                      uint64_t offset, const uint64_t* step, int64_t rows, int32_t d, sf::JoinArgs* a) {
  if (!a_type(h_type) || !std::isfinite(alpha) || !std::isfinite(beta) || !join_sizes(rows, d) ||
      !al16(g_post) || !al16(gate) || !al16(g_next) || !drop_args(p, seed, offset, step, &a->drop))
    return false;
  a->rows = rows;
  a->d = d;
  a->g_post = reinterpret_cast<const bf16*>(g_post);
  a->gate = reinterpret_cast<const bf16*>(gate);
  a->g_next = reinterpret_cast<const bf16*>(g_next);
  a->alpha = alpha;
  a->beta = beta;
  return true;
}

int sf_op_join_fwd(const float* x, const void* h, int32_t h_type, const uint16_t* g_post,
                   const uint16_t* gate, const uint16_t* g_next, float alpha, float beta, float p,
                   uint64_t seed, uint64_t offset, const uint64_t* step, float* xout, uint16_t* y,
                   float* rstd_post, float* rstd_next, int64_t rows, int32_t d, float eps,
                   void* stream) {
  sf::JoinArgs a;
  if (!join_args(h_type, g_post, gate, g_next, alpha, beta, p, seed, offset, step, rows, d, &a))
    return SF_EINVAL;
  if ((g_post || g_next) && !(eps > 0.f)) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!x || !h || !xout || !al16(x) || !al16(h) || !al16(xout)) return SF_EINVAL;
  if (g_post && (!rstd_post || !al1(rstd_post))) return SF_EINVAL;
  if (g_next && (!y || !rstd_next || !al16(y) || !al1(rstd_next))) return SF_EINVAL;
  sf::join_fwd(a, x, h, h_type == SF_F32, xout, reinterpret_cast<bf16*>(y), rstd_post, rstd_next,
               eps, S(stream));
  return launched();
}

int64_t sf_op_join_bwd_scratch(int64_t rows, int32_t d) {
  if (!join_sizes(rows, d)) return -1;
  return (int64_t)sf::join_bwd_parts(rows, d) * 2 * d;
}

int sf_op_join_bwd(const float* xout, const void* h, int32_t h_type, const uint16_t* g_post,
                   const uint16_t* gate, const uint16_t* g_next, float alpha, float beta, float p,
                   uint64_t seed, uint64_t offset, const uint64_t* step, const float* rstd_post,
                   const float* rstd_next, const float* dy, const float* dres, float* dx, void* dh,
                   uint16_t* dg_post, uint16_t* dgate, uint16_t* dg_next, float* scratch,
                   int64_t rows, int32_t d, void* stream) {
  sf::JoinArgs a;
  if (!join_args(h_type, g_post, gate, g_next, alpha, beta, p, seed, offset, step, rows, d, &a) || rows < 1)
    return SF_EINVAL;
  if (!xout || !h || !dx || !dh || !al16(xout) || !al16(h) || !al16(dx) || !al16(dh) || !al16(dres))
    return SF_EINVAL;
  if (dx == xout || dh == h) return SF_EINVAL;
  if (g_next ? (!dy || !rstd_next || !dg_next || !al16(dy) || !al1(rstd_next) || !al1(dg_next)) : !dres)
    return SF_EINVAL;
  if (g_post && (!rstd_post || !dg_post || !al1(rstd_post) || !al1(dg_post))) return SF_EINVAL;
  if (gate && (!dgate || !al1(dgate))) return SF_EINVAL;
  if ((g_post || gate || g_next) && (!scratch || !al16(scratch))) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  if (!sf::join_bwd(a, xout, h, h_type == SF_F32, rstd_post, rstd_next, dy, dres, dx, dh,
                    reinterpret_cast<bf16*>(g_post ? dg_post : nullptr),
                    reinterpret_cast<bf16*>(gate ? dgate : nullptr),
                    reinterpret_cast<bf16*>(g_next ? dg_next : nullptr), scratch, err, S(stream))) {
    cudaGetLastError();
    return SF_ECUDA;
  }
  return launched();
}

int sf_op_swiglu_fwd(const uint16_t* ab, uint16_t* m, int64_t rows, int32_t ffn, void* stream) {
  if (rows < 0 || ffn < 8 || ffn % 8) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!ab || !m || !al16(ab) || !al16(m)) return SF_EINVAL;
  sf::swiglu_fwd(reinterpret_cast<const bf16*>(ab), reinterpret_cast<bf16*>(m), rows, ffn, S(stream));
  return launched();
}

int sf_op_swiglu_bwd(const uint16_t* dm, const uint16_t* ab, uint16_t* dab, int64_t rows,
                     int32_t ffn, void* stream) {
  if (rows < 0 || ffn < 8 || ffn % 8) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!dm || !ab || !dab || !al16(dm) || !al16(ab) || !al16(dab)) return SF_EINVAL;
  sf::swiglu_bwd(reinterpret_cast<const bf16*>(dm), reinterpret_cast<const bf16*>(ab),
                 reinterpret_cast<bf16*>(dab), rows, ffn, S(stream));
  return launched();
}

int64_t sf_op_lce_workspace_bytes(int64_t n, int32_t v, int64_t chunk_rows) {
  if (n < 1 || v < 8 || chunk_rows < 1) return -1;
  const int64_t c = chunk_rows < n ? chunk_rows : n;
  const int64_t logits = (c * v * 4 + 255) / 256 * 256;  // fp32 logits of a chunk
  const int64_t dz = (c * v * 2 + 255) / 256 * 256;      // their bf16 dZ
  const int64_t rows = (n * 4 + 255) / 256 * 256;
  return logits + dz + rows;
}

int sf_op_lce(const uint16_t* h, const uint16_t* w, const int32_t* labels, int64_t n, int32_t d,
              int32_t v, int64_t n_valid, int64_t chunk_rows, void* workspace, float* loss,
              float* dh, float* dw, void* stream) {
  if (n < 1 || d < 8 || d % 8 || v < 8 || v % 8 || chunk_rows < 1 || n_valid < 0 || n_valid > n)
    return SF_EINVAL;
  if (!h || !w || !labels || !workspace || !loss || !dh || !dw) return SF_EINVAL;
  if (!al16(h) || !al16(w) || !al16(dh) || !al16(dw) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  const int64_t c = chunk_rows < n ? chunk_rows : n;
  char* ws = reinterpret_cast<char*>(workspace);
  float* zf = reinterpret_cast<float*>(ws);
  ws += (c * v * 4 + 255) / 256 * 256;
  bf16* dz = reinterpret_cast<bf16*>(ws);
  ws += (c * v * 2 + 255) / 256 * 256;
  float* loss_rows = reinterpret_cast<float*>(ws);
  const bf16* H = reinterpret_cast<const bf16*>(h);
  const bf16* W = reinterpret_cast<const bf16*>(w);
  const float inv_n = n_valid > 0 ? 1.f / (float)n_valid : 0.f;
  char why[128];
  cudaStream_t st = S(stream);
  int count = 0;  // kernels launched, for sf_op_lce_launches
  lce_launches = 0;
  for (int64_t r0 = 0; r0 < n; r0 += c) {
    const int64_t rows = (c < n - r0) ? c : n - r0;
    sf::GemmArgs z;
    z.layout = sf::kNT; z.epi = sf::kEpiF32; z.M = rows; z.N = v; z.K = d;
    z.A = H + r0 * d; z.lda = d; z.B = W; z.ldb = d; z.C = zf; z.ldc = v; z.launched = &count;
    if (sf::gemm(z, err, st, why) != 0) return SF_ECUDA;
    if (sf::ce_rows_f32(zf, dz, labels + r0, rows, v, inv_n, loss_rows + r0, err, st) != 0)
      return SF_ECUDA;
    ++count;
    // dH over up to four vocabulary ranges when that fills the SMs better; the
    // partial sums go to the chunk's fp32 logits, which the row kernel has read
    sf::GemmArgs gx;
    gx.layout = sf::kNN; gx.epi = sf::kEpiF32; gx.M = rows; gx.N = d; gx.K = v;
    gx.A = dz; gx.lda = v; gx.B = W; gx.ldb = d; gx.C = dh + r0 * d; gx.ldc = d;
    gx.splitk_max = (int)std::min<int64_t>(4, 1 + (c * (int64_t)v) / (rows * (int64_t)d));
    gx.ws = zf; gx.launched = &count;
    if (sf::gemm(gx, err, st, why) != 0) return SF_ECUDA;
    sf::GemmArgs gw;
    gw.layout = sf::kTN; gw.epi = r0 == 0 ? sf::kEpiF32 : sf::kEpiF32Acc; gw.M = v; gw.N = d;
    gw.K = rows; gw.A = dz; gw.lda = v; gw.B = H + r0 * d; gw.ldb = d; gw.C = dw; gw.ldc = d;
    gw.launched = &count;
    if (sf::gemm(gw, err, st, why) != 0) return SF_ECUDA;
  }
  sf::sum_f32(loss_rows, n, inv_n, loss, st);
  lce_launches = count + 1;
  return launched();
}

int64_t sf_op_lce_launches(void) { return lce_launches; }

// What both directions of the log probabilities take.
static bool logprob_sizes(int32_t z_type, int64_t ldz, int64_t rows, int32_t vocab, float scale) {
  return a_type(z_type) && rows >= 0 && rows <= INT32_MAX && vocab >= 1 && vocab <= (1 << 20) &&
         ldz >= vocab && ldz % 8 == 0 && scale >= 9.5367431640625e-07f && scale <= 1048576.f;
}
static bool logprob_outputs(float* logp, float* lse, float* entropy, int32_t vocab, int32_t top, int32_t* ids,
                            float* top_logp) {
  if (!logp || !lse || !al1(logp) || !al1(lse) || !al1(entropy)) return false;
  if (top < 0 || top > SF_LOGPROB_TOP_MAX || top > vocab) return false;
  return top == 0 || (ids && top_logp && al1(ids) && al1(top_logp));
}
static bool logprob_gradients(const float* lse, const float* entropy, const float* dlogp, const float* dentropy) {
  return lse && dlogp && al1(lse) && al1(dlogp) && (!dentropy || (entropy && al1(entropy) && al1(dentropy)));
}

static sf::LogprobEpi logprob_epi(const int32_t* tokens, float scale, const float* lse, const float* entropy,
                                  const float* dlogp, const float* dentropy) {
  sf::LogprobEpi a;
  a.tokens = tokens; a.scale = scale; a.lse = lse; a.entropy = entropy; a.dlogp = dlogp; a.dentropy = dentropy;
  return a;
}

int sf_op_logprob_rows(const void* z, int32_t z_type, int64_t ldz, const int32_t* tokens,
                       int64_t rows, int32_t vocab, float scale, float* logp, float* lse,
                       float* entropy, int32_t top, int32_t* ids, float* top_logp, void* stream) {
  if (!logprob_sizes(z_type, ldz, rows, vocab, scale)) return SF_EINVAL;
  if (top < 0 || top > SF_LOGPROB_TOP_MAX || top > vocab) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!z || !tokens || !al16(z) || !al1(tokens)) return SF_EINVAL;
  if (!logprob_outputs(logp, lse, entropy, vocab, top, ids, top_logp)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  if (!sf::logprob_rows(z, z_type == SF_F32, ldz, tokens, rows, vocab, scale, logp, lse, entropy, top,
                        ids, top_logp, err, S(stream))) {
    cudaGetLastError();
    return SF_ECUDA;
  }
  return launched();
}

int sf_op_logprob_rows_bwd(const void* z, int32_t z_type, int64_t ldz, const int32_t* tokens,
                           int64_t rows, int32_t vocab, float scale, const float* lse,
                           const float* entropy, const float* dlogp, const float* dentropy,
                           uint16_t* dz, int64_t lddz, void* stream) {
  if (!logprob_sizes(z_type, ldz, rows, vocab, scale) || lddz < vocab || lddz % 8) return SF_EINVAL;
  if (rows == 0) return SF_OK;
  if (!z || !tokens || !dz || !al16(z) || !al1(tokens) || !al16(dz)) return SF_EINVAL;
  if (!logprob_gradients(lse, entropy, dlogp, dentropy)) return SF_EINVAL;
  if (dz == z && (z_type != SF_BF16 || lddz != ldz)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  sf::logprob_rows_bwd(z, z_type == SF_F32, ldz, logprob_epi(tokens, scale, lse, entropy, dlogp, dentropy), rows,
                       vocab, reinterpret_cast<bf16*>(dz), lddz, err, S(stream));
  return launched();
}

// The head of the log probabilities: sizes, and a chunk's place in the workspace.
static bool lm_logprob_sizes(int64_t n, int32_t d, int32_t v, int64_t chunk_rows) {
  return n >= 1 && n <= INT32_MAX && d >= 8 && d % 8 == 0 && v >= 8 && v % 8 == 0 && v <= (1 << 20) &&
         chunk_rows >= 1;
}
static int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

int64_t sf_op_lm_logprob_workspace_bytes(int64_t n, int32_t v, int64_t chunk_rows) {
  if (!lm_logprob_sizes(n, 8, v, chunk_rows)) return -1;
  return up256(std::min(n, chunk_rows) * v * 4);
}

// Up to this many rows the backward keeps what the rounding of dz left as rows of
// its own: they fit into the same tile of 256 rows, and no other rows average a
// single rounding out (dH and dW of one row were 0.0034 off in the root mean
// square, where rounding the result alone leaves 0.0017).
constexpr int64_t kFewRows = 128;
// Bytes of those rows' products: fp32 dH of both halves, and h twice.
static int64_t few_sums(int64_t n, int32_t d) { return up256(2 * n * d * 4); }
static int64_t lm_bwd_chunk(int64_t n, int64_t chunk_rows) {
  return std::min(n, std::max(chunk_rows, kFewRows));
}

int64_t sf_op_lm_logprob_bwd_workspace_bytes(int64_t n, int32_t d, int32_t v, int64_t chunk_rows) {
  if (!lm_logprob_sizes(n, d, v, chunk_rows)) return -1;
  const int64_t c = lm_bwd_chunk(n, chunk_rows), room = up256(c * v * 4) + up256(c * v * 2);
  if (n <= kFewRows) return room + few_sums(n, d) + up256(2 * n * d * 2);
  return room + (n > c ? up256((int64_t)v * d * 4) : 0);
}

int sf_op_lm_logprob(const uint16_t* h, const uint16_t* w, const int32_t* tokens, int64_t n,
                     int32_t d, int32_t v, float scale, int64_t chunk_rows, void* workspace,
                     float* logp, float* lse, float* entropy, int32_t top, int32_t* ids,
                     float* top_logp, void* stream) {
  if (!lm_logprob_sizes(n, d, v, chunk_rows) || !logprob_sizes(SF_F32, v, n, v, scale)) return SF_EINVAL;
  if (!h || !w || !tokens || !workspace || !al16(h) || !al16(w) || !al1(tokens) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return SF_EINVAL;
  if (!logprob_outputs(logp, lse, entropy, v, top, ids, top_logp)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  const int64_t c = std::min(n, chunk_rows);
  float* zf = static_cast<float*>(workspace);
  char why[128];
  cudaStream_t st = S(stream);
  sf::GemmArgs z;
  z.layout = sf::kNT; z.N = v; z.K = d; z.lda = d; z.B = w; z.ldb = d; z.ldc = v;
  if (top == 0) {
    // The logits leave the product as their sums, 16 bytes for 256 columns of a
    // row: as many rows at a time as the workspace holds of those.
    const int tiles = (v + sf::gemm_tile_cols(v) - 1) / sf::gemm_tile_cols(v);
    const int64_t most = std::min(n, c * v * 4 / (tiles * 16 + 4));
    for (int64_t r0 = 0; r0 < n; r0 += most) {
      const int64_t rows = std::min(most, n - r0);
      sf::LogprobEpi a = logprob_epi(tokens + r0, scale, nullptr, nullptr, nullptr, nullptr);
      a.parts = reinterpret_cast<float4*>(zf);
      a.token_logit = zf + rows * tiles * 4;
      z.epi = sf::kEpiLogprob; z.M = rows; z.A = h + r0 * d; z.lp = a;
      if (sf::gemm(z, err, st, why) != 0) return SF_ECUDA;
      if (!sf::logprob_tiles(a, rows, tiles, v, logp + r0, lse + r0, entropy ? entropy + r0 : nullptr, err, st)) {
        cudaGetLastError();
        return SF_ECUDA;
      }
    }
    return launched();
  }
  for (int64_t r0 = 0; r0 < n; r0 += c) {
    const int64_t rows = std::min(c, n - r0);
    z.epi = sf::kEpiF32; z.M = rows; z.A = h + r0 * d; z.C = zf;
    if (sf::gemm(z, err, st, why) != 0) return SF_ECUDA;
    if (!sf::logprob_rows(zf, true, v, tokens + r0, rows, v, scale, logp + r0, lse + r0,
                          entropy ? entropy + r0 : nullptr, top, ids + r0 * top, top_logp + r0 * top, err, st)) {
      cudaGetLastError();
      return SF_ECUDA;
    }
  }
  return launched();
}

int sf_op_lm_logprob_bwd(const uint16_t* h, const uint16_t* w, const int32_t* tokens, int64_t n,
                         int32_t d, int32_t v, float scale, int64_t chunk_rows, const float* lse,
                         const float* entropy, const float* dlogp, const float* dentropy,
                         void* workspace, uint16_t* dh, uint16_t* dw, void* stream) {
  if (!lm_logprob_sizes(n, d, v, chunk_rows) || !logprob_sizes(SF_F32, v, n, v, scale)) return SF_EINVAL;
  if (!h || !w || !tokens || !workspace || !dh || !dw || !al16(h) || !al16(w) || !al1(tokens) || !al16(dh) ||
      !al16(dw) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return SF_EINVAL;
  if (dh == h) return SF_EINVAL;  // dw's product reads h after dh is written
  if (!logprob_gradients(lse, entropy, dlogp, dentropy)) return SF_EINVAL;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  // The logits leave the product as dz, so a chunk's room holds three chunks' rows;
  // equal passes of whole tiles.  dz is bf16, the type of the other operand of both
  // products: dh and dw are then 0.0024 off in the root mean square, where rounding the
  // results alone leaves 0.0017 (4095 x 2048 x 32000).  Its rest as rows of its own, as
  // few rows have it below, would be two products more.
  const int64_t c = lm_bwd_chunk(n, chunk_rows), most = std::min(n, 3 * c), passes = (n + most - 1) / most;
  const int64_t pass = std::min(most, ((n + passes - 1) / passes + 255) / 256 * 256);
  char* ws = static_cast<char*>(workspace);
  bf16* dz = reinterpret_cast<bf16*>(ws);
  const int64_t room = up256(c * v * 4) + up256(c * v * 2);
  float* sum = reinterpret_cast<float*>(ws + room);
  char why[128];
  cudaStream_t st = S(stream);
  if (n <= kFewRows) {
    float* part = reinterpret_cast<float*>(ws + room);
    bf16* twice = reinterpret_cast<bf16*>(ws + room + few_sums(n, d));
    const int64_t slice = 2 * n * d, used = up256(2 * n * v * 2), fits = (room - used) / (slice * 4);
    for (int half = 0; half < 2; ++half)
      if (cudaMemcpyAsync(twice + half * n * d, h, (size_t)(n * d * 2), cudaMemcpyDeviceToDevice, st) != cudaSuccess) {
        cudaGetLastError();
        return SF_ECUDA;
      }
    sf::GemmArgs z;
    z.layout = sf::kNT; z.epi = sf::kEpiLogprobBwd; z.M = n; z.N = v; z.K = d;
    z.A = h; z.lda = d; z.B = w; z.ldb = d; z.C = dz; z.ldc = v;
    z.lp = logprob_epi(tokens, scale, lse, entropy, dlogp, dentropy);
    z.lp.low = dz + n * v;
    if (sf::gemm(z, err, st, why) != 0) return SF_ECUDA;
    sf::GemmArgs gx;
    gx.layout = sf::kNN; gx.epi = sf::kEpiF32; gx.M = 2 * n; gx.N = d; gx.K = v;
    gx.A = dz; gx.lda = v; gx.B = w; gx.ldb = d; gx.C = part; gx.ldc = d;
    gx.splitk_max = (int)std::min<int64_t>(fits + 1, 64);
    gx.ws = reinterpret_cast<float*>(ws + used);
    if (sf::gemm(gx, err, st, why) != 0) return SF_ECUDA;
    sf::add_halves_bf16(part, reinterpret_cast<bf16*>(dh), n * d, st);
    sf::GemmArgs gw;
    gw.layout = sf::kTN; gw.epi = sf::kEpiBF16Acc; gw.M = v; gw.N = d; gw.K = 2 * n;
    gw.A = dz; gw.lda = v; gw.B = twice; gw.ldb = d; gw.C = dw; gw.ldc = d;
    if (sf::gemm(gw, err, st, why) != 0) return SF_ECUDA;
    return launched();
  }
  for (int64_t r0 = 0; r0 < n; r0 += pass) {
    const int64_t rows = std::min(pass, n - r0);
    const bool first = r0 == 0, last = r0 + rows == n;
    sf::GemmArgs z;
    z.layout = sf::kNT; z.epi = sf::kEpiLogprobBwd; z.M = rows; z.N = v; z.K = d;
    z.A = h + r0 * d; z.lda = d; z.B = w; z.ldb = d; z.C = dz; z.ldc = v;
    z.lp = logprob_epi(tokens + r0, scale, lse + r0, entropy ? entropy + r0 : nullptr, dlogp + r0,
                       dentropy ? dentropy + r0 : nullptr);
    if (sf::gemm(z, err, st, why) != 0) return SF_ECUDA;
    // dH over ranges of the vocabulary where its tiles leave SMs idle and the room
    // behind dz holds their fp32 sums (1 x 4096 x 128256 in one range: 1.2 ms)
    const int64_t slice = rows * d, fits = (room - up256(rows * v * 2)) / (slice * 4);
    const int split = sf::gemm_splitk(rows, d, v, (int)std::min<int64_t>(fits, 64));
    float* part = reinterpret_cast<float*>(ws + up256(rows * v * 2));
    sf::GemmArgs gx;
    gx.layout = sf::kNN; gx.epi = sf::kEpiBF16; gx.M = rows; gx.N = d; gx.K = v;
    gx.A = dz; gx.lda = v; gx.B = w; gx.ldb = d; gx.C = dh + r0 * d; gx.ldc = d;
    if (split > 1) {
      gx.epi = sf::kEpiF32; gx.C = part; gx.splitk_max = split; gx.ws = part + slice;
    }
    if (sf::gemm(gx, err, st, why) != 0) return SF_ECUDA;
    if (split > 1) sf::cast_f32_bf16(part, reinterpret_cast<bf16*>(dh) + r0 * d, slice, st);
    // dW: fp32 sums over the chunks; the last chunk's product adds the sum and rounds it once
    sf::GemmArgs gw;
    gw.layout = sf::kTN; gw.epi = last ? sf::kEpiBF16Acc : first ? sf::kEpiF32 : sf::kEpiF32Acc;
    gw.M = v; gw.N = d; gw.K = rows; gw.A = dz; gw.lda = v; gw.B = h + r0 * d; gw.ldb = d; gw.ldc = d;
    gw.C = last ? static_cast<void*>(dw) : sum;
    gw.R = last && !first ? sum : nullptr;
    gw.ldr = d;
    if (sf::gemm(gw, err, st, why) != 0) return SF_ECUDA;
  }
  return launched();
}

// The fused-epilogue projections: argument checks in sf::gemm_check.
static int run_gemm(const sf::GemmArgs& g, cudaStream_t st) {
  char why[128];
  if (sf::gemm_check(g, why) != 0) return SF_EINVAL;
  if (g.M == 0 || g.N == 0) return SF_OK;
  int* err = dev_err_word();
  if (!err) return SF_ECUDA;
  const int rc = sf::gemm(g, err, st, why);
  if (rc == -1) return SF_EINVAL;
  return rc == 0 ? SF_OK : SF_ECUDA;
}

int sf_op_gemm_qkv(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                   int64_t ldb, uint16_t* C, int64_t ldc, const uint16_t* bias, const float* table,
                   int32_t seq, int32_t rope_cols, int32_t head_dim, void* stream) {
  sf::GemmArgs g;
  g.layout = sf::kNT; g.epi = sf::kEpiQKV; g.M = M; g.N = N; g.K = K;
  g.A = A; g.lda = lda; g.B = B; g.ldb = ldb; g.C = C; g.ldc = ldc; g.bias = bias;
  g.cs = reinterpret_cast<const float2*>(table); g.seq = seq; g.rope_cols = rope_cols; g.hd = head_dim;
  return run_gemm(g, S(stream));
}

int sf_op_gemm_swiglu(int64_t M, int64_t F, int64_t K, const void* A, int64_t lda,
                      const void* B, int64_t ldb, uint16_t* m, int64_t ldm, float* ab,
                      int64_t ldab, void* stream) {
  sf::GemmArgs g;
  g.layout = sf::kNT; g.epi = sf::kEpiGLU; g.M = M; g.N = F; g.K = K;
  g.A = A; g.lda = lda; g.B = B; g.ldb = ldb; g.C = m; g.ldc = ldm; g.aux = ab; g.ldaux = ldab;
  return run_gemm(g, S(stream));
}

int sf_op_gemm_swiglu_bwd(int64_t M, int64_t F, int64_t K, const void* dy, int64_t lddy,
                          const void* wd, int64_t ldw, const float* ab, int64_t ldab,
                          uint16_t* dab, int64_t lddab, void* stream) {
  sf::GemmArgs g;
  g.layout = sf::kNN; g.epi = sf::kEpiGLUBwd; g.M = M; g.N = F; g.K = K;
  g.A = dy; g.lda = lddy; g.B = wd; g.ldb = ldw; g.C = dab; g.ldc = lddab; g.R = ab; g.ldr = ldab;
  return run_gemm(g, S(stream));
}

int sf_op_device_error(int32_t* out) {
  if (!out) return SF_EINVAL;
  int* e = dev_err_word();
  if (!e) return SF_ECUDA;
  int v = 0;
  if (cudaDeviceSynchronize() != cudaSuccess) return SF_ECUDA;
  if (cudaMemcpy(&v, e, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return SF_ECUDA;
  if (cudaMemset(e, 0, sizeof(int)) != cudaSuccess) return SF_ECUDA;
  *out = v;
  return SF_OK;
}

}  // extern "C"
