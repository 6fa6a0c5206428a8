// Internal launchers of the CUDA kernels (host-side declarations).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

namespace sf {

// Codes written to the device error word (the first one a launch meets).
enum DevErr : int {
  kDevOk = 0,
  kDevGemmTimeout = 1,
  kDevAttnTimeout = 2,
  kDevCeTimeout = 3,
  kDevCeBadLabel = 4,  // a label or token at or beyond the vocabulary (the row is ignored)
  kDevBadPosition = 5,  // a position outside the rotation table (the token is not rotated)
  kDevSharedBase = 6,   // an attention backward's shared memory does not start on 1024 bytes (nothing is written)
  kDevJoinTimeout = 7,
};

// Operand layouts of C[M,N] = A * B (all matrices row-major in memory):
//   kNT: A [M,K] (K contiguous), B [N,K] (K contiguous)   -> Y = X W^T
//   kNN: A [M,K] (K contiguous), B [K,N] (N contiguous)   -> dX = dY W
//   kTN: A [K,M] (M contiguous), B [K,N] (N contiguous)   -> dW = dY^T X
enum GemmLayout : int { kNT = 0, kNN = 1, kTN = 2 };
// Epilogues: C bf16 = alpha*acc | C f32 = alpha*acc | C f32 = R + alpha*acc | C f32 += alpha*acc
// | C bf16 = alpha*acc + bias[col] (bias bf16 [N], 64-byte aligned; layout kNT only)
// | C fp16 = alpha*acc (layout kTN only: scaled fp16 weight gradients)
// | kEpiQKV (layout kNT): y = alpha*acc (+ bias[col] when bias != null), then the
//   rotary embedding on the columns below rope_cols (heads of hd columns, pair
//   (j, j + hd/2), position row % seq, (cos, sin) from cs[pos * hd/2 + j]) and
//   one bf16 rounding: the Q/K/V projection with its rotation
// | kEpiGLU (layout kNT): B holds 2N rows, [Bg; Bu]; a = alpha*A Bg^T and
//   b = alpha*A Bu^T share one accumulator tile, C bf16 [M, N] = silu(a) * b;
//   when aux != null, a and b are also stored as fp32: aux[r, j] = a,
//   aux[r, N + j] = b (the SwiGLU forward of the gate/up projection)
// | kEpiGLUBwd (layout kNN): dm = alpha*acc, with a = R[r, j], b = R[r, N + j]
//   (fp32) C[r, j] = bf16(dm b s (1 + a (1 - s))), C[r, N + j] = bf16(dm a s),
//   s = sigmoid(a) (the down projection's input gradient through SwiGLU)
// | kEpiBF16Acc (layout kTN): C bf16 = alpha*acc + R (R fp32, may be null):
//   the last of a chunked sum of weight gradients, rounded once
// | kEpiLogprob (layout kNT): no C; for each row and tile of gemm_tile_cols columns
//   the sums of its logits z = acc as lp.parts[tile * M + row], and the logit of
//   the row's token (0 <= lp.tokens[row] < N) as lp.token_logit[row]
// | kEpiLogprobBwd (layout kNT): C bf16 = the gradient of the logits z = acc from
//   lp's tokens, lse, entropy, dlogp and dentropy
enum GemmEpi : int {
  kEpiBF16 = 0, kEpiF32 = 1, kEpiF32Add = 2, kEpiF32Acc = 3, kEpiBF16Bias = 4, kEpiF16 = 5,
  kEpiQKV = 6, kEpiGLU = 7, kEpiGLUBwd = 8, kEpiBF16Acc = 9, kEpiLogprob = 10, kEpiLogprobBwd = 11
};

// Rows' tokens and scale for the log probabilities (sf.h); backward: lse,
// entropy, dlogp, dentropy (may be null, and entropy with it).  parts and
// token_logit are written by kEpiLogprob and read by logprob_tiles; low, unless it
// is null, gets what the rounding of a kEpiLogprobBwd product's C left, as bf16.
struct LogprobEpi {
  const int32_t* tokens = nullptr;
  float scale = 1.f;
  const float *lse = nullptr, *entropy = nullptr, *dlogp = nullptr, *dentropy = nullptr;
  float4* parts = nullptr;
  float* token_logit = nullptr;
  __nv_bfloat16* low = nullptr;
};

struct GemmArgs {
  int layout = kNT, epi = kEpiBF16;
  int64_t M = 0, N = 0, K = 0;
  const void* A = nullptr;
  int64_t lda = 0;
  const void* B = nullptr;
  int64_t ldb = 0;
  void* C = nullptr;
  int64_t ldc = 0;
  const float* R = nullptr;
  int64_t ldr = 0;
  float alpha = 1.f;
  const void* bias = nullptr;  // kEpiBF16Bias; kEpiQKV (optional)
  // kEpiQKV: rotation table (cos, sin) [seq, hd/2], columns [0, rope_cols) rotated
  const float2* cs = nullptr;
  int seq = 0, rope_cols = 0, hd = 0;
  // kEpiGLU: optional fp32 copy of the gate and up outputs, row stride ldaux
  float* aux = nullptr;
  int64_t ldaux = 0;
  // kEpiF32 only: up to splitk_max ranges of K run as separate work units
  // when that fills the SMs better; split 0 writes C, split s > 0 the fp32
  // slice ws + (s - 1) * M * ldc, and a fixed-order sum adds the slices into
  // C (ws: (splitk_max - 1) * M * ldc floats, or null for no split)
  int splitk_max = 1;
  float* ws = nullptr;
  LogprobEpi lp;  // kEpiLogprob, kEpiLogprobBwd
  // when set, the number of kernels the call launched is added to it
  int* launched = nullptr;
};

// Returns 0, or a negative status with a message in `why` (64 chars at least).
int gemm(const GemmArgs& a, int* dev_err, cudaStream_t st, char* why);
// Columns of a product's tiles.
constexpr int gemm_tile_cols(int64_t N) { return N > 128 ? 256 : 128; }
// The K ranges that a kEpiF32 product with splitk_max = max_split takes.
int gemm_splitk(int64_t M, int64_t N, int64_t K, int max_split);
// Host-side argument check only (no CUDA call): 0 or -1.
int gemm_check(const GemmArgs& a, char* why);

// ---- elementwise / normalisation kernels (elementwise.cu)
void rmsnorm_fwd(const float* x, const __nv_bfloat16* g, __nv_bfloat16* y, float* rstd,
                 int64_t rows, int d, float eps, cudaStream_t st);
// dx = dres + rstd*(g*dy - xhat*mean(g*dy*xhat)); dxb = bf16(dx); dg partials [parts, d]
void rmsnorm_bwd(const float* x, const __nv_bfloat16* g, const float* rstd, const float* dy,
                 const float* dres, float* dx, __nv_bfloat16* dxb, float* dg_part, int parts,
                 int64_t rows, int d, cudaStream_t st);
int rmsnorm_bwd_parts(int64_t rows, int d);
void reduce_parts_bf16(const float* part, int parts, int d, __nv_bfloat16* out, cudaStream_t st);
// The same sum as fp16 after multiplying by scale (a scaled fp16 gradient).
void reduce_parts_f16(const float* part, int parts, int d, uint16_t* out, float scale,
                      cudaStream_t st);
// out1 = bf16 sums of the first n1 columns of part [parts, n1 + n2], out2 of the
// others, in a fixed order.  Call it right after the launch that writes part.
void gain_sums(const float* part, int parts, int n1, __nv_bfloat16* out1, int n2,
               __nv_bfloat16* out2, cudaStream_t st);
// out[c] = bf16(sum over rows of x[r, c]) for x bf16 [rows, cols] (cols even, row
// stride ld, 4-byte aligned rows); part: fp32 scratch [parts, cols]
void bias_grad(const __nv_bfloat16* x, int64_t ld, int64_t rows, int cols, float* part, int parts,
               __nv_bfloat16* out, cudaStream_t st);
// the column sums as fp16 times scale
void bias_grad_f16(const __nv_bfloat16* x, int64_t ld, int64_t rows, int cols, float* part,
                   int parts, uint16_t* out, float scale, cudaStream_t st);
void rope_inplace(__nv_bfloat16* qkv, int64_t ld, int64_t tokens, int seq, int heads,
                  int head_dim, const float2* cs, int inverse, cudaStream_t st);
// The fused cross-entropy rows on fp32 logits z [rows, vocab] (vocab % 8 == 0,
// z 16-byte aligned): loss_rows[r] = lse - z[r, label] (0 when ignored) and
// dz [rows, vocab] bf16 = (softmax(z) - onehot) * inv_n (0 on ignored rows).
// A cluster of CTAs shares a row held in shared memory, so z is read once;
// a wait that runs out writes kDevCeTimeout to *err, and a label >= vocab
// writes kDevCeBadLabel (its row is then ignored).  Returns 0, or -1 when the
// launch fails.
int ce_rows_f32(const float* z, __nv_bfloat16* dz, const int32_t* labels, int64_t rows,
                int64_t vocab, float inv_n, float* loss_rows, int* err, cudaStream_t st);
// CTAs per row of the cross-entropy kernel for this vocabulary (0: one CTA
// reading the row twice, for rows beyond the clusters' shared memory).
int ce_cluster_size(int64_t vocab);
void swiglu_fwd(const __nv_bfloat16* ab, __nv_bfloat16* m, int64_t rows, int ffn,
                cudaStream_t st);
void swiglu_bwd(const __nv_bfloat16* dm, const __nv_bfloat16* ab, __nv_bfloat16* dab,
                int64_t rows, int ffn, cudaStream_t st);
void sum_f32(const float* x, int64_t n, float scale, float* out, cudaStream_t st);
void cast_f32_bf16(const float* x, __nv_bfloat16* y, int64_t n, cudaStream_t st);
// y = fp16(scale * x)
void cast_f32_f16(const float* x, uint16_t* y, int64_t n, float scale, cudaStream_t st);
void cast_bf16_f32(const __nv_bfloat16* x, float* y, int64_t n, cudaStream_t st);

// ---- attention (attention.cu).  qkv [T, (Hq+2Hkv)*hd] bf16, token t = b*S + s.
// Forward on tcgen05 (attention_tc.cu); a bounded wait that runs out writes
// kDevAttnTimeout to *err.
int attn_fwd(const __nv_bfloat16* qkv, __nv_bfloat16* o, float* lse, int B, int S, int Hq,
             int Hkv, int hd, int* err, cudaStream_t st);
// Backward on tcgen05 (attention_tc.cu).  delta: fp32 scratch [B, Hq, S].
// dq_acc: fp32 scratch, [T, Hq*hd] (zeroed inside, partials added in the
// order they arrive) or, when deterministic, [ceil(S/128)][T, Hq*hd] (one slot
// per 128-key block, summed in key order: bit-reproducible).  Writes dQ and dK
// (inverse RoPE applied when cs != null) and dV into dqkv.
int attn_bwd(const __nv_bfloat16* qkv, const __nv_bfloat16* o, const __nv_bfloat16* dout,
             const float* lse, float* delta, float* dq_acc, __nv_bfloat16* dqkv, int B, int S,
             int Hq, int Hkv, int hd, const float2* cs, bool deterministic, int* err,
             cudaStream_t st);
// delta[b, h, s] = sum_j dO * O over one head's row (attention.cu); zeroes
// zero [B*S, Hq*hd] unless it is null
void attn_delta(const __nv_bfloat16* o, const __nv_bfloat16* dout, float* delta, float* zero, int B,
                int S, int Hq, int hd, cudaStream_t st);
// dQ = scale * (accumulated or slot-summed dq_acc), inverse RoPE, into the
// query columns of dqkv (attention.cu); slots = 0 for one accumulated buffer.
// Launched as the dependent of the backward kernel before it.
void attn_dq_finalize(const float* dq_acc, __nv_bfloat16* dqkv, int B, int S, int Hq, int Hkv,
                      int hd, float scale, const float2* cs, int slots, int window, int sinks,
                      cudaStream_t st);
// The same attention with a sliding window and sinks: query q sees key k when
// k <= q and (q - k < window or k < sinks).  window >= 1, sinks >= 0; both are
// clipped to S.  dq_acc when deterministic: attn_window_dq_slots slots.
int attn_window_fwd(const __nv_bfloat16* qkv, __nv_bfloat16* o, float* lse, int B, int S, int Hq,
                    int Hkv, int hd, int window, int sinks, int* err, cudaStream_t st);
int attn_window_bwd(const __nv_bfloat16* qkv, const __nv_bfloat16* o, const __nv_bfloat16* dout,
                    const float* lse, float* delta, float* dq_acc, __nv_bfloat16* dqkv, int B,
                    int S, int Hq, int Hkv, int hd, int window, int sinks, const float2* cs,
                    bool deterministic, int* err, cudaStream_t st);
// Key blocks of 128 that the windows of a query block (128 queries,
// aligned) can reach: its own and those of the window - 1 keys before it.
__host__ __device__ constexpr int attn_window_slots(int window) { return (window + 126) / 128 + 1; }
// dQ slots of the deterministic backward: one for each of the sinks' key
// blocks, and attn_window_slots that the other key blocks take in turn.
__host__ __device__ constexpr int attn_window_dq_slots(int S, int window, int sinks) {
  const int w = window < S ? window : S, k = sinks < S ? sinks : S;
  const int ns = (k + 127) / 128, rest = (S + 127) / 128 - ns, turn = attn_window_slots(w);
  return ns + (rest < turn ? rest : turn);
}
// Items that the queries behind the window of a sinks' key block are split
// into in the backward: each about as many query blocks as another key block
// has, none empty, at most 32 in all; 0 (one item with the rest)
// where there are fewer such queries than another block has, or more than 32
// blocks of sinks, which make enough items anyway.
constexpr int attn_window_splits(int S, int window, int sinks) {
  const int w = window < S ? window : S, k = sinks < S ? sinks : S;
  const int ns = (k + 127) / 128, nq = (S + 127) / 128;
  if (ns == 0 || ns > 32) return 0;
  const int near = (126 + w) / 128 + 1;                         // query blocks of key block 0's window
  const int usual = near > 4 ? near : 4;                        // of an item
  const int far = nq - near;                                    // behind it
  const int least = nq - ((ns - 1) * 128 + 126 + w) / 128 - 1;  // the last sinks' block's
  if (far < usual || least < 1) return 0;
  int f = (far + usual - 1) / usual;
  f = f < 32 / ns ? f : 32 / ns;
  return f < least ? f : least;
}
// Floats of the sinks' partial dK and dV (fp32 [B, Hkv, sinks' blocks, splits +
// 1, dK and dV, 128, hd]).
constexpr int64_t attn_window_part_floats(int B, int S, int Hkv, int hd, int window, int sinks) {
  const int f = attn_window_splits(S, window, sinks), k = sinks < S ? sinks : S;
  return f ? (int64_t)B * Hkv * ((k + 127) / 128) * (f + 1) * 256 * hd : 0;
}
// dK and dV of the sinks' key blocks from those parts, in a fixed order
// (attention.cu).  Launched as the dependent of the backward kernel.
void attn_sink_join(const float* part, __nv_bfloat16* dqkv, int B, int S, int Hq, int Hkv, int hd,
                    float scale, const float2* cs, int splits, int sinks, cudaStream_t st);

// ---- norms of queries and keys with the rotation (qknorm.cu)
// Rows of Hq query, Hkv key and Hkv value heads of hd columns (hd % 16 == 0,
// 16 to 256; row strides multiples of 8).  The position of token t is pos[t],
// or t % seq when pos is null; cs [seq, hd/2].
struct QkNormArgs {
  int64_t tokens = 0;
  int seq = 0, Hq = 0, Hkv = 0, hd = 0;
  const __nv_bfloat16 *gq = nullptr, *gk = nullptr;
  float eps = 0.f;
  const float2* cs = nullptr;
  const int32_t* pos = nullptr;
};
// y = rotated norms of x's query and key heads; value heads copied unless y == x.
void qknorm_rope_fwd(const QkNormArgs& a, const __nv_bfloat16* x, int64_t ldx, __nv_bfloat16* y,
                     int64_t ldy, int* err, cudaStream_t st);
// dx (may be dy) from dy and the raw x; the gains' gradients from fp32
// partials in part [qknorm_parts, 2 * hd], summed in a fixed order.
void qknorm_rope_bwd(const QkNormArgs& a, const __nv_bfloat16* x, int64_t ldx,
                     const __nv_bfloat16* dy, int64_t lddy, __nv_bfloat16* dx, int64_t lddx,
                     float* part, __nv_bfloat16* dgq, __nv_bfloat16* dgk, int* err,
                     cudaStream_t st);
int qknorm_parts(int64_t tokens, int Hq, int hd);

// ---- 8-bit checkpoints (ckpt8.cu): codes [rows, d], fp32 scales
// [rows, ceil(d / 128)], one for each block of 128 columns (sf.h has the rule).
void ckpt8_save(const float* x, uint8_t* q, float* scale, int fmt, int64_t rows, int d,
                cudaStream_t st);
void ckpt8_load(const uint8_t* q, const float* scale, float* x, int fmt, int64_t rows, int d,
                cudaStream_t st);
// rmsnorm_fwd that also saves x.
void rmsnorm_fwd_save8(const float* x, const __nv_bfloat16* g, __nv_bfloat16* y, float* rstd,
                       uint8_t* q, float* scale, int fmt, int64_t rows, int d, float eps,
                       cudaStream_t st);
// rmsnorm_fwd of the saved values; xout (null: none) gets them too.
void rmsnorm_fwd_load8(const uint8_t* q, const float* scale, const __nv_bfloat16* g,
                       __nv_bfloat16* y, float* rstd, float* xout, int fmt, int64_t rows, int d,
                       float eps, cudaStream_t st);
// rmsnorm_bwd at the saved values; dg_part [parts, d] with parts =
// rmsnorm_bwd_load8_parts (at most rmsnorm_bwd_parts).  False: no launch.
int rmsnorm_bwd_load8_parts(int64_t rows, int d);
bool rmsnorm_bwd_load8(const uint8_t* q, const float* scale, const __nv_bfloat16* g,
                       const float* rstd, const float* dy, const float* dres, float* dx,
                       __nv_bfloat16* dxb, float* dg_part, int parts, int fmt, int64_t rows, int d,
                       cudaStream_t st);

// ---- dropout and the join with the residual stream (join.cu)
// Which elements dropout keeps (sf.h has the rule): top = 2^16 T (0: all of
// them), scale = 2^16 / (2^16 - T), and the generator's key and counter.
struct DropArgs {
  uint32_t top = 0;
  float scale = 1.f;
  uint64_t seed = 0, offset = 0;
  const uint64_t* step = nullptr;
};
void dropout(const void* x, void* y, bool f32, int64_t n, const DropArgs& a, cudaStream_t st);

// Rows of d columns (d % 8 == 0, 8 to 16384); g_post, gate and g_next may be null.
struct JoinArgs {
  int64_t rows = 0;
  int d = 0;
  const __nv_bfloat16 *g_post = nullptr, *gate = nullptr, *g_next = nullptr;
  float alpha = 1.f, beta = 1.f;
  DropArgs drop;
};
void join_fwd(const JoinArgs& a, const float* x, const void* h, bool h32, float* xout,
              __nv_bfloat16* y, float* rstd_post, float* rstd_next, float eps, cudaStream_t st);
// part: fp32 [join_bwd_parts, 2, d].  A wait that runs out writes kDevJoinTimeout to
// *err.  False: no launch.
int join_bwd_parts(int64_t rows, int d);
bool join_bwd(const JoinArgs& a, const float* xout, const void* h, bool h32,
              const float* rstd_post, const float* rstd_next, const float* dy, const float* dres,
              float* dx, void* dh, __nv_bfloat16* dg_post, __nv_bfloat16* dgate,
              __nv_bfloat16* dg_next, float* part, int* err, cudaStream_t st);

// ---- log probabilities of given tokens (logprob.cu); z fp32 or bf16, row
// stride ld (a multiple of 8), 16-byte aligned.  entropy may be null; top <= 32
// alternatives; a token at or beyond the vocabulary writes kDevCeBadLabel to
// *err.  False: no launch.
bool logprob_rows(const void* z, bool f32, int64_t ld, const int32_t* tokens, int64_t rows,
                  int vocab, float scale, float* logp, float* lse, float* entropy, int top,
                  int32_t* ids, float* top_logp, int* err, cudaStream_t st);
// dz may be z where z is bf16.
void logprob_rows_bwd(const void* z, bool f32, int64_t ld, const LogprobEpi& a, int64_t rows,
                      int vocab, __nv_bfloat16* dz, int64_t lddz, int* err, cudaStream_t st);
// logp, lse and entropy (may be null) from the sums that a kEpiLogprob product
// left for `tiles` tiles.  Call it right after that launch.  False: no launch.
bool logprob_tiles(const LogprobEpi& a, int64_t rows, int tiles, int vocab, float* logp,
                   float* lse, float* entropy, int* err, cudaStream_t st);

// y[i] = bf16(x[i] + x[n + i]), n a multiple of 8.
void add_halves_bf16(const float* x, __nv_bfloat16* y, int64_t n, cudaStream_t st);

int num_sms();

}  // namespace sf
