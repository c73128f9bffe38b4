// Internal launchers of the denoiser kernels (not part of the public C ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include "common.cuh"
#include "epilogue.cuh"

namespace kd {

// D[M, N] = A[M, K] . B[N, K]^T; A, B row-major with leading dimensions lda, ldb.
struct GemmArgs {
  const void* A = nullptr;
  const void* B = nullptr;
  int M = 0, N = 0, K = 0;
  int lda = 0, ldb = 0;
};

// tcgen05 bf16 GEMM.  bn in {16, 32, 64, 128, 256}; returns cudaErrorInvalidValue for an
// unsupported (bn, kind, output type) combination.
cudaError_t gemm_tc(const GemmArgs& g, int bn, int kind, bool out_f32, const EpiParams& ep, DevError* err,
                    cudaStream_t st, int num_sms);
bool gemm_tc_available();

// TMA descriptor of a row-major bf16 matrix [rows, ld] whose first `cols` columns are
// the K extent; boxes of 64 columns x box_rows rows, 128-byte swizzle, zero fill.
int make_tmap_bf16(CUtensorMap* m, const void* base, int rows, int cols, int ld, int box_rows);
// Row-major fp32 (elem 4) or bf16 (elem 2) matrix, boxes box_cols x box_rows,
// shared-memory swizzle 0, 32, 64 or 128 bytes (= the box row's bytes when nonzero).
int make_tmap_plain(CUtensorMap* m, const void* base, int elem, int rows, int cols, long ld, int box_cols,
                    int box_rows, int swizzle);

// tcgen05 GEMM on CTA pairs (256-row tiles).  bn in {144, 160, 208, 256} for EPI_BIAS /
// EPI_BIAS_GELU with bf16 output, {144, 160} for EPI_BIAS_RESID / EPI_BIAS_RESID_LN with
// fp32 output.
cudaError_t gemm_tc2(const GemmArgs& g, int bn, int kind, bool out_f32, const EpiParams& ep, DevError* err,
                     cudaStream_t st);
cudaError_t gemm_tc2_prepare();
bool gemm_tc2_supports(int kind, bool out_f32);
int gemm_tc2_pick_bn(int M, int N, int kind);
// Set the dynamic shared-memory limits of every kernel instantiation (call once
// per device before any launch or graph capture).
cudaError_t gemm_tc_prepare();

// fp32 SIMT GEMM with the same epilogues (fp32 everywhere).  K % 16 == 0.
cudaError_t gemm_f32(const GemmArgs& g, int kind, const EpiParams& ep, cudaStream_t st);

// Masked multi-head self-attention over the fused QKV matrix (columns Q | K | V,
// head h at h*DH), fp32 path.  Padded layout (tok0 null): sequence s owns rows
// s*S .. s*S + S - 1 and keys at token index >= 1 + lengths[s % len_mod] are excluded.
// Packed layout: sequence s owns rows tok0[s] .. tok0[s + 1] - 1 (its valid tokens
// only; S is then the largest sequence).  out has the rows of qkv, D columns.
cudaError_t attention_f32(const float* qkv, float* out, const int* lengths, int len_mod, int nseq, int S,
                          cudaStream_t st, const int* tok0 = nullptr);

// The same attention on the tcgen05 tensor cores (bf16 path): one CTA per (head, sequence,
// 128-query tile), exact softmax over all keys of the sequence at once.  qkv has M
// rows (16-byte aligned, row stride 3*D); S <= MAX_FRAMES + 1.  pf: weights its CTAs pull
// into L2 for the projections that follow.
cudaError_t attention_tc(const bf16* qkv, bf16* out, int M, const int* lengths, int len_mod, int nseq, int S,
                         DevError* err, cudaStream_t st, const int* tok0 = nullptr, L2Prefetch pf = {});
cudaError_t attention_tc_prepare();
size_t attention_tc_smem(int S);

// Token layout of a batch: tok0[s] = sum over s' < s of (1 + lengths[s' % len_mod]) for
// s <= nseq, and row_seq[r] = s for the rows r of sequence s (one CTA).
cudaError_t build_token_map(const int* lengths, int len_mod, int nseq, int* tok0, int* row_seq, cudaStream_t st);

// Row LayerNorm over D features: y fp32 [M, D] -> out (bf16 or fp32) [M, D], and
// optionally the row statistics (mean, 1/std) into stats [M][2]; pf: weights its CTAs pull
// into L2 for the projections that follow.
cudaError_t layernorm(const float* y, void* out, bool out_bf16, const float* gamma, const float* beta, int M,
                      cudaStream_t st, float* stats = nullptr, L2Prefetch pf = {});

// ---- motion / sampler kernels (element type of the activation matrices: bf16 or fp32)

// A[(row(seq, i)) * lda + col0 + f] = src[((seq % nsrc) * T + i) * ld_src + f0 + f], f < nf, with
// row(seq, i) = seq*S + 1 + i for every i < T (padded layout, tok0 null) or tok0[seq] + 1 + i
// for the valid frames i < lengths[seq % len_mod] only (packed layout).
cudaError_t pack_frames(const float* src, int nsrc, int ld_src, int f0, int nf, void* A, bool a_bf16, int lda,
                        int col0, int nseq, int T, int S, cudaStream_t st, const int* tok0 = nullptr,
                        const int* lengths = nullptr, int len_mod = 1);

// Body-network input of the two-stage step: for seq in [0, nseq), frame i < T (padded
// layout) or i < lengths[seq % B] (packed layout, rows as pack_frames):
//   A[.., 0:274] = x[seq % B, i, 5:279];  A[.., 274:279] = G2L(root_hat[seq])[i]  (0 for padded frames)
cudaError_t g2l_body_input(const float* root_hat, const float* x, const int* lengths, int B, int nseq, int T,
                           int S, void* A, bool a_bf16, int lda, cudaStream_t st, const int* tok0 = nullptr);

// CFG + DDIM update in place on x [B, T, 279]: x0 = u + w (c - u) from the root /
// body predictions of sequences b (cond) and B + b (uncond); x = c0 x0 + c1 x
// (+ c2 z when z [B, T, 279] is given); padded frames 0.  If A_next != nullptr the
// new root features are also packed into the root network's input matrix for
// sequences b and B + b.
cudaError_t cfg_ddim(const float* root_hat, const float* body_hat, float* x, const int* lengths, int B, int T,
                     float w, float c0, float c1, const float* z, float c2, void* A_next, bool a_bf16, int lda, int S,
                     cudaStream_t st, const int* tok0 = nullptr);

// Condition inputs: rows [0, B) = text_emb row r / takes (several takes of one prompt
// share its row), rows [B, B + null_rows) = null_emb row (r - B) % null_batch.
// out (bf16 or fp32) [rows, DTXT].
cudaError_t pack_embeddings(const float* text_emb, int B, const float* null_emb, int null_batch, int null_rows,
                            void* out, bool out_bf16, cudaStream_t st, int takes = 1);

// out[k, :] = pe[t_k, :] for k < n (sinusoid rows of the timesteps): t_k = t_single
// when steps == 0, else the k-th trailing timestep of a `steps`-step sampler,
// floor(N_TRAIN (steps - k) / steps + 1/2) - 1.
cudaError_t gather_timestep_rows(const float* pe, int t_single, int steps, int n, void* out, bool out_bf16,
                                 cudaStream_t st);

// ---- 8-bit projections and attention with scored masks (kernel-level entry points)

// Rows in 8-bit integers: q = rint(127 t / max |t|), scale = max |t| / 127, with t = x or
// (rms_norm_rows_int8) t = h gamma / sqrt(mean h^2 + eps), h = x + r_in (null: h = x), whose
// fp32 sum is stored in r_out (may equal r_in) rounded to the residual's type.  x and the
// residual are fp32 or bf16; leading dimensions in elements; 1 <= cols <= 32768.
struct RowsInt8 {
  const void* x = nullptr;
  long ldx = 0;
  const void* r_in = nullptr;
  long ldr_in = 0;
  void* r_out = nullptr;
  long ldr_out = 0;
  const float* gamma = nullptr;
  int8_t* q = nullptr;
  long ldq = 0;
  float* scale = nullptr;
  int rows = 0, cols = 0;
  float eps = 0.f;
};
constexpr int ROWS_INT8_MAX_COLS = 32768;
cudaError_t quantize_rows_int8(const RowsInt8& a, bool x_bf16, cudaStream_t st);
cudaError_t rms_norm_rows_int8(const RowsInt8& a, bool x_bf16, bool r_bf16, cudaStream_t st);

// out[m, n] = epilogue(a_scale[m] w_scale[n] sum_k A[m, k] W[n, k] + bias[n]); A, W int8 with
// 16-byte aligned rows, bias may be null; kind and output type as the bf16 GEMM.
struct GemmI8 {
  const void* A = nullptr;
  const void* W = nullptr;
  const float* a_scale = nullptr;
  const float* w_scale = nullptr;
  const float* bias = nullptr;
  const float* resid = nullptr;
  void* out = nullptr;
  int M = 0, N = 0, K = 0;
  long lda = 0, ldw = 0, ldr = 0, ldo = 0;
};
cudaError_t gemm_i8(const GemmI8& g, int kind, bool out_f32, DevError* err, cudaStream_t st, int num_sms);
int make_tmap_i8(CUtensorMap* m, const void* base, int rows, int cols, long ld, int box_rows);
int make_tmap_i8_blocks(CUtensorMap* m, const void* base, int rows, int cols, long ld, int box_rows, int blocks);
int make_tmap_heads(CUtensorMap* m, const void* base, int dims, int tokens, int heads, int batch, long s_token,
                    long s_head, long s_batch);

// Attention with scored masks (definition in attention_scored.cu).  q, out [B][Sq][Hq][HD],
// k, v [B][Sk][Hkv][HD] by strides in elements, dims consecutive; HD 64 or 128; null optional
// pointers switch their option off.
struct ScoredAttention {
  const void* q = nullptr;
  const void* k = nullptr;
  const void* v = nullptr;
  void* out = nullptr;
  const float* slopes = nullptr;     // [Hq]
  const int* prefix = nullptr;       // [B], with causal
  const int* q_doc = nullptr;        // [B][Sq], with kv_doc
  const int* kv_doc = nullptr;       // [B][Sk]
  const int* kv_lengths = nullptr;   // [B]
  const int* q_start = nullptr;      // [B]; null: Sk - Sq
  long q_batch = 0, q_token = 0, q_head = 0, k_batch = 0, k_token = 0, k_head = 0;
  long v_batch = 0, v_token = 0, v_head = 0, o_batch = 0, o_token = 0, o_head = 0;
  int B = 0, Sq = 0, Sk = 0, Hq = 0, Hkv = 0, G = 0, HD = 0;
  float scale = 0.f, cap = 0.f;
  int causal = 0;
};
// What the kernels multiply scores by, as pairs (f32x2 operands); computed on the host, so that
// it sits in constant memory and not in the softmax threads' registers.
struct ScoredConst {
  float2 lin;            // |scale| * log2 e (a scale of 0 counts as 1: its scores are made 0)
  float2 c[4];           // tanh(z) / z * lin as a polynomial in s^2, z = |scale| s / cap
  float limit2;          // s^2 up to which it holds
  float z;               // |scale| / cap
  float two, cap2;       // e^(2 z) = 2^(two s); cap * log2 e
};
// Split of a call over CTAs and keys; parts > 1: results of each part and their weights in a
// workspace of `bytes`, joined by a second kernel.
struct ScoredPlan {
  int splits = 1, tiles_per_split = 1, row_blocks = 1, parts = 1;
  int few = 0;   // rows of the kernel for few rows (0: not those)
  int tiles = 2; // row tiles of a CTA of the kernel for many rows
  ScoredConst k;
  float* part_o = nullptr;
  float* part_lse = nullptr;
  int2* doc_tiles = nullptr;   // [B][key_tiles], documents of the key tiles (null: each CTA looks at the keys)
  int key_tiles = 0;
  size_t doc_offset = 0, doc_bytes = 0;   // of doc_tiles in the workspace
  size_t bytes = 0;
};
ScoredPlan scored_attention_plan(const ScoredAttention& a, bool is_bf16, int num_sms);
cudaError_t attention_scored(const ScoredAttention& a, bool is_bf16, ScoredPlan plan, void* workspace, DevError* err,
                             cudaStream_t st);

}  // namespace kd
