/*
 * kimodo_kernels.h -- kernel-level entry points of libkimodo.so.
 *
 * Each call runs exactly one of the kernels that kimodo.h's entry points chain
 * together, so that each can be checked on its own against a reference of the
 * same operation.  All tensor pointers are DEVICE pointers of the current CUDA
 * device, row-major; calls are asynchronous on `stream` (a cudaStream_t, NULL =
 * legacy default stream).  Return value and error message as in kimodo.h
 * (KIMODO_OK or KIMODO_E*, kimodo_last_error()).  The caller owns all memory.
 */
#ifndef KIMODO_KERNELS_H
#define KIMODO_KERNELS_H

#include "kimodo.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Epilogues of the projections ("Kimodo WebGPU", "WGSL compute shaders" table:
 * linear + bias, GELU, SiLU, residual add). */
enum {
  KIMODO_EPI_BIAS = 0,      /* out = A W^T + b                      */
  KIMODO_EPI_BIAS_GELU = 1, /* out = gelu_erf(A W^T + b)            */
  KIMODO_EPI_BIAS_SILU = 2, /* out = silu(A W^T + b)                */
  KIMODO_EPI_BIAS_RESID = 3 /* out = A W^T + b + resid (fp32 out)   */
};

/*
 * Tensor-core (tcgen05) GEMM, bf16 operands, fp32 accumulation:
 *   out[M, N] = epilogue(A[M, K] W[N, K]^T + bias[N]).
 * A: bf16, row stride lda elements; W: bf16, row stride ldw; both 16-byte
 * aligned with lda, ldw multiples of 8 and >= K.  bias: fp32 [N].
 * resid: fp32 [M, ldr] (KIMODO_EPI_BIAS_RESID only, else NULL); may equal out.
 * out: bf16 (out_f32 = 0) or fp32 (out_f32 = 1), row stride ldo.
 * out, resid, bias 16-byte aligned; ldo, ldr multiples of 4.
 * KIMODO_EPI_BIAS_RESID requires out_f32 = 1.  tile_n: 32, 64, 128 or 256
 * (output columns per tile; 32 and 64 are built for the bias and GELU epilogues
 * with bf16 output and the residual epilogue), or 0 to let the library choose.
 */
KIMODO_API int kimodo_gemm_bf16(const void* A, int lda, const void* W, int ldw, const float* bias,
                                const void* resid, int ldr, void* out, int ldo, int M, int N, int K,
                                int epilogue, int out_f32, int tile_n, void* stream);

/*
 * The same product on pairs of SMs (one 256-row output tile per CTA pair,
 * tcgen05 cta_group::2), the kernel the denoiser uses for its large projections.
 * Arguments as kimodo_gemm_bf16; epilogues KIMODO_EPI_BIAS and KIMODO_EPI_BIAS_GELU
 * with bf16 output and KIMODO_EPI_BIAS_RESID with fp32 output; N % 16 == 0 and output
 * rows a multiple of 16 bytes.  tile_n: output
 * columns per pair tile, 144, 160, 208 or 256 (144 or 160 with the residual
 * epilogue), or 0 for the library's choice.
 */
KIMODO_API int kimodo_gemm_bf16_pair(const void* A, int lda, const void* W, int ldw, const float* bias,
                                     const void* resid, int ldr, void* out, int ldo, int M, int N, int K,
                                     int epilogue, int out_f32, int tile_n, void* stream);

/* fp32 SIMT GEMM with the same epilogues; all operands fp32; K % 16 == 0,
 * lda, ldw multiples of 4. */
KIMODO_API int kimodo_gemm_f32(const float* A, int lda, const float* W, int ldw, const float* bias,
                               const float* resid, int ldr, float* out, int ldo, int M, int N, int K,
                               int epilogue, void* stream);

/*
 * Masked multi-head self-attention ("Kimodo WebGPU", "WGSL compute shaders":
 * multi-head self-attention with optional key masking), 8 heads x 128.
 * qkv: [nseq * S, 3072] with columns Q | K | V (head h at h * 128 inside each).
 * Sequence s attends to keys 0 .. lengths[s] (the condition token plus
 * lengths[s] frames; clamped to [1, S] keys).  out: [nseq * S, 1024].
 * 1 <= S <= 301.
 * bf16 variant: bf16 qkv/out (qkv 16-byte aligned), on the tcgen05 tensor cores:
 *   one CTA per (head, sequence, 128-query tile), S = Q K^T and O = P V in TMEM,
 *   exact fp32 softmax over all keys of a sequence.
 * f32 variant: fp32 throughout (SIMT, one warp per query).
 */
KIMODO_API int kimodo_attention_bf16(const void* qkv, void* out, const int* lengths, int nseq, int S,
                                     void* stream);
KIMODO_API int kimodo_attention_f32(const float* qkv, float* out, const int* lengths, int nseq, int S,
                                    void* stream);

/* LayerNorm over 1024 features, eps 1e-5, biased variance: y fp32 [M, 1024] ->
 * out bf16 (out_bf16 = 1) or fp32 [M, 1024]; gamma, beta fp32 [1024]. */
KIMODO_API int kimodo_layernorm(const float* y, void* out, int out_bf16, const float* gamma,
                                const float* beta, int M, void* stream);

/*
 * globalRootToLocalRoot and the body network's input ("Kimodo WebGPU",
 * "Architecture" figure: root model -> globalRootToLocalRoot -> body model), the
 * fp32 form of the kernel the two-stage step runs between its two networks.
 * root: [batch, frames, 5] global root (x, z, sin heading, cos heading, height), the
 *   root network's output for one guidance branch.  x: [batch, frames, 279] state x_t.
 * body_in (output): [batch, frames, 279] = [x[..., 5:279] | local root 5], local root =
 *   (v'x, v'z, sin d, cos d, height): the displacement from the previous frame turned
 *   into the current heading's frame, the heading change, the height; headings are
 *   normalised, and the frame before the first sits at the origin with heading 0.
 *   Frames at index >= lengths[b] get local root 0 (their body columns are copied).
 * lengths: int32 [batch], 1..frames.  1 <= batch, 1 <= frames <= 300.
 */
KIMODO_API int kimodo_global_to_local_root(const float* root, const float* x, const int* lengths, int batch,
                                           int frames, float* body_in, void* stream);

/* ------------------------------------------------------------------ 8-bit projections
 *
 * A projection in 8-bit integers: its input rows are quantised with one scale each
 * (kimodo_rms_norm_int8 or kimodo_quantize_int8), its weight matrix once with one scale per
 * output channel (kimodo_quantize_int8 on its rows), and kimodo_gemm_int8 multiplies them.
 * No counterpart is on the pages; the calls stand beside kimodo_layernorm and
 * kimodo_gemm_bf16.  Every tensor must be memory of the current device (else
 * KIMODO_EINVAL).  All calls may be captured into a CUDA graph; make one call of a kind
 * before the capture, so that its kernels are loaded.
 */

/*
 * Rows in 8-bit integers: scale[r] = max_c |x[r, c]| / 127, q[r, c] = rint(127 x[r, c] /
 * max_c |x[r, c]|) (ties to even), so x is about q * scale.  A row of zeros has q = 0,
 * scale = 0; a row with a NaN or an infinity has q = 0 and scale NaN.
 * x: fp32 (x_bf16 = 0) or bf16 (1) [rows, cols], row stride ldx elements.  q: int8, row
 * stride ldq.  scale: fp32 [rows].  1 <= rows, 1 <= cols <= 32768.  Rows on 16-byte
 * boundaries (8 for q) with cols a multiple of 8 take the faster path; none is required.
 * q must not overlap x.
 */
KIMODO_API int kimodo_quantize_int8(const void* x, long long ldx, int x_bf16, void* q, long long ldq,
                                    float* scale, int rows, int cols, void* stream);

/*
 * RMS norm with the residual's addition, its output in 8-bit integers:
 *   h = x + resid (fp32; resid NULL: h = x), resid_out = h in the residual's type,
 *   t = h gamma / sqrt(mean_c h^2 + eps), q and scale as kimodo_quantize_int8 of t.
 * t is taken from the fp32 sum, not from the rounded resid_out.  A row in which an h or an
 * h gamma leaves fp32's range has q = 0 and scale NaN.
 * x as above; resid, resid_out: fp32 (resid_bf16 = 0) or bf16 (1), strides ldr, ldro; both
 * or neither; resid_out may equal resid (in place, same stride) but not overlap it or x
 * otherwise; q overlaps none of them.  gamma: fp32 [cols].  eps: finite, >= 0.
 */
KIMODO_API int kimodo_rms_norm_int8(const void* x, long long ldx, int x_bf16, const void* resid, long long ldr,
                                    void* resid_out, long long ldro, int resid_bf16, const float* gamma, float eps,
                                    void* q, long long ldq, float* scale, int rows, int cols, void* stream);

/*
 * Product in 8-bit integers on the tcgen05 tensor cores:
 *   out[m, n] = epilogue(a_scale[m] w_scale[n] sum_k A[m, k] W[n, k] + bias[n]).
 * The sum is exact (32-bit integers): results do not depend on how the work is split.
 * A: int8 [M, K], row stride lda; W: int8 [N, K], row stride ldw; both 16-byte aligned with
 * lda, ldw multiples of 16 (columns past K are not read into the sum).  1 <= K <=
 * KIMODO_INT8_MAX_K, the largest K whose sum cannot leave 32 bits; M, N <= KIMODO_INT8_MAX_ROWS.
 * a_scale: fp32 [M]; w_scale: fp32 [N]; bias: fp32 [N] or NULL.
 * epilogue: KIMODO_EPI_*; resid fp32 [M, ldr] with KIMODO_EPI_BIAS_RESID (may equal out),
 * ignored otherwise.  out: bf16 (out_f32 = 0) or fp32 (1), row stride ldo, no alignment
 * beyond its elements; GELU and SiLU write bf16, the residual epilogue fp32.  out must not
 * overlap A or W, nor resid unless it equals it (in place, same stride).
 */
#define KIMODO_INT8_MAX_K 131071
#define KIMODO_INT8_MAX_ROWS 2147483135 /* 2^31 - 513 */
KIMODO_API int kimodo_gemm_int8(const void* A, long long lda, const float* a_scale, const void* W, long long ldw,
                                const float* w_scale, const float* bias, const float* resid, long long ldr,
                                void* out, long long ldo, int M, int N, int K, int epilogue, int out_f32,
                                void* stream);

/* ------------------------------------------------------------------ attention with scored masks
 *
 * kimodo_attention_* with other head layouts, lengths, score forms and masks.  Query i of
 * sequence b has position p_i = q_start[b] + i; for query head h and key j:
 *   x_ij = scale q_i . k_j
 *   x_ij = cap tanh(x_ij / cap)          if cap > 0 (any finite cap of at least |scale| / 1e6)
 *   x_ij = x_ij - slopes[h] |p_i - j|    if slopes
 * Key j is seen if j < kv_lengths[b], and, with causal, j <= p_i or j < prefix[b], and, with
 * documents, q_documents[b, i] == kv_documents[b, j] >= 0 (a negative number: in no
 * document).  o_i = sum_j softmax_j(x_ij) v_j over the keys seen, 0 if there are none.
 * NaN and infinities in keys and values that a query does not see never reach its output.  Behind the
 * last key that any query of the call sees they cost nothing; among the keys of other queries
 * or documents they cost time (such rows are computed again, key by key).
 *
 * q, out: [batch, q_len, q_heads, head_dim]; k, v: [batch, kv_len, kv_heads, head_dim]; head
 *   h reads key head h / (q_heads / kv_heads).  head_dim 64 or 128, its elements
 *   consecutive.  Strides (elements) of batch, token and head: multiples of 16 bytes, at
 *   least head_dim; that of an extent of one is ignored.  Bases 16-byte aligned.  out must
 *   not overlap the inputs.
 * dtype: KIMODO_BF16 (tcgen05 tensor cores; fp32 scores, softmax and sums, weights rounded to
 *   bf16) or KIMODO_FP32 (fp32 throughout; above 16 rows per key head, q_len x q_heads /
 *   kv_heads, products run on the tensor cores with every operand in three bf16 parts, 24
 *   bits as fp32 has, and are summed in fp32).
 * slopes: fp32 [q_heads].  prefix (with causal), kv_lengths, q_start: int32 [batch];
 *   q_documents int32 [batch, q_len], kv_documents int32 [batch, kv_len] (both or
 *   neither).  NULL switches an option off; kv_lengths NULL: kv_len (lengths are clamped to
 *   [0, kv_len]); q_start NULL: kv_len - q_len (the queries are the last tokens).
 *   A row's distances are counted from the nearest position that its length and causal masks let
 *   it see (the softmax cancels the constant), so a query far from all its keys, on either
 *   side, keeps their differences.  A bias is right to |slope| d 2^-20, d that distance: with
 *   documents, to the distance at which the row's own document lies.
 * 1 <= batch, q_len; 0 <= kv_len; q_len, kv_len <= KIMODO_MAX_KEYS.
 * workspace: device memory of at least the bytes that kimodo_attention_scored_workspace
 *   gives for the same arguments (0 for many), 16-byte aligned, the caller's until the call's
 *   work is done; calls that may overlap (streams, captured graphs) need their own.
 */
#define KIMODO_MAX_KEYS 16777216
typedef struct kimodo_scored_attention {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  const float* slopes;
  const int* prefix;
  const int* q_documents;
  const int* kv_documents;
  const int* kv_lengths;
  const int* q_start;
  long long q_strides[3]; /* batch, token, head */
  long long k_strides[3];
  long long v_strides[3];
  long long out_strides[3];
  int batch, q_len, kv_len, q_heads, kv_heads, head_dim;
  int dtype;
  int causal;
  float scale;
  float cap;
} kimodo_scored_attention;
KIMODO_API int kimodo_attention_scored_workspace(const kimodo_scored_attention* args, size_t* bytes);
KIMODO_API int kimodo_attention_scored(const kimodo_scored_attention* args, void* workspace, size_t workspace_bytes,
                                       void* stream);

/* Synchronise `stream` and report (and clear) a bounded wait that ran out in a kernel-level
 * call on the current device since the last check (KIMODO_ETIMEOUT). */
KIMODO_API int kimodo_kernel_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KIMODO_KERNELS_H */
