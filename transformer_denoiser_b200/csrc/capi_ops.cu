// C ABI of the 8-bit projections and of attention with scored masks (declared in
// include/kimodo_kernels.h): argument checks and launches.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kimodo_kernels.h"
#include "kernels.h"
#include "status.h"

using namespace kd;

namespace {

bool misaligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// SM count of the current device, 0 on failure.
int current_sms() {
  static std::atomic<int> sms[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Every given pointer is memory of the current device (a kernel that read host memory or
// another GPU's would fault, or run over the bus).
int check_here(std::initializer_list<const void*> ptrs) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return set_error(KIMODO_EUNSUPPORTED, "no CUDA device available");
  }
  for (const void* p : ptrs) {
    if (p == nullptr) continue;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
      cudaGetLastError();
      return set_error(KIMODO_EINVAL, "a tensor pointer is not CUDA memory");
    }
    if (at.type == cudaMemoryTypeManaged) continue;
    if (at.type != cudaMemoryTypeDevice)
      return set_error(KIMODO_EINVAL, "tensors must be device memory");
    if (at.device != dev)
      return set_error(KIMODO_EINVAL, "a tensor is on device %d, the current device is %d", at.device, dev);
  }
  return KIMODO_OK;
}

int check_rows(const void* x, long long ldx, const void* q, long long ldq, const void* scale, int rows, int cols) {
  if (!x || !q || !scale) return set_error(KIMODO_EINVAL, "NULL tensor argument");
  if (rows < 1) return set_error(KIMODO_EINVAL, "rows must be >= 1 (got %d)", rows);
  if (cols < 1 || cols > ROWS_INT8_MAX_COLS)
    return set_error(KIMODO_EINVAL, "cols must be in [1, %d] (got %d)", ROWS_INT8_MAX_COLS, cols);
  if (ldx < cols || ldq < cols) return set_error(KIMODO_EINVAL, "leading dimensions must cover cols");
  return KIMODO_OK;
}

// Element type sizes of float tensors: 4 (fp32) or 2 (bf16).
int check_type(const char* what, const void* p, int bf16_flag) {
  if (bf16_flag != 0 && bf16_flag != 1) return set_error(KIMODO_EINVAL, "%s_bf16 must be 0 or 1", what);
  if (misaligned(p, bf16_flag ? 2 : 4)) return set_error(KIMODO_EINVAL, "%s is not aligned to its elements", what);
  return KIMODO_OK;
}

using Wide = __int128;   // strides in bytes, and extents times strides, can leave 64 bits

// Where a tensor lies: `width` consecutive bytes, repeated along up to three dimensions.
struct Place {
  const void* p;
  long long width;
  long long extent[3] = {1, 1, 1};
  Wide stride[3] = {0, 0, 0};   // bytes, >= 0
};
Place place_of_rows(const void* p, long long rows, long long cols, long long ld, int elem) {
  return Place{p, cols * elem, {rows, 1, 1}, {(Wide)ld * elem, 0, 0}};
}

// Whether two tensors have no byte in common.  Where their ranges meet, they may still be parts of one
// buffer (columns of the same rows, heads of the same tokens): modulo a stride of either, each
// then stays in a window, and the windows do not meet.
bool apart(const Place& a, const Place& b) {
  const Place* t[2] = {&a, &b};
  const Wide d = (Wide)reinterpret_cast<uintptr_t>(b.p) - (Wide)reinterpret_cast<uintptr_t>(a.p);
  Wide span[2];
  for (int i = 0; i < 2; ++i) {
    span[i] = t[i]->width;
    for (int e = 0; e < 3; ++e) span[i] += (Wide)(t[i]->extent[e] - 1) * t[i]->stride[e];
  }
  if (d >= span[0] || -d >= span[1]) return true;
  for (int c = 0; c < 6; ++c) {
    if (t[c / 3]->extent[c % 3] <= 1) continue;
    const Wide period = t[c / 3]->stride[c % 3];
    if (period <= 0) continue;
    Wide window[2];
    for (int i = 0; i < 2; ++i) {
      window[i] = t[i]->width;
      for (int e = 0; e < 3; ++e)
        if (t[i]->extent[e] > 1 && t[i]->stride[e] % period != 0)
          window[i] += (Wide)(t[i]->extent[e] - 1) * t[i]->stride[e];
    }
    const Wide at = ((d % period) + period) % period;
    if (at >= window[0] && at + window[1] <= period) return true;
  }
  return false;
}

// An output that meets an input: rows would be overwritten that other threads, or the same call again
// (attention's rows with non-finite results), still read.
int check_apart(const char* what, const Place& out, std::initializer_list<Place> inputs) {
  for (const Place& in : inputs)
    if (in.p != nullptr && !apart(out, in)) return set_error(KIMODO_EINVAL, "%s must not overlap the inputs", what);
  return KIMODO_OK;
}

}  // namespace

extern "C" {

int kimodo_quantize_int8(const void* x, long long ldx, int x_bf16, void* q, long long ldq, float* scale, int rows,
                         int cols, void* stream) {
  clear_error();
  KD_TRY(check_rows(x, ldx, q, ldq, scale, rows, cols));
  KD_TRY(check_type("x", x, x_bf16));
  if (misaligned(scale, 4)) return set_error(KIMODO_EINVAL, "scale is not aligned to its elements");
  KD_TRY(check_apart("q", place_of_rows(q, rows, cols, ldq, 1), {place_of_rows(x, rows, cols, ldx, x_bf16 ? 2 : 4)}));
  KD_TRY(check_here({x, q, scale}));
  RowsInt8 a;
  a.x = x; a.ldx = ldx; a.q = static_cast<int8_t*>(q); a.ldq = ldq; a.scale = scale; a.rows = rows; a.cols = cols;
  KD_CUDA(quantize_rows_int8(a, x_bf16 != 0, static_cast<cudaStream_t>(stream)));
  return KIMODO_OK;
}

int kimodo_rms_norm_int8(const void* x, long long ldx, int x_bf16, const void* resid, long long ldr,
                         void* resid_out, long long ldro, int resid_bf16, const float* gamma, float eps, void* q,
                         long long ldq, float* scale, int rows, int cols, void* stream) {
  clear_error();
  KD_TRY(check_rows(x, ldx, q, ldq, scale, rows, cols));
  KD_TRY(check_type("x", x, x_bf16));
  if (!gamma) return set_error(KIMODO_EINVAL, "NULL tensor argument");
  if (!isfinite(eps) || eps < 0.f) return set_error(KIMODO_EINVAL, "eps must be finite and >= 0");
  if ((resid == nullptr) != (resid_out == nullptr))
    return set_error(KIMODO_EINVAL, "resid and resid_out come together");
  if (resid) {
    if (ldr < cols || ldro < cols) return set_error(KIMODO_EINVAL, "leading dimensions must cover cols");
    if (resid == resid_out && ldr != ldro) return set_error(KIMODO_EINVAL, "in place, ldr and ldro must be equal");
    KD_TRY(check_type("resid", resid, resid_bf16));
    KD_TRY(check_type("resid", resid_out, resid_bf16));
  }
  if (misaligned(scale, 4) || misaligned(gamma, 4))
    return set_error(KIMODO_EINVAL, "gamma and scale must be aligned to their elements");
  const Place xs = place_of_rows(x, rows, cols, ldx, x_bf16 ? 2 : 4);
  const Place rs = place_of_rows(resid, rows, cols, ldr, resid_bf16 ? 2 : 4);
  const Place ros = place_of_rows(resid_out, rows, cols, ldro, resid_bf16 ? 2 : 4);
  if (resid) {
    KD_TRY(check_apart("resid_out", ros, {xs}));
    if (resid != resid_out) KD_TRY(check_apart("resid_out", ros, {rs}));
  }
  KD_TRY(check_apart("q", place_of_rows(q, rows, cols, ldq, 1), {xs, rs, ros}));
  KD_TRY(check_here({x, resid, resid_out, gamma, q, scale}));
  RowsInt8 a;
  a.x = x; a.ldx = ldx; a.r_in = resid; a.ldr_in = ldr; a.r_out = resid_out; a.ldr_out = ldro; a.gamma = gamma;
  a.q = static_cast<int8_t*>(q); a.ldq = ldq; a.scale = scale; a.rows = rows; a.cols = cols; a.eps = eps;
  KD_CUDA(rms_norm_rows_int8(a, x_bf16 != 0, resid_bf16 != 0, static_cast<cudaStream_t>(stream)));
  return KIMODO_OK;
}

int kimodo_gemm_int8(const void* A, long long lda, const float* a_scale, const void* W, long long ldw,
                     const float* w_scale, const float* bias, const float* resid, long long ldr, void* out,
                     long long ldo, int M, int N, int K, int epilogue, int out_f32, void* stream) {
  clear_error();
  if (!A || !a_scale || !W || !w_scale || !out) return set_error(KIMODO_EINVAL, "NULL tensor argument");
  if (M < 1 || N < 1 || K < 1) return set_error(KIMODO_EINVAL, "M, N, K must be >= 1");
  // the kernels go past the last row by up to two tiles in 32-bit integers
  if (M > KIMODO_INT8_MAX_ROWS || N > KIMODO_INT8_MAX_ROWS)
    return set_error(KIMODO_EINVAL, "M and N must be at most %d (got %d, %d)", KIMODO_INT8_MAX_ROWS, M, N);
  if (K > KIMODO_INT8_MAX_K)
    return set_error(KIMODO_EINVAL, "K must be at most %d (32-bit sums; got %d)", KIMODO_INT8_MAX_K, K);
  if (lda < K || ldw < K || ldo < N) return set_error(KIMODO_EINVAL, "leading dimensions must cover K / N");
  if (epilogue < 0 || epilogue > 3) return set_error(KIMODO_EINVAL, "unknown epilogue %d", epilogue);
  if (epilogue == KIMODO_EPI_BIAS_RESID) {
    if (!resid) return set_error(KIMODO_EINVAL, "residual epilogue needs resid");
    if (ldr < N) return set_error(KIMODO_EINVAL, "leading dimensions must cover K / N");
    if (!out_f32) return set_error(KIMODO_EINVAL, "residual epilogue writes fp32");
    if (resid == out && ldr != ldo) return set_error(KIMODO_EINVAL, "in place, ldr and ldo must be equal");
  }
  if ((epilogue == KIMODO_EPI_BIAS_GELU || epilogue == KIMODO_EPI_BIAS_SILU) && out_f32)
    return set_error(KIMODO_EINVAL, "GELU/SiLU epilogues write bf16");
  if (lda % 16 || ldw % 16 || misaligned(A, 16) || misaligned(W, 16))
    return set_error(KIMODO_EINVAL, "int8 operands need 16-byte aligned rows (lda, ldw multiples of 16)");
  if (misaligned(out, out_f32 ? 4 : 2) || misaligned(a_scale, 4) || misaligned(w_scale, 4) || misaligned(bias, 4) ||
      misaligned(resid, 4))
    return set_error(KIMODO_EINVAL, "out, resid, bias and scales must be aligned to their elements");
  const bool resid_used = epilogue == KIMODO_EPI_BIAS_RESID && resid != out;
  KD_TRY(check_apart("out", place_of_rows(out, M, N, ldo, out_f32 ? 4 : 2),
                     {place_of_rows(A, M, K, lda, 1), place_of_rows(W, N, K, ldw, 1),
                      place_of_rows(resid_used ? resid : nullptr, M, N, ldr, 4)}));
  if (!gemm_tc_available()) return set_error(KIMODO_EUNSUPPORTED, "cuTensorMapEncodeTiled is unavailable");
  KD_TRY(check_here({A, a_scale, W, w_scale, bias, epilogue == KIMODO_EPI_BIAS_RESID ? resid : nullptr, out}));
  const int sms = current_sms();
  if (sms < 1) return set_error(KIMODO_ECUDA, "the SM count could not be read");
  GemmI8 g;
  g.A = A; g.W = W; g.a_scale = a_scale; g.w_scale = w_scale; g.bias = bias; g.resid = resid; g.out = out;
  g.M = M; g.N = N; g.K = K; g.lda = lda; g.ldw = ldw; g.ldr = ldr; g.ldo = ldo;
  KD_CUDA(gemm_i8(g, epilogue, out_f32 != 0, kernel_error_word(), static_cast<cudaStream_t>(stream), sms));
  return KIMODO_OK;
}

}  // extern "C"

namespace {

// Validates a call and fills the kernel's arguments.
int scored_args(const kimodo_scored_attention* p, ScoredAttention* a) {
  if (!p) return set_error(KIMODO_EINVAL, "arguments are NULL");
  if (!p->q || !p->out || (p->kv_len > 0 && (!p->k || !p->v))) return set_error(KIMODO_EINVAL, "NULL tensor argument");
  if (p->batch < 1 || p->q_len < 1 || p->kv_len < 0)
    return set_error(KIMODO_EINVAL, "need batch >= 1, q_len >= 1, kv_len >= 0");
  if (p->q_heads < 1 || p->kv_heads < 1 || p->q_heads % p->kv_heads)
    return set_error(KIMODO_EINVAL, "q_heads must be a multiple of kv_heads (got %d, %d)", p->q_heads, p->kv_heads);
  if (p->head_dim != 64 && p->head_dim != 128)
    return set_error(KIMODO_EINVAL, "head_dim must be 64 or 128 (got %d)", p->head_dim);
  if (p->dtype != KIMODO_FP32 && p->dtype != KIMODO_BF16)
    return set_error(KIMODO_EINVAL, "dtype must be KIMODO_FP32 or KIMODO_BF16 (got %d)", p->dtype);
  if (p->kv_len > KIMODO_MAX_KEYS || p->q_len > KIMODO_MAX_KEYS)
    return set_error(KIMODO_EINVAL, "q_len and kv_len must be at most %d", KIMODO_MAX_KEYS);
  // (two steps: the product of all three can leave 64 bits)
  if ((long long)p->batch * p->q_len > INT_MAX / 2 || (long long)p->batch * p->q_len * p->q_heads > INT_MAX / 2)
    return set_error(KIMODO_EINVAL, "too many query rows");
  if (!isfinite(p->scale)) return set_error(KIMODO_EINVAL, "scale must be finite");
  if (!isfinite(p->cap) || p->cap < 0.f) return set_error(KIMODO_EINVAL, "cap must be finite and >= 0");
  if (p->cap > 0.f && !(fabsf(p->scale) <= 1e6f * p->cap))
    return set_error(KIMODO_EINVAL, "cap must be at least a millionth of the scale");
  if (p->prefix && !p->causal) return set_error(KIMODO_EINVAL, "prefix needs causal");
  // (without keys there are no documents of keys, whose tensor of no elements has no address)
  if ((p->q_documents == nullptr) != (p->kv_documents == nullptr) && (p->kv_len > 0 || !p->q_documents))
    return set_error(KIMODO_EINVAL, "q_documents and kv_documents come together");
  // strides: an extent of one has none; 16-byte rows (vector loads, TMA)
  const int unit = p->dtype == KIMODO_BF16 ? 8 : 4;
  const long long extents[4][3] = {{p->batch, p->q_len, p->q_heads},
                                   {p->batch, p->kv_len, p->kv_heads},
                                   {p->batch, p->kv_len, p->kv_heads},
                                   {p->batch, p->q_len, p->q_heads}};
  const long long* strides[4] = {p->q_strides, p->k_strides, p->v_strides, p->out_strides};
  const void* bases[4] = {p->q, p->k, p->v, p->out};
  long s[4][3];
  for (int t = 0; t < 4; ++t) {
    if (misaligned(bases[t], 16)) return set_error(KIMODO_EINVAL, "q, k, v and out must be 16-byte aligned");
    for (int d = 0; d < 3; ++d) {
      const bool used = extents[t][d] > 1;
      if (used && (strides[t][d] < p->head_dim || strides[t][d] % unit || strides[t][d] > (1ll << 36)))
        return set_error(KIMODO_EINVAL,
                         "strides must be multiples of 16 bytes, at least head_dim elements and below 2^36");
      s[t][d] = used ? (long)strides[t][d] : 0;
    }
  }
  if (misaligned(p->slopes, 4) || misaligned(p->prefix, 4) || misaligned(p->q_documents, 4) ||
      misaligned(p->kv_documents, 4) || misaligned(p->kv_lengths, 4) || misaligned(p->q_start, 4))
    return set_error(KIMODO_EINVAL, "slopes and index tensors must be aligned to their elements");
  a->q = p->q; a->k = p->k; a->v = p->v; a->out = p->out;
  a->slopes = p->slopes; a->prefix = p->prefix;
  a->q_doc = p->kv_len > 0 ? p->q_documents : nullptr;
  a->kv_doc = p->kv_len > 0 ? p->kv_documents : nullptr;
  a->kv_lengths = p->kv_lengths; a->q_start = p->q_start;
  a->q_batch = s[0][0]; a->q_token = s[0][1]; a->q_head = s[0][2];
  a->k_batch = s[1][0]; a->k_token = s[1][1]; a->k_head = s[1][2];
  a->v_batch = s[2][0]; a->v_token = s[2][1]; a->v_head = s[2][2];
  a->o_batch = s[3][0]; a->o_token = s[3][1]; a->o_head = s[3][2];
  a->B = p->batch; a->Sq = p->q_len; a->Sk = p->kv_len; a->Hq = p->q_heads; a->Hkv = p->kv_heads;
  a->G = p->q_heads / p->kv_heads; a->HD = p->head_dim;
  a->scale = p->scale; a->cap = p->cap; a->causal = p->causal != 0;
  return KIMODO_OK;
}

}  // namespace

extern "C" {

int kimodo_attention_scored_workspace(const kimodo_scored_attention* args, size_t* bytes) {
  clear_error();
  if (!bytes) return set_error(KIMODO_EINVAL, "bytes is NULL");
  *bytes = 0;
  ScoredAttention a;
  KD_TRY(scored_args(args, &a));
  const int sms = current_sms();
  if (sms < 1) return set_error(KIMODO_EUNSUPPORTED, "no CUDA device available");
  *bytes = scored_attention_plan(a, args->dtype == KIMODO_BF16, sms).bytes;
  return KIMODO_OK;
}

int kimodo_attention_scored(const kimodo_scored_attention* args, void* workspace, size_t workspace_bytes,
                            void* stream) {
  clear_error();
  ScoredAttention a;
  KD_TRY(scored_args(args, &a));
  const long long e = args->dtype == KIMODO_BF16 ? 2 : 4, w = a.HD * e;
  const Place out{a.out, w, {a.B, a.Sq, a.Hq}, {a.o_batch * e, a.o_token * e, a.o_head * e}};
  const Place q{a.q, w, {a.B, a.Sq, a.Hq}, {a.q_batch * e, a.q_token * e, a.q_head * e}};
  const Place k{a.Sk > 0 ? a.k : nullptr, w, {a.B, a.Sk, a.Hkv}, {a.k_batch * e, a.k_token * e, a.k_head * e}};
  const Place v{a.Sk > 0 ? a.v : nullptr, w, {a.B, a.Sk, a.Hkv}, {a.v_batch * e, a.v_token * e, a.v_head * e}};
  KD_TRY(check_apart("out", out, {q, k, v}));
  KD_TRY(check_here({a.q, a.k, a.v, a.out, a.slopes, a.prefix, a.q_doc, a.kv_doc, a.kv_lengths, a.q_start}));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = args->dtype == KIMODO_BF16;
  if (bf && !gemm_tc_available()) return set_error(KIMODO_EUNSUPPORTED, "cuTensorMapEncodeTiled is unavailable");
  const int sms = current_sms();
  if (sms < 1) return set_error(KIMODO_ECUDA, "the SM count could not be read");
  const ScoredPlan plan = scored_attention_plan(a, bf, sms);
  if (plan.bytes > 0) {
    if (!workspace || workspace_bytes < plan.bytes)
      return set_error(KIMODO_EINVAL, "this call needs a workspace of %zu bytes (got %zu)", plan.bytes,
                       workspace ? workspace_bytes : (size_t)0);
    if (misaligned(workspace, 16)) return set_error(KIMODO_EINVAL, "the workspace must be 16-byte aligned");
    KD_TRY(check_here({workspace}));
  }
  KD_CUDA(attention_scored(a, bf, plan, workspace, kernel_error_word(), st));
  return KIMODO_OK;
}

int kimodo_kernel_status(void* stream) {
  clear_error();
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return set_error(KIMODO_EUNSUPPORTED, "no CUDA device available");
  }
  KD_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
  DevError* err = kernel_error_word();
  if (!err) return set_error(KIMODO_ECUDA, "the device error word is not available");
  DevError h;
  KD_CUDA(cudaMemcpy(&h, err, sizeof(h), cudaMemcpyDeviceToHost));
  if (h.code != 0) {
    KD_CUDA(cudaMemset(err, 0, sizeof(DevError)));
    return set_error(h.code, "device wait timed out in %s (block %d)", where_name(h.where), h.block);
  }
  return KIMODO_OK;
}

}  // extern "C"
