// Attention whose scores may be capped, biased by distance and masked.  For query i (at
// position p_i = q_start + i) and key j of sequence b, head h:
//   x_ij = scale * q_i . k_j;             x_ij = cap * tanh(x_ij / cap)           (cap > 0)
//   x_ij = x_ij - slope_h * |p_i - j|                                             (slopes)
//   seen: j < kv_len_b, j <= p_i or j < prefix_b (causal), same document >= 0 (documents)
//   o_i = sum_j softmax_j(x_ij over the keys seen) v_j, and 0 where no key is seen.
// Scores, softmax statistics and sums are fp32; the weights p = 2^(x - max) are rounded to
// bf16 (8 bits, as the values they multiply) for the tensor cores, the output once to bf16.
//
// Rows of a tile.  The Sq queries of the G query heads that share a key head are one list of
// Sq * G rows (token-major), so grouped heads share every key tile they load and a few new
// tokens fill one MMA tile together.
//
// Many rows (scored_tc_kernel): an SM works on two tiles of 128 rows, as two CTAs or as one that
// takes both in turn; while the softmax of one runs, the tensor cores work on the other.
// Roles (128 threads and 256 a row tile): warp 0 TMA of K and V tiles (128 keys, 128-byte
// swizzle), warps 1 and 2 MMA issue of tile 0 and 1, warps 4-11 and 12-19 softmax and output
// of tile 0 and 1, two threads a row, each half of the keys (one thread a row left the four
// schedulers two warps each, too few to hide the latencies: 490 against 431 us for 16 heads x
// 8192 tokens).  Per key tile and row tile: S = Q K^T into 128 TMEM columns; the row's threads
// read S, form p and write it in bf16 over S; O += P V with P as the TMEM operand.
//
// Few rows (scored_few_kernel, at most 16: new tokens over a cache): the keys take the MMA's
// rows instead, S^T = K Q^T and O^T = V^T P^T, so that all four TMEM quarters, and with them
// all softmax warps, share a key tile however few the queries are, and an MMA costs N = rows.
//
// Keys are split over CTAs while these do not fill the SMs; a second kernel joins the parts.
// The weights' reference need not be the running maximum: it only has to keep p = 2^(x - ref) in
// range, and fp32 sums and bf16 weights hold 2^10 as well as 1.  So a tile's weights are
// formed with the reference that is there, without its maximum; where their sum (or a cap
// polynomial's range) shows that this was wrong, and in masked tiles, the maximum is taken,
// the reference moved and O rescaled.
//
// Masked places never reach a result: a masked score is replaced, value rows past the last key
// that a CTA's rows see are zeroed in shared memory (a cache may hold anything behind its
// newest token), and a row whose result is still not finite (a NaN or infinity among values
// with weight 0 in its tile) is computed again over the seen keys alone, slowly.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace kd {
namespace {

constexpr int TILE = 128;                    // query rows of a tile, keys of a tile
constexpr int DOC_TILES_MIN = 8;             // key tiles from which their documents are summarised by a kernel of its own
constexpr int MAX_LIST = 4096;               // key tiles that a CTA with documents lists (12 bits of an entry)
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr int KIMODO_ETIMEOUT_CODE = -5;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESCALE_AT = 8.f;            // log2 units the maximum may run ahead of its reference
constexpr float MAX_SUM = 1024.f;            // weights of 64 keys whose sum stays below need no new one

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(x / cap) in log2 units, x = scale s.  For |x| <= cap / 2: s times a polynomial of degree
// 3 in z^2, z = x / cap, for tanh(z) / z (weighted least squares towards the relative minimax on
// [0, 1/4] in z^2; relative error 5.5e-7, on a cap of 50 at most 2e-5 of a weight, a
// hundredth of its rounding to bf16).  It costs no special-function slots, which bound
// the softmax.  Beyond, tanh z = 1 - 2 / (1 + e^(2z)), whose error is that of the cap: a small
// score never takes that form, whatever the other scores of the warp are.
__host__ __device__ constexpr float cap_poly(int i) {
  return i == 0 ? 0.999999463558197f : i == 1 ? -0.33326318860054016f : i == 2 ? 0.13190296292304993f : -0.044402219355106354f;
}
ScoredConst scored_const(float scale, float cap) {
  const float sc = scale == 0.f ? 1.f : fabsf(scale), lin = sc * LOG2E, z = cap > 0.f ? sc / cap : 0.f;
  ScoredConst k;
  k.lin = make_float2(lin, lin);
  float f = lin;
  for (int i = 0; i < 4; ++i) {
    k.c[i] = make_float2(cap_poly(i) * f, cap_poly(i) * f);
    f *= z * z;
  }
  // Below 1e-5 the higher coefficients may underflow; they are not needed while x is below a
  // 64th of the cap (the terms of degree 4 and 6 in z are then below 1e-8).
  const double z2 = (double)z * z;
  k.limit2 = z > 1e-5f ? (float)(0.25 / z2) : z2 > 2.5e-34 ? (float)(2.4e-4 / z2) : 1e30f;
  // scales and caps that take a coefficient out of the floats' range leave every score to capped_any
  if (lin < 1e-6f || !isfinite(k.c[3].x)) k.limit2 = -1.f;
  k.z = z;
  k.two = 2.f * LOG2E * z;
  k.cap2 = cap * LOG2E;
  return k;
}
// two scores at once (f32x2 arithmetic); t = s^2 up to limit2
__device__ __forceinline__ float2 cap_ratio(const ScoredConst& k, float2 t) {
  return __ffma2_rn(__ffma2_rn(__ffma2_rn(k.c[3], t, k.c[2]), t, k.c[1]), t, k.c[0]);
}
// any score
__device__ __forceinline__ float capped_any(const ScoredConst& k, float s) {
  const float zs = s * k.z, t = zs * zs;
  const float ratio = fmaf(fmaf(fmaf(cap_poly(3), t, cap_poly(2)), t, cap_poly(1)), t, cap_poly(0));
  const float far = fmaf(-2.f * k.cap2, rcp_approx(1.f + ex2(s * k.two)), k.cap2);
  return t <= 0.25f ? s * k.lin.x * ratio : far;
}
template <int N>
__device__ __forceinline__ void cap_scores(const ScoredConst& k, float (&x)[N]) {
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) far = fmaxf(far, fabsf(x[e]));
  if (__any_sync(0xffffffffu, !(far * far <= k.limit2))) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = capped_any(k, x[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 v = make_float2(x[e], x[e + 1]);
      const float2 y = __fmul2_rn(v, cap_ratio(k, __fmul2_rn(v, v)));
      x[e] = y.x;
      x[e + 1] = y.y;
    }
  }
}

// 3-operand maximum; a NaN operand gives NaN (and a row whose maximum is NaN is
// done again at the end)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float a[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) a[c] = max3(x[c], x[4 + c], x[8 + c]);
#pragma unroll
  for (int e = 12; e < N - 4; e += 8)
#pragma unroll
    for (int c = 0; c < 4; ++c) a[c] = max3(a[c], x[e + c], x[e + 4 + c]);
#pragma unroll
  for (int c = 0; c < 4; ++c) a[c] = max3(a[c], x[N - 4 + c], x[N - 4 + c]);
  return max3(max3(a[0], a[1], a[2]), a[3], a[3]);
}
__device__ __forceinline__ void record_timeout(DevError* err, volatile int* abort) {
  *abort = 1;
  if (err && atomicCAS(&err->code, 0, KIMODO_ETIMEOUT_CODE) == 0) {
    err->where = WHERE_SCORED_ATTENTION;
    err->block = blockIdx.x;
  }
}

// ---------------------------------------------------------------- what a row sees

struct SeqInfo {
  int kv_len, start, prefix;
};
__device__ __forceinline__ SeqInfo sequence_info(const ScoredAttention& a, int b) {
  SeqInfo s;
  s.kv_len = a.kv_lengths ? min(max(a.kv_lengths[b], 0), a.Sk) : a.Sk;
  s.start = a.q_start ? a.q_start[b] : a.Sk - a.Sq;
  s.prefix = a.prefix ? a.prefix[b] : 0;
  return s;
}
// last key (by length, position and prefix) that query position p sees; -1: none
__device__ __forceinline__ int last_key(const ScoredAttention& a, const SeqInfo& s, long p) {
  int j = s.kv_len - 1;
  if (a.causal) {
    const long c = p > (long)s.prefix - 1 ? p : (long)s.prefix - 1;
    if (c < j) j = c < -1 ? -1 : (int)c;
  }
  return j;
}
// Position that a row's distances are counted from: the nearest one that length, position and prefix
// let it see.  It differs from p by a constant of the row for all its keys, which the softmax
// cancels; counted from p itself, slope * distance would round the differences between keys
// away where all of them are far (a slope of 0.5 at a distance of 10^6: 3 % of a weight).
__device__ __forceinline__ int bias_position(long p, int last) {
  return p > last ? max(last, 0) : p < 0 ? 0 : (int)p;
}

// ---------------------------------------------------------------- one row by one warp, fp32
// The definition, over the seen keys alone: scores by warp-shuffle dot products, online
// softmax.  For the rows whose first result is not finite.
template <typename T, int HD>
__device__ __noinline__ void row_by_warp(const ScoredAttention& a, int b, int hq, int i) {
  constexpr int PER = HD / 32;
  const int lane = threadIdx.x & 31;
  const int hk = hq / a.G;
  const SeqInfo s = sequence_info(a, b);
  const long p = (long)s.start + i;
  const int last = last_key(a, s, p), from = bias_position(p, last);
  const T* q = static_cast<const T*>(a.q) + b * a.q_batch + i * a.q_token + hq * a.q_head + lane * PER;
  const T* k = static_cast<const T*>(a.k) + b * a.k_batch + hk * a.k_head + lane * PER;
  const T* v = static_cast<const T*>(a.v) + b * a.v_batch + hk * a.v_head + lane * PER;
  const int qd = a.q_doc ? a.q_doc[(long)b * a.Sq + i] : 0;
  const float slope = a.slopes ? a.slopes[hq] : 0.f;
  float qv[PER], o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    qv[e] = to_f<T>(q[e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j <= last; ++j) {
    if (a.q_doc && (qd < 0 || a.kv_doc[(long)b * a.Sk + j] != qd)) continue;
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) d = fmaf(qv[e], to_f<T>(k[j * a.k_token + e]), d);
#pragma unroll
    for (int off = 16; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    float x = d * a.scale;
    if (a.cap > 0.f) x = a.cap * tanhf(x / a.cap);
    if (a.slopes) x -= slope * fabsf((float)(from - j));
    if (x == -INFINITY) continue;   // weight 0, whatever the value is
    const float mn = fmaxf(m, x);
    const float f = expf(m - mn), w = expf(x - mn);
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = o[e] * f + w * to_f<T>(v[j * a.v_token + e]);
    m = mn;
  }
  T* out = static_cast<T*>(a.out) + b * a.o_batch + i * a.o_token + hq * a.o_head + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; ++e) out[e] = from_f<T>(l == 0.f ? 0.f : o[e] / l);
}

// ---------------------------------------------------------------- bf16: tcgen05

template <int HD, int TILES>
struct Cfg {
  static constexpr int THREADS = 128 + 256 * TILES;
  // K and V tiles in flight, alternating; two CTAs share an SM where each has one row tile
  static constexpr int STAGES = TILES == 2 || HD == 64 ? 4 : 2;
  static constexpr uint32_t Q_BYTES = TILE * HD * 2;       // one row tile
  static constexpr uint32_t KV_BYTES = TILE * HD * 2;      // one key or value tile
  static constexpr uint32_t HALF = TILE * 128;             // 64 dims of a tile
  static constexpr uint32_t COLS = 256 * TILES;            // TMEM
  static constexpr size_t DATA = TILES * Q_BYTES + (size_t)STAGES * KV_BYTES;
  // two row tiles take all of the TMEM: the size keeps a second CTA of 64-dim heads off the SM
  static constexpr size_t BODY = TILES == 2 && DATA < 119808 ? 119808 : DATA;
  static constexpr size_t LIST = BODY, BARS = LIST + MAX_LIST * 2, DOCS = BARS + 256, XCH = DOCS + 8 * TILES * 64 * 4;
  static constexpr size_t SMEM = 1024 + XCH + 2 * TILES * 2 * TILE * 4;
  static_assert(SMEM <= 232448 / (TILES == 1 ? 2 : 1) - (TILES == 1 ? 1024 : 0), "shared memory");
};
constexpr uint32_t TMEM_COLS = 512;
__device__ __forceinline__ uint32_t s_col(int t) { return 128u * t; }
template <int HD, int TILES> __device__ __forceinline__ uint32_t o_col(int t) { return 128u * TILES + (uint32_t)HD * t; }

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle layout:
// 64-element atoms along MN `lbo` bytes apart, 8-row groups along K 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

struct RowTile {
  int docs_lo, docs_hi;   // smallest and largest document of its rows (lo > hi: none)
  int any_none;           // a row in no document
  int pad;
};

// Summary of a key tile's documents, its keys spread over a warp (-1: no document): x = the
// smallest, its sign bit set where a key is in none; y = the largest (-1: all are in none).
__device__ __forceinline__ int2 docs_of_tile(const int (&d)[TILE / 32]) {
  int lo = INT_MAX, hi = -1;
  bool none = false;
#pragma unroll
  for (int e = 0; e < TILE / 32; ++e) {
    none |= d[e] < 0;
    lo = min(lo, d[e] < 0 ? INT_MAX : d[e]);
    hi = max(hi, d[e]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  none = __any_sync(0xffffffffu, none);
  return make_int2(none ? lo | INT_MIN : lo, hi < 0 ? -1 : hi);
}

// The summaries of all key tiles, one warp each, where every CTA would otherwise read all keys'
// documents to list its tiles (8 heads of 64 dims, documents of up to 301 tokens: one row of 12289 tokens
// 65 us without, 59 with them; 8 of 1536: 55.5 and 54.3).
__global__ void __launch_bounds__(128) scored_docs_kernel(const __grid_constant__ ScoredAttention a,
                                                          const __grid_constant__ ScoredPlan plan) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const long id = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (id >= (long)a.B * plan.key_tiles) return;
  const int b = (int)(id / plan.key_tiles), jt = (int)(id % plan.key_tiles), lane = threadIdx.x & 31;
  const SeqInfo seq = sequence_info(a, b);
  int d[TILE / 32];
#pragma unroll
  for (int e = 0; e < TILE / 32; ++e) {
    const int j = jt * TILE + e * 32 + lane;
    d[e] = j < seq.kv_len ? a.kv_doc[(long)b * a.Sk + j] : -1;
  }
  const int2 v = docs_of_tile(d);
  if (lane == 0) plan.doc_tiles[id] = v;
}

template <int HD, bool CAP, bool BIAS, int TILES>
__global__ void __launch_bounds__(128 + 256 * TILES, TILES == 2 ? 1 : 2)   // 96 or 80 registers a thread
scored_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ ScoredAttention a, const __grid_constant__ ScoredPlan plan,
                 DevError* err) {
  static_assert(CAP || TILES == 1, "two row tiles are taken under a cap only");
  using C = Cfg<HD, TILES>;
  constexpr int STAGES = C::STAGES, NUM_THREADS = C::THREADS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = ptx::smem_u32(smem);
  const uint32_t sKV = sQ + TILES * C::Q_BYTES;
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + C::LIST);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BARS);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto s_bar = [&](int t) { return bar0 + 8u * (2 * STAGES + t); };       // S formed
  auto p_bar = [&](int t) { return bar0 + 8u * (2 * STAGES + 2 + t); };   // P written, O rescaled
  auto o_bar = [&](int t) { return bar0 + 8u * (2 * STAGES + 4 + t); };   // last P V done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 6);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* mma_lock = reinterpret_cast<int*>(tmem_slot + 2);
  int* list_len = mma_lock + 1;
  RowTile* tiles = reinterpret_cast<RowTile*>(tmem_slot + 4);
  int* docs_smem = reinterpret_cast<int*>(smem + C::DOCS);    // [softmax warps][64]
  float* xch = reinterpret_cast<float*>(smem + C::XCH);   // [2 turns][TILES][2 halves][TILE]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // block = ((row block, last first) * Hkv * B + (b * Hkv + hk)) * splits + split
  long id = blockIdx.x;
  const int split = (int)(id % plan.splits);
  id /= plan.splits;
  const int hk = (int)(id % a.Hkv);
  id /= a.Hkv;
  const int b = (int)(id % a.B);
  const int rb = plan.row_blocks - 1 - (int)(id / a.B);
  const int rows = a.Sq * a.G;
  const int row0 = rb * TILE * TILES;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), TILES);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(s_bar(t), 1);
      ptx::mbar_init(p_bar(t), 8);
      ptx::mbar_init(o_bar(t), 1);
      tiles[t].docs_lo = INT_MAX;
      tiles[t].docs_hi = -1;
      tiles[t].any_none = 0;
    }
    ptx::fence_mbar_init();
    *abort = 0;
    *mma_lock = 0;
    ptx::tma_prefetch_desc(&tmK);
    ptx::tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::COLS);
    ptx::tmem_relinquish();
  }
  ptx::pdl_wait();
  ptx::pdl_trigger();
  SeqInfo seq = sequence_info(a, b);
  __syncthreads();

  // ---------------- queries into shared memory (K-major, 128-byte swizzle), rows' documents
  {
    constexpr int CH = HD / 8;                               // 16-byte chunks of a row
    const bf16* qb = static_cast<const bf16*>(a.q) + b * a.q_batch + (long)hk * a.G * a.q_head;
    const int total = TILES * TILE * CH;
    for (int c = threadIdx.x; c < total; c += NUM_THREADS) {
      const int lr = c / CH, ch = c % CH, r = row0 + lr;
      const bool in = r < rows;
      const int i = in ? r / a.G : 0, g = in ? r - i * a.G : 0;
      const int t = lr / TILE, rr = lr % TILE;
      ptx::cp_async_16_zfill(sQ + t * C::Q_BYTES + (ch >> 3) * C::HALF + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4),
                             qb + i * a.q_token + g * a.q_head + ch * 8, in);
    }
    ptx::cp_async_commit();   // waited for below, under the key tiles' documents
  }
  // this softmax thread's row
  const int t_own = TILES == 2 && warp >= 12 ? 1 : 0;
  const int lr_own = (warp & 3) * 32 + lane + t_own * TILE;
  const int r_own = row0 + lr_own;
  const bool row_ok = warp >= 4 && r_own < rows;
  const int i_own = row_ok ? r_own / a.G : 0;
  const int g_own = row_ok ? r_own - i_own * a.G : 0;
  int qdoc = 0;
  if (a.q_doc != nullptr && warp >= 4) {
    qdoc = row_ok ? a.q_doc[(long)b * a.Sq + i_own] : -1;
    const int lo = __reduce_min_sync(0xffffffffu, qdoc >= 0 ? qdoc : INT_MAX);
    const int hi = __reduce_max_sync(0xffffffffu, qdoc);
    const unsigned none = __ballot_sync(0xffffffffu, row_ok && qdoc < 0);
    if (lane == 0) {
      atomicMin(&tiles[t_own].docs_lo, lo);
      atomicMax(&tiles[t_own].docs_hi, hi);
      if (none) tiles[t_own].any_none = 1;
    }
  }
  __syncthreads();

  // ---------------- key tiles of this CTA
  const int row_last = min(row0 + TILES * TILE, rows) - 1;
  const int key_end = 1 + last_key(a, seq, (long)seq.start + row_last / a.G);
  seq.kv_len = key_end;   // what no row of this CTA sees counts as behind the keys
  const int jt_all = (key_end + TILE - 1) / TILE;
  const int jt0 = min(split * plan.tiles_per_split, jt_all);
  const int jt1 = plan.splits == 1 ? jt_all : min(jt0 + plan.tiles_per_split, jt_all);
  const bool docs = a.q_doc != nullptr;
  const bool listed = docs && jt1 - jt0 <= MAX_LIST;
  if (listed) {
    // entry of a key tile: its number above 4 flags, bit 2t = row tile t may see it, bit 2t + 1 =
    // all of t's rows and all of its keys are one document
    auto flags = [&](int lo, int hi, bool none) {
      int f = 0;
      for (int t = 0; t < TILES; ++t) {
        const RowTile& q = tiles[t];
        if (lo <= q.docs_hi && q.docs_lo <= hi) f |= 1 << (2 * t);
        if (!none && !q.any_none && lo == hi && q.docs_lo == q.docs_hi && lo == q.docs_lo) f |= 2 << (2 * t);
      }
      return f;
    };
    const int2* doc_tiles = plan.doc_tiles ? plan.doc_tiles + (long)b * plan.key_tiles : nullptr;
    if (doc_tiles != nullptr) {
      for (int e = threadIdx.x; e < jt1 - jt0; e += NUM_THREADS) {
        const int2 d = doc_tiles[jt0 + e];
        list[e] = (uint16_t)(e << 4 | flags(d.x & INT_MAX, d.y, d.x < 0));
      }
    }
    constexpr int AT_ONCE = 4;   // tiles whose loads a warp has in flight
    for (int jq = jt0 + warp; doc_tiles == nullptr && jq < jt1; jq += AT_ONCE * (NUM_THREADS / 32)) {
      int d[AT_ONCE][TILE / 32];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
        for (int e = 0; e < TILE / 32; ++e) {
          const int jt = jq + u * (NUM_THREADS / 32), j = jt * TILE + e * 32 + lane;
          d[u][e] = jt < jt1 && j < seq.kv_len ? a.kv_doc[(long)b * a.Sk + j] : -1;
        }
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const int jt = jq + u * (NUM_THREADS / 32);
        const int2 v = docs_of_tile(d[u]);
        if (lane == 0 && jt < jt1) {
          list[jt - jt0] = (uint16_t)((jt - jt0) << 4 | flags(v.x & INT_MAX, v.y, v.x < 0));
        }
      }
    }
    __syncthreads();
    if (warp == 0) {   // close the gaps: the tiles that neither row tile sees
      int len = 0;
      for (int e = 0; e < jt1 - jt0; e += 32) {
        const uint32_t v = e + lane < jt1 - jt0 ? list[e + lane] : 0u;
        const unsigned keep = __ballot_sync(0xffffffffu, v & 5u);
        if (v & 5u) list[len + __popc(keep & ((1u << lane) - 1u))] = (uint16_t)v;
        len += __popc(keep);
        __syncwarp();
      }
      if (lane == 0) *list_len = len;
    }
  }
  ptx::cp_async_wait_all();
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // two row tiles have all columns, which start at 0 (a constant the MMA operands are made of)
  const uint32_t tmem_base = TILES == 2 ? 0u : __shfl_sync(0xffffffffu, *tmem_slot, 0);

  // Row tile t takes the key tiles [jt0, end_t) that hold a document of its rows.
  auto end_of = [&](int t) {
    const int r_a = row0 + t * TILE, r_b = min(r_a + TILE, rows) - 1;
    if (r_a >= rows) return 0;
    return min((1 + last_key(a, seq, (long)seq.start + r_b / a.G) + TILE - 1) / TILE, jt1);
  };
  const int end0 = end_of(0), end1 = TILES == 2 ? end_of(1) : 0;
  const int n_tiles = listed ? *list_len : jt1 - jt0;
  // entry n of the tiles to go through: key tile and the flags above
  auto entry = [&](int n) -> int { return listed ? list[n] : n << 4 | (docs ? 5 : 15); };
  auto takes = [&](int t, int e) -> bool { return jt0 + (e >> 4) < (t ? end1 : end0) && ((e >> (2 * t)) & 1); };

  // registers: 640 x 96 at launch cover 128 x 32 + 512 x 112, 384 x 80 cover 128 x 32 + 256 x 104
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 0) {
      if (lane == 0) {
        // ---------------- TMA: K and V tile of every key tile that a row tile takes
        int stage = 0;
        uint32_t phase = 0;
        long issued = 0;
        bool ok = true;
        for (int n = 0; n < n_tiles && ok; ++n) {
          const int e = entry(n), jt = jt0 + (e >> 4);
          if (!takes(0, e) && !takes(1, e)) continue;
          for (int kv = 0; kv < 2; ++kv) {
            if (!ptx::mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort, WAIT_LIMIT_NS)) {
              ok = false;
              break;
            }
            ptx::mbar_arrive_expect_tx(full_bar(stage), C::KV_BYTES);
#pragma unroll
            for (int hf = 0; hf < HD / 64; ++hf)
              ptx::tma_load_4d(sKV + stage * C::KV_BYTES + hf * C::HALF, kv ? &tmV : &tmK, full_bar(stage), hf * 64,
                               jt * TILE, hk, b);
            ++issued;
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
        }
        if (!ok && !*abort) record_timeout(err, abort);
        // every copy issued has landed before the CTA leaves (also after a wait that ran out)
        const long left = issued < STAGES ? issued : STAGES;
        volatile int never = 0;
        for (long i = 0; i < left; ++i) {
          if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
          ptx::mbar_wait_bounded(full_bar(stage), phase, &never, WAIT_LIMIT_NS);
        }
      }
    } else if (warp <= TILES) {
      // ---------------- MMA of row tile t: per key tile first P V of the tile before, then Q K^T,
      // which overwrites that P.  The tiles' MMAs come from two warps, so that neither waits
      // for the other's softmax, and from two schedulers: their issue slots are scarce beside
      // the softmax warps.  Control flow and operands are uniform over the warp.
      const int t = warp - 1;
      const uint32_t idesc_s = ptx::idesc_bf16_f32(TILE, TILE);
      const uint32_t idesc_o = ptx::idesc_bf16_f32(TILE, HD) | (1u << 16);
      // operand descriptors: low words of the first stage, later ones and K steps by additions
      const uint64_t d_k = ptx::smem_desc_sw128(sKV), d_v = desc_mn(sKV, C::HALF);
      const uint32_t k_hi = (uint32_t)(d_k >> 32), v_hi = (uint32_t)(d_v >> 32);
      const uint32_t q_lo = (uint32_t)ptx::smem_desc_sw128(sQ + t * C::Q_BYTES);
      const uint32_t s_tmem = tmem_base + s_col(t), o_tmem = tmem_base + o_col<HD, TILES>(t);
      int stage = 0, v_stage = 0, v_rows = TILE;
      uint32_t phase = 0, v_phase = 0, p_phase = 0, started = 0;
      bool ok = true, pend = false;
      auto wait = [&](uint32_t bar, uint32_t ph) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, ph, abort, WAIT_LIMIT_NS));
        return ok;
      };
      auto p_ready = [&]() {   // the pending key tile's values and weights
        if (!wait(full_bar(v_stage), v_phase)) return;
        if (v_rows < TILE) {   // value rows past the last key that a row of this CTA sees: 0, whatever they hold
          uint8_t* v = smem + TILES * C::Q_BYTES + v_stage * C::KV_BYTES;
          const int n = (TILE - v_rows) * 8;
          for (int c = lane; c < n * (HD / 64); c += 32) {
            const int hf = c / n, e = c % n;
            *reinterpret_cast<uint4*>(v + hf * C::HALF + (v_rows + e / 8) * 128 + (e & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        if (!wait(p_bar(t), p_phase)) return;
        p_phase ^= 1u;
      };
      auto pv = [&]() {   // O (+)= P V of the pending key tile
        const uint32_t v_lo = (uint32_t)d_v + v_stage * (C::KV_BYTES >> 4);
        if (ptx::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < TILE / 16; ++kk)
            ptx::tc_mma_bf16_ta_lo(o_tmem, s_tmem + (kk >> 2) * 64 + (kk & 3) * 8, v_lo + kk * (2048 >> 4), v_hi, idesc_o,
                                   kk != 0 ? 1u : started);
          ptx::tc_commit(empty_bar(v_stage));
        }
        __syncwarp();
        started = 1u;
        pend = false;
      };
      // The two warps take turns in whole blocks (P V and Q K^T of one tile): interleaved, both
      // tiles' scores would come at the same time, and softmax and tensor cores would wait for
      // each other instead of working on one tile each.
      auto lock = [&]() {
        if (TILES == 2 && lane == 0) {
          const uint64_t t0 = ptx::global_timer_ns();
          while (atomicCAS(mma_lock, 0, 1) != 0)
            if (*abort || ptx::global_timer_ns() - t0 > WAIT_LIMIT_NS) {
              if (!*abort) record_timeout(err, abort);
              break;
            }
        }
        __syncwarp();
        ptx::tc_fence_after();
      };
      auto unlock = [&]() {
        __syncwarp();
        if (TILES == 2 && lane == 0) atomicExch(mma_lock, 0);
      };
      for (int n = 0; n < n_tiles; ++n) {
        const int e = __shfl_sync(0xffffffffu, entry(n), 0), jt = jt0 + (e >> 4);
        const bool mine = takes(t, e), other = TILES == 2 && takes(t ^ 1, e);
        if (!mine && !other) continue;
        const int k_stage = stage;
        const uint32_t k_phase = phase;
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        if (mine && !wait(full_bar(k_stage), k_phase)) break;
        if (pend) {
          p_ready();
          if (!ok) break;
        }
        if (mine || pend) {
          lock();
          if (pend) pv();
          if (mine) {
            const uint32_t k_lo = (uint32_t)d_k + k_stage * (C::KV_BYTES >> 4);
            if (ptx::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk)
                ptx::tc_mma_bf16_lo(s_tmem, q_lo + (((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4),
                                    k_lo + (((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4), k_hi, idesc_s, kk != 0);
              ptx::tc_commit(s_bar(t));
              ptx::tc_commit(empty_bar(k_stage));
            }
            __syncwarp();
            pend = true;
            v_stage = stage;
            v_phase = phase;
            v_rows = min(seq.kv_len - jt * TILE, TILE);
          }
          unlock();
        }
        if (!mine) {   // the other tile's alone: hand both stages on, once they have been filled
          if (!wait(full_bar(k_stage), k_phase) || !wait(full_bar(stage), phase)) break;
          if (lane == 0) {
            ptx::mbar_arrive(empty_bar(k_stage));
            ptx::mbar_arrive(empty_bar(stage));
          }
        }
        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
      }
      if (ok && pend) {
        p_ready();
        if (ok) {
          lock();
          pv();
          unlock();
        }
      }
      if (!ok && !*abort && lane == 0) record_timeout(err, abort);
      if (ptx::elect_one()) {
        ptx::tc_commit(o_bar(t));
        volatile int never = 0;
        if (!ptx::mbar_wait_bounded(o_bar(t), 0, &never, WAIT_LIMIT_NS)) record_timeout(err, abort);
      }
      __syncwarp();
    }
  } else {
    if constexpr (TILES == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ---------------- softmax and output of row tile t_own
    const int t = t_own;
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem_base + lane_addr + s_col(t), o_addr = tmem_base + lane_addr + o_col<HD, TILES>(t);
    const int half = ((warp - 4) >> 2) & 1;            // keys 64 half .. of a tile, dims likewise
    constexpr int KH = TILE / 2, DH2 = HD / 2;
    const int lrow = (warp & 3) * 32 + lane;
    const int pair_bar = 1 + t * 4 + (warp & 3);       // the two warps that share 32 rows
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory"); };
    const bool warp_rows = (warp & 3) * 32 + row0 + t * TILE < rows;
    const int last = row_ok ? last_key(a, seq, (long)seq.start + i_own) : -1;
    const int p = bias_position((long)seq.start + i_own, last);
    qdoc = qdoc < 0 ? -2 : qdoc;
    const float slope2 = BIAS && row_ok ? a.slopes[hk * a.G + g_own] * LOG2E : 0.f;
    // the constants are those of |scale|: the products take its sign, and a scale of 0 is products of 0
    const ScoredConst& cc = plan.k;
    const float sc = cc.lin.x;
    const int* kdocs = docs ? a.kv_doc + (long)b * a.Sk : nullptr;
    int* dbuf = docs_smem + (warp - 4) * KH;
    float m = -INFINITY;            // reference of the weights (log2 units)
    float2 l2 = make_float2(0.f, 0.f);   // their sum over this thread's keys
    uint32_t phase = 0;
    bool ok = true, started = false;
    for (int n = 0; n < n_tiles; ++n) {
      const int e = entry(n), jt = jt0 + (e >> 4);
      if (!takes(t, e)) continue;
      const int j0 = jt * TILE + half * KH;
      const bool one_doc = (e >> (2 * t + 1)) & 1;
      if (!one_doc) {   // the documents of these keys, staged before the scores are there
        // (a key in no document: -1, which no row has; a row in none: -2, below)
        dbuf[lane] = max(kdocs[min(j0 + lane, a.Sk - 1)], -1);
        dbuf[32 + lane] = max(kdocs[min(j0 + 32 + lane, a.Sk - 1)], -1);
        __syncwarp();
      }
      // after a wait that ran out the rest is gone through without waiting, so that the
      // barriers of the warp pairs stay matched
      if (ok) ok = ptx::mbar_wait_bounded(s_bar(t), phase, abort, WAIT_LIMIT_NS);
      if (warp_rows) {
        ptx::tc_fence_after();
        float x[KH];
        ptx::tmem_ld32_at<0>(s_addr + half * KH, x);
        ptx::tmem_ld32_at<32>(s_addr + half * KH + 32, x);
        ptx::tmem_ld_wait();
        if (a.scale <= 0.f) {
#pragma unroll
          for (int e = 0; e < KH; ++e) x[e] = a.scale < 0.f ? -x[e] : 0.f;
        }
        float* xm = xch + ((phase * TILES + t) * 2) * TILE;
        // the weights arg(score pair) of this half's 64 keys, in bf16 in the first 32 of their columns
        auto weights = [&](auto arg) {
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < KH; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = arg(make_float2(x[c + e], x[c + e + 1]), c + e);
              const float2 pw = make_float2(ex2(y.x), ex2(y.y));
              sum = __fadd2_rn(sum, pw);
              w[e / 2] = bf16x2_bits(pw.x, pw.y);
            }
            ptx::tmem_st16(s_addr + half * KH + c / 2, w);
          }
          return sum;
        };
        // both warps of the rows decide alike: the conditions are those of the rows
        const bool cut = !__all_sync(0xffffffffu, jt * TILE + TILE - 1 <= last || !row_ok);
        const bool masked = cut || !one_doc;
        bool done = false, tried = false;
        if (!masked && __all_sync(0xffffffffu, m > -INFINITY || !row_ok)) {
          const float2 nref2 = make_float2(-m, -m);
          float2 sum;
          float far = 0.f;
          if constexpr (CAP) {
            if constexpr (BIAS) {
              // -slope |p - j| is linear in j on either side of p; a tile that p cuts takes the other way
              const float d0 = (float)(p - j0), sl = d0 > 0.f ? -slope2 : slope2;
              far = d0 < (float)KH && d0 > 0.f ? INFINITY : 0.f;
              const float2 sl2 = make_float2(-sl, -sl), b2 = make_float2(fmaf(sl, d0, -m), fmaf(sl, d0, -m));
              sum = weights([&](float2 v, int e) {
                const float2 u = __fmul2_rn(v, v);
                far = max3(far, u.x, u.y);
                return __ffma2_rn(v, cap_ratio(cc, u), __ffma2_rn(sl2, make_float2((float)e, (float)(e + 1)), b2));
              });
            } else {
              sum = weights([&](float2 v, int) {
                const float2 u = __fmul2_rn(v, v);
                far = max3(far, u.x, u.y);
                return __ffma2_rn(v, cap_ratio(cc, u), nref2);
              });
            }
          } else if constexpr (BIAS) {
            const float d0 = (float)(p - j0), sl = d0 > 0.f ? -slope2 : slope2;
            far = d0 < (float)KH && d0 > 0.f ? INFINITY : 0.f;
            const float2 sl2 = make_float2(-sl, -sl), b2 = make_float2(fmaf(sl, d0, -m), fmaf(sl, d0, -m));
            sum = weights([&](float2 v, int e) {
              return __ffma2_rn(v, cc.lin, __ffma2_rn(sl2, make_float2((float)e, (float)(e + 1)), b2));
            });
          } else {
            sum = weights([&](float2 v, int) { return __ffma2_rn(v, cc.lin, nref2); });
          }
          const bool good = sum.x + sum.y <= MAX_SUM && far <= (CAP ? cc.limit2 : 0.f);
          const bool all_good = __all_sync(0xffffffffu, good || !row_ok);
          if (lane == 0) xm[half * TILE + lrow] = all_good ? 1.f : 0.f;
          pair_sync();
          done = all_good && xm[(half ^ 1) * TILE + (lrow & ~31)] != 0.f;
          tried = true;
          if (done)
            l2 = __fadd2_rn(l2, sum);
          else
            pair_sync();   // the flags have been read: the maxima go to the same place
        }
        if (!done) {
          if constexpr (CAP) cap_scores(cc, x);
          if constexpr (BIAS) {
            const float d0 = (float)(p - j0);
            if (__all_sync(0xffffffffu, d0 <= 0.f || d0 >= (float)(KH - 1))) {   // linear on one side of p
              const float sl = d0 > 0.f ? -slope2 : slope2, base = sl * d0;
              const float2 sl2 = make_float2(-sl, -sl), b2 = make_float2(base, base);
#pragma unroll
              for (int e = 0; e < KH; e += 2) {
                const float2 v = make_float2(x[e], x[e + 1]);
                const float2 d = __ffma2_rn(sl2, make_float2((float)e, (float)(e + 1)), b2);
                const float2 y = CAP ? __fadd2_rn(v, d) : __ffma2_rn(v, cc.lin, d);
                x[e] = y.x;
                x[e + 1] = y.y;
              }
            } else {
#pragma unroll
              for (int e = 0; e < KH; ++e) x[e] = fmaf(-slope2, fabsf(d0 - (float)e), CAP ? x[e] : x[e] * sc);
            }
          } else if constexpr (!CAP) {
#pragma unroll
            for (int e = 0; e < KH; e += 2) {
              const float2 y = __fmul2_rn(make_float2(x[e], x[e + 1]), cc.lin);
              x[e] = y.x;
              x[e + 1] = y.y;
            }
          }
          if (cut) {
#pragma unroll
            for (int e = 0; e < KH; ++e)
              if (j0 + e > last) x[e] = -INFINITY;
          }
          if (!one_doc) {
#pragma unroll
            for (int e = 0; e < KH; e += 4) {
              const int4 d = *reinterpret_cast<const int4*>(dbuf + e);
              if (d.x != qdoc) x[e] = -INFINITY;
              if (d.y != qdoc) x[e + 1] = -INFINITY;
              if (d.z != qdoc) x[e + 2] = -INFINITY;
              if (d.w != qdoc) x[e + 3] = -INFINITY;
            }
          }
          xm[half * TILE + lrow] = max_of(x);
          pair_sync();
          const float top = max3(xm[lrow], xm[TILE + lrow], m);
          // move the reference: at once while there is none or where it did not do, else only when
          // it falls far behind
          const bool move = !started || !(top <= (tried ? m : m + RESCALE_AT));
          const float m_new = move ? top : m;
          if (started && __any_sync(0xffffffffu, move)) {   // both warps of the rows alike
            const float f = m_new == m ? 1.f : ex2(m - m_new);   // m = -infinity: 0
            l2.x *= f;
            l2.y *= f;
#pragma unroll 1
            for (int c = half * DH2; c < (half + 1) * DH2; c += 16) {
              float v[16];
              uint32_t w[16];
              ptx::tmem_ld(o_addr + c, v);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e] * f);
              ptx::tmem_st16(o_addr + c, w);
            }
          }
          m = m_new;
          const float ref = m == -INFINITY ? 0.f : m;
          const float2 nref2 = make_float2(-ref, -ref);
          l2 = __fadd2_rn(l2, weights([&](float2 v, int) { return __fadd2_rn(v, nref2); }));
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      }
      phase ^= 1u;
      started = true;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(p_bar(t));
    }
    if (ok) ok = ptx::mbar_wait_bounded(o_bar(t), 0, abort, WAIT_LIMIT_NS);
    if (!ok && !*abort) record_timeout(err, abort);
    if (warp_rows) {   // also after a wait that ran out: the pair's barriers stay matched
      float* xs = xch + t * 2 * TILE;
      pair_sync();     // the maxima have been read
      xs[half * TILE + lrow] = l2.x + l2.y;
      pair_sync();
      const float l = xs[lrow] + xs[TILE + lrow];
      ptx::tc_fence_after();
      const bool seen = started && l != 0.f;   // l is NaN where a score is
      const float inv = seen ? 1.f / l : 0.f;
      if (ok && plan.parts == 1) {
        bool finite = true;
        bf16* o = static_cast<bf16*>(a.out) + b * a.o_batch + i_own * a.o_token + (long)(hk * a.G + g_own) * a.o_head;
#pragma unroll 1
        for (int c = half * DH2; c < (half + 1) * DH2; c += 16) {
          float v[16];
          ptx::tmem_ld(o_addr + c, v);
          ptx::tmem_ld_wait();
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float y0 = seen ? v[e] * inv : 0.f, y1 = seen ? v[e + 1] * inv : 0.f;
            finite = finite && fabsf(y0) < INFINITY && fabsf(y1) < INFINITY;
            w[e / 2] = bf16x2_bits(y0, y1);
          }
          if (row_ok) {
            *reinterpret_cast<uint4*>(o + c) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(o + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        pair_sync();   // the sums have been read; both halves are written
        xs[half * TILE + lrow] = finite ? 0.f : 1.f;
        pair_sync();
        unsigned redo = half == 0 ? __ballot_sync(0xffffffffu, row_ok && xs[lrow] + xs[TILE + lrow] != 0.f) : 0u;
        while (redo) {
          const int src = __ffs(redo) - 1;
          redo &= redo - 1;
          row_by_warp<bf16, HD>(a, b, hk * a.G + __shfl_sync(0xffffffffu, g_own, src),
                                __shfl_sync(0xffffffffu, i_own, src));
        }
      } else if (ok) {
        // a part: the result over these keys and the log2 of its weight
        const long prow = ((long)b * a.Hkv + hk) * rows + r_own;
        const long n_rows = (long)a.B * a.Hkv * rows;
        float* o = plan.part_o + ((long)split * n_rows + prow) * HD;
        if (row_ok && half == 0) plan.part_lse[(long)split * n_rows + prow] = seen ? m + log2f(l) : -INFINITY;
#pragma unroll 1
        for (int c = half * DH2; c < (half + 1) * DH2; c += 16) {
          float v[16];
          ptx::tmem_ld(o_addr + c, v);
          ptx::tmem_ld_wait();
          if (row_ok && seen) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(o + c + e) = make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(*tmem_slot, C::COLS);
  }
}

// ---------------------------------------------------------------- bf16, few rows: keys on the MMA's rows
//
// At most NR query rows (all heads of a key head, all new tokens) against a range of keys:
//   S^T [128 keys x NR] = K Q^T,  thread = key: scores, masks, p;  P [NR][128 keys] in shared
//   memory;  O^T [dims x NR] += V^T P^T (V as an MN-major A operand, P K-major B).
// NR = 16: with more rows their maxima, one redux each, cost more than the other kernel's 128 rows
// (8 x 4 key heads, 40 rows over 8192 keys: 135 us against 35).
// The row maxima cross the 128 threads by redux and shared memory; the row sums stay with the
// threads until the end.  Bound by the K and V bytes.  Roles (192 threads): warp 0 TMA, warp
// 1 MMA, warps 2-5 softmax and output.
constexpr int F_THREADS = 192;
template <int HD, int NR>
struct FewCfg {
  static constexpr uint32_t Q_BYTES = NR * HD * 2;
  static constexpr uint32_t P_BYTES = NR * 256;
  static constexpr uint32_t KV_BYTES = TILE * HD * 2;
  static constexpr uint32_t HALF = TILE * 128;
  // two CTAs an SM, so that one's set-up and last tiles run under the other's loads
  static constexpr int NST = HD == 128 ? 3 : 6;
  static constexpr size_t BODY = Q_BYTES + P_BYTES + (size_t)NST * KV_BYTES;
  // rows' last key, position, document, slope; maxima (2 x 4 warps), references and factors (4 warps)
  static constexpr size_t ROWS = NR * 4 * (4 + 8 + 8 + 1);
  static constexpr size_t SMEM = 1024 + BODY + ROWS + (2 * NST + 8) * 8 + 16;
  static constexpr uint32_t COLS = 64;
  static_assert(NR == 16, "one TMEM load a thread, 3 * NR columns");
  static_assert(SMEM <= 232448 / 2 - 1024, "shared memory of two CTAs");
};

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

template <int HD, int NR>
__global__ void __launch_bounds__(F_THREADS, 2)
scored_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ ScoredAttention a, const __grid_constant__ ScoredPlan plan,
                  DevError* err) {
  using C = FewCfg<HD, NR>;
  constexpr int NST = C::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = ptx::smem_u32(smem), sP = sQ + C::Q_BYTES, sKV = sP + C::P_BYTES;
  uint8_t* gP = smem + C::Q_BYTES;
  int* row_last = reinterpret_cast<int*>(smem + C::BODY);
  int* row_pos = row_last + NR;
  int* row_doc = row_pos + NR;
  float* row_slope = reinterpret_cast<float*>(row_doc + NR);
  float* wmax = row_slope + NR;           // [2][4][NR]
  float* wref = wmax + 8 * NR;            // [4][2][NR]: a warp's references and factors
  int* bad = reinterpret_cast<int*>(wref + 8 * NR);   // [NR]
  uint64_t* bars = reinterpret_cast<uint64_t*>(bad + NR);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (NST + s); };
  auto s_bar = [&](int i) { return bar0 + 8u * (2 * NST + i); };
  const uint32_t p_bar = bar0 + 8u * (2 * NST + 2), o_bar = bar0 + 8u * (2 * NST + 3),
                 drain_bar = bar0 + 8u * (2 * NST + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NST + 5);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long id = blockIdx.x;
  const int split = (int)(id % plan.splits);
  id /= plan.splits;
  const int hk = (int)(id % a.Hkv);
  const int b = (int)(id / a.Hkv);
  const int rows = a.Sq * a.G;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    ptx::mbar_init(s_bar(0), 1);
    ptx::mbar_init(s_bar(1), 1);
    ptx::mbar_init(p_bar, 4);
    ptx::mbar_init(o_bar, 1);
    ptx::mbar_init(drain_bar, 1);
    ptx::fence_mbar_init();
    *abort = 0;
    ptx::tma_prefetch_desc(&tmK);
    ptx::tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::COLS);
    ptx::tmem_relinquish();
  }
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const SeqInfo seq = sequence_info(a, b);
  {
    constexpr int CH = HD / 8;
    const bf16* qb = static_cast<const bf16*>(a.q) + b * a.q_batch + (long)hk * a.G * a.q_head;
    for (int c = threadIdx.x; c < NR * CH; c += F_THREADS) {
      const int r = c / CH, ch = c % CH;
      uint4 val = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const int i = r / a.G, g = r - i * a.G;
        val = *reinterpret_cast<const uint4*>(qb + i * a.q_token + g * a.q_head + ch * 8);
      }
      *reinterpret_cast<uint4*>(smem + (ch >> 3) * (NR * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = val;
    }
    ptx::fence_proxy_async_smem();
    for (int r = threadIdx.x; r < NR; r += F_THREADS) {
      const bool ok = r < rows;
      const int i = ok ? r / a.G : 0, g = ok ? r - i * a.G : 0;
      row_last[r] = ok ? last_key(a, seq, (long)seq.start + i) : -1;
      row_pos[r] = bias_position((long)seq.start + i, row_last[r]);
      row_doc[r] = ok && a.q_doc ? a.q_doc[(long)b * a.Sq + i] : 0;
      row_slope[r] = ok && a.slopes ? a.slopes[hk * a.G + g] * LOG2E : 0.f;
      bad[r] = 0;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // keys of this CTA: up to the last one that any row sees (the last token's)
  const int key_end = 1 + row_last[rows - 1];
  const int jt_all = (key_end + TILE - 1) / TILE;
  const int jt0 = min(split * plan.tiles_per_split, jt_all), jt1 = min(jt0 + plan.tiles_per_split, jt_all);
  const int n_tiles = jt1 - jt0;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      long issued = 0;
      for (int n = 0; n < 2 * n_tiles; ++n) {
        ok = ptx::mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort, WAIT_LIMIT_NS);
        if (!ok) break;
        ptx::mbar_arrive_expect_tx(full_bar(stage), C::KV_BYTES);
#pragma unroll
        for (int hf = 0; hf < HD / 64; ++hf)
          ptx::tma_load_4d(sKV + stage * C::KV_BYTES + hf * C::HALF, n & 1 ? &tmV : &tmK, full_bar(stage), hf * 64,
                           (jt0 + (n >> 1)) * TILE, hk, b);
        ++issued;
        if (++stage == NST) { stage = 0; phase ^= 1u; }
      }
      if (!ok && !*abort) record_timeout(err, abort);
      // every copy issued has landed before the CTA leaves
      const long n = issued < NST ? issued : NST;
      volatile int never = 0;
      for (long i = 0; i < n; ++i) {
        if (--stage < 0) { stage = NST - 1; phase ^= 1u; }
        ptx::mbar_wait_bounded(full_bar(stage), phase, &never, WAIT_LIMIT_NS);
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc_s = ptx::idesc_bf16_f32(TILE, NR);
    const uint32_t idesc_o = ptx::idesc_bf16_f32(TILE, NR) | (1u << 15);
    // 64 dims: both 64-row halves of the MMA read the same values, the second half is not used
    constexpr uint32_t V_ATOM = HD == 128 ? C::HALF : 0u;
    const uint64_t q_desc = ptx::smem_desc_sw128(sQ), p_desc = ptx::smem_desc_sw128(sP);
    const uint64_t k_desc0 = ptx::smem_desc_sw128(sKV), v_desc0 = desc_mn(sKV, V_ATOM);
    bool ok = true;
    auto stage_of = [](int i) { return i % NST; };
    auto phase_of = [](int i) { return (uint32_t)((i / NST) & 1); };
    auto qk = [&](int n) {   // S^T of tile n into buffer n & 1, whose last use P V of tile n - 2 precedes
      ok = ptx::mbar_wait_bounded(full_bar(stage_of(2 * n)), phase_of(2 * n), abort, WAIT_LIMIT_NS);
      if (!ok) return;
      ptx::tc_fence_after();
      const uint64_t k = k_desc0 + (uint64_t)(stage_of(2 * n) * (C::KV_BYTES >> 4));
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          ptx::tc_mma_bf16(tmem_base + (n & 1) * NR, k + (uint64_t)(((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4),
                           q_desc + (uint64_t)(((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4), idesc_s, kk != 0);
        ptx::tc_commit(empty_bar(stage_of(2 * n)));
        ptx::tc_commit(s_bar(n & 1));
      }
      __syncwarp();
    };
    if (n_tiles > 0) qk(0);
    for (int n = 0; n < n_tiles && ok; ++n) {
      if (n + 1 < n_tiles) qk(n + 1);
      const int vs = stage_of(2 * n + 1);
      if (ok) ok = ptx::mbar_wait_bounded(full_bar(vs), phase_of(2 * n + 1), abort, WAIT_LIMIT_NS);
      if (!ok) break;
      const int v_rows = min(key_end - (jt0 + n) * TILE, TILE);
      if (v_rows < TILE) {   // value rows past the last key that a row of this CTA sees: 0, whatever they hold
        uint8_t* v = smem + C::Q_BYTES + C::P_BYTES + (size_t)vs * C::KV_BYTES;
        const int cnt = (TILE - v_rows) * 8;
        for (int c = lane; c < cnt * (HD / 64); c += 32) {
          const int hf = c / cnt, e = c % cnt;
          *reinterpret_cast<uint4*>(v + hf * C::HALF + (v_rows + e / 8) * 128 + (e & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      ok = ptx::mbar_wait_bounded(p_bar, n & 1, abort, WAIT_LIMIT_NS);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint64_t v = v_desc0 + (uint64_t)(vs * (C::KV_BYTES >> 4));
      const uint32_t more = n != 0 ? 1u : 0u;
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          ptx::tc_mma_bf16(tmem_base + 2 * NR, v + (uint64_t)(kk * (2048 >> 4)),
                           p_desc + (uint64_t)(((kk >> 2) * (NR * 128) + (kk & 3) * 32) >> 4), idesc_o,
                           kk != 0 ? 1u : more);
        ptx::tc_commit(empty_bar(vs));
        ptx::tc_commit(o_bar);
      }
      __syncwarp();
    }
    if (!ok && !*abort && lane == 0) record_timeout(err, abort);
    if (ptx::elect_one()) {
      ptx::tc_commit(drain_bar);
      volatile int never = 0;
      if (!ptx::mbar_wait_bounded(drain_bar, 0, &never, WAIT_LIMIT_NS)) record_timeout(err, abort);
    }
    __syncwarp();
  } else {
    // ---------------- softmax: this thread's key of the tile, then this thread's dim of the output
    const int quarter = warp & 3, sw = warp - 2, key = quarter * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_addr = tmem_base + lane_addr + 2 * NR;
    const bool cap = a.cap > 0.f, bias = a.slopes != nullptr, docs = a.q_doc != nullptr;
    const ScoredConst& cc = plan.k;
    const float sc = a.scale == 0.f ? 0.f : copysignf(cc.lin.x, a.scale);
    const int all_see = row_last[0];            // keys up to here are seen by every row
    float* refs = wref + sw * 2 * NR;
    float* facs = refs + NR;
    float my_ref = -INFINITY, l[NR];            // reference of row `lane`
#pragma unroll
    for (int r = 0; r < NR; ++r) l[r] = 0.f;
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      const int j = (jt0 + n) * TILE + key;
      const int kd = docs ? a.kv_doc[(long)b * a.Sk + min(j, a.Sk - 1)] : 0;
      // (after a wait that ran out the rest is gone through without waiting, so that the
      // barriers of the four warps stay matched)
      if (ok) ok = ptx::mbar_wait_bounded(s_bar(n & 1), (n >> 1) & 1, abort, WAIT_LIMIT_NS);
      ptx::tc_fence_after();
      float x[NR];
      const uint32_t s_addr = tmem_base + lane_addr + (n & 1) * NR;
      ptx::tmem_ld16_at<0>(s_addr, x);
      ptx::tmem_ld_wait();
      if (cap) {
        cap_scores(cc, x);
        if (a.scale <= 0.f) {   // the constants are those of |scale|
#pragma unroll
          for (int r = 0; r < NR; ++r) x[r] = a.scale < 0.f ? -x[r] : 0.f;
        }
      } else {
#pragma unroll
        for (int r = 0; r < NR; ++r) x[r] *= sc;
      }
      if (bias) {
#pragma unroll
        for (int r = 0; r < NR; ++r) x[r] = fmaf(-row_slope[r], fabsf((float)(row_pos[r] - j)), x[r]);
      }
      if ((jt0 + n) * TILE + TILE - 1 > all_see) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (j > row_last[r]) x[r] = -INFINITY;
      }
      if (docs) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (kd < 0 || row_doc[r] != kd) x[r] = -INFINITY;
      }
      // row maxima over the tile: within the warp, then over the four
      float* wm = wmax + (n & 1) * 4 * NR;
      float keep = -INFINITY;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float v = warp_max(x[r]);
        if (lane == r) keep = v;
      }
      if (lane < NR) wm[sw * NR + lane] = keep;
      asm volatile("bar.sync 1, 128;" ::: "memory");
      bool any = false;
      if (lane < NR) {
        const float top = fmaxf(fmaxf(wm[lane], wm[NR + lane]), fmaxf(wm[2 * NR + lane], wm[3 * NR + lane]));
        any = n == 0 || top > my_ref + RESCALE_AT;
        const float next = any ? fmaxf(my_ref, top) : my_ref;
        facs[lane] = next == my_ref ? 1.f : ex2(my_ref - next);
        my_ref = next;
        refs[lane] = next == -INFINITY ? 0.f : next;
      }
      any = __any_sync(0xffffffffu, any);   // the same in all four warps
      __syncwarp();
      if (n > 0) {
        if (ok) ok = ptx::mbar_wait_bounded(o_bar, (n - 1) & 1, abort, WAIT_LIMIT_NS);   // P and O of tile n - 1
        if (any) {
          ptx::tc_fence_after();
          float v[NR];
          uint32_t w[NR];
          ptx::tmem_ld(o_addr, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            w[r] = __float_as_uint(v[r] * facs[r]);
            l[r] *= facs[r];
          }
          ptx::tmem_st16(o_addr, w);
          ptx::tmem_st_wait();
        }
      }
      // weights: P row r, this key (K-major, 128-byte swizzle, 64 keys a block)
      uint8_t* pk = gP + (key >> 6) * (NR * 128) + (key & 7) * 2;
      const int ch = (key & 63) >> 3;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float w = ex2(x[r] - refs[r]);
        l[r] += w;
        *reinterpret_cast<bf16*>(pk + r * 128 + ((ch ^ (r & 7)) << 4)) = __float2bfloat16_rn(w);
      }
      ptx::fence_proxy_async_smem();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(p_bar);
    }
    // row sums over the threads: in the warp, then over the four (the maxima's first buffer)
    if (n_tiles > 0 && ok) ok = ptx::mbar_wait_bounded(o_bar, (n_tiles - 1) & 1, abort, WAIT_LIMIT_NS);
    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float v = l[r];
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == r) wmax[sw * NR + r] = v;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (!ok && !*abort) record_timeout(err, abort);
    {
      ptx::tc_fence_after();
      const long n_rows = (long)a.B * a.Hkv * rows, prow = ((long)b * a.Hkv + hk) * rows;
      const int d = quarter * 32 + lane;       // output dim (HD 64: quarters 0 and 1)
      if (plan.parts > 1) {
        for (int r = threadIdx.x - 64; r < rows; r += 128) {
          const float sum = wmax[r] + wmax[NR + r] + wmax[2 * NR + r] + wmax[3 * NR + r];
          const float ref = wref[r];           // any warp's copy
          plan.part_lse[(long)split * n_rows + prow + r] = n_tiles > 0 && sum != 0.f ? ref + log2f(sum) : -INFINITY;
        }
      }
      float v[NR];
      ptx::tmem_ld(o_addr, v);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (r < rows && d < HD) {
          const float sum = wmax[r] + wmax[NR + r] + wmax[2 * NR + r] + wmax[3 * NR + r];
          const bool seen = n_tiles > 0 && sum != 0.f;
          const float y = seen ? v[r] / sum : 0.f;
          if (plan.parts > 1) {
            if (seen) plan.part_o[((long)split * n_rows + prow + r) * HD + d] = y;
          } else {
            const int i = r / a.G, g = r - i * a.G;
            static_cast<bf16*>(a.out)[b * a.o_batch + i * a.o_token + (long)(hk * a.G + g) * a.o_head + d] =
                __float2bfloat16_rn(y);
            if (!(fabsf(y) < INFINITY)) bad[r] = 1;
          }
        }
      }
      if (plan.parts == 1) {
        asm volatile("bar.sync 1, 128;" ::: "memory");
        for (int r = sw; r < rows; r += 4)
          if (bad[r]) row_by_warp<bf16, HD>(a, b, hk * a.G + r % a.G, r / a.G);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, C::COLS);
  }
}

// ---------------------------------------------------------------- fp32
//
// At most 16 rows (new tokens over a cache) on the FMA units, whose rate such a call does not need:
// a CTA of 128 threads takes 16 rows and walks key tiles of 64; thread (row group,
// column group) holds 2 x 4 scores and 2 x HD / 16 outputs in registers.  Rows are padded by
// 16 bytes, so that the eight lanes of a load's phase read different banks; the weights take
// the keys' place.  A row's statistics live in the 16 lanes that share it.  (2 x 32 heads over
// 8000 keys, 8 key heads: 58 us for 131 MB, 35 % of the copy rate: keys and values have one
// buffer each, which is filled again only after the whole CTA has read both.)
constexpr int FT = 64, TM = 2, NT = 128;
template <int HD>
struct F32Cfg {
  static constexpr int CG = FT / 4, RG = NT / CG, BM = RG * TM, LD = HD + 4, LP = FT + 4;
  static_assert(BM * (FT + 4) <= FT * (HD + 4), "the weights fit in the keys' place");
  static constexpr size_t SMEM = (size_t)(BM * LD + 2 * FT * LD) * 4;
};

template <int HD>
__global__ void __launch_bounds__(NT, 2) scored_f32_kernel(const __grid_constant__ ScoredAttention a,
                                                            const __grid_constant__ ScoredPlan plan) {
  using C = F32Cfg<HD>;
  constexpr int CG = C::CG, RG = C::RG, BM = C::BM, LD = C::LD, LP = C::LP;
  constexpr int ND = HD / (4 * CG);   // float4 of outputs per row and thread
  extern __shared__ float fsm[];
  float* sQ = fsm;
  float* sK = sQ + BM * LD;
  float* sP = sK;
  float* sV = sK + FT * LD;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  long id = blockIdx.x;
  const int split = (int)(id % plan.splits);
  id /= plan.splits;
  const int hk = (int)(id % a.Hkv);
  id /= a.Hkv;
  const int b = (int)(id % a.B);
  const int rb = plan.row_blocks - 1 - (int)(id / a.B);
  const int rows = a.Sq * a.G, row0 = rb * BM;
  const SeqInfo seq = sequence_info(a, b);
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
  const int row_end = min(row0 + BM, rows);

  const int key_end = 1 + last_key(a, seq, (long)seq.start + (row_end - 1) / a.G);
  const int jt_all = (key_end + FT - 1) / FT;
  const int jt0 = min(split * plan.tiles_per_split, jt_all), jt1 = min(jt0 + plan.tiles_per_split, jt_all);
  const bool docs = a.q_doc != nullptr;
  const float* kb = static_cast<const float*>(a.k) + b * a.k_batch + hk * a.k_head;
  const float* vb = static_cast<const float*>(a.v) + b * a.v_batch + hk * a.v_head;
  // one tile's rows into shared memory, those past the last key that a row sees as zeros
  auto fetch = [&](float* dst, const float* src, long stride, int j0) {
    const uint32_t d0 = ptx::smem_u32(dst);
#pragma unroll 4
    for (int c = threadIdx.x; c < FT * (HD / 4); c += NT) {
      const int lj = c / (HD / 4), ch = c % (HD / 4), j = j0 + lj;
      const bool in = j < key_end;
      ptx::cp_async_16_zfill(d0 + (uint32_t)(lj * LD + ch * 4) * 4, src + (in ? j : 0) * stride + ch * 4, in);
    }
    ptx::cp_async_commit();
  };
  if (jt0 < jt1) {
    fetch(sK, kb, a.k_token, jt0 * FT);
    fetch(sV, vb, a.v_token, jt0 * FT);
  }
  const float* qb = static_cast<const float*>(a.q) + b * a.q_batch + (long)hk * a.G * a.q_head;
  for (int c = threadIdx.x; c < BM * (HD / 4); c += NT) {
    const int lr = c / (HD / 4), ch = c % (HD / 4), r = row0 + lr;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      const int i = r / a.G, g = r - i * a.G;
      v = *reinterpret_cast<const float4*>(qb + i * a.q_token + g * a.q_head + ch * 4);
    }
    *reinterpret_cast<float4*>(sQ + lr * LD + ch * 4) = v;
  }
  // row u of this thread: local row rg + 8 u
  int last[TM], pos[TM], doc[TM];
  float slope[TM], m[TM], l[TM];
  float4 o[TM][ND];
#pragma unroll
  for (int u = 0; u < TM; ++u) {
    const int r = row0 + rg + RG * u;
    const bool ok = r < rows;
    const int i = ok ? r / a.G : 0, g = ok ? r - i * a.G : 0;
    last[u] = ok ? last_key(a, seq, (long)seq.start + i) : -1;
    pos[u] = bias_position((long)seq.start + i, last[u]);
    doc[u] = ok && a.q_doc ? a.q_doc[(long)b * a.Sq + i] : 0;
    slope[u] = ok && a.slopes ? a.slopes[hk * a.G + g] * LOG2E : 0.f;
    m[u] = -INFINITY;
    l[u] = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[u][d] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int jt = jt0; jt < jt1; ++jt) {
    const int j0 = jt * FT;
    asm volatile("cp.async.wait_group 1;" ::: "memory");   // the keys
    __syncthreads();
    // scores of keys cg + 16 w, two key halves of the products a register pair
    float2 acc[TM][4];
#pragma unroll
    for (int u = 0; u < TM; ++u)
#pragma unroll
      for (int w = 0; w < 4; ++w) acc[u][w] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int d = 0; d < HD; d += 4) {
      float4 k4[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) k4[w] = *reinterpret_cast<const float4*>(sK + (cg + CG * w) * LD + d);
#pragma unroll
      for (int u = 0; u < TM; ++u) {
        const float4 q4 = *reinterpret_cast<const float4*>(sQ + (rg + RG * u) * LD + d);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          acc[u][w] = __ffma2_rn(make_float2(q4.x, q4.y), make_float2(k4[w].x, k4[w].y), acc[u][w]);
          acc[u][w] = __ffma2_rn(make_float2(q4.z, q4.w), make_float2(k4[w].z, k4[w].w), acc[u][w]);
        }
      }
    }
    int kd[4];
#pragma unroll
    for (int w = 0; w < 4; ++w)
      kd[w] = docs && j0 + cg + CG * w < a.Sk ? a.kv_doc[(long)b * a.Sk + j0 + cg + CG * w] : -1;
    __syncthreads();   // all have read the keys: the weights take their place
#pragma unroll
    for (int u = 0; u < TM; ++u) {
      float x[4], top = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int j = j0 + cg + CG * w;
        float y = (acc[u][w].x + acc[u][w].y) * a.scale;
        y = a.cap > 0.f ? a.cap * tanhf(y / a.cap) * LOG2E : y * LOG2E;
        if (a.slopes) y = fmaf(-slope[u], fabsf((float)(pos[u] - j)), y);
        const bool seen = j <= last[u] && (!docs || (doc[u] >= 0 && kd[w] == doc[u]));
        x[w] = seen ? y : -INFINITY;
        top = fmaxf(top, x[w]);
      }
#pragma unroll
      for (int s = 1; s < CG; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      const float mn = fmaxf(m[u], top), ref = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[u] - ref);
      m[u] = mn;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float p = exp2f(x[w] - ref);
        sum += p;
        sP[(rg + RG * u) * LP + cg + CG * w] = p;
      }
      l[u] = l[u] * f + sum;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        o[u][d].x *= f; o[u][d].y *= f; o[u][d].z *= f; o[u][d].w *= f;
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");   // the values
    __syncthreads();
    // outputs: dims 4 cg + 64 d
#pragma unroll 1
    for (int j = 0; j < FT; j += 4) {
      float4 v4[4][ND];
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int d = 0; d < ND; ++d) v4[w][d] = *reinterpret_cast<const float4*>(sV + (j + w) * LD + 4 * CG * d + 4 * cg);
#pragma unroll
      for (int u = 0; u < TM; ++u) {
        const float4 p4 = *reinterpret_cast<const float4*>(sP + (rg + RG * u) * LP + j);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float p = w == 0 ? p4.x : w == 1 ? p4.y : w == 2 ? p4.z : p4.w;
          const float2 pp = make_float2(p, p);
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const float2 lo = __ffma2_rn(pp, make_float2(v4[w][d].x, v4[w][d].y), make_float2(o[u][d].x, o[u][d].y));
            const float2 hi = __ffma2_rn(pp, make_float2(v4[w][d].z, v4[w][d].w), make_float2(o[u][d].z, o[u][d].w));
            o[u][d] = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
        }
      }
    }
    __syncthreads();   // all have read weights and values: the next tile may come
    if (jt + 1 < jt1) {
      fetch(sK, kb, a.k_token, j0 + FT);
      fetch(sV, vb, a.v_token, j0 + FT);
    }
  }
  const long n_rows = (long)a.B * a.Hkv * rows, prow = ((long)b * a.Hkv + hk) * rows;
#pragma unroll
  for (int u = 0; u < TM; ++u) {
    const int r = row0 + rg + RG * u;
    const bool row_ok = r < rows;
    float sum = l[u];
#pragma unroll
    for (int s = 1; s < CG; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    const bool seen = sum != 0.f;
    const int i = row_ok ? r / a.G : 0, g = row_ok ? r - i * a.G : 0;
    bool finite = true;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const float4 y = seen ? make_float4(o[u][d].x / sum, o[u][d].y / sum, o[u][d].z / sum, o[u][d].w / sum)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
      finite = finite && fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY && fabsf(y.w) < INFINITY;
      if (row_ok) {
        if (plan.parts == 1)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + b * a.o_batch + i * a.o_token +
                                     (long)(hk * a.G + g) * a.o_head + 4 * CG * d + 4 * cg) = y;
        else if (seen)
          *reinterpret_cast<float4*>(plan.part_o + ((long)split * n_rows + prow + r) * HD + 4 * CG * d + 4 * cg) = y;
      }
    }
    if (plan.parts == 1) {
      unsigned redo = __ballot_sync(0xffffffffu, row_ok && !finite);
      while (redo) {
        const int src = __ffs(redo) - 1;
        redo &= ~(((1u << CG) - 1u) << (src / CG * CG));   // the lanes of that row
        row_by_warp<float, HD>(a, b, hk * a.G + __shfl_sync(0xffffffffu, g, src), __shfl_sync(0xffffffffu, i, src));
      }
    } else if (row_ok && cg == 0) {
      plan.part_lse[(long)split * n_rows + prow + r] = seen ? m[u] + log2f(sum) : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- fp32 on the tensor cores
//
// For more than 16 rows the fp32 path runs on the bf16 tensor cores with every operand in
// three bf16 parts, x = x0 + x1 + x2, each the rounding of what the parts before leave: 24
// bits, as fp32 has.  Of the nine products of two such sums the six down to 2^-16 are formed
// (those left out are below 2^-24 of the largest) and added in fp32, smallest first.  Six
// MMAs at over 16 times the FMA units' rate: 16 heads x 1000 tokens 65 us against 262 in register
// tiles on the FMA units, 32 x 8 heads x 151 tokens 84 against 137 (two CTAs a head, the
// second with 23 rows: set-up and latencies).  A warp whose rows see none of its keys, or which has
// no rows, skips the scores (that call 88 -> 84 us; the bf16 kernel, short of registers, got
// slower by it: 16 heads x 4096 causal 78 -> 88 us).
// One 128-row tile a CTA, key tiles of 64.  Roles (544 threads): warps 0-7 softmax and output
// (two threads a row, 32 keys each), warps 8-11 and 12-15 load keys and values, split them and
// write them as the MMAs read them (128-byte swizzle), warp 16 MMA.  TMEM: two score buffers
// of 64 columns, the three weight parts in 32 each, the output.
constexpr int S3_THREADS = 544;
constexpr int S3_KEYS = 64;
template <int HD>
struct Split3Cfg {
  static constexpr uint32_t Q_PART = TILE * HD * 2, KV_PART = S3_KEYS * HD * 2;
  static constexpr uint32_t Q_HALF = TILE * 128, KV_HALF = S3_KEYS * 128;   // 64 dims
  static constexpr size_t BODY = 3 * Q_PART + 6 * KV_PART;
  // exchange of maxima and sums (2 turns x 2 halves x 128 rows), documents (8 warps x 32 keys)
  static constexpr size_t XCH = 4 * TILE * 4 + 8 * 32 * 4;
  static constexpr size_t SMEM = 1024 + BODY + XCH + 16 * 8 + 16;
  static_assert(SMEM <= 232448, "shared memory");
};
// (part of the first operand, part of the second), smallest products first
__device__ constexpr int S3_A[6] = {2, 0, 1, 1, 0, 0}, S3_B[6] = {0, 2, 1, 0, 1, 0};

// Eight floats in three bf16 parts.
__device__ __forceinline__ void split3(const float (&v)[8], uint4 (&out)[3]) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = bf16x2_bits(r[2 * e], r[2 * e + 1]);
      r[2 * e] -= __uint_as_float(w[e] << 16);
      r[2 * e + 1] -= __uint_as_float(w[e] & 0xffff0000u);
    }
    out[t] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int HD>
__global__ void __launch_bounds__(S3_THREADS, 1)
scored_split3_kernel(const __grid_constant__ ScoredAttention a, const __grid_constant__ ScoredPlan plan, DevError* err) {
  using C = Split3Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = ptx::smem_u32(smem), sK = sQ + 3 * C::Q_PART, sV = sK + 3 * C::KV_PART;
  float* xch = reinterpret_cast<float*>(smem + C::BODY);
  int* docs_smem = reinterpret_cast<int*>(xch + 4 * TILE);
  uint64_t* bars = reinterpret_cast<uint64_t*>(docs_smem + 8 * 32);
  const uint32_t bar0 = ptx::smem_u32(bars);
  // full (loaders' warps), empty (MMA) of keys and values; scores; weights; output; drain
  const uint32_t k_full = bar0, k_empty = bar0 + 8, v_full = bar0 + 16, v_empty = bar0 + 24, p_bar = bar0 + 48,
                 o_bar = bar0 + 56, drain_bar = bar0 + 64, q_bar = bar0 + 72;
  auto s_bar = [&](int i) { return bar0 + 32u + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 10);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t tmem_base = 0, P_COL = 128, O_COL = 256;   // all columns are this CTA's

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long id = blockIdx.x;
  const int split = (int)(id % plan.splits);
  id /= plan.splits;
  const int hk = (int)(id % a.Hkv);
  id /= a.Hkv;
  const int b = (int)(id % a.B);
  const int rb = plan.row_blocks - 1 - (int)(id / a.B);
  const int rows = a.Sq * a.G, row0 = rb * TILE;
  if (threadIdx.x == 0) {
    ptx::mbar_init(k_full, 4);
    ptx::mbar_init(k_empty, 1);
    ptx::mbar_init(v_full, 4);
    ptx::mbar_init(v_empty, 1);
    ptx::mbar_init(s_bar(0), 1);
    ptx::mbar_init(s_bar(1), 1);
    ptx::mbar_init(p_bar, 8);
    ptx::mbar_init(o_bar, 1);
    ptx::mbar_init(drain_bar, 1);
    ptx::mbar_init(q_bar, 8);
    ptx::fence_mbar_init();
    *abort = 0;
  }
  if (warp == 16) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const SeqInfo seq = sequence_info(a, b);
  constexpr int CH = HD / 8;                                // 8-dim chunks of a row
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const int row_last = min(row0 + TILE, rows) - 1;
  const int key_end = 1 + last_key(a, seq, (long)seq.start + row_last / a.G);
  const int jt_all = (key_end + S3_KEYS - 1) / S3_KEYS;
  const int jt0 = min(split * plan.tiles_per_split, jt_all), jt1 = min(jt0 + plan.tiles_per_split, jt_all);
  const int n_tiles = jt1 - jt0;

  if (warp >= 8 && warp < 16) {
    // ---------------- loads: one operand's tile, split into its parts
    const bool values = warp >= 12;
    const int l = threadIdx.x - (values ? 384 : 256);
    const long stride = values ? a.v_token : a.k_token;
    const float* src = values ? static_cast<const float*>(a.v) + b * a.v_batch + hk * a.v_head
                              : static_cast<const float*>(a.k) + b * a.k_batch + hk * a.k_head;
    uint8_t* dst = smem + 3 * C::Q_PART + (values ? 3 * C::KV_PART : 0);
    const uint32_t full = values ? v_full : k_full, empty = values ? v_empty : k_empty;
    constexpr int TASKS = S3_KEYS * CH / 128;
    bool ok = true;
    for (int n = 0; n < n_tiles && ok; ++n) {
      const int j0 = (jt0 + n) * S3_KEYS;
      float4 lo[TASKS], hi[TASKS];
#pragma unroll
      for (int u = 0; u < TASKS; ++u) {
        const int task = l + 128 * u, j = j0 + task / CH;
        lo[u] = hi[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < key_end) {   // the last key that a row of this CTA sees; zeros behind it
          const float* p = src + j * stride + (task % CH) * 8;
          lo[u] = *reinterpret_cast<const float4*>(p);
          hi[u] = *reinterpret_cast<const float4*>(p + 4);
        }
      }
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(empty, (n & 1) ^ 1u, abort, WAIT_LIMIT_NS));
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < TASKS; ++u) {
        const int task = l + 128 * u, r = task / CH, ch = task % CH;
        const float v[8] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w, hi[u].x, hi[u].y, hi[u].z, hi[u].w};
        uint4 w[3];
        split3(v, w);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          *reinterpret_cast<uint4*>(dst + t * C::KV_PART + (ch >> 3) * C::KV_HALF + r * 128 +
                                    (((ch & 7) ^ (r & 7)) << 4)) = w[t];
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full);
    }
    if (!ok && !*abort && lane == 0) record_timeout(err, abort);
  } else if (warp == 16) {
    // ---------------- MMA: S of a tile ahead of P V of the one before
    const uint32_t idesc_s = ptx::idesc_bf16_f32(TILE, S3_KEYS);
    const uint32_t idesc_o = ptx::idesc_bf16_f32(TILE, HD) | (1u << 16);
    const uint64_t d_q = ptx::smem_desc_sw128(sQ), d_k = ptx::smem_desc_sw128(sK), d_v = desc_mn(sV, C::KV_HALF);
    const uint32_t k_hi = (uint32_t)(d_k >> 32), v_hi = (uint32_t)(d_v >> 32);
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t ph) {
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, ph, abort, WAIT_LIMIT_NS));
      return ok;
    };
    auto qk = [&](int n) {
      if (!wait(k_full, n & 1)) return;
      ptx::tc_fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int t = 0; t < 6; ++t) {
          const uint32_t q = (uint32_t)d_q + S3_A[t] * (C::Q_PART >> 4), k = (uint32_t)d_k + S3_B[t] * (C::KV_PART >> 4);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            ptx::tc_mma_bf16_lo(tmem_base + (n & 1) * S3_KEYS, q + (((kk >> 2) * C::Q_HALF + (kk & 3) * 32) >> 4),
                                k + (((kk >> 2) * C::KV_HALF + (kk & 3) * 32) >> 4), k_hi, idesc_s, (t | kk) != 0);
        }
        ptx::tc_commit(s_bar(n & 1));
        ptx::tc_commit(k_empty);
      }
      __syncwarp();
    };
    if (n_tiles > 0 && wait(q_bar, 0)) qk(0);
    for (int n = 0; n < n_tiles && ok; ++n) {
      if (n + 1 < n_tiles) qk(n + 1);
      if (!ok || !wait(v_full, n & 1) || !wait(p_bar, n & 1)) break;
      ptx::tc_fence_after();
      const uint32_t more = n != 0 ? 1u : 0u;
      if (ptx::elect_one()) {
#pragma unroll
        for (int t = 0; t < 6; ++t) {
          const uint32_t v = (uint32_t)d_v + S3_B[t] * (C::KV_PART >> 4);
#pragma unroll
          for (int kk = 0; kk < S3_KEYS / 16; ++kk)
            ptx::tc_mma_bf16_ta_lo(tmem_base + O_COL, tmem_base + P_COL + S3_A[t] * 32 + kk * 8, v + kk * (2048 >> 4), v_hi,
                                   idesc_o, (t | kk) != 0 ? 1u : more);
        }
        ptx::tc_commit(v_empty);
        ptx::tc_commit(o_bar);
      }
      __syncwarp();
    }
    if (!ok && !*abort && lane == 0) record_timeout(err, abort);
    if (ptx::elect_one()) {
      ptx::tc_commit(drain_bar);
      volatile int never = 0;
      if (!ptx::mbar_wait_bounded(drain_bar, 0, &never, WAIT_LIMIT_NS)) record_timeout(err, abort);
    }
    __syncwarp();
  } else {
    // ---------------- queries in their parts, while the first keys and values are on their way
    {
      const float* qb = static_cast<const float*>(a.q) + b * a.q_batch + (long)hk * a.G * a.q_head;
#pragma unroll 4
      for (int c = threadIdx.x; c < TILE * CH; c += 256) {
        const int lr = c / CH, ch = c % CH, r = row0 + lr;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < rows) {
          const int i = r / a.G, g = r - i * a.G;
          const float* q = qb + i * a.q_token + g * a.q_head + ch * 8;
          const float4 x = *reinterpret_cast<const float4*>(q), y = *reinterpret_cast<const float4*>(q + 4);
          v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        }
        uint4 w[3];
        split3(v, w);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          *reinterpret_cast<uint4*>(smem + t * C::Q_PART + (ch >> 3) * C::Q_HALF + lr * 128 +
                                    (((ch & 7) ^ (lr & 7)) << 4)) = w[t];
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(q_bar);
    }
    // ---------------- softmax and output: row lrow, keys 32 half .. of a tile, dims HD / 2 half ..
    const int quarter = warp & 3, half = warp >> 2, lrow = quarter * 32 + lane;
    constexpr int KH = S3_KEYS / 2, DH2 = HD / 2;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t o_addr = tmem_base + lane_addr + O_COL;
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory"); };
    const int r_own = row0 + lrow;
    const bool row_ok = r_own < rows;
    const int i_own = row_ok ? r_own / a.G : 0, g_own = row_ok ? r_own - i_own * a.G : 0;
    const int last = row_ok ? last_key(a, seq, (long)seq.start + i_own) : -1;
    const int p = bias_position((long)seq.start + i_own, last);
    const bool docs = a.q_doc != nullptr;
    int qdoc = docs && row_ok ? a.q_doc[(long)b * a.Sq + i_own] : 0;
    // documents of this warp's rows: from docs_lo to docs_hi (lo > hi: none)
    const int docs_lo = __reduce_min_sync(0xffffffffu, row_ok && qdoc >= 0 ? qdoc : INT_MAX);
    const int docs_hi = __reduce_max_sync(0xffffffffu, row_ok ? qdoc : -1);
    qdoc = qdoc < 0 ? -2 : qdoc;   // a key in no document is staged as -1
    const float slope2 = a.slopes && row_ok ? a.slopes[hk * a.G + g_own] * LOG2E : 0.f;
    int* dbuf = docs_smem + warp * 32;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      const int j0 = (jt0 + n) * S3_KEYS + half * KH;
      // no row of this warp sees any of its keys (or it has no rows): their weights are 0 and
      // nothing is computed
      bool none = __all_sync(0xffffffffu, j0 > last);
      if (docs) {
        __syncwarp();   // the documents before have been read
        const int d = max(a.kv_doc[(long)b * a.Sk + min(j0 + lane, a.Sk - 1)], -1);
        dbuf[lane] = d;
        const int lo = __reduce_min_sync(0xffffffffu, d < 0 ? INT_MAX : d), hi = __reduce_max_sync(0xffffffffu, d);
        none = none || lo > docs_hi || hi < docs_lo;
        __syncwarp();
      }
      // (after a wait that ran out the rest is gone through without waiting, so that the
      // barriers of the warp pairs stay matched)
      if (ok) ok = ptx::mbar_wait_bounded(s_bar(n & 1), (n >> 1) & 1, abort, WAIT_LIMIT_NS);
      ptx::tc_fence_after();
      float x[KH];
      float top = -INFINITY;
      if (!none) {
        ptx::tmem_ld32(tmem_base + lane_addr + (n & 1) * S3_KEYS + half * KH, x);
        ptx::tmem_ld_wait();
        if (a.cap > 0.f) {
#pragma unroll
          for (int e = 0; e < KH; ++e) x[e] = a.cap * tanhf(x[e] * a.scale / a.cap) * LOG2E;
        } else {
#pragma unroll
          for (int e = 0; e < KH; ++e) x[e] = x[e] * a.scale * LOG2E;
        }
        if (a.slopes) {
#pragma unroll
          for (int e = 0; e < KH; ++e) x[e] = fmaf(-slope2, fabsf((float)(p - j0 - e)), x[e]);
        }
        if (!__all_sync(0xffffffffu, j0 + KH - 1 <= last)) {
#pragma unroll
          for (int e = 0; e < KH; ++e)
            if (j0 + e > last) x[e] = -INFINITY;
        }
        if (docs) {
#pragma unroll
          for (int e = 0; e < KH; ++e)
            if (dbuf[e] != qdoc) x[e] = -INFINITY;
        }
        top = max_of(x);
      }
      float* xm = xch + (n & 1) * 2 * TILE;
      xm[half * TILE + lrow] = top;
      pair_sync();
      top = max3(xm[lrow], xm[TILE + lrow], m);
      const bool move = n == 0 || !(top <= m + RESCALE_AT);
      const float m_new = move ? top : m;
      if (n > 0) {
        if (ok) ok = ptx::mbar_wait_bounded(o_bar, (n - 1) & 1, abort, WAIT_LIMIT_NS);   // weights and output of tile n - 1
        if (__any_sync(0xffffffffu, move)) {
          ptx::tc_fence_after();
          const float f = m_new == m ? 1.f : exp2f(m - m_new);   // m = -infinity: 0
          l *= f;
#pragma unroll 1
          for (int c = half * DH2; c < (half + 1) * DH2; c += 16) {
            float v[16];
            uint32_t w[16];
            ptx::tmem_ld(o_addr + c, v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e] * f);
            ptx::tmem_st16(o_addr + c, w);
          }
        }
      }
      m = m_new;
      const float ref = m == -INFINITY ? 0.f : m;
      if (none) {
        const uint32_t w[16] = {};
#pragma unroll
        for (int t = 0; t < 3; ++t) ptx::tmem_st16(tmem_base + lane_addr + P_COL + t * 32 + half * 16, w);
      } else {
#pragma unroll
        for (int e = 0; e < KH; ++e) {
          x[e] = exp2f(x[e] - ref);
          l += x[e];
        }
#pragma unroll
        for (int t = 0; t < 3; ++t) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            w[e] = bf16x2_bits(x[2 * e], x[2 * e + 1]);
            x[2 * e] -= __uint_as_float(w[e] << 16);
            x[2 * e + 1] -= __uint_as_float(w[e] & 0xffff0000u);
          }
          ptx::tmem_st16(tmem_base + lane_addr + P_COL + t * 32 + half * 16, w);
        }
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(p_bar);
    }
    if (ok && n_tiles > 0) ok = ptx::mbar_wait_bounded(o_bar, (n_tiles - 1) & 1, abort, WAIT_LIMIT_NS);
    if (!ok && !*abort) record_timeout(err, abort);
    pair_sync();   // the maxima have been read
    xch[half * TILE + lrow] = l;
    pair_sync();
    l = xch[lrow] + xch[TILE + lrow];
    ptx::tc_fence_after();
    const bool seen = n_tiles > 0 && l != 0.f;   // l is NaN where a score is
    bool finite = true;
    const long n_rows = (long)a.B * a.Hkv * rows, prow = ((long)b * a.Hkv + hk) * rows + r_own;
    float* o = plan.part_o + ((long)split * n_rows + prow) * HD;
    if (plan.parts == 1)
      o = static_cast<float*>(a.out) + b * a.o_batch + i_own * a.o_token + (long)(hk * a.G + g_own) * a.o_head;
    const bool write = ok && row_ok && (plan.parts == 1 || seen);
    const float inv = 1.f / l;
#pragma unroll 1
    for (int c = half * DH2; c < (half + 1) * DH2; c += 16) {
      float v[16];
      ptx::tmem_ld(o_addr + c, v);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        v[e] = seen ? v[e] * inv : 0.f;
        finite = finite && fabsf(v[e]) < INFINITY;
      }
      if (write) {
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4*>(o + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
    if (plan.parts == 1) {
      pair_sync();   // the sums have been read; both halves are written
      xch[half * TILE + lrow] = finite ? 0.f : 1.f;
      pair_sync();
      unsigned redo = half == 0 && ok ? __ballot_sync(0xffffffffu, row_ok && xch[lrow] + xch[TILE + lrow] != 0.f) : 0u;
      while (redo) {
        const int src = __ffs(redo) - 1;
        redo &= redo - 1;
        row_by_warp<float, HD>(a, b, hk * a.G + __shfl_sync(0xffffffffu, g_own, src), __shfl_sync(0xffffffffu, i_own, src));
      }
    } else if (row_ok && half == 0) {
      plan.part_lse[(long)split * n_rows + prow] = seen ? m + log2f(l) : -INFINITY;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(*tmem_slot, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- join of the parts
// o = sum 2^(lse - max) o_part / sum 2^(lse - max).  One CTA a row: warp w takes parts w, w + 4, ...
template <typename T, int HD>
__global__ void __launch_bounds__(128) scored_join_kernel(const __grid_constant__ ScoredAttention a,
                                                          const ScoredPlan plan) {
  constexpr int PER = HD / 32;
  __shared__ float sm[4], st[4], so[4][HD];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int rows = a.Sq * a.G;
  const long n_rows = (long)a.B * a.Hkv * rows;
  const long r = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int s = threadIdx.x; s < plan.parts; s += 128) top = fmaxf(top, plan.part_lse[s * n_rows + r]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sm[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f, o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int s = warp; s < plan.parts; s += 4) {
    const float w = exp2f(plan.part_lse[s * n_rows + r] - ref);
    float v[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) v[e] = 0.f;
    if (w != 0.f) {   // a part that saw nothing has no values
      const float* po = plan.part_o + (s * n_rows + r) * HD + lane * PER;
#pragma unroll
      for (int e = 0; e < PER; ++e) v[e] = po[e];
    }
    total += w;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = fmaf(w, v[e], o[e]);
  }
  if (lane == 0) st[warp] = total;
#pragma unroll
  for (int e = 0; e < PER; ++e) so[warp][lane * PER + e] = o[e];
  __syncthreads();
  if (warp != 0) return;
  total = st[0] + st[1] + st[2] + st[3];
  const int rr = (int)(r % rows), i = rr / a.G, g = rr - i * a.G;
  const int bh = (int)(r / rows), hk = bh % a.Hkv, b = bh / a.Hkv, hq = hk * a.G + g;
  T* out = static_cast<T*>(a.out) + b * a.o_batch + i * a.o_token + hq * a.o_head + lane * PER;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int d = lane * PER + e;
    const float y = total == 0.f ? 0.f : (so[0][d] + so[1][d] + so[2][d] + so[3][d]) / total;
    finite = finite && fabsf(y) < INFINITY;
    out[e] = from_f<T>(y);
  }
  if (!__all_sync(0xffffffffu, finite)) row_by_warp<T, HD>(a, b, hq, i);
}

// The same with one warp a row, for few parts: all of them in flight at once.
constexpr int JOIN_WARP_PARTS = 8;
template <typename T, int HD>
__global__ void __launch_bounds__(128) scored_join_warp_kernel(const __grid_constant__ ScoredAttention a,
                                                               const __grid_constant__ ScoredPlan plan) {
  constexpr int PER = HD / 32;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int rows = a.Sq * a.G, lane = threadIdx.x & 31;
  const long n_rows = (long)a.B * a.Hkv * rows, r = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= n_rows) return;
  const float mine = lane < plan.parts ? plan.part_lse[lane * n_rows + r] : -INFINITY;
  float top = mine;
#pragma unroll
  for (int o = 4; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  top = __shfl_sync(0xffffffffu, top, 0);
  const float w_mine = exp2f(mine - (top == -INFINITY ? 0.f : top));
  float w[JOIN_WARP_PARTS], v[JOIN_WARP_PARTS][PER], total = 0.f, y[PER];
#pragma unroll
  for (int s = 0; s < JOIN_WARP_PARTS; ++s) {
    w[s] = __shfl_sync(0xffffffffu, w_mine, s);
    const float* po = plan.part_o + (s * n_rows + r) * HD + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) v[s][e] = 0.f;
    if (s < plan.parts && w[s] != 0.f) {   // a part that saw nothing has no values
      if constexpr (PER == 4) {
        const float4 t = *reinterpret_cast<const float4*>(po);
        v[s][0] = t.x; v[s][1] = t.y; v[s][2] = t.z; v[s][3] = t.w;
      } else {
        const float2 t = *reinterpret_cast<const float2*>(po);
        v[s][0] = t.x; v[s][1] = t.y;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) y[e] = 0.f;
#pragma unroll
  for (int s = 0; s < JOIN_WARP_PARTS; ++s) {
    if (s < plan.parts) total += w[s];
#pragma unroll
    for (int e = 0; e < PER; ++e) y[e] = fmaf(s < plan.parts ? w[s] : 0.f, v[s][e], y[e]);
  }
  const int rr = (int)(r % rows), i = rr / a.G, g = rr - i * a.G;
  const int bh = (int)(r / rows), hk = bh % a.Hkv, b = bh / a.Hkv, hq = hk * a.G + g;
  T* out = static_cast<T*>(a.out) + b * a.o_batch + i * a.o_token + hq * a.o_head + lane * PER;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    y[e] = total == 0.f ? 0.f : y[e] / total;
    finite = finite && fabsf(y[e]) < INFINITY;
    out[e] = from_f<T>(y[e]);
  }
  if (!__all_sync(0xffffffffu, finite)) row_by_warp<T, HD>(a, b, hq, i);
}

// ---------------------------------------------------------------- host side

template <typename T, int HD>
cudaError_t join(const ScoredAttention& a, const ScoredPlan& plan, cudaStream_t st) {
  if (plan.parts == 1) return cudaSuccess;
  const long n_rows = (long)a.B * a.Hq * a.Sq;
  if (plan.parts <= JOIN_WARP_PARTS)
    return launch_kernel(scored_join_warp_kernel<T, HD>, dim3((unsigned)((n_rows + 3) / 4)), dim3(128), 0, st, a, plan);
  return launch_kernel(scored_join_kernel<T, HD>, dim3((unsigned)n_rows), dim3(128), 0, st, a, plan);
}

template <typename K>
cudaError_t launch_maps(K kern, int threads, size_t smem, const ScoredAttention& a, const ScoredPlan& plan,
                        DevError* err, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  CUtensorMap tk, tv;
  // without keys no copy is issued; the maps then describe one token of q
  const bool keys = a.Sk > 0;
  const int tokens = keys ? a.Sk : 1;
  if (make_tmap_heads(&tk, keys ? a.k : a.q, a.HD, tokens, a.Hkv, a.B, a.k_token, a.k_head, a.k_batch) ||
      make_tmap_heads(&tv, keys ? a.v : a.q, a.HD, tokens, a.Hkv, a.B, a.v_token, a.v_head, a.v_batch))
    return cudaErrorInvalidValue;
  const long grid = (long)plan.row_blocks * a.Hkv * a.B * plan.splits;
  if (grid > INT_MAX) return cudaErrorInvalidValue;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(threads), smem, st, tk, tv, a, plan, err);
}

// The register counts that setmaxnreg moves between the warps are those of a launch with 96 (two
// row tiles) or 80 registers a thread; with fewer the increase would never be granted, so a
// build that came out otherwise is refused here.
template <int HD, bool CAP, bool BIAS, int TILES>
cudaError_t launch_rows_kernel(const ScoredAttention& a, const ScoredPlan& plan, DevError* err, cudaStream_t st) {
  using C = Cfg<HD, TILES>;
  struct One {   // a type of its own for each kernel
    static bool ok() {
      static std::atomic<int> state{0};
      int s = state.load(std::memory_order_relaxed);
      if (s == 0) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, scored_tc_kernel<HD, CAP, BIAS, TILES>) != cudaSuccess) {
          cudaGetLastError();
          return false;
        }
        s = at.numRegs == (TILES == 2 ? 96 : 80) ? 1 : 2;
        state.store(s, std::memory_order_relaxed);
      }
      return s == 1;
    }
  };
  if (!One::ok()) return cudaErrorInvalidConfiguration;
  return launch_maps(scored_tc_kernel<HD, CAP, BIAS, TILES>, C::THREADS, C::SMEM, a, plan, err, st);
}

template <int HD, int TILES>
cudaError_t launch_rows(const ScoredAttention& a, const ScoredPlan& plan, DevError* err, cudaStream_t st) {
  if constexpr (TILES == 1)   // the plan takes two under a cap only
    if (!(a.cap > 0.f))
      return a.slopes ? launch_rows_kernel<HD, false, true, 1>(a, plan, err, st)
                      : launch_rows_kernel<HD, false, false, 1>(a, plan, err, st);
  return a.slopes ? launch_rows_kernel<HD, true, true, TILES>(a, plan, err, st)
                  : launch_rows_kernel<HD, true, false, TILES>(a, plan, err, st);
}

template <int HD>
cudaError_t run_tc(const ScoredAttention& a, const ScoredPlan& plan, DevError* err, cudaStream_t st) {
  cudaError_t e;
  if (plan.doc_tiles) {
    const long tiles = (long)a.B * plan.key_tiles;
    e = launch_kernel(scored_docs_kernel, dim3((unsigned)((tiles + 3) / 4)), dim3(128), 0, st, a, plan);
    if (e != cudaSuccess) return e;
  }
  if (plan.few)
    e = launch_maps(scored_few_kernel<HD, 16>, F_THREADS, FewCfg<HD, 16>::SMEM, a, plan, err, st);
  else if (plan.tiles == 1)
    e = launch_rows<HD, 1>(a, plan, err, st);
  else
    e = launch_rows<HD, 2>(a, plan, err, st);
  return e != cudaSuccess ? e : join<bf16, HD>(a, plan, st);
}

template <int HD>
cudaError_t launch_split3(const ScoredAttention& a, const ScoredPlan& plan, DevError* err, cudaStream_t st) {
  using C = Split3Cfg<HD>;
  auto kern = scored_split3_kernel<HD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const long grid = (long)plan.row_blocks * a.Hkv * a.B * plan.splits;
  if (grid > INT_MAX) return cudaErrorInvalidValue;
  e = launch_kernel(kern, dim3((unsigned)grid), dim3(S3_THREADS), C::SMEM, st, a, plan, err);
  return e != cudaSuccess ? e : join<float, HD>(a, plan, st);
}

template <int HD>
cudaError_t launch_f32(const ScoredAttention& a, const ScoredPlan& plan, cudaStream_t st) {
  using C = F32Cfg<HD>;
  auto kern = scored_f32_kernel<HD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const long grid = (long)plan.row_blocks * a.Hkv * a.B * plan.splits;
  if (grid > INT_MAX) return cudaErrorInvalidValue;
  e = launch_kernel(kern, dim3((unsigned)grid), dim3(NT), C::SMEM, st, a, plan);
  return e != cudaSuccess ? e : join<float, HD>(a, plan, st);
}

}  // namespace

// How a call is laid out over the GPU: row blocks by the number of rows a key head has, and
// keys split where that takes less time by this estimate (us): the CTAs in turn on the slots
// of all SMs, each `start` and `step` a key tile, and the join its launch, a little for each
// part and the parts written and read again.  (32 x 8 key heads over 2000 keys, one token: one
// part 47 us, two 56; 4 x 8 heads x 100 rows over 2000 keys: one part 37 us, eight 21; 4 x 8
// heads x 512 tokens: one part 15 us, two 24.)
ScoredPlan scored_attention_plan(const ScoredAttention& a, bool is_bf16, int num_sms) {
  ScoredPlan p;
  const long rows = (long)a.Sq * a.G;
  const bool wide = a.HD == 128;
  int block, tile, slots;
  double start, step;
  p.few = rows <= 16 ? 16 : 0;
  if (p.few) {
    block = 16;
    tile = is_bf16 ? TILE : FT;
    slots = 2 * num_sms;
    start = 4;
    step = wide ? 2.9 : 1.5;   // 64 KB of keys and values (128 dims) at two CTAs' share of the bandwidth
  } else if (is_bf16) {
    // One row tile a CTA, two CTAs an SM: their set-up, loads and last steps overlap, and short calls
    // have twice the CTAs (16 heads x 4096: 145 us against 154 with two tiles, 4 x 8 heads x
    // 512: 15 against 40).  With a cap, whose polynomial keeps the FMA units busy too, tiles in
    // turn do better once they fill the SMs (16 heads x 4096: 176 us against 204).
    p.tiles = a.cap > 0.f && (rows + 2 * TILE - 1) / (2 * TILE) * a.Hkv * a.B >= num_sms ? 2 : 1;
    block = p.tiles * TILE;
    tile = TILE;
    slots = p.tiles == 1 ? 2 * num_sms : num_sms;
    start = 6;
    step = wide ? 2.0 : 1.5;
  } else {
    block = TILE;
    tile = S3_KEYS;
    slots = num_sms;
    start = 12;
    step = wide ? 4.0 : 2.5;
  }
  p.k = scored_const(a.scale, a.cap);
  p.row_blocks = (int)((rows + block - 1) / block);
  const int key_tiles = (a.Sk + tile - 1) / tile;
  const double ctas = (double)p.row_blocks * a.Hkv * a.B;
  const double part_mb = (double)a.B * a.Hq * a.Sq * a.HD * 4e-6;
  double least = 1e30;
  for (int rounds = 0; rounds <= 4; ++rounds) {   // one part, or as many as fill 1 to 4 rounds of CTAs
    long s = rounds == 0 ? 1 : (long)(rounds * slots / ctas);
    if (s > key_tiles / 2) s = key_tiles / 2;
    if (s < 1 || (rounds > 0 && s == 1) || (s > 1 && s * part_mb > 256)) continue;
    const int per = key_tiles > 0 ? (int)((key_tiles + s - 1) / s) : 1;
    const int parts = key_tiles > 0 ? (key_tiles + per - 1) / per : 1;
    // (a last round that is partly filled takes part of a round's time)
    const double w = ctas * parts / slots, waves = w <= 1 ? 1 : (w + ceil(w)) / 2;
    const double us = waves * (start + per * step) + (parts > 1 ? 3 + 0.1 * parts + parts * part_mb * 2 / 3 : 0);
    if (us < least) {
      least = us;
      p.tiles_per_split = per;
      p.splits = p.parts = parts;
    }
  }
  p.bytes = p.parts > 1 ? (size_t)p.parts * a.B * a.Hkv * rows * (a.HD + 1) * 4 : 0;
  p.key_tiles = key_tiles;
  if (is_bf16 && !p.few && a.q_doc != nullptr && key_tiles >= DOC_TILES_MIN) {
    p.doc_offset = (p.bytes + 15) / 16 * 16;
    p.doc_bytes = (size_t)a.B * key_tiles * sizeof(int2);
    p.bytes = p.doc_offset + p.doc_bytes;
  }
  return p;
}

cudaError_t attention_scored(const ScoredAttention& a, bool is_bf16, ScoredPlan plan, void* workspace, DevError* err,
                             cudaStream_t st) {
  if (plan.parts > 1) {
    plan.part_o = static_cast<float*>(workspace);
    plan.part_lse = plan.part_o + (size_t)plan.parts * a.B * a.Hq * a.Sq * a.HD;
  }
  if (plan.doc_bytes > 0) plan.doc_tiles = reinterpret_cast<int2*>(static_cast<char*>(workspace) + plan.doc_offset);
  if (is_bf16) return a.HD == 64 ? run_tc<64>(a, plan, err, st) : run_tc<128>(a, plan, err, st);
  if (!plan.few) return a.HD == 64 ? launch_split3<64>(a, plan, err, st) : launch_split3<128>(a, plan, err, st);
  return a.HD == 64 ? launch_f32<64>(a, plan, st) : launch_f32<128>(a, plan, st);
}

}  // namespace kd
