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
// tokens fill one MMA tile together.  A CTA takes 256 rows as two 128-row tiles: while the
// softmax of one runs, the tensor cores work on the other.  With at most 128 rows (new
// tokens over a cache) both halves take the same rows and alternate over the key tiles;
// keys are also split over CTAs, and a second kernel joins the parts.
//
// Roles (384 threads): warp 0 TMA of K and V tiles (128 keys, 128-byte swizzle), warp 1 MMA
// issue, warps 4-7 and 8-11 softmax and output of tile 0 and 1, one row a thread.  Per key
// tile and row tile: S = Q K^T into 128 TMEM columns; the row's thread reads S, forms p and
// writes it in bf16 over S; O += P V with P as the TMEM operand.  The running maximum is a
// reference that moves only when it falls 2^8 behind (p stays below 2^8, which fp32 sums
// and bf16 weights hold as well as 1), so O is rarely rescaled.
//
// Masked places never reach a result: a masked score is replaced, value rows past kv_len are
// zeroed in shared memory, and a row whose result is not finite (a NaN or infinity among
// values with weight 0 in its tile) is computed again over the seen keys alone.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace kd {
namespace {

constexpr int TILE = 128;                    // query rows of a tile, keys of a tile
constexpr int NUM_THREADS = 384;
constexpr int STAGES = 4;                    // K and V tiles in flight, alternating
constexpr int MAX_FLAGS = 8192;              // key tiles whose document ranges a CTA keeps
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr int KIMODO_ETIMEOUT_CODE = -5;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESCALE_AT = 8.f;            // log2 units the maximum may run ahead of its reference

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(x / cap) in log2 units: tanh z = 1 - 2 / (1 + e^(2z)), absolute error a few 2^-23
__device__ __forceinline__ float capped(float s, float two_log2e_scale_over_cap, float cap_log2) {
  const float e = ex2(s * two_log2e_scale_over_cap);
  return fmaf(-2.f * cap_log2, rcp_approx(1.f + e), cap_log2);
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

// ---------------------------------------------------------------- one row by one warp, fp32
// The definition, over the seen keys alone: scores by warp-shuffle dot products, online
// softmax.  The fp32 path, and the rows of the bf16 path whose first result is not finite.
template <typename T, int HD>
__device__ __noinline__ void row_by_warp(const ScoredAttention& a, int b, int hq, int i) {
  constexpr int PER = HD / 32;
  const int lane = threadIdx.x & 31;
  const int hk = hq / a.G;
  const SeqInfo s = sequence_info(a, b);
  const long p = (long)s.start + i;
  const int last = last_key(a, s, p);
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
    if (a.slopes) {
      const long dist = p - j;
      x -= slope * (float)(dist < 0 ? -dist : dist);
    }
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

template <int HD>
__global__ void __launch_bounds__(128) scored_f32_kernel(const __grid_constant__ ScoredAttention a) {
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const long rows = (long)a.B * a.Sq * a.Hq;
  const long r = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const int hq = (int)(r % a.Hq);
  const long bi = r / a.Hq;
  row_by_warp<float, HD>(a, (int)(bi / a.Sq), hq, (int)(bi % a.Sq));
}

// ---------------------------------------------------------------- bf16: tcgen05

template <int HD>
struct Cfg {
  static constexpr uint32_t Q_BYTES = TILE * HD * 2;       // one row tile
  static constexpr uint32_t KV_BYTES = TILE * HD * 2;      // one key or value tile
  static constexpr uint32_t HALF = TILE * 128;             // 64 dims of a tile
  // HD 64 would let two CTAs share an SM, whose TMEM holds one: the size keeps them apart
  static constexpr size_t BODY = 2 * Q_BYTES + (size_t)STAGES * KV_BYTES;
  static constexpr size_t SMEM = 1024 + (BODY < 120000 ? 120000 / 1024 * 1024 : BODY) + MAX_FLAGS + 256;
};
constexpr uint32_t TMEM_COLS = 512;
__device__ __forceinline__ uint32_t s_col(int t) { return 128u * t; }
template <int HD> __device__ __forceinline__ uint32_t o_col(int t) { return 256u + (uint32_t)HD * t; }

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

template <int HD, bool CAP, bool BIAS>
__global__ void __launch_bounds__(NUM_THREADS, 1)
scored_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ ScoredAttention a, const ScoredPlan plan, DevError* err) {
  using C = Cfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = ptx::smem_u32(smem);
  const uint32_t sKV = sQ + 2 * C::Q_BYTES;
  uint8_t* flags = smem + C::BODY;
  uint64_t* bars = reinterpret_cast<uint64_t*>(flags + MAX_FLAGS);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto s_bar = [&](int t) { return bar0 + 8u * (2 * STAGES + t); };       // S formed
  auto p_bar = [&](int t) { return bar0 + 8u * (2 * STAGES + 2 + t); };   // P written, O rescaled
  auto o_bar = [&](int t) { return bar0 + 8u * (2 * STAGES + 4 + t); };   // last P V done
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 6);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 7);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  RowTile* tiles = reinterpret_cast<RowTile*>(tmem_slot + 2);

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
  const int n_tiles_q = plan.alternate ? 1 : 2;             // row tiles of this CTA
  const int row0 = rb * TILE * n_tiles_q;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(s_bar(t), 1);
      ptx::mbar_init(p_bar(t), 4);
      ptx::mbar_init(o_bar(t), 1);
      tiles[t].docs_lo = INT_MAX;
      tiles[t].docs_hi = -1;
      tiles[t].any_none = 0;
    }
    ptx::mbar_init(drain_bar, 1);
    ptx::fence_mbar_init();
    *abort = 0;
    ptx::tma_prefetch_desc(&tmK);
    ptx::tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), TMEM_COLS);
    ptx::tmem_relinquish();
  }
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const SeqInfo seq = sequence_info(a, b);
  __syncthreads();

  // ---------------- queries into shared memory (K-major, 128-byte swizzle), rows' documents
  {
    constexpr int CH = HD / 8;                               // 16-byte chunks of a row
    const bf16* qb = static_cast<const bf16*>(a.q) + b * a.q_batch + (long)hk * a.G * a.q_head;
    const int total = n_tiles_q * TILE * CH;
    for (int c = threadIdx.x; c < total; c += NUM_THREADS) {
      const int lr = c / CH, ch = c % CH, r = row0 + lr;
      uint4 val = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        const int i = r / a.G, g = r - i * a.G;
        val = *reinterpret_cast<const uint4*>(qb + i * a.q_token + g * a.q_head + ch * 8);
      }
      const int t = lr / TILE, rr = lr % TILE;
      *reinterpret_cast<uint4*>(smem + t * C::Q_BYTES + (ch >> 3) * C::HALF + rr * 128 +
                                (((ch & 7) ^ (rr & 7)) << 4)) = val;
    }
    ptx::fence_proxy_async_smem();
  }
  // this softmax thread's row
  const int t_own = warp >= 8 ? 1 : 0;
  const int lr_own = ((warp & 3) * 32 + lane) + (plan.alternate ? 0 : t_own * TILE);
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
  const int row_last = min(row0 + n_tiles_q * TILE, rows) - 1;
  const int key_end = 1 + last_key(a, seq, (long)seq.start + row_last / a.G);
  const int jt_all = (key_end + TILE - 1) / TILE;
  const int jt0 = min(split * plan.tiles_per_split, jt_all);
  const int jt1 = plan.splits == 1 ? jt_all : min(jt0 + plan.tiles_per_split, jt_all);
  const bool docs = a.q_doc != nullptr;
  const bool listed = docs && jt1 - jt0 <= MAX_FLAGS;
  if (listed) {
    // flags of a key tile: bit 2t = row tile t may see it, bit 2t + 1 = all of t's rows and all
    // of its keys are one document
    for (int jt = jt0 + warp; jt < jt1; jt += NUM_THREADS / 32) {
      int lo = INT_MAX, hi = -1;
      bool none = false;
#pragma unroll
      for (int e = 0; e < TILE / 32; ++e) {
        const int j = jt * TILE + e * 32 + lane;
        const int d = j < seq.kv_len ? a.kv_doc[(long)b * a.Sk + j] : -1;
        none |= d < 0;
        if (d >= 0) {
          lo = min(lo, d);
          hi = max(hi, d);
        }
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      none = __any_sync(0xffffffffu, none);
      if (lane == 0) {
        uint8_t f = 0;
        for (int t = 0; t < 2; ++t) {
          const RowTile& q = tiles[t];
          if (lo <= q.docs_hi && q.docs_lo <= hi) f |= 1u << (2 * t);
          if (!none && !q.any_none && lo == hi && q.docs_lo == q.docs_hi && lo == q.docs_lo) f |= 2u << (2 * t);
        }
        flags[jt - jt0] = f;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // Which of the row tiles take key tile jt (bits 0 and 1); `turn` counts the tiles taken so
  // far, by whose parity the halves alternate.
  int last_pos[2];
  bool alive[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r_a = row0 + (plan.alternate ? 0 : t * TILE);
    const int r_b = min(r_a + TILE, rows) - 1;
    alive[t] = r_a < rows;
    last_pos[t] = seq.start + max(r_b, 0) / a.G;
  }
  auto needed = [&](int jt, int turn) -> int {
    const int j0 = jt * TILE;
    int need = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      bool n = alive[t] && (!a.causal || j0 <= last_pos[t] || j0 < seq.prefix);
      if (listed) n = n && ((flags[jt - jt0] >> (2 * t)) & 1);
      need |= n ? 1 << t : 0;
    }
    if (plan.alternate && need) need = 1 << (turn & 1);
    return need;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA: K and V tile of every key tile taken, in turn
      int stage = 0, turn = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      for (int jt = jt0; jt < jt1 && ok; ++jt) {
        if (!needed(jt, turn)) continue;
        ++turn;
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
      const long n = issued < STAGES ? issued : STAGES;
      volatile int never = 0;
      for (long i = 0; i < n; ++i) {
        if (--stage < 0) { stage = STAGES - 1; phase ^= 1u; }
        ptx::mbar_wait_bounded(full_bar(stage), phase, &never, WAIT_LIMIT_NS);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA: per key tile and row tile t, first P V of the tile before, then Q K^T
    // (which overwrites that P); the other row tile's products run while t's softmax does
    const uint32_t idesc_s = ptx::idesc_bf16_f32(TILE, TILE);
    const uint32_t idesc_o = ptx::idesc_bf16_f32(TILE, HD) | (1u << 16);
    int stage = 0, turn = 0, pend = 0, v_stage = 0, v_rows = TILE;
    uint32_t phase = 0, v_phase = 0, p_phase[2] = {0, 0};
    bool started[2] = {false, false}, ok = true;
    auto advance = [&](int& s, uint32_t& ph) { if (++s == STAGES) { s = 0; ph ^= 1u; } };
    auto pv = [&](int t) -> bool {   // O_t (+)= P_t V of the pending value tile
      if (!ptx::mbar_wait_bounded(p_bar(t), p_phase[t], abort, WAIT_LIMIT_NS)) return false;
      p_phase[t] ^= 1u;
      ptx::tc_fence_after();
      if (lane == 0) {
        const uint32_t v = sKV + v_stage * C::KV_BYTES;
#pragma unroll
        for (int kk = 0; kk < TILE / 16; ++kk)
          ptx::tc_mma_bf16_ta(tmem_base + o_col<HD>(t), tmem_base + s_col(t) + kk * 8, desc_mn(v + kk * 2048, C::HALF),
                              idesc_o, started[t] || kk != 0);
      }
      started[t] = true;
      __syncwarp();
      return true;
    };
    auto values_ready = [&]() -> bool {
      if (!ptx::mbar_wait_bounded(full_bar(v_stage), v_phase, abort, WAIT_LIMIT_NS)) return false;
      if (v_rows < TILE) {   // value rows past the last key: 0, whatever they hold
        uint8_t* v = smem + 2 * C::Q_BYTES + v_stage * C::KV_BYTES;
        const int n = (TILE - v_rows) * 8;
        for (int c = lane; c < n * (HD / 64); c += 32) {
          const int hf = c / n, e = c % n;
          *reinterpret_cast<uint4*>(v + hf * C::HALF + (v_rows + e / 8) * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      return true;
    };
    for (int jt = jt0; jt <= jt1 && ok; ++jt) {
      const bool end = jt == jt1;
      const int need = end ? 0 : needed(jt, turn);
      if (!end && !need) continue;
      int k_stage = stage;
      if (!end) {
        ++turn;
        ok = ptx::mbar_wait_bounded(full_bar(stage), phase, abort, WAIT_LIMIT_NS);
        if (!ok) break;
        advance(stage, phase);
      }
      ptx::tc_fence_after();
      auto qk = [&](int t) {
        if (lane == 0) {
          const uint32_t q = sQ + (plan.alternate ? 0u : t * C::Q_BYTES), k = sKV + k_stage * C::KV_BYTES;
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            ptx::tc_mma_bf16(tmem_base + s_col(t), ptx::smem_desc_sw128(q + (kk >> 2) * C::HALF + (kk & 3) * 32),
                             ptx::smem_desc_sw128(k + (kk >> 2) * C::HALF + (kk & 3) * 32), idesc_s, kk != 0);
          ptx::tc_commit(s_bar(t));
        }
        __syncwarp();
      };
      // scores of a row tile with no weights outstanding first: they wait for nothing
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if ((need & ~pend) >> t & 1) qk(t);
      if (pend) ok = values_ready();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (ok && (pend >> t & 1)) ok = pv(t);
        if (ok && ((need & pend) >> t & 1)) qk(t);
      }
      if (!ok) break;
      if (lane == 0) {
        if (!end) ptx::tc_commit(empty_bar(k_stage));
        if (pend) ptx::tc_commit(empty_bar(v_stage));
      }
      __syncwarp();
      if (!end) {
        pend = need;
        v_stage = stage;
        v_phase = phase;
        v_rows = min(seq.kv_len - jt * TILE, TILE);
        advance(stage, phase);
      }
    }
    if (!ok && !*abort && lane == 0) record_timeout(err, abort);
    if (lane == 0) {
      ptx::tc_commit(o_bar(0));
      ptx::tc_commit(o_bar(1));
      ptx::tc_commit(drain_bar);
      volatile int never = 0;
      if (!ptx::mbar_wait_bounded(drain_bar, 0, &never, WAIT_LIMIT_NS)) record_timeout(err, abort);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- softmax and output of row tile t_own
    const int t = t_own;
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem_base + lane_addr + s_col(t), o_addr = tmem_base + lane_addr + o_col<HD>(t);
    const bool warp_rows = (warp & 3) * 32 + row0 + (plan.alternate ? 0 : t * TILE) < rows;
    const int p = seq.start + i_own;
    const int last = row_ok ? last_key(a, seq, (long)seq.start + i_own) : -1;
    const float slope2 = BIAS && row_ok ? a.slopes[hk * a.G + g_own] * LOG2E : 0.f;
    const float sc = CAP ? 2.f * LOG2E * a.scale / a.cap : a.scale * LOG2E;
    const float cap2 = CAP ? a.cap * LOG2E : 0.f;
    float m = -INFINITY, l = 0.f;   // reference of the weights (log2 units) and their sum
    uint32_t phase = 0;
    bool ok = true, started = false;
    int turn = 0;
    for (int jt = jt0; jt < jt1; ++jt) {
      const int need = needed(jt, turn);
      if (need) ++turn;
      if (!(need >> t & 1)) continue;
      ok = ptx::mbar_wait_bounded(s_bar(t), phase, abort, WAIT_LIMIT_NS);
      if (!ok) break;
      phase ^= 1u;
      if (warp_rows) {
        ptx::tc_fence_after();
        const int j0 = jt * TILE;
        const bool one_doc = !docs || (listed && ((flags[jt - jt0] >> (2 * t + 1)) & 1));
        // scores in log2 units, masked ones -infinity
        float x[TILE];
#pragma unroll
        for (int c = 0; c < TILE; c += 32) {
          float v[32];
          ptx::tmem_ld(s_addr + c, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float y = CAP ? capped(v[e], sc, cap2) : v[e] * sc;
            if (BIAS) y = fmaf(-slope2, fabsf((float)(p - (j0 + c + e))), y);
            x[c + e] = y;
          }
        }
        if (!__all_sync(0xffffffffu, j0 + TILE - 1 <= last || !row_ok)) {
#pragma unroll
          for (int e = 0; e < TILE; ++e)
            if (j0 + e > last) x[e] = -INFINITY;
        }
        if (!one_doc) {
          const int* kd_ = a.kv_doc + (long)b * a.Sk;
#pragma unroll
          for (int e = 0; e < TILE; ++e) {
            const int d = kd_[min(j0 + e, a.Sk - 1)];
            if (d != qdoc || qdoc < 0) x[e] = -INFINITY;
          }
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < TILE; ++e) top = fmaxf(top, x[e]);
        // move the reference: at once while there is none, later only when it falls far behind
        const bool move = !started || top > m + RESCALE_AT;
        const float m_new = move ? fmaxf(m, top) : m;
        if (started && __any_sync(0xffffffffu, move)) {
          const float f = m_new == m ? 1.f : ex2(m - m_new);   // m = -infinity: 0
          l *= f;
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
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
#pragma unroll
        for (int c = 0; c < TILE; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = ex2(x[c + e] - ref), p1 = ex2(x[c + e + 1] - ref);
            l += p0 + p1;
            w[e / 2] = bf16x2_bits(p0, p1);
          }
          ptx::tmem_st16(s_addr + c / 2, w);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      }
      started = true;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(p_bar(t));
    }
    if (ok) ok = ptx::mbar_wait_bounded(o_bar(t), 0, abort, WAIT_LIMIT_NS);
    if (!ok && !*abort) record_timeout(err, abort);
    if (ok && warp_rows) {
      ptx::tc_fence_after();
      const bool seen = started && l != 0.f;   // l is NaN where a score is
      const float inv = seen ? 1.f / l : 0.f;
      bool finite = true;
      if (plan.parts == 1) {
        bf16* o = static_cast<bf16*>(a.out) + b * a.o_batch + i_own * a.o_token + (long)(hk * a.G + g_own) * a.o_head;
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
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
        unsigned redo = __ballot_sync(0xffffffffu, row_ok && !finite);
        while (redo) {
          const int src = __ffs(redo) - 1;
          redo &= redo - 1;
          row_by_warp<bf16, HD>(a, b, hk * a.G + __shfl_sync(0xffffffffu, g_own, src),
                                __shfl_sync(0xffffffffu, i_own, src));
        }
      } else {
        // a part: the result over these keys and the log2 of its weight
        const int part = plan.alternate ? 2 * split + t : split;
        const long prow = ((long)b * a.Hkv + hk) * rows + r_own;
        const long n_rows = (long)a.B * a.Hkv * rows;
        float* o = plan.part_o + ((long)part * n_rows + prow) * HD;
        if (row_ok) plan.part_lse[(long)part * n_rows + prow] = seen ? m + log2f(l) : -INFINITY;
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          float v[16];
          ptx::tmem_ld(o_addr + c, v);
          ptx::tmem_ld_wait();
          if (row_ok) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(o + c + e) =
                  seen ? make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Join of the parts of a row: o = sum 2^(lse - max) o_part / sum 2^(lse - max).  One warp a row.
template <int HD>
__global__ void __launch_bounds__(128) scored_join_kernel(const __grid_constant__ ScoredAttention a,
                                                          const ScoredPlan plan) {
  constexpr int PER = HD / 32;
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int rows = a.Sq * a.G;
  const long n_rows = (long)a.B * a.Hkv * rows;
  const long r = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= n_rows) return;
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int s = lane; s < plan.parts; s += 32) top = fmaxf(top, plan.part_lse[s * n_rows + r]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f, o[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = 0.f;
  for (int s = 0; s < plan.parts; ++s) {
    const float lse = plan.part_lse[s * n_rows + r];
    if (lse == -INFINITY) continue;
    const float w = exp2f(lse - ref);
    total += w;
    const float* po = plan.part_o + (s * n_rows + r) * HD + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = fmaf(w, po[e], o[e]);
  }
  const int rr = (int)(r % rows), i = rr / a.G, g = rr - i * a.G;
  const int bh = (int)(r / rows), hk = bh % a.Hkv, b = bh / a.Hkv, hq = hk * a.G + g;
  bf16* out = static_cast<bf16*>(a.out) + b * a.o_batch + i * a.o_token + hq * a.o_head + lane * PER;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const float y = total == 0.f ? 0.f : o[e] / total;
    finite = finite && fabsf(y) < INFINITY;
    out[e] = __float2bfloat16_rn(y);
  }
  if (!__all_sync(0xffffffffu, finite)) row_by_warp<bf16, HD>(a, b, hq, i);
}

template <int HD, bool CAP, bool BIAS>
cudaError_t launch_tc(const ScoredAttention& a, const ScoredPlan& plan, DevError* err, cudaStream_t st) {
  using C = Cfg<HD>;
  auto kern = scored_tc_kernel<HD, CAP, BIAS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap tk, tv;
  // without keys no copy is issued; the maps then describe one token of q
  const bool keys = a.Sk > 0;
  const int tokens = keys ? a.Sk : 1;
  if (make_tmap_heads(&tk, keys ? a.k : a.q, HD, tokens, a.Hkv, a.B, a.k_token, a.k_head, a.k_batch) ||
      make_tmap_heads(&tv, keys ? a.v : a.q, HD, tokens, a.Hkv, a.B, a.v_token, a.v_head, a.v_batch))
    return cudaErrorInvalidValue;
  const long grid = (long)plan.row_blocks * a.Hkv * a.B * plan.splits;
  if (grid > INT_MAX) return cudaErrorInvalidValue;
  e = launch_kernel(kern, dim3((unsigned)grid), dim3(NUM_THREADS), C::SMEM, st, tk, tv, a, plan, err);
  if (e != cudaSuccess || plan.parts == 1) return e;
  const long n_rows = (long)a.B * a.Hq * a.Sq;
  return launch_kernel(scored_join_kernel<HD>, dim3((unsigned)((n_rows + 3) / 4)), dim3(128), 0, st, a, plan);
}

template <int HD>
cudaError_t run_tc(const ScoredAttention& a, const ScoredPlan& plan, DevError* err, cudaStream_t st) {
  if (a.cap > 0.f)
    return a.slopes ? launch_tc<HD, true, true>(a, plan, err, st) : launch_tc<HD, true, false>(a, plan, err, st);
  return a.slopes ? launch_tc<HD, false, true>(a, plan, err, st) : launch_tc<HD, false, false>(a, plan, err, st);
}

}  // namespace

// How a bf16 call is laid out over the GPU.  At most 128 rows a key head leave one row tile,
// whose key tiles the two halves of a CTA take in turn; keys are split further while the
// CTAs do not fill the SMs and every part keeps two tiles.
ScoredPlan scored_attention_plan(const ScoredAttention& a, int num_sms) {
  ScoredPlan p;
  const long rows = (long)a.Sq * a.G;
  const int key_tiles = (a.Sk + TILE - 1) / TILE;
  p.alternate = rows <= TILE && key_tiles > 1;
  p.row_blocks = (int)((rows + 2 * TILE - 1) / (2 * TILE));
  const long ctas = (long)p.row_blocks * a.Hkv * a.B;
  long splits = ctas < num_sms ? num_sms / ctas : 1;
  if (splits > (key_tiles + 1) / 2) splits = (key_tiles + 1) / 2;
  if (splits < 1) splits = 1;
  p.tiles_per_split = (int)((key_tiles + splits - 1) / splits);
  if (p.tiles_per_split < 1) p.tiles_per_split = 1;
  p.splits = key_tiles > 0 ? (key_tiles + p.tiles_per_split - 1) / p.tiles_per_split : 1;
  p.parts = p.splits * (p.alternate ? 2 : 1);
  const long n_rows = (long)a.B * a.Hkv * rows;
  p.bytes = p.parts > 1 ? (size_t)p.parts * n_rows * (a.HD + 1) * 4 : 0;
  return p;
}

cudaError_t attention_scored_bf16(const ScoredAttention& a, ScoredPlan plan, void* workspace, DevError* err,
                                  cudaStream_t st) {
  if (plan.parts > 1) {
    plan.part_o = static_cast<float*>(workspace);
    plan.part_lse = plan.part_o + (size_t)plan.parts * a.B * a.Hq * a.Sq * a.HD;
  }
  return a.HD == 64 ? run_tc<64>(a, plan, err, st) : run_tc<128>(a, plan, err, st);
}

cudaError_t attention_scored_f32(const ScoredAttention& a, cudaStream_t st) {
  const long rows = (long)a.B * a.Sq * a.Hq;
  const dim3 grid((unsigned)((rows + 3) / 4));
  return a.HD == 64 ? launch_kernel(scored_f32_kernel<64>, grid, dim3(128), 0, st, a)
                    : launch_kernel(scored_f32_kernel<128>, grid, dim3(128), 0, st, a);
}

}  // namespace kd
