// Matrix product in 8-bit integers with a scale for each token and each output channel:
//   y[m, n] = a_scale[m] * w_scale[n] * sum_k a[m, k] w[n, k] + bias[n],
// then GELU, SiLU or a residual, on the tcgen05 tensor cores (kind::i8).  The sum is exact
// in 32-bit integers (K <= 131071 keeps it below 2^31), so neither the order of K nor a
// split of it changes a bit; it is rounded once to fp32 (24 bits) when it meets the scales.
//
// Both kernels put the WEIGHTS on the rows of the MMA (TMEM lanes) and the tokens on its
// columns.  A thread of the epilogue then owns one output channel, whose scale and bias
// are two registers, and a warp stores 32 consecutive channels of a token at once: whole
// sectors with no staging and no rule on the alignment of the output, so odd N costs
// nothing.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <type_traits>

#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace kd {
namespace {

constexpr int BK = 128;                      // K of one 128-byte swizzle atom
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr int KIMODO_ETIMEOUT_CODE = -5;

struct I8Epi {
  const float* a_scale;
  const float* w_scale;
  const float* bias;     // [N] or null
  const float* resid;    // [M, ldr] (EPI_BIAS_RESID)
  long ldr;
  void* out;
  long ldo;
  int M, N;
};

__device__ __forceinline__ void record_timeout(DevError* err, int where, volatile int* abort) {
  *abort = 1;
  if (err && atomicCAS(&err->code, 0, KIMODO_ETIMEOUT_CODE) == 0) {
    err->where = where;
    err->block = blockIdx.x;
  }
}

// What a chunk of NV tokens from m0 needs besides its accumulators, loaded a chunk ahead: lane l's
// token scale and, with a residual, channel n of every token.
template <int KIND, int NV>
struct Ahead {
  float scale;
  float resid[KIND == EPI_BIAS_RESID ? NV : 1];
  __device__ __forceinline__ void load(const I8Epi& e, int n, int m0, int lane) {
    scale = lane < NV && m0 + lane < e.M ? e.a_scale[m0 + lane] : 0.f;
    if constexpr (KIND == EPI_BIAS_RESID) {
      const float* r = e.resid + (long)m0 * e.ldr + n;
      if (n < e.N && m0 + NV <= e.M) {
#pragma unroll
        for (int j = 0; j < NV; ++j) resid[j] = r[j * e.ldr];
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) resid[j] = n < e.N && m0 + j < e.M ? r[j * e.ldr] : 0.f;
      }
    }
  }
};

// Finish and store the accumulators v (32-bit integers) of channel n for the tokens
// m0 .. m0 + NV - 1.
template <int KIND, typename OutT, int NV>
__device__ __forceinline__ void store_tokens(const I8Epi& e, int n, float sn, float bn, int m0,
                                             const Ahead<KIND, NV>& ahead, const int (&v)[NV]) {
  const bool col = n < e.N;
  float y[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    y[j] = fmaf((float)v[j], __shfl_sync(0xffffffffu, ahead.scale, j) * sn, bn);
    if constexpr (KIND == EPI_BIAS_RESID) y[j] += ahead.resid[j];
  }
  if constexpr (KIND == EPI_BIAS_GELU) {
#pragma unroll
    for (int j = 0; j < NV; j += 2) gelu2_as7128(y[j], y[j + 1]);
  }
  if constexpr (KIND == EPI_BIAS_SILU) {
#pragma unroll
    for (int j = 0; j < NV; ++j) y[j] = silu_f(y[j]);
  }
  OutT* o = static_cast<OutT*>(e.out) + (long)m0 * e.ldo + n;
  if (!col) return;
  if (m0 + NV <= e.M) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      *o = from_f<OutT>(y[j]);
      o += e.ldo;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (m0 + j < e.M) o[j * e.ldo] = from_f<OutT>(y[j]);
  }
}

// ====================================================================== CTA pairs (many tokens)
//
// A cluster of two CTAs computes 256 channels x BN tokens: each CTA stages 128 weight rows
// and BN / 2 token rows (TMA, 128-byte swizzle, no multicast), the leader issues
// 256 x BN x 32 MMAs that read both CTAs' shared memory.  Persistent; two accumulators in
// TMEM, so the epilogue of a tile runs under the MMAs of the next.
// Roles (320 threads): warp 0 TMA, warp 1 TMEM allocation and (leader) MMA, warps 2-9
// epilogue.  Every wait is bounded.
constexpr int P_EPI_WARPS = 8;
constexpr int P_THREADS = 64 + 32 * P_EPI_WARPS;

template <int BN>
struct PairCfg {
  static constexpr int KA = 2;               // atoms (128 K) per stage: halves the hand-offs
  static constexpr uint32_t ATOM_A = 128 * 128;
  static constexpr uint32_t ATOM_B = (BN / 2) * 128;
  static constexpr uint32_t STAGE_BYTES = KA * (ATOM_A + ATOM_B);
  static constexpr int STAGES = (int)((232448 - 1024 - 256) / STAGE_BYTES) > 6 ? 6 : (int)((232448 - 1024 - 256) / STAGE_BYTES);
  static constexpr uint32_t NUM_BARS = 2 * STAGES + 5;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + NUM_BARS * 8 + 16;
  static constexpr uint32_t TMEM_COLS = 2 * BN <= 32 ? 32 : 2 * BN <= 64 ? 64 : 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
  static constexpr uint32_t IDESC = ptx::idesc_i8_s32(256, BN);
  static_assert(BN % 32 == 0 && BN <= 256, "MMA N of the pair, whole 32-token chunks");
  static_assert(SMEM <= 232448, "shared memory");
};

// Tile order: groups of GROUP_W channel blocks, all token blocks of a group in turn, so that
// the tiles in flight share both operands in L2.
constexpr int GROUP_W = 8;
__device__ __forceinline__ void tile_at(int tile, int nw, int nt, int& w, int& t) {
  const int per = GROUP_W * nt, g = tile / per, in = tile - g * per;
  const int first = g * GROUP_W, gw = min(GROUP_W, nw - first);
  w = first + in % gw;
  t = in / gw;
}

template <int BN, int KIND, typename OutT>
__global__ void __launch_bounds__(P_THREADS, 1)
gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, int nw, int nt,
                    int num_kb, I8Epi ep, DevError* err) {
  using C = PairCfg<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sW = ptx::smem_u32(smem);
  const uint32_t sA = sW + STAGES * C::KA * C::ATOM_A;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES);
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NUM_BARS);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(tfull_bar(a), 1);
      ptx::mbar_init(tempty_bar(a), 2 * P_EPI_WARPS);
    }
    ptx::mbar_init(drain_bar, 1);
    ptx::fence_mbar_init();
    *abort = 0;
    ptx::tma_prefetch_desc(&tmW);
    ptx::tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_u32(tmem_slot), C::TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::pdl_trigger();
  ptx::pdl_wait();
  ptx::tc_fence_before();
  __syncwarp();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int num_tiles = nw * nt;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      for (int tile = pair; tile < num_tiles && ok; tile += npairs) {
        int w, t;
        tile_at(tile, nw, nt, w, t);
        const int wrow = w * 256 + (int)rank * 128, arow = t * BN + (int)rank * (BN / 2);
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!ptx::mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort, WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          if (rank == 0) ptx::mbar_arrive_expect_tx(full_bar(stage), 2 * C::STAGE_BYTES);
          const uint32_t lbar = ptx::mapa_shared(full_bar(stage), 0);
#pragma unroll
          for (int at = 0; at < C::KA; ++at) {
            const int k = (kb * C::KA + at) * BK;
            ptx::tma_load_2d_pair(sW + (stage * C::KA + at) * C::ATOM_A, &tmW, lbar, k, wrow);
            ptx::tma_load_2d_pair(sA + (stage * C::KA + at) * C::ATOM_B, &tmA, lbar, k, arow);
          }
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        if (!*abort) record_timeout(err, WHERE_GEMM_PRODUCER, abort);
        if (rank == 0) {   // the leader's full barriers count both CTAs' loads
          const long n = issued < STAGES ? issued : STAGES;
          int s = stage;
          uint32_t ph = phase;
          volatile int never = 0;
          for (long i = 0; i < n; ++i) {
            if (--s < 0) { s = STAGES - 1; ph ^= 1u; }
            ptx::mbar_wait_bounded(full_bar(s), ph, &never, WAIT_LIMIT_NS);
          }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // operand descriptors of the first stage; later ones and K steps by additions (16-byte units)
      const uint64_t w_desc0 = ptx::smem_desc_sw128(sW), a_desc0 = ptx::smem_desc_sw128(sA);
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair; tile < num_tiles && ok; tile += npairs, ++local) {
        const int acc = local & 1;
        if (!ptx::mbar_wait_bounded(tempty_bar(acc), ((local >> 1) & 1) ^ 1u, abort, WAIT_LIMIT_NS)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!ptx::mbar_wait_bounded(full_bar(stage), phase, abort, WAIT_LIMIT_NS)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t w0 = w_desc0 + (uint64_t)(stage * (C::KA * C::ATOM_A >> 4));
          const uint64_t a0 = a_desc0 + (uint64_t)(stage * (C::KA * C::ATOM_B >> 4));
          const uint32_t more = kb != 0 ? 1u : 0u;
          if (ptx::elect_one()) {
#pragma unroll
            for (int k = 0; k < C::KA * 4; ++k)
              ptx::tc_mma_i8_pair(d_tmem, w0 + (uint64_t)(((k >> 2) * C::ATOM_A + (k & 3) * 32) >> 4),
                                  a0 + (uint64_t)(((k >> 2) * C::ATOM_B + (k & 3) * 32) >> 4), C::IDESC,
                                  k != 0 ? 1u : more);
            ptx::tc_commit_pair(empty_bar(stage), 0x3);
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (ptx::elect_one()) ptx::tc_commit_pair(tfull_bar(acc), 0x3);
        __syncwarp();
      }
      if (ptx::elect_one()) {
        if (!ok && !*abort) record_timeout(err, WHERE_GEMM_MMA, abort);
        ptx::tc_commit_pair(drain_bar, 0x1);
        volatile int never = 0;
        if (!ptx::mbar_wait_bounded(drain_bar, 0, &never, WAIT_LIMIT_NS)) record_timeout(err, WHERE_GEMM_DRAIN, abort);
      }
      __syncwarp();
    }
  } else {
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const uint32_t leader_tempty0 = ptx::mapa_shared(tempty_bar(0), 0);
    const uint32_t leader_tempty1 = ptx::mapa_shared(tempty_bar(1), 0);
    int local = 0;
    for (int tile = pair; tile < num_tiles; tile += npairs, ++local) {
      const int acc = local & 1;
      int w, t;
      tile_at(tile, nw, nt, w, t);
      const int n = w * 256 + (int)rank * 128 + quarter * 32 + lane;
      const float sn = n < ep.N ? ep.w_scale[n] : 0.f;
      const float bn = n < ep.N && ep.bias != nullptr ? ep.bias[n] : 0.f;
      // 32-token chunks part, part + 2, ...
      Ahead<KIND, 32> next;
      next.load(ep, n, t * BN + part * 32, lane);
      if (!ptx::mbar_wait_bounded(tfull_bar(acc), (local >> 1) & 1, abort, WAIT_LIMIT_NS)) {
        if (!*abort) record_timeout(err, WHERE_GEMM_EPILOGUE, abort);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * BN;
#pragma unroll 1
      for (int c = part * 32; c < BN; c += 64) {
        const int m0 = t * BN + c;
        if (m0 >= ep.M) break;
        float f[32];
        int v[32];
        ptx::tmem_ld(taddr + c, f);
        const Ahead<KIND, 32> now = next;
        if (c + 64 < BN) next.load(ep, n, m0 + 64, lane);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __float_as_int(f[j]);
        store_tokens<KIND, OutT, 32>(ep, n, sn, bn, m0, now, v);
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_remote(acc ? leader_tempty1 : leader_tempty0);
    }
  }
  // both CTAs finish every access to the pair's shared memory and TMEM before either leaves
  ptx::tc_fence_before();
  __syncwarp();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

// ====================================================================== single CTAs (few tokens)
//
// One CTA computes `ct` channels x BN tokens over the whole K.  With few tokens the time is that of
// the weights' bytes, and one SM takes in about 60 bytes a cycle, so the channels are cut as
// narrow as gives every SM a CTA (1 x 4096 x 4096: 128 CTAs of 32 channels), with the whole
// ring of stages in flight.  The MMA still has 128 rows; those past ct read whatever follows in
// shared memory and are not looked at.  (Slices of K over a cluster, exchanged through
// distributed shared memory, measured 9.2 us there against 7.9 us for one CTA of 128
// channels and all of K.)
// Roles (192 threads): warp 0 TMA, warp 1 MMA, warps 2-5 epilogue.
constexpr int S_THREADS = 192;
constexpr int S_MAX_STAGES = 16;
constexpr uint32_t S_SMEM_MAX = 232448;
struct SmallPlan {
  int ct;        // channels of a CTA: 16, 32, 64 or 128
  int ka;        // 128-column blocks of a stage
  int stages;
  int num_kb;    // blocks of K, the last one perhaps partial
  int whole;     // whole blocks
};
__host__ __device__ inline uint32_t small_stage_bytes(const SmallPlan& p, int bn) {
  return (uint32_t)p.ka * (uint32_t)(p.ct + bn) * 128;
}
// behind the stages, room for the rows past ct of the last one's MMAs, then barriers
__host__ __device__ inline uint32_t small_pad_bytes(const SmallPlan& p) { return (uint32_t)(128 - p.ct) * 128; }
inline size_t small_smem(const SmallPlan& p, int bn) {
  return 1024 + (size_t)p.stages * small_stage_bytes(p, bn) + small_pad_bytes(p) + (2 * S_MAX_STAGES + 1) * 8 + 16;
}

template <int BN, int KIND, typename OutT>
__global__ void __launch_bounds__(S_THREADS)
gemm_i8_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmWt, const __grid_constant__ CUtensorMap tmAt, SmallPlan p,
                     I8Epi ep, DevError* err) {
  constexpr uint32_t COLS = BN <= 32 ? 32 : BN <= 64 ? 64 : 128;
  constexpr uint32_t IDESC = ptx::idesc_i8_s32(128, BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t atom_w = (uint32_t)p.ct * 128, atom_a = BN * 128;
  // token stages first: what the weight stages' MMAs read past ct rows lies behind them
  const uint32_t sA = ptx::smem_u32(smem), sW = sA + p.stages * p.ka * atom_a;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * small_stage_bytes(p, BN) + small_pad_bytes(p));
  const uint32_t bar0 = ptx::smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S_MAX_STAGES + s); };
  const uint32_t done_bar = bar0 + 8u * (2 * S_MAX_STAGES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S_MAX_STAGES + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * p.ct, t0 = blockIdx.y * BN;
  const int steps = (p.num_kb + p.ka - 1) / p.ka;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    ptx::mbar_init(done_bar, 1);
    ptx::fence_mbar_init();
    *abort = 0;
    ptx::tma_prefetch_desc(&tmW);
    ptx::tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), COLS);
    ptx::tmem_relinquish();
  }
  ptx::pdl_wait();
  ptx::pdl_trigger();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; i < steps; ++i) {
        if (i >= p.stages) {
          ok = ptx::mbar_wait_bounded(empty_bar(stage), phase ^ 1u, abort, WAIT_LIMIT_NS);
          if (!ok) break;
        }
        const int kb = i * p.ka, n = min(p.ka, p.num_kb - kb);
        const uint32_t dw = sW + stage * p.ka * atom_w, da = sA + stage * p.ka * atom_a;
        ptx::mbar_arrive_expect_tx(full_bar(stage), (uint32_t)n * (atom_w + atom_a));
        if (kb + p.ka <= p.whole) {   // whole blocks only: one box an operand
          ptx::tma_load_3d(dw, &tmW, full_bar(stage), 0, n0, kb);
          ptx::tma_load_3d(da, &tmA, full_bar(stage), 0, t0, kb);
        } else {
          for (int a = 0; a < n; ++a) {
            ptx::tma_load_2d(dw + a * atom_w, &tmWt, full_bar(stage), (kb + a) * BK, n0);
            ptx::tma_load_2d(da + a * atom_a, &tmAt, full_bar(stage), (kb + a) * BK, t0);
          }
        }
        ++issued;
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) {
        if (!*abort) record_timeout(err, WHERE_GEMM_PRODUCER, abort);
        volatile int never = 0;   // every copy issued has landed before the CTA leaves
        for (int i = 0; i < issued && i < p.stages; ++i) {
          if (--stage < 0) { stage = p.stages - 1; phase ^= 1u; }
          ptx::mbar_wait_bounded(full_bar(stage), phase, &never, WAIT_LIMIT_NS);
        }
      }
    }
  } else if (warp == 1) {
    const uint64_t w_desc0 = ptx::smem_desc_sw128(sW), a_desc0 = ptx::smem_desc_sw128(sA);
    int stage = 0;
    uint32_t phase = 0, more = 0;
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
      ok = __all_sync(0xffffffffu, ptx::mbar_wait_bounded(full_bar(stage), phase, abort, WAIT_LIMIT_NS));
      if (!ok) break;
      ptx::tc_fence_after();
      const int n = min(p.ka, p.num_kb - i * p.ka);
      for (int a = 0; a < n; ++a) {
        const uint64_t w0 = w_desc0 + (uint64_t)((stage * p.ka + a) * (atom_w >> 4));
        const uint64_t a0 = a_desc0 + (uint64_t)((stage * p.ka + a) * (atom_a >> 4));
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::tc_mma_i8(tmem_base, w0 + (uint64_t)(k * 2), a0 + (uint64_t)(k * 2), IDESC, k != 0 ? 1u : more);
        }
        __syncwarp();
        more = 1u;
      }
      if (ptx::elect_one()) ptx::tc_commit(empty_bar(stage));
      __syncwarp();
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
    if (ptx::elect_one()) {
      if (!ok && !*abort) record_timeout(err, WHERE_GEMM_MMA, abort);
      ptx::tc_commit(done_bar);
      volatile int never = 0;
      if (!ptx::mbar_wait_bounded(done_bar, 0, &never, WAIT_LIMIT_NS)) record_timeout(err, WHERE_GEMM_DRAIN, abort);
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    if (quarter * 32 < p.ct) {   // whole warps past the channels have nothing to do
      const int n = row < p.ct ? n0 + row : ep.N;   // ep.N: no channel
      const float sn = n < ep.N ? ep.w_scale[n] : 0.f;
      const float bn = n < ep.N && ep.bias != nullptr ? ep.bias[n] : 0.f;
      constexpr int CH = BN % 32 == 0 ? 32 : 16;   // tokens of a chunk
      Ahead<KIND, CH> next;
      next.load(ep, n, t0, lane);
      const bool ok = ptx::mbar_wait_bounded(done_bar, 0, abort, WAIT_LIMIT_NS);
      if (!ok && !*abort) record_timeout(err, WHERE_GEMM_EPILOGUE, abort);
      ptx::tc_fence_after();
      if (__all_sync(0xffffffffu, ok)) {
        const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < BN; c += CH) {
          const int m0 = t0 + c;
          if (m0 >= ep.M) break;
          float f[CH];
          int v[CH];
          ptx::tmem_ld(taddr + c, f);
          const Ahead<KIND, CH> now = next;
          if (c + CH < BN) next.load(ep, n, m0 + CH, lane);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < CH; ++j) v[j] = __float_as_int(f[j]);
          store_tokens<KIND, OutT, CH>(ep, n, sn, bn, m0, now, v);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, COLS);
  }
}

// ---------------------------------------------------------------- host side

template <int BN, int KIND, typename OutT>
cudaError_t launch_pair(const GemmI8& g, const I8Epi& ep, DevError* err, cudaStream_t st, int num_sms) {
  using C = PairCfg<BN>;
  auto kern = gemm_i8_pair_kernel<BN, KIND, OutT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap tw, ta;
  if (make_tmap_i8(&tw, g.W, g.N, g.K, g.ldw, 128) || make_tmap_i8(&ta, g.A, g.M, g.K, g.lda, BN / 2))
    return cudaErrorInvalidValue;
  const int nw = (g.N + 255) / 256, nt = (g.M + BN - 1) / BN;
  const long tiles = (long)nw * nt;
  if (tiles > INT_MAX - num_sms) return cudaErrorInvalidValue;   // (a CTA steps past the last tile by the grid)
  const int pairs = (int)(tiles < num_sms / 2 ? tiles : num_sms / 2);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(P_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tw, ta, nw, nt, (g.K + C::KA * BK - 1) / (C::KA * BK), ep, err);
}

template <int BN, int KIND, typename OutT>
cudaError_t launch_small(const GemmI8& g, const I8Epi& ep, int ct, DevError* err, cudaStream_t st) {
  SmallPlan p;
  p.ct = ct;
  p.num_kb = (g.K + BK - 1) / BK;
  p.whole = g.K / BK;
  p.ka = ct + BN <= 64 ? 4 : ct + BN <= 128 ? 2 : 1;   // 16 to 32 KB a stage
  const int steps = (p.num_kb + p.ka - 1) / p.ka;
  const long room = (long)S_SMEM_MAX - 1024 - small_pad_bytes(p) - (2 * S_MAX_STAGES + 1) * 8 - 16;
  p.stages = (int)(room / small_stage_bytes(p, BN));
  if (p.stages > S_MAX_STAGES) p.stages = S_MAX_STAGES;
  if (p.stages > steps) p.stages = steps;
  auto kern = gemm_i8_small_kernel<BN, KIND, OutT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S_SMEM_MAX);
  if (e != cudaSuccess) return e;
  CUtensorMap tw, ta, twt, tat;
  if (make_tmap_i8(&twt, g.W, g.N, g.K, g.ldw, ct) || make_tmap_i8(&tat, g.A, g.M, g.K, g.lda, BN))
    return cudaErrorInvalidValue;
  tw = twt;
  ta = tat;
  if (p.whole > 0 && (make_tmap_i8_blocks(&tw, g.W, g.N, g.K, g.ldw, ct, p.ka) ||
                      make_tmap_i8_blocks(&ta, g.A, g.M, g.K, g.lda, BN, p.ka)))
    return cudaErrorInvalidValue;
  return launch_kernel(kern, dim3((unsigned)((g.N + ct - 1) / ct), (unsigned)((g.M + BN - 1) / BN)), dim3(S_THREADS),
                       small_smem(p, BN), st, tw, ta, twt, tat, p, ep, err);
}

// Tile and kernel of a call, by estimated cycles.  An SM takes about 48 bytes a cycle from L2 and
// does 16384 8-bit MMA operations; a 32-token chunk of an epilogue warp takes about 1500
// cycles, and a tile's set-up and first loads 3000.
struct Choice {
  bool pair;
  int bn, ct;
};
Choice choose(int M, int N, int K, int num_sms) {
  const double atoms = (K + BK - 1) / BK;
  Choice best{true, 256, 256};
  double least = 1e30;
  auto offer = [&](double cost, Choice c) {
    if (cost < least) {
      least = cost;
      best = c;
    }
  };
  for (int bn : {64, 96, 128, 160, 192, 224, 256}) {
    const double tiles = (double)((N + 255) / 256) * ((M + bn - 1) / bn);
    const double rounds = ceil(tiles / (num_sms / 2));
    const double main = atoms * fmax(2.0 * bn, (16384 + 64.0 * bn) / 48), epi = 500 + 1500.0 * ((bn + 63) / 64);
    offer(3000 + rounds * fmax(main, epi) + epi, Choice{true, bn, 256});
  }
  for (int bn : {16, 32, 48, 64, 96, 128})
    for (int ct : {16, 32, 64, 128}) {
      if ((M + bn - 1) / bn > 65535) continue;
      const double tiles = (double)((N + ct - 1) / ct) * ((M + bn - 1) / bn);
      const double rounds = ceil(tiles / num_sms);
      const double main = atoms * fmax(4.0 * bn, 128.0 * (ct + bn) / 48), epi = 500 + 1500.0 * ((bn + 31) / 32);
      offer(rounds * (3000 + main + epi), Choice{false, bn, ct});
    }
  return best;
}

template <int KIND, typename OutT>
cudaError_t run(const GemmI8& g, DevError* err, cudaStream_t st, int num_sms) {
  I8Epi ep{g.a_scale, g.w_scale, g.bias, g.resid, g.ldr, g.out, g.ldo, g.M, g.N};
  const Choice c = choose(g.M, g.N, g.K, num_sms);
  if (c.pair) {
    switch (c.bn) {
      case 64: return launch_pair<64, KIND, OutT>(g, ep, err, st, num_sms);
      case 96: return launch_pair<96, KIND, OutT>(g, ep, err, st, num_sms);
      case 128: return launch_pair<128, KIND, OutT>(g, ep, err, st, num_sms);
      case 160: return launch_pair<160, KIND, OutT>(g, ep, err, st, num_sms);
      case 192: return launch_pair<192, KIND, OutT>(g, ep, err, st, num_sms);
      case 224: return launch_pair<224, KIND, OutT>(g, ep, err, st, num_sms);
      default: return launch_pair<256, KIND, OutT>(g, ep, err, st, num_sms);
    }
  }
  switch (c.bn) {
    case 16: return launch_small<16, KIND, OutT>(g, ep, c.ct, err, st);
    case 32: return launch_small<32, KIND, OutT>(g, ep, c.ct, err, st);
    case 48: return launch_small<48, KIND, OutT>(g, ep, c.ct, err, st);
    case 64: return launch_small<64, KIND, OutT>(g, ep, c.ct, err, st);
    case 96: return launch_small<96, KIND, OutT>(g, ep, c.ct, err, st);
    default: return launch_small<128, KIND, OutT>(g, ep, c.ct, err, st);
  }
}

}  // namespace

cudaError_t gemm_i8(const GemmI8& g, int kind, bool out_f32, DevError* err, cudaStream_t st, int num_sms) {
  switch (kind) {
    case EPI_BIAS:
      return out_f32 ? run<EPI_BIAS, float>(g, err, st, num_sms) : run<EPI_BIAS, bf16>(g, err, st, num_sms);
    case EPI_BIAS_GELU: return run<EPI_BIAS_GELU, bf16>(g, err, st, num_sms);
    case EPI_BIAS_SILU: return run<EPI_BIAS_SILU, bf16>(g, err, st, num_sms);
    case EPI_BIAS_RESID: return run<EPI_BIAS_RESID, float>(g, err, st, num_sms);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kd
