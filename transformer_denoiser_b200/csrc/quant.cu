// Rows in 8-bit integers with one scale each: the plain quantisation of rows (weights per
// output channel, activations per token) and the RMS norm that adds the residual and
// quantises its result.
//
// For a row t: scale = max |t| / 127, q = rint(127 t / max |t|).  The norm's row is
// t = h gamma / rms(h), h = x + residual, and since the rms divides every t alike it
// cancels in q: one pass over the row in registers gives sum h^2 and max |h gamma|
// together, q follows from the second and only the scale needs the first.  So the row is
// read once, reduced once and written once; the kernel is bound by DRAM traffic.
//
// A row is spread over TPR threads, NG groups of 8 values each.  Where every row starts
// on a 16-byte boundary (8 for q) and the columns divide by 8, a group is 8 consecutive
// values (vector loads); otherwise its values lie TPR columns apart, so that the scalar
// loads of a warp still fall on consecutive addresses.
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "ptx.cuh"

namespace kd {
namespace {

struct NoResidual {};

template <typename T> struct Elem { static constexpr int size = sizeof(T); };
template <> struct Elem<NoResidual> { static constexpr int size = 0; };

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// Sum and maximum (of non-negative floats, compared as bits, so that a NaN wins) over the
// TPR threads of a row.
template <int TPR>
__device__ __forceinline__ void row_reduce(float& s, uint32_t& m, float* xs, uint32_t* xm) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();   // the arrays may still be read from an earlier reduction
    if ((threadIdx.x & 31) == 0) {
      xs[warp] = s;
      xm[warp] = m;
    }
    __syncthreads();
    s = 0.f;
    m = 0;
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) {
      s += xs[w];
      m = max(m, xm[w]);
    }
  }
}

// Rows in flight hide the latency of their one pass, so registers are held down where the
// compiler would take more than these CTAs an SM leave (norm of 8192 x 4096: 59 -> 49 us;
// quantisation of 12289 x 2731 fp32: 41 -> 38 us).
constexpr int ctas_per_sm(bool norm, int tpr) { return norm ? (tpr == 256 ? 5 : tpr == 64 ? 20 : 1) : tpr == 128 ? 8 : 1; }

template <typename TX, typename TR, bool NORM, int TPR, int NG, bool VEC>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR, ctas_per_sm(NORM, TPR)) rows_int8_kernel(RowsInt8 a) {
  constexpr bool RES = Elem<TR>::size != 0;
  __shared__ float xs[TPR / 32];
  __shared__ uint32_t xm[TPR / 32];
  ptx::pdl_wait();
  ptx::pdl_trigger();
  const int t = TPR == 32 ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const long row = TPR == 32 ? (long)blockIdx.x * 4 + (threadIdx.x >> 5) : (long)blockIdx.x;
  if (row >= a.rows) return;   // whole warps (TPR 32) or never
  const int cols = a.cols;
  const TX* x = static_cast<const TX*>(a.x) + row * a.ldx;
  auto column = [&](int i, int e) { return VEC ? (i * TPR + t) * 8 + e : (i * 8 + e) * TPR + t; };
  float h[NG][8], g[NORM ? NG : 1][8];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    if constexpr (VEC) {
      const int c = column(i, 0);
      if (c < cols) {
        load8(x + c, h[i]);
        if constexpr (NORM) load8(a.gamma + c, g[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[i][e] = 0.f;
          if constexpr (NORM) g[i][e] = 0.f;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column(i, e);
        h[i][e] = c < cols ? load1(x + c) : 0.f;
        if constexpr (NORM) g[i][e] = c < cols ? a.gamma[c] : 0.f;
      }
    }
  }
  if constexpr (RES) {
    const TR* r = static_cast<const TR*>(a.r_in) + row * a.ldr_in;
    TR* ro = static_cast<TR*>(a.r_out) + row * a.ldr_out;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if constexpr (VEC) {
        const int c = column(i, 0);
        if (c < cols) {
          float v[8];
          load8(r + c, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[i][e] += v[e];
          store8(ro + c, h[i]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = column(i, e);
          if (c < cols) {
            h[i][e] += load1(r + c);
            store1(ro + c, h[i][e]);
          }
        }
      }
    }
  }
  float s = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (NORM) s = fmaf(h[i][e], h[i][e], s);
      const float v = NORM ? h[i][e] * g[NORM ? i : 0][e] : h[i][e];
      top = max(top, __float_as_uint(fabsf(v)));
    }
  row_reduce<TPR>(s, top, xs, xm);
  const bool finite = top < 0x7f800000u;
  const float amax = __uint_as_float(top);
  float scale = amax / 127.f;
  if constexpr (NORM) {
    const float mean = s / (float)cols + a.eps;
    if (mean >= 1e-30f && s < INFINITY) {
      scale = amax / (127.f * sqrtf(mean));
    } else {
      // squares past the largest float, or so small that those which underflow would count (above
      // 1e-30 they are less than 2^-26 of the mean): the sum of the squares of h / max |h| instead
      float hs = 0.f;
      uint32_t ht = 0;
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ht = max(ht, __float_as_uint(fabsf(h[i][e])));
      float zero = 0.f;
      row_reduce<TPR>(zero, ht, xs, xm);
      const float hm = __uint_as_float(ht);
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = h[i][e] / hm;
          hs = fmaf(v, v, hs);
        }
      ht = 0;
      row_reduce<TPR>(hs, ht, xs, xm);
      // (NaN where a value is not finite; eps so far above the squares that its share leaves the range: eps alone)
      const float e = a.eps / hm / hm;
      scale = e < INFINITY ? amax / hm / (127.f * sqrtf(hs / (float)cols + e)) : amax / (127.f * sqrtf(a.eps));
    }
  }
  if (t == 0) a.scale[row] = !finite ? __uint_as_float(0x7fc00000u) : top == 0 ? 0.f : scale;
  // q = rint(t * (127 / max |t|)), quotient and product in fp32: adding 1.5 * 2^23 leaves the
  // rounded integer (ties to even) in the low bits of the sum.  A maximum near the smallest
  // floats is scaled up first, so that 127 / max stays finite.
  const float up = amax < 0x1p-100f ? 0x1p100f : 1.f;
  const float inv = finite && top != 0 ? 127.f / (amax * up) : 0.f;
  int8_t* q = a.q + row * a.ldq;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = (NORM ? h[i][e] * g[NORM ? i : 0][e] : h[i][e]) * up;
      b[e] = finite ? __float_as_uint(__fadd_rn(__fmul_rn(v, inv), 12582912.f)) : 0u;
    }
    if constexpr (VEC) {
      const int c = column(i, 0);
      if (c < cols) {
        const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
        *reinterpret_cast<uint2*>(q + c) = make_uint2(lo, hi);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column(i, e);
        if (c < cols) q[c] = (int8_t)(b[e] & 0xffu);
      }
    }
  }
}

bool aligned(const void* p, long ld, int elem, int to) {
  return (reinterpret_cast<uintptr_t>(p) % to) == 0 && (ld * elem) % to == 0;
}

template <typename TX, typename TR, bool NORM>
cudaError_t run_rows(const RowsInt8& a, cudaStream_t st) {
  constexpr int rsz = Elem<TR>::size;
  const bool vec = a.cols % 8 == 0 && aligned(a.x, a.ldx, sizeof(TX), 16) && aligned(a.q, a.ldq, 1, 8) &&
                   (!NORM || aligned(a.gamma, 0, 4, 16)) &&
                   (rsz == 0 || (aligned(a.r_in, a.ldr_in, rsz, 16) && aligned(a.r_out, a.ldr_out, rsz, 16)));
#define KD_ROWS(TPR_, NG_)                                                                                  \
  if (a.cols <= TPR_ * NG_ * 8) {                                                                           \
    const long grid = TPR_ == 32 ? ((long)a.rows + 3) / 4 : (long)a.rows;                                   \
    const int block = TPR_ == 32 ? 128 : TPR_;                                                              \
    return vec ? launch_kernel(rows_int8_kernel<TX, TR, NORM, TPR_, NG_, true>, dim3((unsigned)grid), dim3(block), \
                               0, st, a)                                                                    \
               : launch_kernel(rows_int8_kernel<TX, TR, NORM, TPR_, NG_, false>, dim3((unsigned)grid),      \
                               dim3(block), 0, st, a);                                                      \
  }
  // The quantisation alone runs best with a row in one warp or few (38528 x 1024 bf16: 19.6 us with
  // 32 threads a row, 40 with 64 or 128); the norm, which holds gamma and reads the residual too,
  // with fewer values a thread (38528 x 1024: 67.8 us with 64 threads, 86.8 with 32;
  // 8192 x 4096: 53 us with 256, 59 with 128).
  if constexpr (NORM) {
    KD_ROWS(64, 2)
    KD_ROWS(256, 2)
    KD_ROWS(1024, 2)
  } else {
    KD_ROWS(32, 4)
    KD_ROWS(128, 4)
    KD_ROWS(512, 4)
  }
  KD_ROWS(1024, 4)
#undef KD_ROWS
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t quantize_rows_int8(const RowsInt8& a, bool x_bf16, cudaStream_t st) {
  return x_bf16 ? run_rows<bf16, NoResidual, false>(a, st) : run_rows<float, NoResidual, false>(a, st);
}

cudaError_t rms_norm_rows_int8(const RowsInt8& a, bool x_bf16, bool r_bf16, cudaStream_t st) {
  if (a.r_in == nullptr)
    return x_bf16 ? run_rows<bf16, NoResidual, true>(a, st) : run_rows<float, NoResidual, true>(a, st);
  if (r_bf16) return x_bf16 ? run_rows<bf16, bf16, true>(a, st) : run_rows<float, bf16, true>(a, st);
  return x_bf16 ? run_rows<bf16, float, true>(a, st) : run_rows<float, float, true>(a, st);
}

}  // namespace kd
