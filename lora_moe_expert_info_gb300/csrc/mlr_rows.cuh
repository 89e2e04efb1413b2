// mlr_rows.cuh -- 16-byte vectors of rows as fp32 values, and sums and maxima
// over warps, for the operators that work row by row.
#pragma once
#include "mlr_common.cuh"

namespace mlr {

// bf16 (as uint16_t) and float32 elements and vectors as fp32 values, and back
// (rounded to nearest, ties to even).
__device__ __forceinline__ float row_widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float row_widen(float v) { return v; }
__device__ __forceinline__ void row_narrow(float f, uint16_t& o) { o = f32_to_bf16_bits(f); }
__device__ __forceinline__ void row_narrow(float f, float& o) { o = f; }
__device__ __forceinline__ void row_widen(const uint4& q, float (&v)[4]) {
  v[0] = __uint_as_float(q.x);
  v[1] = __uint_as_float(q.y);
  v[2] = __uint_as_float(q.z);
  v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void row_widen(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t row_narrow2(float a, float b) {
  uint32_t o;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(b), "f"(a));
  return o;
}
__device__ __forceinline__ void row_narrow(const float (&v)[4], uint4& q) {
  q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void row_narrow(const float (&v)[8], uint4& q) {
  q = make_uint4(row_narrow2(v[0], v[1]), row_narrow2(v[2], v[3]), row_narrow2(v[4], v[5]), row_narrow2(v[6], v[7]));
}

// Elementwise fp32 operations on the values of a vector, two to an instruction; each is
// rounded as the single operation is.
template <int N>
__device__ __forceinline__ void row_add(float (&a)[N], const float (&b)[N]) {
  if constexpr (N == 1) a[0] += b[0];
  else
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 s = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      a[i] = s.x;
      a[i + 1] = s.y;
    }
}
template <int N>
__device__ __forceinline__ void row_mul(float (&a)[N], const float (&b)[N]) {
  if constexpr (N == 1) a[0] *= b[0];
  else
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 s = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      a[i] = s.x;
      a[i + 1] = s.y;
    }
}
template <int N>
__device__ __forceinline__ void row_scale(float (&a)[N], float b) {
  if constexpr (N == 1) a[0] *= b;
  else
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 s = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b, b));
      a[i] = s.x;
      a[i + 1] = s.y;
    }
}
// c[i] + a[i] b[i], and the sum over i of a[i] b[i] (two chains).
template <int N>
__device__ __forceinline__ void row_fma(const float (&a)[N], const float (&b)[N], float (&c)[N]) {
  if constexpr (N == 1) c[0] = fmaf(a[0], b[0], c[0]);
  else
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 s = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
      c[i] = s.x;
      c[i + 1] = s.y;
    }
}
template <int N>
__device__ __forceinline__ float row_dot(const float (&a)[N], const float (&b)[N]) {
  if constexpr (N == 1) return a[0] * b[0];
  else {
    float2 s = __fmul2_rn(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
#pragma unroll
    for (int i = 2; i < N; i += 2) s = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), s);
    return s.x + s.y;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

inline bool aligned_to(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// SMs of the current device (152 where it cannot be asked).
inline int current_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return 152;
  }
  return n;
}

}  // namespace mlr
