// mlr_router.cuh -- what the router's choice and the balance loss have in common:
// logits as fp32, their exponentials and sigmoids, and a token's logits in the lanes of a
// part of a warp.
#pragma once
#include <math_constants.h>

#include <initializer_list>

#include "mlr_profile.cuh"
#include "mlr_rows.cuh"

namespace mlr {

constexpr int kMaxRouteExperts = 4096;
constexpr int kMaxRouteTopk = 32;
constexpr int kPartExperts = 1024;  // a part of a warp holds a token of up to this many experts

enum Scoring { kSoftmax = 0, kSigmoid = 1 };

// A logit as fp32, -inf where it is not finite.
__device__ __forceinline__ float finite_logit(float v) { return fabsf(v) < CUDART_INF_F ? v : -CUDART_INF_F; }
template <typename E_>
__device__ __forceinline__ float finite_logit(const E_* p) {
  return finite_logit(row_widen(*p));
}
// By e^-|v|, which does not overflow: fp32's bits down to -87, 0 below -103.
__device__ __forceinline__ float sigmoid_f(float v) {
  const float e = expf(-fabsf(v));
  return (v < 0.f ? e : 1.f) / (1.f + e);
}
// Sums of sigmoids down to the smallest float are divisors: what is multiplied by this
// first, divisor and dividends, has a reciprocal.
__device__ __forceinline__ float lift_of(float total) { return total < 0x1p-100f ? 0x1p100f : 1.f; }
// The same with the hardware's exponential and reciprocal: relative error below
// (|v| + 5) 2^-23, at most 2.25 2^-23 as a difference.
__device__ __forceinline__ float quick_sigmoid(float v) {
  float e, r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(v * -1.44269504f));
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
// e^x for x <= 0 in a few instructions, whatever x within 5 2^-24 of itself (3.3 measured from
// -87 to 0; 64 without the remainder): 2^h with h = x / ln 2 rounded, times 1 plus x - h ln 2,
// which the rounding leaves.  0 below 2^-126.
__device__ __forceinline__ float share_exp(float x) {
  x = fmaxf(x, -100.f);  // -inf has no remainder
  const float h = x * 1.44269504f, left = fmaf(h, 1.90465421e-9f, fmaf(h, -0x1.62e43p-1f, x));  // ln 2 in two parts
  float p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(h));
  return fmaf(p, left, p);
}
// The sigmoid within 9 2^-24 of itself down to -87; in `slope` s (1 - s) from the smaller of
// the two, as 1 - s from s would cancel.
__device__ __forceinline__ float share_sigmoid(float v, float& slope) {
  const float e = share_exp(-fabsf(v));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  slope = e * r * r;
  return v < 0.f ? e * r : r;
}
__device__ __forceinline__ float share_sigmoid(float v) {
  float slope;
  return share_sigmoid(v, slope);
}

// A token's logits in LPT lanes, V each: unit j of lane ll is number ll + LPT j, VEC
// logits (16 bytes, or one where rows lie off that grid).
template <typename E_, int VEC>
__device__ __forceinline__ void load_unit(const E_* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) v[0] = row_widen(__ldg(p));
  else row_widen(__ldg(reinterpret_cast<const uint4*>(p)), v);
}
// NaN if one of them is not finite, else 0.
template <int V>
__device__ __forceinline__ float check_finite(const float (&v)[V]) {
  float2 check = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < V; i += 2) check = __ffma2_rn(make_float2(v[i], v[i + 1]), make_float2(0.f, 0.f), check);
  return check.x + check.y;
}
// The larger of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest of v[FIRST], v[FIRST + STEP], ...
template <int FIRST, int STEP, int V>
__device__ __forceinline__ float max_of(const float (&v)[V]) {
  float m = v[FIRST];
#pragma unroll
  for (int i = FIRST + STEP; i < V; i += 2 * STEP) m = i + STEP < V ? max3(m, v[i], v[i + STEP < V ? i + STEP : i]) : fmaxf(m, v[i]);
  return m;
}
// Loads them: zeros past E, and all where `active` is not set.
template <int VEC, int LPT, int V, typename E_>
__device__ __forceinline__ void load_logits(const E_* row, int E, int ll, bool active, float (&v)[V]) {
  if (E == LPT * V && __all_sync(0xffffffffu, active)) {  // nothing to put in the place of any
#pragma unroll
    for (int j = 0; j < V / VEC; ++j) {
      float u[VEC];
      load_unit<E_, VEC>(row + (ll + LPT * j) * VEC, u);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j * VEC + i] = u[i];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V / VEC; ++j) {
    const int e = (ll + LPT * j) * VEC;
    float u[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) u[i] = 0.f;
    if (active && e < E) load_unit<E_, VEC>(row + e, u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[j * VEC + i] = u[i];
  }
}
// Logits on the 16-byte grid can be fetched a turn ahead: every thread of a block of
// THREADS copies the units that it takes to places of its own in shared memory (16 bytes
// each, one for every unit and thread), which asks for no barrier; once they are in
// registers their places are free for the next turn's.
template <int VEC, int LPT, int V, int THREADS, typename E_>
__device__ __forceinline__ void fetch_logits(uint4* ring, const E_* row, int E, int ll, bool have) {
  if (have)
#pragma unroll
    for (int j = 0; j < V / VEC; ++j) {
      const int e = (ll + LPT * j) * VEC;
      if (e < E)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(ring + j * THREADS + threadIdx.x)), "l"(row + e)
                     : "memory");
    }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int VEC, int LPT, int V, int THREADS>
__device__ __forceinline__ void take_logits(const uint4* ring, int E, int ll, bool active, float (&v)[V]) {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int j = 0; j < V / VEC; ++j) {
    float u[VEC] = {};
    if (active && (ll + LPT * j) * VEC < E) row_widen(ring[j * THREADS + threadIdx.x], u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[j * VEC + i] = u[i];
  }
}
// -inf past E.
template <int VEC, int LPT, int V>
__device__ __forceinline__ void close_past(int E, int ll, float (&v)[V]) {
  if (E < LPT * V)
#pragma unroll
    for (int j = 0; j < V / VEC; ++j)
      if ((ll + LPT * j) * VEC >= E)
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j * VEC + i] = -CUDART_INF_F;
}

template <int LPT>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPT>
__device__ __forceinline__ float part_max(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Launches with `smem` bytes of dynamic shared memory.  Above what needs no opt-in the
// kernel is given `most`, which all of its calls stay below, not what this one needs: a
// smaller call in another thread must not lower the limit before this one's launch.
template <typename Kernel, typename... Args>
int launch_with_smem(Kernel kernel, dim3 grid, dim3 block, size_t smem, int most, cudaStream_t stream, Args... args) {
  cudaError_t err = cudaSuccess;
  if (smem > 46 * 1024) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (err == cudaSuccess) err = launch_pdl(kernel, grid, block, smem, stream, args...);
  return launched(err);
}

inline int check_logits(const void* logits, int32_t T, int32_t E, int32_t K, int32_t dtype, int32_t scoring) {
  if (T < 0 || E < 1 || K < 1 || (dtype != MLR_DTYPE_BF16 && dtype != MLR_DTYPE_F32) ||
      (scoring != kSoftmax && scoring != kSigmoid))
    return MLR_ERR_INVALID;
  if (E > kMaxRouteExperts || K > kMaxRouteTopk || (int64_t)T * K >= INT32_MAX) return MLR_ERR_UNSUPPORTED;
  if (T > 0 && (logits == nullptr || !aligned_to(logits, dtype == MLR_DTYPE_BF16 ? 2 : 4))) return MLR_ERR_INVALID;
  return MLR_OK;
}
// Whether arrays of 32-bit elements lie on their grid (those not given do).
inline bool on_word_grid(std::initializer_list<const void*> arrays) {
  for (const void* p : arrays)
    if (!aligned_to(p, 4)) return false;
  return true;
}

}  // namespace mlr
