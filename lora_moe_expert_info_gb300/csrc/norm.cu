// norm.cu -- the residual's addition and a root-mean-square norm, its output
// also in 8 bits, and the gradients.
//
// Per row of H columns, with r = x + residual rounded to the rows' type (r = x
// without a residual) and m = 1 / sqrt(mean(r^2) + eps):
//   y = r m w                                              rounded to the type
//   8 bits per group of 128 columns, from y so rounded: scale 2^s with s the
//   smallest integer >= -127 with max|y| <= 448 2^s (0 for zeros), code the
//   nearest E4M3 value of y 2^-s -- the W8A8 layer's own quantisation of x
//   dr = m (h - r m^2 mean(h r)) + d_r,  h = dy w           (d_r: what reaches r otherwise)
//   dw = sum over rows of dy r m
// Sums, m and dw are held in fp32.
//
// A row stays in the registers of its threads (the gradients': in their places of
// shared memory) between the pass that reads it and the one that writes it, so every
// tensor is moved once, and HBM bounds all of it.  8192 rows of 7168 bf16: residual and
// norm 71 us (97% of the copy rate), with the 8 bits 87 (89%: 47% of the issue slots at 20
// warps an SM, whose 96 registers spill 88 bytes a thread), gradients 76 (91%), 8 bits
// back 27 (97%).  float32: 144 (96%), gradients 136.  1 to 256 rows: 2 to 4 us.  Rows off the
// 16-byte grid go element by element, 24 to 84% of the rate, their gradients 14 to 63%.
#include <cuda_fp16.h>

#include <initializer_list>
#include <type_traits>

#include "mlr_profile.cuh"
#include "mlr_rows.cuh"

namespace mlr {
namespace {

constexpr int kMaxNormHidden = 16384;
constexpr int kGroupCols = 128;  // columns of an 8-bit scale

// How the threads of a row hold it: LPT threads (a multiple of 32), NV units
// each.  VEC > 1: a unit is 16 bytes, VEC elements; unit j of thread lt is number
// lt + j LPT.  VEC == 1 (rows or bases off the 16-byte grid): a unit is one
// element, and a warp takes 128 columns at a time, four units a lane, so that
// here too a group's columns lie in one warp.
template <int VEC>
__device__ __forceinline__ int unit_col(int lt, int j, int lpt) {
  if (VEC > 1) return (lt + j * lpt) * VEC;
  return ((lt >> 5) + (j >> 2) * (lpt >> 5)) * kGroupCols + (j & 3) * 32 + (lt & 31);
}

template <typename E_, int VEC> struct Unit { using T = uint4; };
template <typename E_> struct Unit<E_, 1> { using T = E_; };

__device__ __forceinline__ void widen_unit(const uint4& q, float (&v)[8]) { row_widen(q, v); }
__device__ __forceinline__ void widen_unit(const uint4& q, float (&v)[4]) { row_widen(q, v); }
__device__ __forceinline__ void widen_unit(uint16_t q, float (&v)[1]) { v[0] = row_widen(q); }
__device__ __forceinline__ void widen_unit(float q, float (&v)[1]) { v[0] = q; }
__device__ __forceinline__ void narrow_unit(const float (&v)[8], uint4& q) { row_narrow(v, q); }
__device__ __forceinline__ void narrow_unit(const float (&v)[4], uint4& q) { row_narrow(v, q); }
__device__ __forceinline__ void narrow_unit(const float (&v)[1], uint16_t& q) { row_narrow(v[0], q); }
__device__ __forceinline__ void narrow_unit(const float (&v)[1], float& q) { q = v[0]; }

// VEC columns of the weight (bf16 or float32, whatever the rows' type) as they lie in
// memory, so that they take few registers while a row's sum is found.
template <typename W_, int VEC>
struct WeightUnit {
  uint32_t w[VEC * sizeof(W_) / 4];
  __device__ __forceinline__ void load(const W_* p) {
    if constexpr (VEC * sizeof(W_) == 8) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = q.x; w[1] = q.y;
    } else {
#pragma unroll
      for (int i = 0; i < (int)(VEC * sizeof(W_) / 16); ++i) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(W_) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};
template <typename W_>
struct WeightUnit<W_, 1> {
  W_ w;
  __device__ __forceinline__ void load(const W_* p) { w = __ldg(p); }
  __device__ __forceinline__ float at(int) const { return row_widen(w); }
};

// The exponent s of a group from the fp32 bits of its largest magnitude: the
// smallest integer with amax 2^-s <= 448 = 1.75 2^8, not below -127; 0 for zeros.
__device__ __forceinline__ int group_exp(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = (int)(amax >> 23);
  if (e == 0) return -127;
  return max(-127, e - 127 - ((amax & 0x7fffffu) <= 0x600000u ? 8 : 7));
}

// Sum of two values over the LPT threads of a row; `red` has 2 floats per warp
// of the block.  Every thread of the block calls it.
__device__ __forceinline__ float2 row_sum2(float a, float b, int lpt, float2* red) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (lpt == 32) return make_float2(a, b);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wpr = lpt >> 5;
  if (lane == 0) red[warp] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < wpr ? red[warp / wpr * wpr + lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

// Two sums of bf16, each rounded once from the exact sum.  That is the fp32 sum rounded:
// where 24 bits do not hold it exactly, one term is below 2^-16 of the other and neither
// rounding moves the larger one.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t s;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(s) : "r"(a), "r"(b));
  return s;
}

// 1 / sqrt(mean + eps) of a row as up (hi + lo), from its threads' sums of squares.  The
// rounding errors of threads and warps average out over a row; what is left of fp32's
// errors from there on would move values over rounding borders of bf16 or of the 8 bits, so
// the last sums, the quotient and the root carry their remainders, and y is rounded once
// (8192 x 7168 bf16: 140 values off a border, 480 without).  up is a power of two and hi + lo
// in [1, 2]; lo > 2^-20, so that what it gives has the sign of what hi does and products of
// infinity stay infinite.  No branch: one costs 3 to 13% of the time of a row.
// `red`: a float per warp of the block; every thread of the block calls it.
struct InverseRms { float up, hi, lo; };
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x;
  return make_float2(s, (a.x - (s - t)) + (b.x - t) + a.y + b.y);
}
__device__ __forceinline__ InverseRms row_inverse_rms(float sum, int H, float eps, int lpt, float* red) {
  float2 s = make_float2(warp_sum(sum), 0.f);
  if (lpt > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wpr = lpt >> 5;
    if (lane == 0) red[warp] = s.x;
    __syncthreads();
    s.x = lane < wpr ? red[warp / wpr * wpr + lane] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)  // of at most 16 warps
      s = add2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
    s = make_float2(__shfl_sync(0xffffffffu, s.x, 0), __shfl_sync(0xffffffffu, s.y, 0));
  }
  const float h = (float)H, q = s.x / h;
  const float2 v = add2(make_float2(q, (fmaf(-q, h, s.x) + s.y) / h), make_float2(eps, 0.f));
  const float m = 1.f / sqrtf(v.x), p = m * m;
  // one step of Newton's, from the exact square of m (none where that is out of range)
  float left = fmaf(-v.y, p, fmaf(-v.x, fmaf(m, m, -p), fmaf(-v.x, p, 1.f)));
  if (!(fabsf(left) < 0x1p-20f)) left = 0.f;  // m is within two units of the last place
  const uint32_t b = __float_as_uint(m);
  const float hi = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);  // up is 0 or infinite where m is
  return {m == m ? __uint_as_float(b & 0x7f800000u) : m, hi - 0x1p-19f, fmaf(0.5f * hi, left, 0x1p-19f)};
}
// a w up (hi + lo), rounded once; what is multiplied first is a row near 1, so that it passes
// fp32's range only where y does.  EXACT (rows and weight in bf16): a w needs no more than
// fp32's bits.
template <bool EXACT, int N>
__device__ __forceinline__ void row_output(float (&a)[N], const float (&w)[N], InverseRms m) {
  if constexpr (EXACT) row_scale(a, m.up);
  const float h = EXACT ? m.hi : m.up * m.hi, l = EXACT ? m.lo : m.up * m.lo;
  if constexpr (N == 1) {
    const float p = a[0] * (EXACT ? w[0] : h);
    a[0] = EXACT ? fmaf(p, h, p * l) : fmaf(p, w[0], fmaf(a[0], l, fmaf(a[0], h, -p)) * w[0]);
  } else {
    const float2 hi = make_float2(h, h), lo = make_float2(l, l);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 x = make_float2(a[i], a[i + 1]), v = make_float2(w[i], w[i + 1]), p = __fmul2_rn(x, EXACT ? v : hi);
      float2 y;
      if constexpr (EXACT) {
        y = __ffma2_rn(p, hi, __fmul2_rn(p, lo));
      } else {
        const float2 left = __ffma2_rn(x, lo, __ffma2_rn(x, hi, make_float2(-p.x, -p.y)));
        y = __ffma2_rn(p, v, __fmul2_rn(left, v));
      }
      a[i] = y.x;
      a[i + 1] = y.y;
    }
  }
}

template <typename E_, typename W_, int VEC, int NV, bool QUANT, int MOST>
__global__ void __launch_bounds__(MOST, (NV <= (VEC == 1 ? 8 : 4) ? 1024 : VEC == 8 && QUANT ? 640 : 512) / MOST)
norm_kernel(const E_* x, const E_* residual, const W_* __restrict__ w, int T, int H, int lpt, float eps, E_* y, E_* r_out,
            uint8_t* codes, uint8_t* exps) {
  using U = typename Unit<E_, VEC>::T;
  __shared__ float red[16];
  const int sub = threadIdx.x / lpt, lt = threadIdx.x - sub * lpt;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / lpt) + sub;
  const bool in = row < T;
  const int64_t at = row * H;
  pdl_wait();
  pdl_trigger();
  constexpr bool kEarly = NV * VEC <= 32;  // the weight's columns are loaded before the sum is known
  U r[NV];
  WeightUnit<W_, VEC> wu[kEarly ? NV : 1];
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
    r[j] = in && c < H ? *reinterpret_cast<const U*>(x + at + c) : U{};
  }
  if (residual != nullptr) {
    U q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
      q[j] = in && c < H ? *reinterpret_cast<const U*>(residual + at + c) : U{};
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (VEC == 8) {
        r[j] = make_uint4(add_bf16x2(r[j].x, q[j].x), add_bf16x2(r[j].y, q[j].y), add_bf16x2(r[j].z, q[j].z),
                          add_bf16x2(r[j].w, q[j].w));
      } else {
        float a[VEC], b[VEC];
        widen_unit(r[j], a);
        widen_unit(q[j], b);
        row_add(a, b);
        narrow_unit(a, r[j]);
      }
      const int c = unit_col<VEC>(lt, j, lpt);
      if (in && c < H) *reinterpret_cast<U*>(r_out + at + c) = r[j];
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
    float a[VEC];
    widen_unit(r[j], a);
    sum += row_dot(a, a);
    if (kEarly && c < H) wu[kEarly ? j : 0].load(w + c);
  }
  const InverseRms m = row_inverse_rms(sum, H, eps, lpt, red);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
    float a[VEC];
    WeightUnit<W_, VEC>& wj = wu[kEarly ? j : 0];
    if (!kEarly && c < H) wj.load(w + c);
    if (c < H) {
      float wf[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) wf[i] = wj.at(i);
      widen_unit(r[j], a);
      row_output<sizeof(E_) == 2 && sizeof(W_) == 2>(a, wf, m);
      narrow_unit(a, r[j]);
    }
    if (in && c < H && y != nullptr) *reinterpret_cast<U*>(y + at + c) = r[j];
  }
  if constexpr (QUANT) {
    const int groups = (H + kGroupCols - 1) / kGroupCols;
    constexpr int UPG = VEC > 1 ? 1 : 4;           // units of a lane in a group
    constexpr int LANES = VEC > 1 ? kGroupCols / VEC : 32;  // lanes of a group
#pragma unroll
    for (int j = 0; j < NV; j += UPG) {
      float a[UPG][VEC];
      uint32_t most = 0;
#pragma unroll
      for (int u = 0; u < UPG; ++u) widen_unit(r[j + u], a[u]);
      if constexpr (VEC == 8) {  // magnitudes of bf16 are ordered as their bits: two at a time
        most = __vmaxu2(__vmaxu2(r[j].x & 0x7fff7fffu, r[j].y & 0x7fff7fffu), __vmaxu2(r[j].z & 0x7fff7fffu, r[j].w & 0x7fff7fffu));
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
        most = max(most & 0xffff0000u, most << 16);
      } else {
#pragma unroll
        for (int u = 0; u < UPG; ++u)
#pragma unroll
          for (int i = 0; i < VEC; ++i) most = max(most, __float_as_uint(a[u][i]) & 0x7fffffffu);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      }
      const int s = group_exp(most);
      const int c = unit_col<VEC>(lt, j, lpt);
#pragma unroll
      for (int u = 0; u < UPG; ++u) row_scale(a[u], exp2_neg(s));
      if constexpr (VEC > 1) {
        uint32_t q[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
          q[i] = f32x2_to_e4m3x2(a[0][4 * i], a[0][4 * i + 1]) | (f32x2_to_e4m3x2(a[0][4 * i + 2], a[0][4 * i + 3]) << 16);
        if (in && c < H) {
          if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes + at + c) = make_uint2(q[0], q[1]);
          else *reinterpret_cast<uint32_t*>(codes + at + c) = q[0];
        }
      } else {
#pragma unroll
        for (int u = 0; u < UPG; ++u)
          if (in && c + 32 * u < H) codes[at + c + 32 * u] = (uint8_t)f32x2_to_e4m3x2(a[u][0], 0.f);
      }
      if (in && c < H && (lt & (LANES - 1)) == 0) exps[row * groups + c / kGroupCols] = (uint8_t)(s + 127);
    }
  }
}

// The gradients.  A block takes rows blockIdx.x, + gridDim.x, ... (several at a
// time where rows are short) and its threads keep the same columns, so that dw's
// terms add up in registers; the blocks' sums go to `part` [blocks][H] and are added
// in order by sum_parts_kernel.
//
// One thread's units of a row: its gradient, and its terms of dw.
template <typename E_, int VEC, typename U>
__device__ __forceinline__ void row_terms(const U& ru, const U& gu, const float (&w)[VEC], float& ss, float& hr) {
  float a[VEC], g[VEC];
  widen_unit(ru, a);
  widen_unit(gu, g);
  ss += row_dot(a, a);
  row_mul(g, w);
  hr += row_dot(g, a);
}
template <typename E_, int VEC, typename U>
__device__ __forceinline__ U row_gradient(const U& ru, const U& gu, const U& eu, bool add, const float (&w)[VEC], float m,
                                          float k, float (&acc)[VEC]) {
  float a[VEC], g[VEC], d[VEC];
  widen_unit(ru, a);
  widen_unit(gu, g);
#pragma unroll
  for (int i = 0; i < VEC; ++i) d[i] = a[i];
  row_scale(d, m);
  row_fma(g, d, acc);
  // m g w - m^3 mean(h r) r, with k = -m^2 mean(h r)
  row_scale(d, k);
  row_mul(g, w);
  row_scale(g, m);
  row_add(d, g);
  if (add) {
    float e[VEC];
    widen_unit(eu, e);
    row_add(d, e);
  }
  U o;
  narrow_unit(d, o);
  return o;
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Rows on the 16-byte grid: every thread copies its own units of the next rows to
// shared memory (DEPTH rows in flight with the one in work, about 190 KB per SM), so
// that neither a barrier nor the sums wait for HBM.
template <typename E_, typename W_, int NV, int DEPTH, int MOST, int PER_SM>
__global__ void __launch_bounds__(MOST, PER_SM)
norm_backward_kernel(const E_* dy, const E_* r, const W_* __restrict__ w, const E_* d_r, int T, int H, int lpt, float eps,
                     E_* dx, float* __restrict__ part) {
  constexpr int VEC = 16 / sizeof(E_);
  extern __shared__ uint4 ring[];  // [DEPTH][3][NV][threads]
  __shared__ float2 red[2][32];
  const int threads = blockDim.x, rpb = threads / lpt;
  const int sub = threadIdx.x / lpt, lt = threadIdx.x - sub * lpt;
  auto slot = [&](int stage, int which, int j) { return ring + ((stage * 3 + which) * NV + j) * threads + threadIdx.x; };
  const int64_t step = (int64_t)gridDim.x * rpb;
  auto fetch = [&](int64_t row, int stage) {
    if (row < T) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = unit_col<VEC>(lt, j, lpt);
        if (c >= H) continue;
        copy_async16(slot(stage, 0, j), r + row * H + c);
        copy_async16(slot(stage, 1, j), dy + row * H + c);
        if (d_r != nullptr) copy_async16(slot(stage, 2, j), d_r + row * H + c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (unit_col<VEC>(lt, j, lpt) >= H)
      for (int i = 0; i < DEPTH * 3; ++i) *slot(i / 3, i % 3, j) = make_uint4(0, 0, 0, 0);  // never fetched
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * rpb + sub;
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) fetch(row0 + i * step, i);
  float wv[NV][VEC] = {}, acc[NV][VEC] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
    WeightUnit<W_, VEC> u;
    if (c < H) {
      u.load(w + c);
#pragma unroll
      for (int i = 0; i < VEC; ++i) wv[j][i] = u.at(i);
    }
  }
  int stage = 0, turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpb; base < T; base += step, turn ^= 1) {
    const int64_t row = base + sub;
    fetch(row + (DEPTH - 1) * step, stage == 0 ? DEPTH - 1 : stage - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    float ss = 0.f, hr = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) row_terms<E_, VEC>(*slot(stage, 0, j), *slot(stage, 1, j), wv[j], ss, hr);
    const float2 s = row_sum2(ss, hr, lpt, red[turn]);
    const float m = 1.f / sqrtf(s.x / (float)H + eps);
    const float k = -m * m * (s.y / (float)H);
    if (row < T) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = unit_col<VEC>(lt, j, lpt);
        if (c >= H) continue;
        *reinterpret_cast<uint4*>(dx + row * H + c) = row_gradient<E_, VEC>(
            *slot(stage, 0, j), *slot(stage, 1, j), *slot(stage, 2, j), d_r != nullptr, wv[j], m, k, acc[j]);
      }
    }
    stage = stage == DEPTH - 1 ? 0 : stage + 1;
  }
  float* p = part + (int64_t)blockIdx.x * H;
  if (rpb == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        if (c < H) *reinterpret_cast<float4*>(p + c + i) = make_float4(acc[j][i], acc[j][i + 1], acc[j][i + 2], acc[j][i + 3]);
    }
    return;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* sums = reinterpret_cast<float*>(ring);  // [rpb][H]: no more than the ring of a row
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c < H) sums[sub * H + c + i] = acc[j][i];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < H; c += threads) {
    float v = sums[c];
    for (int i = 1; i < rpb; ++i) v += sums[i * H + c];
    p[c] = v;
  }
}

template <typename W_, int VEC>
__device__ __forceinline__ void load_weight(const W_* w, int c, float (&v)[VEC]) {
  WeightUnit<W_, VEC> u;
  u.load(w + c);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = u.at(i);
}
// Rows off the 16-byte grid, and those too long for the ring: from registers, short
// ones with the next row loaded ahead (8192 rows of 1111 fp32: 64 -> 34 us).
template <typename E_, typename W_, int VEC, int NV, int MOST>
__global__ void __launch_bounds__(MOST)
norm_backward_plain_kernel(const E_* dy, const E_* r, const W_* __restrict__ w, const E_* d_r, int T, int H, int lpt,
                           float eps, E_* dx, float* __restrict__ part) {
  using U = typename Unit<E_, VEC>::T;
  __shared__ float2 red[2][32];
  const int lt = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  constexpr bool kNext = NV * VEC <= 8;  // the next row is loaded while this one is in work
  float acc[NV][VEC] = {};
  U rn[kNext ? NV : 1], gn[kNext ? NV : 1], en[kNext ? NV : 1];
  auto load = [&](int64_t row, U(&ru)[NV], U(&gu)[NV], U(&eu)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
      const bool have = row < T && c < H;
      ru[j] = have ? *reinterpret_cast<const U*>(r + row * H + c) : U{};
      gu[j] = have ? *reinterpret_cast<const U*>(dy + row * H + c) : U{};
      eu[j] = have && d_r != nullptr ? *reinterpret_cast<const U*>(d_r + row * H + c) : U{};
    }
  };
  if constexpr (kNext) load(blockIdx.x, rn, gn, en);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < T; row += gridDim.x, turn ^= 1) {
    const int64_t at = row * H;
    U ru[NV], gu[NV], eu[NV];
    if constexpr (kNext) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        ru[j] = rn[j];
        gu[j] = gn[j];
        eu[j] = en[j];
      }
      load(row + gridDim.x, rn, gn, en);
    } else {
      load(row, ru, gu, eu);
    }
    float ss = 0.f, hr = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
      float wv[VEC] = {};
      if (c < H) load_weight<W_, VEC>(w, c, wv);
      row_terms<E_, VEC>(ru[j], gu[j], wv, ss, hr);
    }
    const float2 s = row_sum2(ss, hr, lpt, red[turn]);
    const float m = 1.f / sqrtf(s.x / (float)H + eps);
    const float k = -m * m * (s.y / (float)H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
      if (c >= H) continue;
      float wv[VEC];
      load_weight<W_, VEC>(w, c, wv);
      *reinterpret_cast<U*>(dx + at + c) = row_gradient<E_, VEC>(ru[j], gu[j], eu[j], d_r != nullptr, wv, m, k, acc[j]);
    }
  }
  float* p = part + (int64_t)blockIdx.x * H;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c < H) p[c + i] = acc[j][i];
  }
}

// dw[c] = sum over i of part[i][c], in a fixed order: a block takes 32 columns,
// warp k the rows k, k + 32, ...
__global__ void __launch_bounds__(1024)
sum_parts_kernel(const float* __restrict__ part, int n, int H, float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  pdl_wait();
  pdl_trigger();
  float v = 0.f;
  if (c < H)
#pragma unroll 8
    for (int i = warp; i < n; i += 32) v += part[(int64_t)i * H + c];
  s[warp][lane] = v;
  __syncthreads();
  v = warp_sum(s[lane][warp]);
  const int o = blockIdx.x * 32 + warp;
  if (lane == 0 && o < H) dw[o] = v;
}

// Codes and exponents back to numbers, in units of VEC codes, as many as fill 16 bytes
// of the output, so that a warp's store has whole lines.
constexpr int kBackThreads = 256;

// 2^(e - 127); a byte of 255 stands for NaN
__device__ __forceinline__ float scale_of(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23);
}
__device__ __forceinline__ float2 widen_codes(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
template <int VEC> using Codes = std::conditional_t<VEC == 8, uint2, std::conditional_t<VEC == 4, uint32_t, uint8_t>>;
// The numbers of a unit, code k times scale(k).
template <int VEC, typename E_, typename F>
__device__ __forceinline__ void write_back(Codes<VEC> q, F scale, E_* out) {
  if constexpr (VEC == 1) {
    row_narrow(widen_codes(q).x * scale(0), *out);
  } else {
    uint32_t w[2];
    if constexpr (VEC == 8) w[0] = q.x, w[1] = q.y;
    else w[0] = q;
    float v[VEC];
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      const float2 f = widen_codes(w[k / 2] >> (16 * (k & 1)));
      v[2 * k] = f.x * scale(2 * k);
      v[2 * k + 1] = f.y * scale(2 * k + 1);
    }
    uint4 o;
    row_narrow(v, o);
    *reinterpret_cast<uint4*>(out) = o;
  }
}

// Rows of whole units, two to a thread (8192 x 7168 to bf16: 26.8 us; one 32.1; four 27.1
// and slower for few rows; 16 codes to a thread, whose stores have half sectors, 29.7).
constexpr int kBackUnits = 2;
template <typename E_, int VEC>
__global__ void __launch_bounds__(kBackThreads)
fp8_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t units, int per_row, int groups,
                      E_* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t first = (int64_t)blockIdx.x * (kBackThreads * kBackUnits) + threadIdx.x;
  Codes<VEC> q[kBackUnits];
  uint32_t e[kBackUnits];
#pragma unroll
  for (int j = 0; j < kBackUnits; ++j) {
    const int64_t u = first + j * kBackThreads;
    if (u >= units) break;
    const int64_t row = units <= UINT32_MAX ? (uint32_t)u / (uint32_t)per_row : u / per_row;
    q[j] = __ldg(reinterpret_cast<const Codes<VEC>*>(codes) + u);
    e[j] = __ldg(exps + row * groups + (int)(u - row * per_row) * VEC / kGroupCols);
  }
#pragma unroll
  for (int j = 0; j < kBackUnits; ++j) {
    const int64_t u = first + j * kBackThreads;
    if (u >= units) break;
    const float scale = scale_of(e[j]);
    write_back<VEC>(q[j], [&](int) { return scale; }, out + u * VEC);
  }
}

// Rows of other lengths: a unit may begin in one group and end in the next one, which is
// the next exponent, of the next row too.  Where that one ends as well (the last group of a
// row has fewer than VEC columns), and for the last codes, they are taken one by one.
template <typename E_, int VEC>
__global__ void __launch_bounds__(kBackThreads)
fp8_dequantize_ragged_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n, int H, int groups,
                             E_* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = ((int64_t)blockIdx.x * kBackThreads + threadIdx.x) * VEC;
  if (i >= n) return;
  const int64_t row = n <= UINT32_MAX ? (uint32_t)i / (uint32_t)H : i / H;
  const int c = (int)(i - row * H);
  int64_t at = row * groups + c / kGroupCols;
  const int first = min(kGroupCols - c % kGroupCols, H - c);  // columns left of the unit's group
  const int second = first == H - c ? min(kGroupCols, H) : min(kGroupCols, H - c - first);
  if (i + VEC <= n && first + second >= VEC) {
    const Codes<VEC> q = __ldg(reinterpret_cast<const Codes<VEC>*>(codes + i));
    const float s0 = scale_of(__ldg(exps + at)), s1 = scale_of(__ldg(exps + at + (first < VEC ? 1 : 0)));
    write_back<VEC>(q, [&](int k) { return k < first ? s0 : s1; }, out + i);
    return;
  }
  int left = first, col = c;
  for (int64_t k = i; k < min(i + VEC, n); ++k) {
    row_narrow(widen_codes(__ldg(codes + k)).x * scale_of(__ldg(exps + at)), out[k]);
    if (++col == H) col = 0;
    if (--left == 0) {
      ++at;
      left = min(kGroupCols, H - col);
    }
  }
}

// Threads of a row of `units` units, nv of them a thread.
int row_lanes(int units, int nv) { return (int)ceil_div(units, 32 * nv) * 32; }
// Short rows share a block of 128 threads.
int rows_per_block(int lpt) { return lpt <= 64 ? 128 / lpt : 1; }

template <typename E_, typename W_, int VEC, bool QUANT, typename... Args>
cudaError_t launch_norm(int T, int H, cudaStream_t stream, const E_* x, const E_* res, const W_* w, float eps, Args... out) {
  const int units = VEC > 1 ? H / VEC : (int)round_up(H, kGroupCols);
  auto run = [&](auto kernel, int nv) {
    const int lpt = row_lanes(units, nv), rpb = rows_per_block(lpt);
    return launch_pdl(kernel, dim3((unsigned)ceil_div(T, rpb)), dim3(lpt * rpb), 0, stream, x, res, w, T, H, lpt, eps,
                      out...);
  };
  if constexpr (VEC > 1) {
    // With many rows few threads take each, which wait for one another less; with few
    // rows many do, as there is nothing else to run meanwhile (us, 1, 256 and 16384 rows
    // of bf16: 7168 columns in two units a thread 2.1, 3.1, 159, in eight 3.2, 3.8, 135;
    // 1024 columns in one 1.5, 1.7, 24.0, in two 1.7, 1.8, 21.1; 512 columns in two at
    // all sizes).
    const bool many = T > 1024;
    if (units > 64 && units <= 128 && !many) return run(norm_kernel<E_, W_, VEC, 1, QUANT, 128>, 1);
    if (units <= 512) return run(norm_kernel<E_, W_, VEC, 2, QUANT, 256>, 2);
    if constexpr (VEC == 8) {
      if (units <= 1024)
        return many ? run(norm_kernel<E_, W_, 8, 8, QUANT, 128>, 8) : run(norm_kernel<E_, W_, 8, 2, QUANT, 512>, 2);
      return many ? run(norm_kernel<E_, W_, 8, 8, QUANT, 256>, 8) : run(norm_kernel<E_, W_, 8, 4, QUANT, 512>, 4);
    } else {
      // Four units a thread for all (us, 64, 1100 and 16384 rows of 7168 columns: 2.9, 22.7, 289,
      // in eight 3.1, 20.2, 265; with a bf16 weight 2.7, 18.8, 264, in eight 3.0, 20.0, 264; with
      // the 8 bits 3.6, 25.6, 313, in eight 4.6, 26.0, 303; 16384 rows of 2560 columns with them
      // 105 and 111).
      if (units <= 2048) return run(norm_kernel<E_, W_, 4, 4, QUANT, 512>, 4);
      return run(norm_kernel<E_, W_, 4, 8, QUANT, 512>, 8);
    }
  } else {
    if (units <= 2048) return run(norm_kernel<E_, W_, 1, 4, QUANT, 512>, 4);
    if (units <= 4096) return run(norm_kernel<E_, W_, 1, 8, QUANT, 512>, 8);
    if (units <= 8192) return run(norm_kernel<E_, W_, 1, 16, QUANT, 512>, 16);
    return run(norm_kernel<E_, W_, 1, 32, QUANT, 512>, 32);
  }
}

// How the gradient kernel is launched.  On the 16-byte grid a thread has one unit of
// rows up to 256 units, then two, the ring holding four or two rows; longer rows (and
// all that lie off the grid) go without it.
struct BackPlan {
  bool ring;
  int nv, lpt, rpb;  // units a thread, threads a row, rows a block
  int64_t blocks;
};
BackPlan back_plan(int32_t T, int32_t H, int vec) {
  BackPlan b{};
  const int units = vec > 1 ? H / vec : (int)round_up(H, kGroupCols);
  b.ring = vec > 1 && units <= 2048;
  if (b.ring) b.nv = units <= 256 ? 1 : 2;
  else if (vec > 1) b.nv = 8;
  else b.nv = units <= 2048 ? 4 : units <= 8192 ? 8 : 16;
  b.lpt = row_lanes(units, b.nv);
  b.rpb = b.ring ? rows_per_block(b.lpt) : 1;
  const int threads = b.lpt * b.rpb;
  // threads that an SM's registers hold
  const int per_sm = (!b.ring && (vec > 1 || (b.nv == 8 && b.lpt <= 512)) ? 576 : 1024) / threads;
  const int64_t most = (int64_t)(per_sm < 1 ? 1 : per_sm > 8 ? 8 : per_sm) * current_sms(), want = ceil_div(T, b.rpb);
  b.blocks = want < most ? want : most;
  return b;
}

template <typename E_, typename W_>
cudaError_t launch_backward_ring(const BackPlan& b, cudaStream_t stream, const E_* dy, const E_* r, const W_* w, const E_* d_r,
                                 int T, int H, float eps, E_* dx, float* part) {
  // the shared memory that the largest block of the kernel takes, whatever this
  // call's: a call in another thread does not lower it
  auto run = [&](auto kernel, int most) {
    const size_t per = 4 * 3 * sizeof(uint4), smem = per * b.lpt * b.rpb;  // NV DEPTH = 4
    cudaError_t err = cudaSuccess;
    if (smem > 46 * 1024) err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(per * most));
    return err != cudaSuccess ? err
                              : launch_pdl(kernel, dim3((unsigned)b.blocks), dim3(b.lpt * b.rpb), smem, stream, dy, r, w, d_r, T,
                                           H, b.lpt, eps, dx, part);
  };
  if (b.nv == 1) return run(norm_backward_kernel<E_, W_, 1, 4, 256, 4>, 256);
  if (b.lpt <= 512) return run(norm_backward_kernel<E_, W_, 2, 2, 512, 2>, 512);
  return run(norm_backward_kernel<E_, W_, 2, 2, 1024, 1>, 1024);
}
template <typename E_, typename W_, int VEC>
cudaError_t launch_backward_plain(const BackPlan& b, cudaStream_t stream, const E_* dy, const E_* r, const W_* w, const E_* d_r,
                                  int T, int H, float eps, E_* dx, float* part) {
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)b.blocks), dim3(b.lpt), 0, stream, dy, r, w, d_r, T, H, b.lpt, eps, dx, part);
  };
  if constexpr (VEC > 1) {
    return run(norm_backward_plain_kernel<E_, W_, VEC, 8, 512>);  // float32 rows of more than 8192 columns
  } else {
    // (us, 8192 rows of 5001 bf16 in eight elements a thread 234, in sixteen of half as
    // many threads 431; 4096 of 11317 in sixteen 257, in thirty-two 450)
    return b.nv == 4       ? run(norm_backward_plain_kernel<E_, W_, 1, 4, 512>)
           : b.nv == 16    ? run(norm_backward_plain_kernel<E_, W_, 1, 16, 1024>)
           : b.lpt <= 512 ? run(norm_backward_plain_kernel<E_, W_, 1, 8, 512>)
                          : run(norm_backward_plain_kernel<E_, W_, 1, 8, 1024>);
  }
}

// Common checks; the element size in *es and whether rows lie on the 16-byte grid.
int check_norm(int32_t T, int32_t H, int32_t dtype, int32_t w_dtype, const void* w, std::initializer_list<const void*> rows,
               int* es, bool* whole) {
  if (T < 0 || H < 1) return MLR_ERR_INVALID;
  for (int d : {dtype, w_dtype})
    if (d != MLR_DTYPE_BF16 && d != MLR_DTYPE_F32) return MLR_ERR_INVALID;
  if (H > kMaxNormHidden) return MLR_ERR_UNSUPPORTED;
  *es = dtype == MLR_DTYPE_BF16 ? 2 : 4;
  *whole = (int64_t)H * *es % 16 == 0 && aligned_to(w, 16);
  if (w == nullptr || !aligned_to(w, w_dtype == MLR_DTYPE_BF16 ? 2 : 4)) return MLR_ERR_INVALID;
  for (const void* p : rows) {
    if (p == nullptr) continue;
    if (!aligned_to(p, *es)) return MLR_ERR_INVALID;
    if (!aligned_to(p, 16)) *whole = false;
  }
  return MLR_OK;
}

template <typename E_, typename W_, bool QUANT>
int run_norm(bool whole, const void* x, const void* residual, const void* weight, int T, int H, float eps, void* y, void* r_out,
             uint8_t* codes, uint8_t* exps, cudaStream_t stream) {
  const E_ *xp = static_cast<const E_*>(x), *rp = static_cast<const E_*>(residual);
  const W_* w = static_cast<const W_*>(weight);
  E_ *yp = static_cast<E_*>(y), *op = static_cast<E_*>(r_out);
  constexpr int VEC = 16 / sizeof(E_);
  return launched(whole ? launch_norm<E_, W_, VEC, QUANT>(T, H, stream, xp, rp, w, eps, yp, op, codes, exps)
                        : launch_norm<E_, W_, 1, QUANT>(T, H, stream, xp, rp, w, eps, yp, op, codes, exps));
}

template <typename E_, typename W_>
int run_backward(bool whole, const BackPlan& b, cudaStream_t stream, const void* dy, const void* r, const void* weight,
                 const void* d_r, int T, int H, float eps, void* dx, float* part) {
  const E_ *g = static_cast<const E_*>(dy), *a = static_cast<const E_*>(r), *e = static_cast<const E_*>(d_r);
  const W_* w = static_cast<const W_*>(weight);
  E_* o = static_cast<E_*>(dx);
  if (b.ring) return launched(launch_backward_ring<E_, W_>(b, stream, g, a, w, e, T, H, eps, o, part));
  if constexpr (sizeof(E_) == 4)
    if (whole) return launched(launch_backward_plain<E_, W_, 4>(b, stream, g, a, w, e, T, H, eps, o, part));
  return launched(launch_backward_plain<E_, W_, 1>(b, stream, g, a, w, e, T, H, eps, o, part));
}

// f<E_, W_>() for the types of rows and weight.
template <typename F>
int by_types(int32_t dtype, int32_t weight_dtype, F f) {
  const bool w32 = weight_dtype == MLR_DTYPE_F32;
  if (dtype == MLR_DTYPE_BF16) return w32 ? f(uint16_t{}, float{}) : f(uint16_t{}, uint16_t{});
  return w32 ? f(float{}, float{}) : f(float{}, uint16_t{});
}

}  // namespace
}  // namespace mlr

extern "C" int moe_rms_norm(const void* x, const void* residual, const void* weight, int32_t num_tokens, int32_t hidden,
                            int32_t dtype, int32_t weight_dtype, float eps, void* y, void* residual_out, uint8_t* codes,
                            uint8_t* exps, void* stream_) {
  using namespace mlr;
  int es = 0;
  bool whole = false;
  const int code = check_norm(num_tokens, hidden, dtype, weight_dtype, weight, {x, residual, y, residual_out}, &es, &whole);
  if (code != MLR_OK) return code;
  if (!(eps >= 0.f)) return MLR_ERR_INVALID;
  if (num_tokens == 0) return MLR_OK;  // empty tensors may have no address
  if (x == nullptr || (residual == nullptr) != (residual_out == nullptr) || (codes == nullptr) != (exps == nullptr) ||
      (y == nullptr && codes == nullptr) || (y != nullptr && y == residual_out))
    return MLR_ERR_INVALID;
  // a vector's codes are stored together
  if (codes != nullptr && !aligned_to(codes, 16)) whole = false;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  return by_types(dtype, weight_dtype, [&](auto e, auto w) {
    auto run = codes != nullptr ? run_norm<decltype(e), decltype(w), true> : run_norm<decltype(e), decltype(w), false>;
    return run(whole, x, residual, weight, num_tokens, hidden, eps, y, residual_out, codes, exps, stream);
  });
}

extern "C" size_t moe_rms_norm_backward_workspace_bytes(int32_t num_tokens, int32_t hidden, int32_t dtype) {
  using namespace mlr;
  if (num_tokens < 0 || hidden < 1 || hidden > kMaxNormHidden || (dtype != MLR_DTYPE_BF16 && dtype != MLR_DTYPE_F32)) return 0;
  // the kernel for rows off the grid may be the one that runs, whatever the size
  const int64_t a = back_plan(num_tokens, hidden, 1).blocks, b = back_plan(num_tokens, hidden, dtype == MLR_DTYPE_BF16 ? 8 : 4).blocks;
  const int64_t parts = a > b ? a : b;
  return (size_t)(parts > 0 ? parts : 1) * hidden * 4;
}

extern "C" int moe_rms_norm_backward(const void* dy, const void* r, const void* weight, const void* d_r, int32_t num_tokens,
                                     int32_t hidden, int32_t dtype, int32_t weight_dtype, float eps, void* dx,
                                     float* d_weight, void* workspace, size_t ws_bytes, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int es = 0;
  bool whole = false;
  const int code = check_norm(num_tokens, hidden, dtype, weight_dtype, weight, {dy, r, d_r, dx}, &es, &whole);
  if (code != MLR_OK) return code;
  if (!(eps >= 0.f) || d_weight == nullptr || !aligned_to(d_weight, 4)) return MLR_ERR_INVALID;
  if (num_tokens == 0) {
    if (cudaMemsetAsync(d_weight, 0, (size_t)hidden * 4, stream) == cudaSuccess) return MLR_OK;
    (void)cudaGetLastError();
    return MLR_ERR_CUDA;
  }
  if (dy == nullptr || r == nullptr || dx == nullptr) return MLR_ERR_INVALID;
  const BackPlan b = back_plan(num_tokens, hidden, whole ? 16 / es : 1);
  if (workspace == nullptr || ws_bytes < (size_t)b.blocks * hidden * 4) return MLR_ERR_CAPACITY;
  if (!aligned_to(workspace, 256)) return MLR_ERR_INVALID;
  float* part = static_cast<float*>(workspace);
  const int c = by_types(dtype, weight_dtype, [&](auto e, auto w) {
    return run_backward<decltype(e), decltype(w)>(whole, b, stream, dy, r, weight, d_r, num_tokens, hidden, eps, dx, part);
  });
  if (c != MLR_OK) return c;
  return launched(launch_pdl(sum_parts_kernel, dim3((unsigned)ceil_div(hidden, 32)), dim3(1024), 0, stream,
                             (const float*)part, (int)b.blocks, (int)hidden, d_weight));
}

extern "C" int moe_fp8_dequantize(const uint8_t* codes, const uint8_t* exps, int32_t rows, int32_t cols, int32_t dtype,
                                  void* out, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (rows < 0 || cols < 1 || (dtype != MLR_DTYPE_BF16 && dtype != MLR_DTYPE_F32)) return MLR_ERR_INVALID;
  const int64_t n = (int64_t)rows * cols;
  if (n == 0) return MLR_OK;
  if (codes == nullptr || exps == nullptr || out == nullptr || !aligned_to(out, dtype == MLR_DTYPE_BF16 ? 2 : 4))
    return MLR_ERR_INVALID;
  const int groups = (int)ceil_div(cols, kGroupCols);
  auto run = [&](auto kernel, int64_t blocks, int64_t count, int per_row, auto* o) {
    if (blocks > INT32_MAX) return (int)MLR_ERR_UNSUPPORTED;
    return launched(launch_pdl(kernel, dim3((unsigned)blocks), dim3(kBackThreads), 0, stream, codes, exps, count, per_row, groups, o));
  };
  auto pick = [&](auto vec, auto* o) {
    using E_ = std::remove_pointer_t<decltype(o)>;
    constexpr int V = vec.value;
    if (!aligned_to(codes, V) || !aligned_to(out, 16))
      return run(fp8_dequantize_kernel<E_, 1>, ceil_div(n, kBackThreads * kBackUnits), n, (int)cols, o);
    if (cols % V == 0)
      return run(fp8_dequantize_kernel<E_, V>, ceil_div(n / V, kBackThreads * kBackUnits), n / V, (int)(cols / V), o);
    return run(fp8_dequantize_ragged_kernel<E_, V>, ceil_div(n, kBackThreads * V), n, (int)cols, o);
  };
  if (dtype == MLR_DTYPE_BF16) return pick(std::integral_constant<int, 8>{}, static_cast<uint16_t*>(out));
  return pick(std::integral_constant<int, 4>{}, static_cast<float*>(out));
}
