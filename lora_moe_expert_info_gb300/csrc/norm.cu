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
// A row stays in the registers of its threads between the pass that reads it and
// the one that writes it, so every tensor is moved once.
#include <cuda_fp16.h>

#include <initializer_list>

#include "mlr_profile.cuh"
#include "mlr_rows.cuh"

namespace mlr {
namespace {

constexpr int kMaxNormHidden = 32768;
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

// The weight's columns c to c + VEC - 1.  bf16 or float32, whatever the rows' type.
template <int VEC>
__device__ __forceinline__ void load_weight(const void* w, bool w32, int c, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = w32 ? __ldg(static_cast<const float*>(w) + c) : row_widen(__ldg(static_cast<const uint16_t*>(w) + c));
  } else if (w32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 q = __ldg(p + i);
      v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
    }
  } else if constexpr (VEC == 8) {
    row_widen(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c)), v);
  } else {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + c));
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
}

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

template <typename E_, int VEC, int NV, bool QUANT>
__global__ void __launch_bounds__(1024)
norm_kernel(const E_* x, const E_* residual, const void* __restrict__ w, bool w32, int T, int H, int lpt, float eps,
            E_* y, E_* r_out, uint8_t* codes, uint8_t* exps) {
  using U = typename Unit<E_, VEC>::T;
  __shared__ float2 red[32];
  const int sub = threadIdx.x / lpt, lt = threadIdx.x - sub * lpt;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / lpt) + sub;
  const bool in = row < T;
  const int64_t at = row * H;
  pdl_wait();
  pdl_trigger();
  U r[NV];
  float wv[NV][VEC];
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
      float a[VEC], b[VEC];
      widen_unit(r[j], a);
      widen_unit(q[j], b);
#pragma unroll
      for (int i = 0; i < VEC; ++i) a[i] += b[i];
      narrow_unit(a, r[j]);
      const int c = unit_col<VEC>(lt, j, lpt);
      if (in && c < H) *reinterpret_cast<U*>(r_out + at + c) = r[j];
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
    float a[VEC];
    widen_unit(r[j], a);
#pragma unroll
    for (int i = 0; i < VEC; ++i) sum = fmaf(a[i], a[i], sum);
    if (c < H) load_weight<VEC>(w, w32, c, wv[j]);
  }
  const float m = 1.f / sqrtf(row_sum2(sum, 0.f, lpt, red).x / (float)H + eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
    float a[VEC];
    widen_unit(r[j], a);
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = c < H ? a[i] * m * wv[j][i] : 0.f;
    narrow_unit(a, r[j]);
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
      for (int u = 0; u < UPG; ++u) {
        widen_unit(r[j + u], a[u]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) most = max(most, __float_as_uint(a[u][i]) & 0x7fffffffu);
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      const int s = group_exp(most);
      const float up = exp2_neg(s);
      const int c = unit_col<VEC>(lt, j, lpt);
      if constexpr (VEC > 1) {
        uint32_t q[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
          q[i] = f32x2_to_e4m3x2(a[0][4 * i] * up, a[0][4 * i + 1] * up) |
                 (f32x2_to_e4m3x2(a[0][4 * i + 2] * up, a[0][4 * i + 3] * up) << 16);
        if (in && c < H) {
          if constexpr (VEC == 8) *reinterpret_cast<uint2*>(codes + at + c) = make_uint2(q[0], q[1]);
          else *reinterpret_cast<uint32_t*>(codes + at + c) = q[0];
        }
      } else {
#pragma unroll
        for (int u = 0; u < UPG; ++u)
          if (in && c + 32 * u < H) codes[at + c + 32 * u] = (uint8_t)f32x2_to_e4m3x2(a[u][0] * up, 0.f);
      }
      if (in && c < H && (lt & (LANES - 1)) == 0) exps[row * groups + c / kGroupCols] = (uint8_t)(s + 127);
    }
  }
}

// The gradients.  A block takes rows blockIdx.x, + gridDim.x, ... (several at a
// time where rows are short) and its threads keep the same columns, so that dw's
// terms add up in registers; the sums of each place of a row in a block go to
// `part` [places][H] and are added in order by sum_parts_kernel.
template <typename E_, int VEC, int NV>
__global__ void __launch_bounds__(1024)
norm_backward_kernel(const E_* dy, const E_* __restrict__ r, const void* __restrict__ w, bool w32, const E_* d_r, int T,
                     int H, int lpt, float eps, E_* dx, float* __restrict__ part) {
  using U = typename Unit<E_, VEC>::T;
  __shared__ float2 red[2][32];
  const int rpb = blockDim.x / lpt;
  const int sub = threadIdx.x / lpt, lt = threadIdx.x - sub * lpt;
  pdl_wait();
  pdl_trigger();
  float acc[NV][VEC] = {};
  int turn = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rpb; row0 < T; row0 += (int64_t)gridDim.x * rpb, turn ^= 1) {
    const int64_t row = row0 + sub;
    const bool in = row < T;
    const int64_t at = row * H;
    U ru[NV], gu[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
      const bool have = in && c < H;
      ru[j] = have ? *reinterpret_cast<const U*>(r + at + c) : U{};
      gu[j] = have ? *reinterpret_cast<const U*>(dy + at + c) : U{};
    }
    float ss = 0.f, hr = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
      float a[VEC], g[VEC], wv[VEC] = {};
      if (c < H) load_weight<VEC>(w, w32, c, wv);
      widen_unit(ru[j], a);
      widen_unit(gu[j], g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        ss = fmaf(a[i], a[i], ss);
        hr = fmaf(g[i] * wv[i], a[i], hr);
      }
    }
    const float2 s = row_sum2(ss, hr, lpt, red[turn]);
    const float m = 1.f / sqrtf(s.x / (float)H + eps);
    const float k = m * m * (s.y / (float)H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = unit_col<VEC>(lt, j, lpt);
      if (!(in && c < H)) continue;
      float a[VEC], g[VEC], wv[VEC], d[VEC];
      load_weight<VEC>(w, w32, c, wv);
      widen_unit(ru[j], a);
      widen_unit(gu[j], g);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        acc[j][i] = fmaf(g[i], a[i] * m, acc[j][i]);
        d[i] = m * (g[i] * wv[i] - a[i] * k);
      }
      if (d_r != nullptr) {
        float e[VEC];
        widen_unit(*reinterpret_cast<const U*>(d_r + at + c), e);
#pragma unroll
        for (int i = 0; i < VEC; ++i) d[i] += e[i];
      }
      U o;
      narrow_unit(d, o);
      *reinterpret_cast<U*>(dx + at + c) = o;
    }
  }
  float* p = part + ((int64_t)blockIdx.x * rpb + sub) * H;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = unit_col<VEC>(lt, j, lpt);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c < H) p[c + i] = acc[j][i];
  }
}

// dw[c] = sum over i of part[i][c], in a fixed order: a block takes 32 columns,
// warp k the rows k, k + 8, ...
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(kSumWarps * 32)
sum_parts_kernel(const float* __restrict__ part, int n, int H, float* __restrict__ dw) {
  __shared__ float s[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  pdl_wait();
  pdl_trigger();
  float v = 0.f;
  if (c < H)
    for (int i = warp; i < n; i += kSumWarps) v += part[(int64_t)i * H + c];
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < H) {
#pragma unroll
    for (int k = 1; k < kSumWarps; ++k) v += s[k][lane];
    dw[c] = v;
  }
}

// Codes and exponents back to numbers.  VEC codes a thread (16 on the 16-byte
// grid, which one group holds; else 1).
template <typename E_, int VEC>
__global__ void __launch_bounds__(256)
fp8_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, int64_t n, int H, int groups,
                      E_* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (i >= n) return;
  const int64_t row = i / H;
  const uint32_t e = __ldg(exps + row * groups + (int)(i - row * H) / kGroupCols);
  // 2^(e - 127); a byte of 255 stands for NaN
  const float scale = __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23);
  if constexpr (VEC == 1) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)__ldg(codes + i)));
    row_narrow(__half2float(__ushort_as_half((uint16_t)h)) * scale, out[i]);
  } else {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(codes + i));
    const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
    constexpr int N = 16 / sizeof(E_);  // numbers of an output vector
    float v[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(qw[k / 2] >> (16 * (k & 1)))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * k] = f.x * scale;
      v[2 * k + 1] = f.y * scale;
    }
#pragma unroll
    for (int k = 0; k < 16 / N; ++k) {
      float p[N];
#pragma unroll
      for (int u = 0; u < N; ++u) p[u] = v[k * N + u];
      uint4 o;
      row_narrow(p, o);
      reinterpret_cast<uint4*>(out + i)[k] = o;
    }
  }
}

int launched(cudaError_t err) {
  if (err != cudaSuccess) {
    (void)cudaGetLastError();  // not left for the next call to find
    return MLR_ERR_CUDA;
  }
  note_launch();
  return MLR_OK;
}

// Threads of a row that holds `units` units, nv of them (a multiple of `step`) a thread.
int row_lanes(int units, int nv) { return (int)ceil_div(units, 32 * nv) * 32; }
// Short rows share a block of 128 threads.
int rows_per_block(int lpt) { return lpt <= 64 ? 128 / lpt : 1; }

template <typename E_, int VEC, bool QUANT, typename... Args>
cudaError_t launch_norm(int T, int H, cudaStream_t stream, const E_* x, const E_* res, const void* w, bool w32, float eps,
                        Args... out) {
  const int units = VEC > 1 ? H / VEC : (int)round_up(H, kGroupCols);
  auto run = [&](auto kernel, int nv) {
    const int lpt = row_lanes(units, nv), rpb = rows_per_block(lpt);
    return launch_pdl(kernel, dim3((unsigned)ceil_div(T, rpb)), dim3(lpt * rpb), 0, stream, x, res, w, w32, T, H, lpt,
                      eps, out...);
  };
  if constexpr (VEC > 1) {
    if (units <= 128) return run(norm_kernel<E_, VEC, 1, QUANT>, 1);
    if (units <= 512) return run(norm_kernel<E_, VEC, 2, QUANT>, 2);
    if (units <= 4096) return run(norm_kernel<E_, VEC, 4, QUANT>, 4);
    return run(norm_kernel<E_, VEC, 8, QUANT>, 8);
  } else {
    if (units <= 1024) return run(norm_kernel<E_, 1, 4, QUANT>, 4);
    if (units <= 8192) return run(norm_kernel<E_, 1, 8, QUANT>, 8);
    return run(norm_kernel<E_, 1, 32, QUANT>, 32);
  }
}

// How the gradient kernel is launched: units a thread, threads a row, rows a
// block, blocks.
struct BackPlan {
  int nv, lpt, rpb;
  int64_t blocks;
};
BackPlan back_plan(int32_t T, int32_t H, int vec) {
  BackPlan b{};
  const int units = vec > 1 ? H / vec : (int)round_up(H, kGroupCols);
  b.nv = vec > 1 ? (units <= 512 ? 1 : units <= 2048 ? 2 : units <= 4096 ? 4 : 8) : (units <= 2048 ? 4 : units <= 8192 ? 8 : 32);
  b.lpt = row_lanes(units, b.nv);
  b.rpb = rows_per_block(b.lpt);
  const int64_t per_sm = b.lpt * b.rpb <= 256 ? 4 : b.lpt * b.rpb <= 512 ? 2 : 1;
  const int64_t most = per_sm * current_sms(), want = ceil_div(T, b.rpb);
  b.blocks = want < most ? want : most;
  return b;
}

template <typename E_, int VEC>
cudaError_t launch_backward(const BackPlan& b, cudaStream_t stream, const E_* dy, const E_* r, const void* w, bool w32,
                            const E_* d_r, int T, int H, float eps, E_* dx, float* part) {
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)b.blocks), dim3(b.lpt * b.rpb), 0, stream, dy, r, w, w32, d_r, T, H, b.lpt,
                      eps, dx, part);
  };
  if constexpr (VEC > 1) {
    return b.nv == 1 ? run(norm_backward_kernel<E_, VEC, 1>) : b.nv == 2 ? run(norm_backward_kernel<E_, VEC, 2>)
           : b.nv == 4 ? run(norm_backward_kernel<E_, VEC, 4>) : run(norm_backward_kernel<E_, VEC, 8>);
  } else {
    return b.nv == 4 ? run(norm_backward_kernel<E_, 1, 4>) : b.nv == 8 ? run(norm_backward_kernel<E_, 1, 8>)
                                                                      : run(norm_backward_kernel<E_, 1, 32>);
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

template <typename E_, bool QUANT>
int run_norm(bool whole, const void* x, const void* residual, const void* w, bool w32, int T, int H, float eps, void* y,
             void* r_out, uint8_t* codes, uint8_t* exps, cudaStream_t stream) {
  const E_ *xp = static_cast<const E_*>(x), *rp = static_cast<const E_*>(residual);
  E_ *yp = static_cast<E_*>(y), *op = static_cast<E_*>(r_out);
  constexpr int VEC = 16 / sizeof(E_);
  return launched(whole ? launch_norm<E_, VEC, QUANT>(T, H, stream, xp, rp, w, w32, eps, yp, op, codes, exps)
                        : launch_norm<E_, 1, QUANT>(T, H, stream, xp, rp, w, w32, eps, yp, op, codes, exps));
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
      (y == nullptr && codes == nullptr))
    return MLR_ERR_INVALID;
  // a vector's codes are stored together
  if (codes != nullptr && !aligned_to(codes, 16)) whole = false;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const bool w32 = weight_dtype == MLR_DTYPE_F32;
  auto run = [&](auto f) {
    return f(whole, x, residual, weight, w32, num_tokens, hidden, eps, y, residual_out, codes, exps, stream);
  };
  if (dtype == MLR_DTYPE_BF16) return codes != nullptr ? run(run_norm<uint16_t, true>) : run(run_norm<uint16_t, false>);
  return codes != nullptr ? run(run_norm<float, true>) : run(run_norm<float, false>);
}

extern "C" size_t moe_rms_norm_backward_workspace_bytes(int32_t num_tokens, int32_t hidden, int32_t dtype) {
  using namespace mlr;
  if (num_tokens < 0 || hidden < 1 || hidden > kMaxNormHidden || (dtype != MLR_DTYPE_BF16 && dtype != MLR_DTYPE_F32)) return 0;
  // the kernel for rows off the grid may be the one that runs, whatever the size
  const BackPlan a = back_plan(num_tokens, hidden, 1), b = back_plan(num_tokens, hidden, dtype == MLR_DTYPE_BF16 ? 8 : 4);
  const int64_t parts = a.blocks * a.rpb > b.blocks * b.rpb ? a.blocks * a.rpb : b.blocks * b.rpb;
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
  if (workspace == nullptr || ws_bytes < (size_t)(b.blocks * b.rpb) * hidden * 4) return MLR_ERR_CAPACITY;
  if (!aligned_to(workspace, 256)) return MLR_ERR_INVALID;
  float* part = static_cast<float*>(workspace);
  const bool w32 = weight_dtype == MLR_DTYPE_F32;
  const int T = num_tokens, H = hidden;
  cudaError_t err;
  if (dtype == MLR_DTYPE_BF16) {
    const uint16_t *g = static_cast<const uint16_t*>(dy), *a = static_cast<const uint16_t*>(r), *e = static_cast<const uint16_t*>(d_r);
    uint16_t* o = static_cast<uint16_t*>(dx);
    err = whole ? launch_backward<uint16_t, 8>(b, stream, g, a, weight, w32, e, T, H, eps, o, part)
                : launch_backward<uint16_t, 1>(b, stream, g, a, weight, w32, e, T, H, eps, o, part);
  } else {
    const float *g = static_cast<const float*>(dy), *a = static_cast<const float*>(r), *e = static_cast<const float*>(d_r);
    float* o = static_cast<float*>(dx);
    err = whole ? launch_backward<float, 4>(b, stream, g, a, weight, w32, e, T, H, eps, o, part)
                : launch_backward<float, 1>(b, stream, g, a, weight, w32, e, T, H, eps, o, part);
  }
  if (const int c = launched(err); c != MLR_OK) return c;
  return launched(launch_pdl(sum_parts_kernel, dim3((unsigned)ceil_div(H, 32)), dim3(kSumWarps * 32), 0, stream,
                             (const float*)part, (int)(b.blocks * b.rpb), H, d_weight));
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
  const bool whole = cols % 16 == 0 && aligned_to(codes, 16) && aligned_to(out, 16);
  const int64_t blocks = ceil_div(n, 256 * (whole ? 16 : 1));
  if (blocks > INT32_MAX) return MLR_ERR_UNSUPPORTED;
  const int groups = (int)ceil_div(cols, kGroupCols);
  auto run = [&](auto kernel, auto* o) {
    return launched(launch_pdl(kernel, dim3((unsigned)blocks), dim3(256), 0, stream, codes, exps, n, (int)cols, groups, o));
  };
  if (dtype == MLR_DTYPE_BF16) {
    uint16_t* o = static_cast<uint16_t*>(out);
    return whole ? run(fp8_dequantize_kernel<uint16_t, 16>, o) : run(fp8_dequantize_kernel<uint16_t, 1>, o);
  }
  float* o = static_cast<float*>(out);
  return whole ? run(fp8_dequantize_kernel<float, 16>, o) : run(fp8_dequantize_kernel<float, 1>, o);
}
