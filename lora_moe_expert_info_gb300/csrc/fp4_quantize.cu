// fp4_quantize.cu -- quantisation to microscaled 4-bit floats and back.
//
// Per row and block of consecutive columns (32 for MXFP4, 16 for NVFP4), with
// m = max |x| over the block:
//   MXFP4  scale 2^s, s the smallest integer in [-127, 126] with m <= 6 * 2^s
//          (s = 0 for m = 0), stored as the byte s + 127
//   NVFP4  E4M3 scale q = rn(min(m / (6 g), 448)) for the matrix's fp32 tensor
//          scale g (1 if none), and r = 1 / (q g), each step rounded to fp32
//          (r = 0 for q = 0, at most the largest float)
// and the code of x is x * 2^-s or x * r rounded to the nearest E2M1 value
// (0, 0.5, 1, 1.5, 2, 3, 4, 6; ties to the even code, saturating, sign kept).
// A block that holds an infinity or a NaN gets a NaN scale and zero codes, so
// that what is computed from it is NaN.  Layouts: mlr_fp4.cuh.
//
// One thread holds 16 consecutive columns of a row (MXFP4: two neighbours
// exchange their maxima), so a row is read once and nothing is kept outside
// registers; bound by HBM: reads x, writes half a byte per value plus one byte
// per block.  65536 rows of 7168 bf16, MXFP4: quantised 169 us (105% of the copy
// rate), back 181 us (98%), from [gate | up] 367 us (87%; without exponential
// and division 300), 8192 tokens to those 65536 sorted rows 73 us (76%: their
// scales go through arrange_kernel).
#include <cuda_fp16.h>

#include "mlr_fp4.cuh"
#include "mlr_profile.cuh"

namespace mlr {
namespace {

constexpr int kQThreads = 128;
constexpr int kQDests = 512;  // (row, destination) pairs a block keeps in shared memory
enum Source { kMatrix, kTokens, kSwiglu };

// What a block's rows are and where their codes and scales go.
struct QuantParams {
  const void* x;
  const void* x_end;
  int64_t rows;        // source rows
  int cols, ng, nga;   // columns; 16-column groups of the code pitch; of the atoms
  int rpb;             // source rows per block
  uint32_t ng_magic;   // ceil(2^32 / nga)
  int64_t group_rows;  // kMatrix: rows per matrix
  int64_t group_blocks;
  const float* tensor_scale;  // kMatrix: one per matrix; else one; null: 1
  const int32_t* ids;         // kTokens: [T, K]
  const int32_t* pair_pos;
  const int32_t* offsets;     // kTokens, kSwiglu: [E + 1]
  int K, E;
  int64_t P;  // sorted rows
  uint8_t* codes;
  uint8_t* scales;
  int64_t pitch, block_bytes;  // bytes of a code row; of a 128-row block's atoms
  int arrange;                 // kTokens: a row's scales one after another, for arrange_kernel
  int32_t* status;
};

// A destination of a quantised row: its code row (-1: none) and the byte of
// its first scale (-1: a masked row, codes zero and no scales).
struct Dest {
  int64_t row, scale;
};

template <int SRC>
__device__ __forceinline__ Dest sorted_dest(const QuantParams& p, int64_t r, int e) {
  const int o0 = __ldg(p.offsets + e), o1 = __ldg(p.offsets + e + 1);
  if (o0 < 0 || r < o0 || r >= o1 || r >= p.P) {
    set_status(p.status, MLR_STATUS_INDEX);
    return Dest{-1, -1};
  }
  const int j = (int)r - o0;
  const int in_block = SRC == kTokens && p.arrange ? (j & 127) * (int)(p.block_bytes / 128) : fp4_scale_byte(j);
  return Dest{r, (int64_t)(o0 / 128 + e + j / 128) * p.block_bytes + in_block};
}

// The expert of sorted row r: the last e with offsets[e] <= r; E if r is before
// the first expert's rows or past the last one's.
__device__ __forceinline__ int row_expert(const int32_t* __restrict__ offsets, int E, int64_t r) {
  if (r < __ldg(offsets) || r >= __ldg(offsets + E)) return E;
  int lo = 0, hi = E;  // offsets[lo] <= r < offsets[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid) <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int SRC>
__device__ __forceinline__ Dest dest_of(const QuantParams& p, int64_t row, int k) {
  if (SRC == kMatrix) {
    const int64_t g = row / p.group_rows;
    const int64_t r = row - g * p.group_rows;
    return Dest{row, (g * p.group_blocks + r / 128) * p.block_bytes + fp4_scale_byte((int)(r & 127))};
  }
  if (SRC == kTokens) {
    const int q = __ldg(p.pair_pos + row * p.K + k);
    if (q < 0) return Dest{~q < p.P ? (int64_t)~q : -1, -1};
    const int e = __ldg(p.ids + row * p.K + k);
    if (e < 0 || e >= p.E) {
      set_status(p.status, MLR_STATUS_INDEX);
      return Dest{-1, -1};
    }
    return sorted_dest<SRC>(p, q, e);
  }
  const int e = row_expert(p.offsets, p.E, row);
  return e == p.E ? Dest{row, -1} : sorted_dest<SRC>(p, row, e);
}

// 32 bytes at a 32-byte boundary, one instruction.
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The 32-bit words of n bytes at p, which no vector divides, from the 16-byte
// vectors that hold them: W words, moved down by the misalignment in two steps
// of words and one of bytes.  The caller sees to it that the vectors lie in the
// tensor; words past the n bytes hold whatever follows.  50440 rows of 900 bf16
// to NVFP4: 33 us, from [gate | up] 66 (element by element through shared
// memory, half a warp to a group of 16 columns, 44 and 90).
template <int W>
__device__ __forceinline__ void load_shifted(const void* p, int n, uint32_t (&w)[W]) {
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
  const uint4* base = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - off);
  uint32_t t[W + 4] = {};
#pragma unroll
  for (int i = 0; i < W / 4 + 1; ++i)
    if (16 * i < off + n) {
      const uint4 q = __ldg(base + i);
      t[4 * i] = q.x;
      t[4 * i + 1] = q.y;
      t[4 * i + 2] = q.z;
      t[4 * i + 3] = q.w;
    }
#pragma unroll
  for (int i = 0; i < W + 2; ++i) t[i] = off & 8 ? t[i + 2] : t[i];
#pragma unroll
  for (int i = 0; i < W + 1; ++i) t[i] = off & 4 ? t[i + 1] : t[i];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(t[i], t[i + 1], 8 * (off & 3));
}
// Whether all those vectors lie in the tensor [lo, hi).
__device__ __forceinline__ bool vectors_inside(const void* p, int n, const void* lo, const void* hi) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return (a & ~(uintptr_t)15) >= reinterpret_cast<uintptr_t>(lo) &&
         ((a + n + 15) & ~(uintptr_t)15) <= reinterpret_cast<uintptr_t>(hi);
}

// 16 columns of a row as fp32, zeros past the end.  VB: the bytes of a vector
// that divide a row and the base's address (32, 16, or 0: none, the vectors
// around them, and element by element at the ends of the tensor [lo, hi)).
template <int VB>
__device__ __forceinline__ void load16(const uint16_t* p, int n, float (&v)[16], const void* lo, const void* hi) {
  uint32_t w[8] = {};
  if (VB == 32) {
    if (n > 0) load32(p, w);
  } else if (VB == 16) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (8 * h < n) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + h);
        w[4 * h] = q.x;
        w[4 * h + 1] = q.y;
        w[4 * h + 2] = q.z;
        w[4 * h + 3] = q.w;
      }
  } else if (n > 0) {
    if (vectors_inside(p, 2 * n, lo, hi)) {
      load_shifted(p, 2 * n, w);
      if (n < 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xffffu : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) w[i / 2] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int VB>
__device__ __forceinline__ void load16(const float* p, int n, float (&v)[16], const void* lo, const void* hi) {
  if (VB == 32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[8] = {};
      if (8 * h < n) load32(p + 8 * h, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] = __uint_as_float(w[i]);
    }
  } else if (VB == 16) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (4 * h < n) q = __ldg(reinterpret_cast<const float4*>(p) + h);
      v[4 * h] = q.x;
      v[4 * h + 1] = q.y;
      v[4 * h + 2] = q.z;
      v[4 * h + 3] = q.w;
    }
  } else {
    uint32_t w[16] = {};
    if (n > 0) {
      if (vectors_inside(p, 4 * n, lo, hi)) {
        load_shifted(p, 4 * n, w);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < n) w[i] = __float_as_uint(__ldg(p + i));
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? __uint_as_float(w[i]) : 0.f;
  }
}

// v[j] = 4 u[j] (v[j] / (1 + exp(-v[j]))), each operation rounded to fp32; not
// finite where exp(-v[j]), 4 v[j] or the result overflows.
//
// The quotient g / d, d = 1 + exp(-g) >= 1, is one approximate reciprocal r and
// one residual step with fused multiply-adds (Markstein's division): q = g r,
// q + (g - d q) r, where g - d q is exact.  r is within 1 ulp, so the result is
// within 1 ulp of the quotient.  d is taken a quarter as large, which keeps 1 / d
// a normal number as long as exp(-g) is finite; the quotient's factor of 4 is
// left to the block's scale.  8192 x 8 rows of 7168 bf16 took 584 us with
// __fdiv_rn, 406 us so; without any division or exponential 300 us, what their
// bytes take.
__device__ __forceinline__ void swiglu16(float (&v)[16], const float (&u)[16]) {
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float2 ng = make_float2(-v[j], -v[j + 1]);
    const float2 d = __ffma2_rn(make_float2(expf(ng.x), expf(ng.y)), make_float2(0.25f, 0.25f),
                                make_float2(0.25f, 0.25f));
    float2 r;  // -1 / d
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-d.y));
    const float2 q = __fmul2_rn(ng, r);
    const float2 m = __ffma2_rn(d, q, ng);  // d q - g
    const float2 h = __fmul2_rn(__ffma2_rn(m, r, q), make_float2(u[j], u[j + 1]));
    v[j] = h.x;
    v[j + 1] = h.y;
  }
}
// u g / (1 + exp(-g)) of any g and u.  Where exp(-g) may overflow (from about
// g = -88.7 down) it is u g exp(g) in three factors,
//   (u w) (g / exp(80)) w,  w = exp((g + 80) / 2),
// none above 1 and none that underflows but where the result does.
__device__ __forceinline__ float swiglu1(float g, float u) {
  if (!(g < -80.f)) return u * __fdiv_rn(g, 1.f + expf(-g));
  constexpr float kExp = 1.8048513878454153e-35f;  // exp(-80)
  const float w = expf(0.5f * (g + 80.f));
  return u * w * (g * kExp) * w;
}
__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }

// Eight values times r as E2M1 codes, value i in bits [4i, 4i + 4).
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v, float r) {
  float2 m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(r, r));
  uint32_t o;
  asm("{\n\t"
      ".reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t"
      "}"
      : "=r"(o)
      : "f"(m[0].x), "f"(m[0].y), "f"(m[1].x), "f"(m[1].y), "f"(m[2].x), "f"(m[2].y), "f"(m[3].x), "f"(m[3].y));
  return o;
}
// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float o;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(o) : "f"(a), "f"(b), "f"(c));
  return o;
}

// MXFP4: the scale byte of a block from the bits of its largest magnitude, and
// the exact reciprocal of the scale.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax, float* r) {
  int s = 0;
  if (amax != 0) {
    // amax = 1.f x 2^(ef - 127): 2^(s + 2) x 1.5 covers it from f = 0.5 down
    const int ef = (int)(amax >> 23);
    s = ef - 127 - ((amax & 0x7fffffu) <= 0x400000u ? 2 : 1);
    if (ef == 0 || s < -127) s = -127;
  }
  *r = __int_as_float((127 - s) << 23);
  return (uint32_t)(s + 127);
}
// NVFP4: the same for an E4M3 scale under the tensor scale g.
__device__ __forceinline__ uint32_t nv_scale(float amax, float g, float* r) {
  // a block of zeros has scale 0 even under the scale 0 of a matrix of zeros
  const float t = amax > 0.f ? fminf(__fdiv_rn(amax, __fmul_rn(6.f, g)), 448.f) : 0.f;
  const uint32_t q = f32x2_to_e4m3x2(t, 0.f) & 0xffu;
  float qf;
  asm("{\n\t"
      ".reg .b32 p;\n\t.reg .f16 a, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 p, %1;\n\t"
      "mov.b32 {a, b}, p;\n\t"
      "cvt.f32.f16 %0, a;\n\t"
      "}"
      : "=f"(qf)
      : "h"((uint16_t)q));
  const float d = __fmul_rn(qf, g);
  *r = d > 0.f ? fminf(__fdiv_rn(1.f, d), 3.4028234663852886e38f) : 0.f;
  return q;
}

// A block's rows.  SwiGLU: whether the thread met a block of columns that holds a
// value that swiglu16 does not give, or an infinity or a NaN; it has a NaN scale.
template <typename E_, int FMT, int SRC, int VB>
__device__ __forceinline__ bool quantize_rows(const QuantParams& p, const Dest* dest, int64_t r0, int nr) {
  const int K = SRC == kTokens ? p.K : 1;
  const E_* x = static_cast<const E_*>(p.x);
  const int total = nr * p.nga;
  bool beyond = false;
  // whole warps stay in the loop: neighbours exchange maxima and scales
  for (int i0 = 0; i0 < total; i0 += kQThreads) {
    const int i = i0 + threadIdx.x;
    const bool in = i < total;
    const int lr = in ? (int)__umulhi((uint32_t)i, p.ng_magic) : 0;
    const int g = in ? i - lr * p.nga : 0;
    const int64_t row = r0 + lr;
    const int c = 16 * g;
    const int n = in ? min(16, p.cols - c) : 0;  // <= 0 past the last column
    // v holds `unit` times the values
    constexpr float unit = SRC == kSwiglu ? 4.f : 1.f;
    float v[16];
    if (SRC == kSwiglu) {
      float u[16];
      load16<VB>(x + row * 2 * p.cols + c, n, v, p.x, p.x_end);
      load16<VB>(x + row * 2 * p.cols + p.cols + c, n, u, p.x, p.x_end);
      swiglu16(v, u);
    } else {
      load16<VB>(x + row * p.cols + c, n, v, p.x, p.x_end);
    }
    float most = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 2) most = max3_abs(most, v[j], v[j + 1]);
    uint32_t amax = __float_as_uint(most * (1.f / unit));  // as bits a NaN counts above infinity
    if (FMT == MLR_FP4_MX) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    float r;
    uint32_t s;
    if (FMT == MLR_FP4_MX) {
      s = mx_scale(amax, &r);
    } else {
      const float ts = p.tensor_scale == nullptr ? 1.f : __ldg(p.tensor_scale + (SRC == kMatrix ? row / p.group_rows : 0));
      s = nv_scale(__uint_as_float(amax), ts, &r);
    }
    r *= 1.f / unit;
    uint2 q = make_uint2(to_e2m1x8(v, r), to_e2m1x8(v + 8, r));
    if (amax >= 0x7f800000u) {
      s = FMT == MLR_FP4_MX ? 0xffu : 0x7fu;
      q = make_uint2(0, 0);
      beyond = true;
    }
    if (n <= 0) s = 0;  // scale blocks past the last column
    // four scales of the row's atom in one word
    if (FMT == MLR_FP4_MX) {
      s |= __shfl_down_sync(0xffffffffu, s, 2) << 8;
      s |= __shfl_down_sync(0xffffffffu, s, 4) << 16;
    } else {
      s |= __shfl_down_sync(0xffffffffu, s, 1) << 8;
      s |= __shfl_down_sync(0xffffffffu, s, 2) << 16;
    }
    if (!in) continue;
    constexpr int kLanes = FMT == MLR_FP4_MX ? 8 : 4;  // 16-column groups per atom
    const int step = SRC == kTokens && p.arrange ? 4 : kAtomBytes;
    for (int k = 0; k < K; ++k) {
      const Dest d = dest[lr * K + k];
      if (d.row < 0) continue;
      if (g < p.ng)
        *reinterpret_cast<uint2*>(p.codes + d.row * p.pitch + 8 * g) = d.scale < 0 ? make_uint2(0, 0) : q;
      if (g % kLanes == 0 && d.scale >= 0)
        *reinterpret_cast<uint32_t*>(p.scales + d.scale + (int64_t)(g / kLanes) * step) = s;
    }
  }
  return beyond;
}

// The blocks of columns of the warp's rows that have a NaN scale once more, value
// by value, any gate.  A pass of its own and short, for the sake of the first
// one's registers: 8192 x 8 rows of 7168 take 367 us (MXFP4) and 363 (NVFP4) so,
// 376 and 393 where the first pass turns to such values itself in a branch that
// is not taken, 360 and 393 with this pass unrolled as the first.
template <typename E_, int FMT>
__device__ __forceinline__ void swiglu_rows_again(const QuantParams& p, const Dest* dest, int64_t r0, int nr) {
  const E_* x = static_cast<const E_*>(p.x);
  const int total = nr * p.nga;
  __syncwarp();  // the scales of the first pass
#pragma unroll 1
  for (int i0 = 0; i0 < total; i0 += kQThreads) {
    const int i = i0 + threadIdx.x;
    const int lr = i < total ? (int)__umulhi((uint32_t)i, p.ng_magic) : 0;
    const int g = i < total ? i - lr * p.nga : 0;
    const int n = i < total ? min(16, p.cols - 16 * g) : 0;
    const E_* gate = x + (r0 + lr) * 2 * p.cols + 16 * g;
    const Dest d = dest[lr];
    const int b = FMT == MLR_FP4_MX ? g / 2 : g;
    uint8_t* const scale = p.scales + d.scale + (int64_t)(b / 4) * kAtomBytes + b % 4;
    constexpr uint32_t kNan = FMT == MLR_FP4_MX ? 0xffu : 0x7fu;
    const bool again = n > 0 && d.row >= 0 && d.scale >= 0 && *scale == kNan;
    float most = 0.f;
#pragma unroll 1
    for (int j = 0; again && j < n; ++j) most = max3_abs(most, swiglu1(load1(gate + j), load1(gate + p.cols + j)), 0.f);
    uint32_t amax = __float_as_uint(most);
    if (FMT == MLR_FP4_MX) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (!again || amax >= 0x7f800000u) continue;
    float r;
    uint32_t s;
    if (FMT == MLR_FP4_MX) s = mx_scale(amax, &r);
    else s = nv_scale(most, p.tensor_scale == nullptr ? 1.f : __ldg(p.tensor_scale), &r);
    uint64_t q = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const float h[8] = {swiglu1(load1(gate + j), load1(gate + p.cols + j))};
      q |= (uint64_t)(to_e2m1x8(h, r) & 15u) << (4 * j);
    }
    *reinterpret_cast<uint64_t*>(p.codes + d.row * p.pitch + 8 * g) = q;
    *scale = (uint8_t)s;
  }
}

// Ten blocks per SM (at most 51 registers): the exponentials of the SwiGLU form
// need the warps (8192 x 8 rows of 7168, before the pass above: 359 us, 386 with twelve).
template <typename E_, int FMT, int SRC, int VB>
__global__ void __launch_bounds__(kQThreads, 10)
quantize_kernel(const QuantParams p) {
  __shared__ Dest dest[kQDests];
  pdl_wait();
  pdl_trigger();
  const int K = SRC == kTokens ? p.K : 1;
  const int64_t r0 = (int64_t)blockIdx.x * p.rpb;
  const int nr = (int)min((int64_t)p.rpb, p.rows - r0);
  for (int i = threadIdx.x; i < nr * K; i += kQThreads) dest[i] = dest_of<SRC>(p, r0 + i / K, i % K);
  __syncthreads();
  const bool beyond = quantize_rows<E_, FMT, SRC, VB>(p, dest, r0, nr);
  if constexpr (SRC == kSwiglu)
    if (__any_sync(0xffffffffu, beyond)) swiglu_rows_again<E_, FMT>(p, dest, r0, nr);
}

// Sorted rows' scales from row after row to atoms, in place, a 128-row block at
// a time: through shared memory (rows an odd number of words apart), 512 bytes
// a warp's store.
//
// Written straight to the atoms, each word of four scales of a token's K rows is
// a 32-byte sector of its own in L2: of 8192 x 8 rows of 7168 bf16 in MXFP4 17 of
// 80 us, in NVFP4, with twice the scales, 44 of 107.  Row after row and arranged
// here it is 73 and 83 us (with 256 threads 80 and 84, with 1024 78 and 85).
constexpr int kArrangeThreads = 512;

__global__ void __launch_bounds__(kArrangeThreads)
arrange_kernel(const QuantParams p, int atoms, uint32_t atoms_magic) {
  extern __shared__ uint32_t words[];  // [128][atoms | 1]
  __shared__ int rows;                 // of block b; 0: none
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  if (threadIdx.x == 0) rows = 0;
  __syncthreads();
  // the expert whose row blocks hold b: all of them at once, a search takes their latency in turn
  for (int e = threadIdx.x; e < p.E; e += kArrangeThreads) {
    const int o0 = __ldg(p.offsets + e), o1 = __ldg(p.offsets + e + 1);
    const int64_t left = (int64_t)o1 - o0 - 128 * ((int64_t)b - (o0 / 128 + e));
    if (b >= o0 / 128 + e && b < o1 / 128 + e + 1 && left > 0) rows = (int)min(left, (int64_t)128);
  }
  __syncthreads();
  const int n = rows;
  if (n == 0) return;
  uint32_t* const scales = reinterpret_cast<uint32_t*>(p.scales + b * p.block_bytes);
  const int pitch = atoms | 1;
  for (int i = threadIdx.x; i < n * atoms; i += kArrangeThreads) {
    const int r = (int)__umulhi((uint32_t)i, atoms_magic);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(words + r * pitch + (i - r * atoms))),
                 "l"(scales + i)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int a = threadIdx.x >> 5; a < atoms; a += kArrangeThreads / 32) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = lane + 32 * i < n ? words[(lane + 32 * i) * pitch + a] : 0;
    reinterpret_cast<uint4*>(scales + a * (kAtomBytes / 4))[lane] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------- back again --
struct DequantParams {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tensor_scale;
  const int32_t* offsets;  // null: matrices of group_rows rows
  int64_t rows, group_rows, group_blocks;
  int E, cols, ng, rpb;
  uint32_t ng_magic;
  int64_t pitch, block_bytes;
  void* out;
};

// Eight E2M1 codes as four pairs of halves (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t (&f)[4]) {
  asm("{\n\t"
      ".reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t"
      "}"
      : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
      : "r"(w));
}

// The number of a scale byte.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t b) {
  if (FMT == MLR_FP4_MX) return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
  float s;
  asm("{\n\t.reg .b32 p;\n\t.reg .f16 a, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 p, %1;\n\tmov.b32 {a, b}, p;\n\tcvt.f32.f16 %0, a;\n\t}"
      : "=f"(s)
      : "h"((uint16_t)b));
  return s;
}

// Where the scales of a row are (.scale, -1: the row is no expert's) and
// the matrix whose tensor scale it has (.row).
__device__ __forceinline__ Dest row_source(const DequantParams& p, int64_t row) {
  if (p.offsets == nullptr) {
    const int64_t g = row / p.group_rows, r = row - g * p.group_rows;
    return Dest{g, (g * p.group_blocks + r / 128) * p.block_bytes + fp4_scale_byte((int)(r & 127))};
  }
  Dest d{0, -1};
  const int e = row_expert(p.offsets, p.E, row);
  if (e < p.E) {
    const int o0 = __ldg(p.offsets + e);
    const int j = (int)row - o0;
    if (o0 >= 0 && j >= 0) d.scale = (int64_t)(o0 / 128 + e + j / 128) * p.block_bytes + fp4_scale_byte(j);
  }
  return d;
}
template <int FMT>
__device__ __forceinline__ float source_scale(const DequantParams& p, const Dest& d, int block) {
  return scale_value<FMT>(__ldg(p.scales + d.scale + (int64_t)(block / 4) * kAtomBytes + block % 4));
}
template <int FMT>
__device__ __forceinline__ float matrix_scale(const DequantParams& p, const Dest& d) {
  return FMT == MLR_FP4_NV && p.tensor_scale != nullptr ? __ldg(p.tensor_scale + d.row) : 1.f;
}
// n bytes in W words to p, which no vector divides, as the 16-byte vectors from
// p's next boundary on: the last one takes its rest from the next lane, if that
// lane's bytes follow.  What no vector covers (at the ends of a warp's or a
// row's run) goes value by value.  T: the values' unsigned type; n = 0: none.
// All lanes of the warp call it.  50440 rows of 900 bf16 from NVFP4: 34 us
// (value by value through shared memory 42; a thread to eight values from a
// boundary on, whatever their blocks and rows, 46).
template <typename T, int W>
__device__ __forceinline__ void store_shifted(void* p, int n, const uint32_t (&w)[W]) {
  const unsigned long long a = reinterpret_cast<unsigned long long>(p);
  const int lane = threadIdx.x & 31;
  const int next_n = __shfl_down_sync(0xffffffffu, n, 1);
  const bool joined = __shfl_down_sync(0xffffffffu, a, 1) == a + n && n == 4 * W && lane < 31;
  const bool follows = __shfl_up_sync(0xffffffffu, joined, 1) && lane > 0;
  uint32_t t[W + 4];
#pragma unroll
  for (int i = 0; i < W; ++i) t[i] = w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[W + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
  const int head = (int)(-a & 15), held = n + (joined ? min(next_n, 16) : 0);
#pragma unroll
  for (int i = 0; i < W + 2; ++i) t[i] = head & 8 ? t[i + 2] : t[i];
#pragma unroll
  for (int i = 0; i < W + 1; ++i) t[i] = head & 4 ? t[i + 1] : t[i];
  uint4* const base = reinterpret_cast<uint4*>(a + head);
  int done = min(head, n);  // the bytes from `done` on are neither the head nor in a vector
#pragma unroll
  for (int i = 0; i < W / 4; ++i)
    if (head + 16 * (i + 1) <= held) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = __funnelshift_r(t[4 * i + j], t[4 * i + j + 1], 8 * (head & 3));
      base[i] = make_uint4(u[0], u[1], u[2], u[3]);
      done = head + 16 * (i + 1);
    }
  const int skip = follows && n >= head ? head : 0;  // the lane before has written the head
  if (skip < min(head, n) || done < n) {
#pragma unroll
    for (int i = 0; i < 4 * W / (int)sizeof(T); ++i) {
      const int b = i * (int)sizeof(T);
      if (b < n && b >= skip && (b < head || b >= done))
        reinterpret_cast<T*>(p)[i] = (T)(sizeof(T) == 4 ? w[i * sizeof(T) / 4] : w[i / 2] >> (16 * (i & 1)));
    }
  }
}

// value = (code x block scale) x tensor scale, rounded once to the output type
// (code x block scale is exact).  Rows that are no expert's are zeros.
template <typename O, int FMT, int VB>
__global__ void __launch_bounds__(kQThreads)
dequantize_kernel(const DequantParams p) {
  __shared__ Dest src[kQDests];
  pdl_wait();
  pdl_trigger();
  const int64_t r0 = (int64_t)blockIdx.x * p.rpb;
  const int nr = (int)min((int64_t)p.rpb, p.rows - r0);
  for (int i = threadIdx.x; i < nr; i += kQThreads) src[i] = row_source(p, r0 + i);
  __syncthreads();
  O* out = static_cast<O*>(p.out);
  const int total = nr * p.ng;
  for (int i0 = 0; i0 < total; i0 += kQThreads) {  // whole warps: store_shifted
    const int i = i0 + threadIdx.x;
    const bool in = i < total;
    const int lr = in ? (int)__umulhi((uint32_t)i, p.ng_magic) : 0;
    const int g = in ? i - lr * p.ng : 0;
    const int64_t row = r0 + lr;
    const int c = 16 * g, n = in ? max(0, min(16, p.cols - c)) : 0;
    const Dest d = src[lr];
    float s = 0.f, ts = 1.f;
    uint2 q = make_uint2(0, 0);
    if (d.scale >= 0 && n > 0) {
      q = __ldg(reinterpret_cast<const uint2*>(p.codes + row * p.pitch + 8 * g));
      const int b = FMT == MLR_FP4_MX ? g / 2 : g;
      s = source_scale<FMT>(p, d, b);
      ts = matrix_scale<FMT>(p, d);
    }
    float2 v[8];
    const float2 s2 = make_float2(s, s), t2 = make_float2(ts, ts);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t f[4];
      from_e2m1x8(h ? q.y : q.x, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[4 * h + j] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&f[j])), s2);
        if (FMT == MLR_FP4_NV) v[4 * h + j] = __fmul2_rn(v[4 * h + j], t2);
      }
    }
    O* o = out + row * p.cols + c;
    if constexpr (sizeof(O) == 4) {
      if (VB == 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[2 * j] = __float_as_uint(v[4 * h + j].x);
            w[2 * j + 1] = __float_as_uint(v[4 * h + j].y);
          }
          if (8 * h < n) store32(o + 8 * h, w);
        }
      } else if (VB == 0) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[2 * j] = __float_as_uint(v[j].x);
          w[2 * j + 1] = __float_as_uint(v[j].y);
        }
        store_shifted<uint32_t>(o, 4 * n, w);
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          if (4 * h < n)
            reinterpret_cast<float4*>(o)[h] = make_float4(v[2 * h].x, v[2 * h].y, v[2 * h + 1].x, v[2 * h + 1].y);
      }
    } else {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[j].y), "f"(v[j].x));
      if (VB == 32) {
        if (n > 0) store32(o, w);
      } else if (VB == 0) {
        store_shifted<uint16_t>(o, 2 * n, w);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (8 * h < n) reinterpret_cast<uint4*>(o)[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
      }
    }
  }
}

// ------------------------------------------------------------------ host side --
// Source rows per block: of at most eight passes of the block (and few enough
// to leave every SM its blocks, at most kQDests destinations) the count that
// leaves the fewest threads idle in the last pass.
int rows_per_block(int64_t rows, int groups, int K) {
  int64_t most = 8 * kQThreads / groups;
  const int64_t spread = ceil_div(rows, 16 * 152);
  if (most > spread) most = spread;
  if (most > kQDests / K) most = kQDests / K;
  int best = 1;
  double used = 0;
  for (int r = 1; r <= most; ++r) {
    const double u = (double)(r * groups) / (double)round_up(r * groups, kQThreads);
    if (u >= used - 0.01) {  // of equals the larger: the destinations are looked up once per block
      used = u > used ? u : used;
      best = r;
    }
  }
  return best;
}

bool fmt_ok(int32_t fmt) { return fmt == MLR_FP4_MX || fmt == MLR_FP4_NV; }
bool dtype_ok(int32_t d) { return d == MLR_DTYPE_BF16 || d == MLR_DTYPE_F32; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int kMaxCols = 1 << 19;

// Whether tokens' scales take the way through arrange_kernel: only many words
// repay its launch and its pass (8 rows per token, NVFP4: 1.8 M words 33.5 -> 30.1
// us, 1.0 M 16.7 -> 17.3), and only where a token's words are written several
// times (2 rows per token, 2.1 M words: 43 -> 49 us; 4 rows, 1.8 M: 45 -> 43).  A
// block's words have to fit into shared memory (up to 25536 columns in NVFP4).
constexpr int64_t kArrangeWords = 3 << 19;
constexpr int kArrangeTopk = 4;
constexpr int kArrangeSmem = 200 << 10;
int arrange_smem(int atoms) { return 128 * 4 * (atoms | 1); }
bool arranged(int64_t P, int K, int atoms) {
  return K >= kArrangeTopk && P * atoms >= kArrangeWords && arrange_smem(atoms) <= kArrangeSmem;
}

// The widest vector that divides a row and its base's address; one thread's 16
// bf16 columns are 32 bytes, which one 32-byte access moves in whole sectors.
int vector_bytes(const void* base, int64_t row_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(base) | (uintptr_t)row_bytes;
  return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : 0;
}

template <typename E_, int FMT, int SRC>
int launch_quantize(const QuantParams& p, int vb, cudaStream_t stream) {
  const int64_t blocks = ceil_div(p.rows, p.rpb);
  if (blocks > INT32_MAX) return MLR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(kQThreads);
  const cudaError_t err = vb == 32   ? launch_pdl(quantize_kernel<E_, FMT, SRC, 32>, grid, block, 0, stream, p)
                          : vb == 16 ? launch_pdl(quantize_kernel<E_, FMT, SRC, 16>, grid, block, 0, stream, p)
                                     : launch_pdl(quantize_kernel<E_, FMT, SRC, 0>, grid, block, 0, stream, p);
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return MLR_ERR_CUDA;
  }
  note_launch();
  return MLR_OK;
}

int launch_arrange(const QuantParams& p, int atoms, cudaStream_t stream) {
  const int smem = arrange_smem(atoms);
  cudaError_t err = cudaFuncSetAttribute(arrange_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kArrangeSmem);
  if (err == cudaSuccess)
    err = launch_pdl(arrange_kernel, dim3((unsigned)(p.P / 128 + p.E)), dim3(kArrangeThreads), smem, stream, p, atoms,
                     (uint32_t)ceil_div(int64_t{1} << 32, atoms));
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return MLR_ERR_CUDA;
  }
  note_launch();
  return MLR_OK;
}

// Fills the layout fields and launches; p has its source and destination set.
template <int SRC>
int quantize(QuantParams& p, int32_t dtype, int32_t fmt, cudaStream_t stream) {
  if (p.rows == 0) return MLR_OK;
  const int es = dtype == MLR_DTYPE_BF16 ? 2 : 4;
  if (p.x == nullptr || p.codes == nullptr || p.scales == nullptr ||
      (reinterpret_cast<uintptr_t>(p.x) & (es - 1)) != 0 || !aligned16(p.codes) || !aligned16(p.scales))
    return MLR_ERR_INVALID;
  p.x_end = static_cast<const char*>(p.x) + p.rows * p.cols * (SRC == kSwiglu ? 2 : 1) * es;
  p.pitch = fp4_pitch(p.cols);
  p.ng = (int)(p.pitch / 8);
  const int atoms = fp4_atoms(p.cols, fmt);
  p.nga = atoms * (fmt == MLR_FP4_MX ? 8 : 4);
  p.block_bytes = (int64_t)atoms * kAtomBytes;
  p.rpb = rows_per_block(p.rows, p.nga, SRC == kTokens ? p.K : 1);
  p.ng_magic = (uint32_t)ceil_div(int64_t{1} << 32, p.nga);
  p.arrange = SRC == kTokens && arranged(p.P, p.K, atoms);
  const int vb = vector_bytes(p.x, (int64_t)p.cols * es);
  int code;
  if (dtype == MLR_DTYPE_BF16)
    code = fmt == MLR_FP4_MX ? launch_quantize<uint16_t, MLR_FP4_MX, SRC>(p, vb, stream)
                             : launch_quantize<uint16_t, MLR_FP4_NV, SRC>(p, vb, stream);
  else
    code = fmt == MLR_FP4_MX ? launch_quantize<float, MLR_FP4_MX, SRC>(p, vb, stream)
                             : launch_quantize<float, MLR_FP4_NV, SRC>(p, vb, stream);
  return code == MLR_OK && p.arrange ? launch_arrange(p, atoms, stream) : code;
}

int check_quantize(int64_t cols, int32_t dtype, int32_t fmt, const float* tensor_scale) {
  if (cols < 1 || !dtype_ok(dtype) || !fmt_ok(fmt)) return MLR_ERR_INVALID;
  if (fmt == MLR_FP4_MX && tensor_scale != nullptr) return MLR_ERR_INVALID;
  return cols > kMaxCols ? MLR_ERR_UNSUPPORTED : MLR_OK;
}

template <typename O, int FMT>
int launch_dequantize(const DequantParams& p, int vb, cudaStream_t stream) {
  const int64_t blocks = ceil_div(p.rows, p.rpb);
  if (blocks > INT32_MAX) return MLR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(kQThreads);
  const cudaError_t err = vb == 32   ? launch_pdl(dequantize_kernel<O, FMT, 32>, grid, block, 0, stream, p)
                          : vb == 16 ? launch_pdl(dequantize_kernel<O, FMT, 16>, grid, block, 0, stream, p)
                                     : launch_pdl(dequantize_kernel<O, FMT, 0>, grid, block, 0, stream, p);
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return MLR_ERR_CUDA;
  }
  note_launch();
  return MLR_OK;
}

}  // namespace
}  // namespace mlr

extern "C" int64_t moe_fp4_pitch(int32_t cols) { return cols < 1 ? -1 : mlr::fp4_pitch(cols); }

extern "C" int32_t moe_fp4_scale_atoms(int32_t cols, int32_t fmt) {
  return cols < 1 || !mlr::fmt_ok(fmt) ? -1 : mlr::fp4_atoms(cols, fmt);
}

extern "C" int moe_fp4_quantize(const void* x, int32_t num_matrices, int32_t rows, int32_t cols, int32_t dtype,
                                int32_t fmt, const float* tensor_scale, uint8_t* codes, uint8_t* scales,
                                void* stream) {
  using namespace mlr;
  const int code = check_quantize(cols, dtype, fmt, tensor_scale);
  if (code != MLR_OK) return code;
  if (num_matrices < 0 || rows < 0) return MLR_ERR_INVALID;
  QuantParams p{};
  p.x = x;
  p.rows = (int64_t)num_matrices * rows;
  p.cols = cols;
  p.group_rows = rows;
  p.group_blocks = ceil_div(rows, 128);
  p.tensor_scale = tensor_scale;
  p.codes = codes;
  p.scales = scales;
  return quantize<kMatrix>(p, dtype, fmt, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_fp4_quantize_permuted(const void* x, const int32_t* topk_ids, const int32_t* pair_pos,
                                         const int32_t* expert_offsets, int32_t num_tokens, int32_t topk,
                                         int32_t cols, int32_t num_experts, int32_t dtype, int32_t fmt,
                                         const float* tensor_scale, uint8_t* codes, uint8_t* scales,
                                         int32_t* d_status, void* stream) {
  using namespace mlr;
  const int code = check_quantize(cols, dtype, fmt, tensor_scale);
  if (code != MLR_OK) return code;
  if (num_tokens < 0 || topk < 1 || num_experts < 1) return MLR_ERR_INVALID;
  if (topk > kQDests || (int64_t)num_tokens * topk >= INT32_MAX) return MLR_ERR_UNSUPPORTED;
  if (num_tokens > 0 && (topk_ids == nullptr || pair_pos == nullptr || expert_offsets == nullptr))
    return MLR_ERR_INVALID;
  QuantParams p{};
  p.x = x;
  p.rows = num_tokens;
  p.cols = cols;
  p.tensor_scale = tensor_scale;
  p.ids = topk_ids;
  p.pair_pos = pair_pos;
  p.offsets = expert_offsets;
  p.K = topk;
  p.E = num_experts;
  p.P = (int64_t)num_tokens * topk;
  p.codes = codes;
  p.scales = scales;
  p.status = d_status;
  return quantize<kTokens>(p, dtype, fmt, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_fp4_quantize_swiglu(const void* gate_up, const int32_t* expert_offsets, int32_t num_rows,
                                       int32_t cols, int32_t num_experts, int32_t dtype, int32_t fmt,
                                       const float* tensor_scale, uint8_t* codes, uint8_t* scales,
                                       int32_t* d_status, void* stream) {
  using namespace mlr;
  const int code = check_quantize(cols, dtype, fmt, tensor_scale);
  if (code != MLR_OK) return code;
  if (num_rows < 0 || num_experts < 1) return MLR_ERR_INVALID;
  if (num_rows > 0 && expert_offsets == nullptr) return MLR_ERR_INVALID;
  QuantParams p{};
  p.x = gate_up;
  p.rows = num_rows;
  p.cols = cols;
  p.tensor_scale = tensor_scale;
  p.offsets = expert_offsets;
  p.E = num_experts;
  p.P = num_rows;
  p.codes = codes;
  p.scales = scales;
  p.status = d_status;
  return quantize<kSwiglu>(p, dtype, fmt, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_fp4_dequantize(const uint8_t* codes, const uint8_t* scales, const int32_t* expert_offsets,
                                  int32_t num_matrices, int32_t rows, int32_t cols, int32_t fmt,
                                  const float* tensor_scale, int32_t dtype, void* out, void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int code = check_quantize(cols, dtype, fmt, tensor_scale);
  if (code != MLR_OK) return code;
  if (num_matrices < 0 || rows < 0) return MLR_ERR_INVALID;
  DequantParams p{};
  p.rows = expert_offsets != nullptr ? rows : (int64_t)num_matrices * rows;
  if (p.rows == 0) return MLR_OK;
  const int es = dtype == MLR_DTYPE_BF16 ? 2 : 4;
  if (codes == nullptr || scales == nullptr || out == nullptr || !aligned16(codes) || !aligned16(scales) ||
      (reinterpret_cast<uintptr_t>(out) & (es - 1)) != 0 || (expert_offsets != nullptr && num_matrices < 1))
    return MLR_ERR_INVALID;
  p.codes = codes;
  p.scales = scales;
  p.tensor_scale = tensor_scale;
  p.offsets = expert_offsets;
  p.group_rows = rows;
  p.group_blocks = ceil_div(rows, 128);
  p.E = num_matrices;
  p.cols = cols;
  p.pitch = fp4_pitch(cols);
  p.ng = (int)(p.pitch / 8);
  p.block_bytes = (int64_t)fp4_atoms(cols, fmt) * kAtomBytes;
  p.rpb = rows_per_block(p.rows, p.ng, 1);
  p.ng_magic = (uint32_t)ceil_div(int64_t{1} << 32, p.ng);
  p.out = out;
  const int vb = vector_bytes(out, (int64_t)cols * es);
  if (dtype == MLR_DTYPE_BF16)
    return fmt == MLR_FP4_MX ? launch_dequantize<uint16_t, MLR_FP4_MX>(p, vb, stream)
                             : launch_dequantize<uint16_t, MLR_FP4_NV>(p, vb, stream);
  return fmt == MLR_FP4_MX ? launch_dequantize<float, MLR_FP4_MX>(p, vb, stream)
                           : launch_dequantize<float, MLR_FP4_NV>(p, vb, stream);
}
