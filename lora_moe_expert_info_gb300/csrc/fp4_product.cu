// fp4_product.cu -- sorted 4-bit rows times their expert's 4-bit matrix.
//
//   y[r, n] = g_a g_w[e] sum_c A[r, c] W[e, n, c],   e the expert of row r
//
// with A and W given as E2M1 codes and block scales (mlr_fp4.cuh), products
// and sums in fp32, y rounded once to bf16.  Rows past the last expert's are
// zeros.  One block per expert and 64 outputs walks the expert's rows, 64 at a
// time, with both operands dequantised into shared memory.
#include "mlr_fp4.cuh"
#include "mlr_profile.cuh"

namespace mlr {
namespace {

constexpr int kPT = 64, kPC = 32, kPThreads = 256;

struct ProductParams {
  const uint8_t *a, *sa, *w, *sw;
  const float *ga, *gw;
  const int32_t* offsets;
  int P, E, N, cols;
  int64_t pitch, block_bytes, w_blocks;
  uint16_t* y;
  int32_t* status;
};

template <int FMT>
__device__ __forceinline__ float fp4_value(const uint8_t* row, const uint8_t* scale_row, int c) {
  const uint32_t w = (row[c >> 1] >> (4 * (c & 1))) & 15u;
  const uint32_t m = w & 7u;
  const float a = m < 2 ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  const int b = c / fp4_block(FMT);
  const uint32_t sb = scale_row[(int64_t)(b / 4) * kAtomBytes + b % 4];
  float s;
  if (FMT == MLR_FP4_MX) s = __uint_as_float(sb == 0 ? 0x00400000u : sb == 255 ? 0x7fc00000u : sb << 23);
  else {
    const uint32_t e = sb >> 3, f = sb & 7u;
    s = sb == 0x7f ? __uint_as_float(0x7fc00000u)
                   : e == 0 ? (float)f * 0.001953125f : __uint_as_float((e + 120u) << 23 | f << 20);
  }
  return (w & 8u ? -a : a) * s;
}

template <int FMT>
__global__ void __launch_bounds__(kPThreads)
product_kernel(const ProductParams p) {
  __shared__ float as[kPC][kPT + 1], ws[kPC][kPT + 1];
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.y, n0 = blockIdx.x * kPT, tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;
  int bad = 0;
  for (int i = tid; i < p.E; i += kPThreads) bad |= p.offsets[i] < 0 || p.offsets[i] > p.offsets[i + 1];
  bad |= p.offsets[p.E] > p.P;
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_status(p.status, MLR_STATUS_INDEX);
    return;
  }
  const int lo = p.offsets[e], hi = p.offsets[e + 1];
  for (int r0 = lo; r0 < hi; r0 += kPT) {
    float acc[4][4] = {};
    for (int c0 = 0; c0 < p.cols; c0 += kPC) {
      for (int i = tid; i < kPT * kPC; i += kPThreads) {
        const int r = i / kPC, c = c0 + i % kPC;
        float va = 0.f, vw = 0.f;
        if (c < p.cols && r0 + r < hi) {
          const int j = r0 + r - lo;
          va = fp4_value<FMT>(p.a + (int64_t)(r0 + r) * p.pitch,
                              p.sa + (int64_t)(lo / 128 + e + j / 128) * p.block_bytes + fp4_scale_byte(j), c);
        }
        if (c < p.cols && n0 + r < p.N)
          vw = fp4_value<FMT>(p.w + ((int64_t)e * p.N + n0 + r) * p.pitch,
                              p.sw + (e * p.w_blocks + (n0 + r) / 128) * p.block_bytes + fp4_scale_byte(n0 + r), c);
        as[i % kPC][r] = va;
        ws[i % kPC][r] = vw;
      }
      __syncthreads();
      for (int c = 0; c < kPC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[c][ty + 16 * i], ws[c][tx + 16 * j], acc[i][j]);
      __syncthreads();
    }
    const float g = (p.ga ? *p.ga : 1.f) * (p.gw ? p.gw[e] : 1.f);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (r < hi && n < p.N) p.y[(int64_t)r * p.N + n] = f32_to_bf16_bits(g * acc[i][j]);
      }
  }
  for (int r = p.offsets[p.E] + e; r < p.P; r += p.E)
    if (tid < kPT && n0 + tid < p.N) p.y[(int64_t)r * p.N + n0 + tid] = 0;
}

}  // namespace
}  // namespace mlr

extern "C" int moe_fp4_expert_product(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_tensor_scale,
                                      const uint8_t* w_codes, const uint8_t* w_scales, const float* w_tensor_scale,
                                      const int32_t* expert_offsets, int32_t num_rows, int32_t num_experts,
                                      int32_t outputs, int32_t cols, int32_t fmt, mlr_bf16* y, int32_t* d_status,
                                      void* stream_) {
  using namespace mlr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (num_rows < 0 || num_experts < 1 || outputs < 1 || cols < 1 || (fmt != MLR_FP4_MX && fmt != MLR_FP4_NV))
    return MLR_ERR_INVALID;
  if (fmt == MLR_FP4_MX && (a_tensor_scale != nullptr || w_tensor_scale != nullptr)) return MLR_ERR_INVALID;
  if (num_experts > 16384) return MLR_ERR_UNSUPPORTED;
  if (num_rows == 0) return MLR_OK;
  for (const void* q : {static_cast<const void*>(a_codes), static_cast<const void*>(a_scales),
                        static_cast<const void*>(w_codes), static_cast<const void*>(w_scales)})
    if (q == nullptr || (reinterpret_cast<uintptr_t>(q) & 15) != 0) return MLR_ERR_INVALID;
  if (expert_offsets == nullptr || y == nullptr) return MLR_ERR_INVALID;
  ProductParams p{a_codes, a_scales, w_codes, w_scales, a_tensor_scale, w_tensor_scale, expert_offsets,
                  num_rows, num_experts, outputs, cols, fp4_pitch(cols),
                  (int64_t)fp4_atoms(cols, fmt) * kAtomBytes, ceil_div(outputs, 128), y, d_status};
  const dim3 grid((unsigned)ceil_div(outputs, kPT), (unsigned)num_experts);
  const cudaError_t err =
      fmt == MLR_FP4_MX ? launch_pdl(product_kernel<MLR_FP4_MX>, grid, dim3(kPThreads), 0, stream, p)
                        : launch_pdl(product_kernel<MLR_FP4_NV>, grid, dim3(kPThreads), 0, stream, p);
  if (err != cudaSuccess) return MLR_ERR_CUDA;
  note_launch();
  return MLR_OK;
}
