// mlr_fp4.cuh -- layouts of microscaled 4-bit (E2M1) matrices, shared by the
// quantisation kernels and the product.
//
// Codes: two per byte, the even column in the low half; a row takes
// fp4_pitch(cols) bytes (a multiple of 16, so that rows can be copied by TMA),
// its columns past the last one hold zero codes.  Block scales lie in 512-byte
// atoms of 128 rows x 4 scale blocks, row r of the atom and block c at byte
// 16 (r % 32) + 4 (r / 32) + c -- the order in which the tensor cores take
// them from TMEM, 16 bytes a lane -- with the atoms of a 128-row block one after
// another along the columns.
#pragma once
#include "mlr_common.cuh"

namespace mlr {

constexpr int kAtomBytes = 512;

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == MLR_FP4_NV ? 16 : 32; }
__host__ __device__ constexpr int64_t fp4_pitch(int64_t cols) { return ceil_div(cols, 32) * 16; }
// atoms of a 128-row block: one per 64 (NVFP4) or 128 (MXFP4) columns
__host__ __device__ constexpr int fp4_atoms(int64_t cols, int fmt) { return (int)ceil_div(cols, 4 * fp4_block(fmt)); }

// Byte of scale block 0 of a row within its 128-row block's atoms.
__device__ __forceinline__ int fp4_scale_byte(int r) { return 16 * (r & 31) + 4 * ((r >> 5) & 3); }

// ---- block-scaled FP4 MMAs ----

// Instruction descriptor of kind::mxf4 / kind::mxf4nvf4: E2M1 A and B, both
// K-major (K = 64), fp32 D; UE8M0 scales (bit 23) for MXFP4, UE4M3 for NVFP4.
// sf: byte of the scale cells where this MMA's scales begin (0 or 2).
template <int FMT>
__device__ __forceinline__ uint32_t idesc_fp4(uint32_t M, uint32_t N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((FMT == MLR_FP4_MX ? 1u : 0u) << 23) |
         ((M >> 7) << 27) | (sf << 29);
}
// D[tmem] (+)= (A x scales) (B x scales)^T over 64 columns: two (MXFP4) or four
// (NVFP4) scales per row, bytes of one TMEM cell; the cell of A's row m is at
// lane m, column sfa + m / 32, that of B's row n at lane n % 32 of every lane
// quarter, column sfb + n / 32.
template <int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if (FMT == MLR_FP4_MX)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

}  // namespace mlr
