// mlr_fp4.cuh -- layouts of microscaled 4-bit (E2M1) matrices, shared by the
// quantisation kernels and the product.
//
// Codes: two per byte, the even column in the low half; a row takes
// fp4_pitch(cols) bytes (a multiple of 16, so that rows can be copied by TMA),
// its columns past the last one hold zero codes.  Block scales lie in 512-byte
// atoms of 128 rows x 4 scale blocks, row r of the atom and block c at byte
// 16 (r % 32) + 4 (r / 32) + c -- the order in which the tensor cores take
// them from TMEM after one copy of the atom -- with the atoms of a 128-row
// block one after another along the columns.
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

}  // namespace mlr
