// kernels8.h -- host-side launchers of the 8-bit operators' kernels (see
// kernels.h: each enqueues on `stream`, never synchronises, returns a QL_*
// status; arguments are validated by the C ABI layer before).
#pragma once

#include "../../include/qlora_8bit.h"
#include "kernels.h"

namespace qlora {

// leading dimensions of an 8-bit matrix: bytes of a row of codes, and bytes
// of one block column of scales
inline int64_t fp8_ld(int64_t cols) { return (cols + QL_FP8_BLOCK - 1) / QL_FP8_BLOCK * QL_FP8_BLOCK; }
inline int64_t fp8_rp(int64_t rows) { return (rows + 15) / 16 * 16; }

// Maxima of unsigned values across lanes, in every lane, without LDS: within a
// row of 16 lanes by pairs, quads, and the mirrored halves of 8 and of 16;
// then by exchanging odd rows with even ones and the wave's two halves.
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max_u32(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max_dpp<0xB1>(v);      // quad_perm 1 0 3 2
  v = max_dpp<0x4E>(v);      // quad_perm 2 3 0 1
  v = max_dpp<0x141>(v);     // row_half_mirror
  return max_dpp<0x140>(v);  // row_mirror
}
__device__ __forceinline__ uint32_t across_rows_max(uint32_t v) {
  auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max_u32(a[0], a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max_u32(b[0], b[1]);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) { return across_rows_max(row_max(v)); }

// fp8_quant.hip: q and qt as in fp8_quantize (either may be NULL)
int launch_fp8_quantize(const void *x, int x_dtype, int64_t R, int64_t C, int block_rows,
                        const ql_fp8 *q, const ql_fp8 *qt, hipStream_t stream);

// fp8_gemm.hip: out [M, N] = a b^T; part holds fp8_matmul_partial_floats
// floats (any output type)
size_t fp8_matmul_partial_floats(int64_t M, int64_t N, int64_t K);
int launch_fp8_matmul(const ql_fp8 *a, const ql_fp8 *b, void *out, int out_dtype, bool accumulate,
                      float *part, hipStream_t stream);

// adam_many.hip: t holds count checked tensors, table the same in device memory,
// byte for byte (the kernel takes n from there)
constexpr int kAdamTable = 960;               // tensors per launch (4 bytes of arguments each)
constexpr int64_t kAdamMaxN = 1ll << 33;      // values of one tensor
int launch_adamw_many(int32_t count, const ql_adamw_tensor *t, const ql_adamw_tensor *table,
                      int grad_dtype, int state_bits, int copy_dtype, const float *grad_scale, double lr, double beta1,
                      double beta2, double eps, double weight_decay, int64_t step, uint64_t seed,
                      hipStream_t stream);

}  // namespace qlora
