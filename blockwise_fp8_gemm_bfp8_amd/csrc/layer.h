// Internal interface of the kernels behind bfp8_layer.h (not part of the ABI).
#pragma once

#include "codes.h"

namespace bfp8 {

// A launch has fewer than 2^32 threads along an axis.
inline bool threads_fit(int64_t blocks, int64_t threads) {
  return blocks < (int64_t(1) << 32) / threads;
}

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* residual;  // null: none, and sum is not written
  int64_t ldres;
  const void* w;
  bool w_f32;
  void* sum;
  int64_t ldsum;
  void* y;  // null where codes are written
  int64_t ldy;
  float* rstd;
  int64_t rows;
  int cols;
  float eps;
  // set by the launch: 1 / cols as a sum of two, and whether the rows are read past the caches
  float per_col, per_col_low;
  bool large;
};
bfp8_status launch_rmsnorm(const NormArgs& a, bfp8_in_dtype dt, hipStream_t stream);
bfp8_status launch_rmsnorm_quantize(const NormArgs& a, bfp8_in_dtype dt, bfp8_code_format format,
                                    const CodesOut& o, hipStream_t stream);

struct NormGradArgs {
  const void* dy;
  int64_t lddy;
  const void* r;
  int64_t ldr;
  const void* w;
  bool w_f32;
  const float* rstd;
  const void* dsum;  // null: none
  int64_t lddsum;
  void* dx;
  int64_t lddx;
  float* dw;
  float* partial;  // [norm_grad_groups(rows, cols)][norm_grad_ld(cols)]
  int64_t rows;
  int cols;
};
int64_t norm_grad_groups(int64_t rows, int64_t cols);
__host__ __device__ inline int64_t norm_grad_ld(int64_t cols) { return (cols + 7) / 8 * 8; }
bfp8_status launch_rmsnorm_backward(const NormGradArgs& a, bfp8_in_dtype dt, hipStream_t stream);

struct GluArgs {
  const void* gate;
  int64_t ldg;
  const void* up;
  int64_t ldu;
  const void* dh;  // null: forward
  int64_t lddh;
  void* a;  // h, or dgate; null where codes are written
  int64_t lda;
  void* b;  // dup
  int64_t ldb;
  int64_t rows, cols;  // of gate
};
bfp8_status launch_swiglu(const GluArgs& a, bfp8_in_dtype dt, hipStream_t stream);
bfp8_status launch_swiglu_quantize(const GluArgs& a, bfp8_in_dtype dt, bfp8_code_format format,
                                   const CodesOut& o, hipStream_t stream);

size_t grad_norm_workspace(const bfp8_grad_job* jobs, int64_t n);
bfp8_status launch_grad_norm(const bfp8_grad_job* jobs, int64_t n, float* norm, double* partial,
                             hipStream_t stream);
bfp8_status launch_grad_clip(const bfp8_grad_job* jobs, int64_t n, float* norm, float max_norm,
                             hipStream_t stream);
bfp8_status launch_grad_norm_clip(const bfp8_grad_job* jobs, int64_t n, float* norm, float max_norm,
                                  double* partial, hipStream_t stream);

// The format chosen at run time as a template argument F.
#define BFP8_WITH_FORMAT(format, CALL)                                             \
  ((format) == BFP8_CODES_F32    ? [&] { constexpr int F = BFP8_CODES_F32; return CALL; }()   \
   : (format) == BFP8_CODES_E8M0 ? [&] { constexpr int F = BFP8_CODES_E8M0; return CALL; }()  \
                                 : [&] { constexpr int F = BFP8_CODES_E8M0_32; return CALL; }())

}  // namespace bfp8
