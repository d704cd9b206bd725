// libbfp8 C ABI, third part: argument validation and dispatch of the entry
// points of include/bfp8_layer.h.  As in api.cpp, every argument is checked on
// the host before the first HIP call.

#include <float.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "layer.h"

using namespace bfp8;

namespace {

constexpr int64_t kMaxNormCols = 16384;
constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxLd = int64_t(1) << 40;  // elements

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t bytes_of(bfp8_in_dtype dt) { return dt == BFP8_IN_F32 ? 4 : 2; }

bool is_dtype(int64_t dt) { return dt == BFP8_IN_BF16 || dt == BFP8_IN_F32; }

// A matrix of rows of `cols` values of `size` bytes.
bfp8_status check_matrix(const void* p, int64_t ld, int64_t cols, int64_t size) {
  if (p == nullptr) return BFP8_ERR_NULL;
  if (!aligned16(p)) return BFP8_ERR_ALIGN;
  if (ld < cols || ld > kMaxLd) return BFP8_ERR_SHAPE;
  return ld * size % 16 == 0 ? BFP8_OK : BFP8_ERR_ALIGN;
}

// An output that is an input itself has to have its rows where the input has them.
bool shifted(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t rows) {
  return out == in && rows > 1 && ldo != ldi;
}

bfp8_status check_sizes(bfp8_in_dtype dt, int64_t rows, int64_t cols) {
  if (!is_dtype(dt)) return BFP8_ERR_DTYPE;
  if (rows < 0 || rows >= kMaxRows || cols < 0) return BFP8_ERR_SHAPE;
  // vectors of 8 values are counted in 32 bits
  if (rows > 0 && (cols + 7) / 8 >= (int64_t(1) << 32) / rows) return BFP8_ERR_SHAPE;
  return BFP8_OK;
}

// The codes of a rows x cols result: the format, then both layouts.
bfp8_status check_codes(const CodesOut& o, bfp8_code_format format) {
  if (format < BFP8_CODES_F32 || format > BFP8_CODES_E8M0_32) return BFP8_ERR_SCALE_MODE;
  if (o.cols % 128 != 0 || (o.qt != nullptr && o.rows % 128 != 0)) return BFP8_ERR_SHAPE;
  if (o.rows == 0 || o.cols == 0) return BFP8_OK;
  bfp8_status st = check_matrix(o.q, o.ldq, o.cols, 1);
  if (st != BFP8_OK) return st;
  if (o.s == nullptr || (o.qt != nullptr && o.st == nullptr)) return BFP8_ERR_NULL;
  if (!aligned16(o.s) || !aligned16(o.st)) return BFP8_ERR_ALIGN;
  if (o.qt == nullptr) return BFP8_OK;
  // a tile has 512 threads
  if (o.rows / 128 * (o.cols / 128) >= (int64_t(1) << 32) / kTileThreads) return BFP8_ERR_SHAPE;
  return check_matrix(o.qt, o.ldqt, o.rows, 1);
}

bfp8_status scan(const void* p, int64_t ld, bfp8_in_dtype dt, int64_t rows, int64_t cols,
                 hipStream_t stream) {
  return p == nullptr ? BFP8_OK : check_finite(p, dt, rows, cols, ld, stream);
}

bfp8_status check_norm(const NormArgs& a, bfp8_in_dtype wdt, bfp8_in_dtype dt) {
  const int64_t size = bytes_of(dt);
  bfp8_status st = check_matrix(a.x, a.ldx, a.cols, size);
  if (st == BFP8_OK && a.residual != nullptr) {
    st = check_matrix(a.residual, a.ldres, a.cols, size);
    if (st == BFP8_OK) st = check_matrix(a.sum, a.ldsum, a.cols, size);
    if (st == BFP8_OK && (shifted(a.sum, a.ldsum, a.x, a.ldx, a.rows) ||
                          shifted(a.sum, a.ldsum, a.residual, a.ldres, a.rows)))
      st = BFP8_ERR_SHAPE;
  }
  if (st != BFP8_OK) return st;
  if (a.w == nullptr || a.rstd == nullptr) return BFP8_ERR_NULL;
  return aligned16(a.w) && aligned16(a.rstd) ? BFP8_OK : BFP8_ERR_ALIGN;
}

bfp8_status check_norm_sizes(bfp8_in_dtype wdt, bfp8_in_dtype dt, int64_t rows, int64_t cols) {
  if (!is_dtype(wdt)) return BFP8_ERR_DTYPE;
  const bfp8_status st = check_sizes(dt, rows, cols);
  return st == BFP8_OK && cols > kMaxNormCols ? BFP8_ERR_SHAPE : st;
}

// From the smallest normal number on: the reciprocal root takes what is less for 0.
bool valid_eps(float eps) { return eps >= FLT_MIN && !isinf(eps); }

bfp8_status check_jobs(const bfp8_grad_job* jobs, int64_t n, bool outputs) {
  if (n < 0) return BFP8_ERR_SHAPE;
  if (n > 0 && jobs == nullptr) return BFP8_ERR_NULL;
  for (int64_t i = 0; i < n; ++i) {
    const bfp8_grad_job& j = jobs[i];
    if (!is_dtype(j.dt)) return BFP8_ERR_DTYPE;
    if (j.rows < 0 || j.cols < 0) return BFP8_ERR_SHAPE;
    if (j.rows == 0 || j.cols == 0) continue;
    if (j.cols >= (int64_t(1) << 40) / j.rows) return BFP8_ERR_SHAPE;
    const uintptr_t mask = static_cast<uintptr_t>(bytes_of(static_cast<bfp8_in_dtype>(j.dt)) - 1);
    if (j.g == nullptr) return BFP8_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(j.g) & mask) != 0) return BFP8_ERR_ALIGN;
    if (j.ldg < j.cols || j.ldg > kMaxLd) return BFP8_ERR_SHAPE;
    if (!outputs) continue;
    if (j.out == nullptr) return BFP8_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(j.out) & mask) != 0) return BFP8_ERR_ALIGN;
    if (j.ldo < j.cols || j.ldo > kMaxLd) return BFP8_ERR_SHAPE;
    if (j.out == j.g && j.rows > 1 && j.ldo != j.ldg) return BFP8_ERR_SHAPE;
  }
  return BFP8_OK;
}

}  // namespace

extern "C" {

bfp8_status bfp8_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldres,
                         const void* w, bfp8_in_dtype wdt, bfp8_in_dtype dt, int64_t rows,
                         int64_t cols, float eps, void* sum, int64_t ldsum, void* y, int64_t ldy,
                         float* rstd, hipStream_t stream) {
  bfp8_status st = check_norm_sizes(wdt, dt, rows, cols);
  if (st != BFP8_OK) return st;
  if (!valid_eps(eps)) return BFP8_ERR_SHAPE;
  if (rows == 0 || cols == 0) return BFP8_OK;
  const NormArgs a{x, ldx, residual, ldres, w, wdt == BFP8_IN_F32, sum, ldsum, y, ldy, rstd, rows,
                   static_cast<int>(cols), eps, 0.0f, 0.0f, false};
  if ((st = check_norm(a, wdt, dt)) != BFP8_OK) return st;
  if ((st = check_matrix(y, ldy, cols, bytes_of(dt))) != BFP8_OK) return st;
  if (shifted(y, ldy, x, ldx, rows) ||
      (residual != nullptr && (shifted(y, ldy, residual, ldres, rows) || y == sum)))
    return BFP8_ERR_SHAPE;
  return launch_rmsnorm(a, dt, stream);
}

bfp8_status bfp8_rmsnorm_quantize(const void* x, int64_t ldx, const void* residual, int64_t ldres,
                                  const void* w, bfp8_in_dtype wdt, bfp8_in_dtype dt, int64_t rows,
                                  int64_t cols, float eps, void* sum, int64_t ldsum, float* rstd,
                                  bfp8_code_format format, uint8_t* q, int64_t ldq, void* s,
                                  uint8_t* qt, int64_t ldqt, void* st_, hipStream_t stream) {
  bfp8_status st = check_norm_sizes(wdt, dt, rows, cols);
  if (st != BFP8_OK) return st;
  if (!valid_eps(eps)) return BFP8_ERR_SHAPE;
  const CodesOut o{q, ldq, s, qt, ldqt, st_, rows, cols};
  if ((st = check_codes(o, format)) != BFP8_OK) return st;
  if (rows == 0 || cols == 0) return BFP8_OK;
  const NormArgs a{x, ldx, residual, ldres, w, wdt == BFP8_IN_F32, sum, ldsum, nullptr, 0, rstd,
                   rows, static_cast<int>(cols), eps, 0.0f, 0.0f, false};
  if ((st = check_norm(a, wdt, dt)) != BFP8_OK) return st;
  if (debug_checks_enabled()) {
    if ((st = scan(x, ldx, dt, rows, cols, stream)) != BFP8_OK) return st;
    if ((st = scan(residual, ldres, dt, rows, cols, stream)) != BFP8_OK) return st;
    if ((st = scan(w, cols, wdt, 1, cols, stream)) != BFP8_OK) return st;
  }
  return launch_rmsnorm_quantize(a, dt, format, o, stream);
}

size_t bfp8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (check_norm_sizes(BFP8_IN_F32, BFP8_IN_F32, rows, cols) != BFP8_OK) return static_cast<size_t>(-1);
  return static_cast<size_t>(norm_grad_groups(rows, cols) * norm_grad_ld(cols)) * sizeof(float);
}

bfp8_status bfp8_rmsnorm_backward(const void* dy, int64_t lddy, const void* r, int64_t ldr,
                                  const void* w, bfp8_in_dtype wdt, const float* rstd,
                                  const void* dsum, int64_t lddsum, bfp8_in_dtype dt, int64_t rows,
                                  int64_t cols, void* dx, int64_t lddx, float* dw, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
  bfp8_status st = check_norm_sizes(wdt, dt, rows, cols);
  if (st != BFP8_OK) return st;
  if (cols == 0) return BFP8_OK;
  if (dw == nullptr) return BFP8_ERR_NULL;
  if (!aligned16(dw)) return BFP8_ERR_ALIGN;
  if (rows > 0) {
    const int64_t size = bytes_of(dt);
    if ((st = check_matrix(dy, lddy, cols, size)) != BFP8_OK) return st;
    if ((st = check_matrix(r, ldr, cols, size)) != BFP8_OK) return st;
    if ((st = check_matrix(dx, lddx, cols, size)) != BFP8_OK) return st;
    if (dsum != nullptr && (st = check_matrix(dsum, lddsum, cols, size)) != BFP8_OK) return st;
    if (shifted(dx, lddx, dy, lddy, rows) || shifted(dx, lddx, r, ldr, rows) ||
        (dsum != nullptr && shifted(dx, lddx, dsum, lddsum, rows)))
      return BFP8_ERR_SHAPE;
    if (w == nullptr || rstd == nullptr) return BFP8_ERR_NULL;
    if (!aligned16(w) || !aligned16(rstd) || !aligned16(workspace)) return BFP8_ERR_ALIGN;
    if (workspace == nullptr || workspace_bytes < bfp8_rmsnorm_backward_workspace_bytes(rows, cols))
      return BFP8_ERR_WORKSPACE;
  }
  const NormGradArgs a{dy, lddy, r, ldr, w, wdt == BFP8_IN_F32, rstd, dsum, lddsum, dx, lddx, dw,
                       static_cast<float*>(workspace), rows, static_cast<int>(cols)};
  return launch_rmsnorm_backward(a, dt, stream);
}

bfp8_status bfp8_swiglu(const void* gate, int64_t ldg, const void* up, int64_t ldu,
                        bfp8_in_dtype dt, int64_t rows, int64_t cols, void* h, int64_t ldh,
                        hipStream_t stream) {
  bfp8_status st = check_sizes(dt, rows, cols);
  if (st != BFP8_OK || rows == 0 || cols == 0) return st;
  const int64_t size = bytes_of(dt);
  if ((st = check_matrix(gate, ldg, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(up, ldu, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(h, ldh, cols, size)) != BFP8_OK) return st;
  if (shifted(h, ldh, gate, ldg, rows) || shifted(h, ldh, up, ldu, rows)) return BFP8_ERR_SHAPE;
  const GluArgs a{gate, ldg, up, ldu, nullptr, 0, h, ldh, nullptr, 0, rows, cols};
  return launch_swiglu(a, dt, stream);
}

bfp8_status bfp8_swiglu_backward(const void* dh, int64_t lddh, const void* gate, int64_t ldg,
                                 const void* up, int64_t ldu, bfp8_in_dtype dt, int64_t rows,
                                 int64_t cols, void* dgate, int64_t lddg, void* dup, int64_t lddu,
                                 hipStream_t stream) {
  bfp8_status st = check_sizes(dt, rows, cols);
  if (st != BFP8_OK || rows == 0 || cols == 0) return st;
  const int64_t size = bytes_of(dt);
  if ((st = check_matrix(dh, lddh, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(gate, ldg, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(up, ldu, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(dgate, lddg, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(dup, lddu, cols, size)) != BFP8_OK) return st;
  if (dgate == dup) return BFP8_ERR_SHAPE;
  for (const auto& in : {std::pair{dh, lddh}, std::pair{gate, ldg}, std::pair{up, ldu}})
    if (shifted(dgate, lddg, in.first, in.second, rows) || shifted(dup, lddu, in.first, in.second, rows))
      return BFP8_ERR_SHAPE;
  const GluArgs a{gate, ldg, up, ldu, dh, lddh, dgate, lddg, dup, lddu, rows, cols};
  return launch_swiglu(a, dt, stream);
}

bfp8_status bfp8_swiglu_quantize(const void* gate, int64_t ldg, const void* up, int64_t ldu,
                                 bfp8_in_dtype dt, int64_t rows, int64_t cols,
                                 bfp8_code_format format, uint8_t* q, int64_t ldq, void* s,
                                 uint8_t* qt, int64_t ldqt, void* st_, hipStream_t stream) {
  bfp8_status st = check_sizes(dt, rows, cols);
  if (st != BFP8_OK) return st;
  const CodesOut o{q, ldq, s, qt, ldqt, st_, rows, cols};
  if ((st = check_codes(o, format)) != BFP8_OK) return st;
  if (rows == 0 || cols == 0) return BFP8_OK;
  const int64_t size = bytes_of(dt);
  if ((st = check_matrix(gate, ldg, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(up, ldu, cols, size)) != BFP8_OK) return st;
  if (debug_checks_enabled()) {
    if ((st = scan(gate, ldg, dt, rows, cols, stream)) != BFP8_OK) return st;
    if ((st = scan(up, ldu, dt, rows, cols, stream)) != BFP8_OK) return st;
  }
  const GluArgs a{gate, ldg, up, ldu, nullptr, 0, nullptr, 0, nullptr, 0, rows, cols};
  return launch_swiglu_quantize(a, dt, format, o, stream);
}

bfp8_status bfp8_swiglu_backward_quantize(const void* dh, int64_t lddh, const void* gate,
                                          int64_t ldg, const void* up, int64_t ldu,
                                          bfp8_in_dtype dt, int64_t rows, int64_t cols,
                                          bfp8_code_format format, uint8_t* q, int64_t ldq,
                                          void* s, uint8_t* qt, int64_t ldqt, void* st_,
                                          hipStream_t stream) {
  bfp8_status st = check_sizes(dt, rows, cols);
  if (st != BFP8_OK) return st;
  if (cols % 128 != 0) return BFP8_ERR_SHAPE;
  const CodesOut o{q, ldq, s, qt, ldqt, st_, rows, 2 * cols};
  if ((st = check_codes(o, format)) != BFP8_OK) return st;
  if (rows == 0 || cols == 0) return BFP8_OK;
  const int64_t size = bytes_of(dt);
  if ((st = check_matrix(dh, lddh, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(gate, ldg, cols, size)) != BFP8_OK) return st;
  if ((st = check_matrix(up, ldu, cols, size)) != BFP8_OK) return st;
  if (debug_checks_enabled()) {
    if ((st = scan(dh, lddh, dt, rows, cols, stream)) != BFP8_OK) return st;
    if ((st = scan(gate, ldg, dt, rows, cols, stream)) != BFP8_OK) return st;
    if ((st = scan(up, ldu, dt, rows, cols, stream)) != BFP8_OK) return st;
  }
  const GluArgs a{gate, ldg, up, ldu, dh, lddh, nullptr, 0, nullptr, 0, rows, cols};
  return launch_swiglu_quantize(a, dt, format, o, stream);
}

size_t bfp8_grad_norm_workspace_bytes(const bfp8_grad_job* jobs, int64_t n) {
  if (check_jobs(jobs, n, false) != BFP8_OK) return static_cast<size_t>(-1);
  return grad_norm_workspace(jobs, n);
}

// The norm's place and the workspace of its partial sums.
static bfp8_status check_norm_out(const bfp8_grad_job* jobs, int64_t n, const float* norm,
                                  const void* workspace, size_t workspace_bytes) {
  if (norm == nullptr) return BFP8_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(norm) & 3u) != 0 || !aligned16(workspace)) return BFP8_ERR_ALIGN;
  const size_t need = grad_norm_workspace(jobs, n);
  return need > 0 && (workspace == nullptr || workspace_bytes < need) ? BFP8_ERR_WORKSPACE : BFP8_OK;
}

bfp8_status bfp8_grad_norm(const bfp8_grad_job* jobs, int64_t n, float* norm, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  bfp8_status st = check_jobs(jobs, n, false);
  if (st == BFP8_OK) st = check_norm_out(jobs, n, norm, workspace, workspace_bytes);
  if (st != BFP8_OK) return st;
  return launch_grad_norm(jobs, n, norm, static_cast<double*>(workspace), stream);
}

bfp8_status bfp8_grad_clip(const bfp8_grad_job* jobs, int64_t n, const float* norm, float max_norm,
                           hipStream_t stream) {
  const bfp8_status st = check_jobs(jobs, n, true);
  if (st != BFP8_OK) return st;
  if (!(max_norm >= 0.0f)) return BFP8_ERR_SHAPE;
  if (n == 0) return BFP8_OK;
  if (norm == nullptr) return BFP8_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(norm) & 3u) != 0) return BFP8_ERR_ALIGN;
  return launch_grad_clip(jobs, n, const_cast<float*>(norm), max_norm, stream);
}

bfp8_status bfp8_grad_norm_clip(const bfp8_grad_job* jobs, int64_t n, float* norm, float max_norm,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  bfp8_status st = check_jobs(jobs, n, true);
  if (st != BFP8_OK) return st;
  if (!(max_norm >= 0.0f)) return BFP8_ERR_SHAPE;
  if ((st = check_norm_out(jobs, n, norm, workspace, workspace_bytes)) != BFP8_OK) return st;
  return launch_grad_norm_clip(jobs, n, norm, max_norm, static_cast<double*>(workspace), stream);
}

}  // extern "C"
