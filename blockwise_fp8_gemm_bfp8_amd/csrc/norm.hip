// RMS norm with the residual's addition, its codes, and its gradient
// (bfp8_layer.h).  All of it is memory-bound: a handful of VALU operations per
// value, so a row is read once, kept in registers between its sum of squares
// and its use, and nothing but outputs is written.

#include <float.h>

#include <algorithm>

#include "layer.h"

namespace bfp8 {
namespace {

// Sum over the 16 lanes of a DPP row, in every lane.
__device__ __forceinline__ float row16_sum(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));
  return v;
}

// Sum over the TPR threads of a row, in every one of them.  Rows of more than
// a wave are a workgroup's, and its `parts` in LDS are free again only after
// the next barrier: two are used in turn (and a third between two of those).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* parts) {
  v = row16_sum(v);
  if (TPR == 16) return v;
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  if (TPR == 64) return v;
  if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < TPR / 64; ++w) v += parts[w];
  return v;
}

// The weight's values of this thread's columns.
template <int TPR, int NV>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int lane, int cols,
                                            float (&v)[NV][8]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + lane) * 8, n = valid8(c, cols);
    if (f32) Load8<float>::run(static_cast<const float*>(w) + c, v[j], n);
    else Load8<uint16_t>::run(static_cast<const uint16_t*>(w) + c, v[j], n);
  }
}

constexpr int block_threads(int tpr) { return tpr <= 64 ? 256 : tpr; }

// What a pass over the rows leaves beside r and rstd: values, or else the row codes
// of a bfp8_code_format.
constexpr int kValues = -1;

// TPR threads a row, NV vectors of 8 values a thread: vector j of a thread
// holds columns 8 (j TPR + lane), so that a wave's loads are contiguous and 16
// lanes hold a 128-group.
template <typename T, int TPR, int NV, int OUT>
__global__ __launch_bounds__(block_threads(TPR)) void norm_rows_kernel(NormArgs a, CodesOut o) {
  __shared__ float parts[3][TPR <= 64 ? 1 : TPR / 64];
  constexpr int kRows = block_threads(TPR) / TPR;  // of a workgroup at once
  const int lane = threadIdx.x % TPR;
  float w[NV][8];
  load_weight<TPR, NV>(a.w, a.w_f32, lane, a.cols, w);
  int turn = 0;
  const int64_t place = a.large ? xcd_run(blockIdx.x, gridDim.x) : blockIdx.x;
  for (int64_t row = place * kRows + threadIdx.x / TPR; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
    Raw8<T> x[NV], y[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * 8, n = valid8(c, a.cols);
      if (a.large && n == 8) {
        x[j].load_once(a.x, row * a.ldx + c);
        if (a.residual != nullptr) y[j].load_once(a.residual, row * a.ldres + c);
      } else {
        x[j].load(a.x, row * a.ldx + c, n);
        if (a.residual != nullptr) y[j].load(a.residual, row * a.ldres + c, n);
      }
    }
    float r[NV][8], square = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * 8, n = valid8(c, a.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[j][i] = x[j].get(i);
      if (a.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] += y[j].get(i);
        if (sizeof(T) == 2) {  // the norm is of the stored sum
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const uint32_t b = pack_bf16x2(r[j][i], r[j][i + 1]);
            r[j][i] = __uint_as_float(b << 16);
            r[j][i + 1] = __uint_as_float(b & 0xFFFF0000u);
          }
        }
        store8(static_cast<T*>(a.sum) + row * a.ldsum + c, r[j], n);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) square = fmaf(r[j][i], r[j][i], square);
    }
    square = row_sum<TPR>(square, parts[turn]);
    // The sum of a row whose mean is within float32's range may be past it: again with
    // values 2^-72 of their size, of which all that matter to such a sum are normal.  (The
    // condition is the same in all of the row's threads.)
    float unit = 1.0f, eps = a.eps;
    if (__builtin_expect(square > FLT_MAX, 0)) {
      unit = 0x1p-72f;
      eps = eps * unit * unit;
      square = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) square = fmaf(r[j][i] * unit, r[j][i] * unit, square);
      square = row_sum<TPR>(square, parts[2]);
    }
    // mean + eps rounded once, the estimate of its root within 2 U (U = 2^-24) squared away:
    // within 2 U (measured 1.5; with 1 / cols rounded and the estimate alone it was 2.3, and
    // two divisions and a root took up to 4 % longer).  An infinite mean leaves 0.
    const float mean = fmaf(square, a.per_col, fmaf(square, a.per_col_low, eps));
    float rstd = __builtin_amdgcn_rsqf(mean);
    rstd = fmaf(rstd * 0.5f, fmaf(-fminf(mean, FLT_MAX) * rstd, rstd, 1.0f), rstd) * unit;
    if (lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * 8, n = valid8(c, a.cols);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r[j][i] * rstd * w[j][i];
      if (OUT == kValues) store8(static_cast<T*>(a.y) + row * a.ldy + c, v, n);
      else if (n > 0) emit_row_chunk<OUT < 0 ? 0 : OUT>(o, row, c & ~127, lane & 15, v);
    }
  }
}

// The threads P and vectors V of a row: one vector a thread as far as a workgroup
// goes.  (Two or four were as fast only before large rows went past the caches: 16384 x
// 2048 with both codes 55 us, 57 and 61; 32768 x 1024 53 and, with two, 58; 8192 x 4096
// 56 and 59.  A few rows are done sooner, too: 16 x 2048 3.3 us against 3.7 and 4.1.)  Up
// to 128 channels 16 lanes, up to 512 a wave: 131072 x 64 11 us, and 33 with a wave a row;
// 65536 x 512 25, and 36 with two.  (Half of the 16 lanes idle at 64 channels, half of the
// wave at 256.)
#define BFP8_WITH_ROW(cols, CALL)                                             \
  ((cols) <= 128    ? [&] { constexpr int P = 16, V = 1; return CALL; }()     \
   : (cols) <= 512  ? [&] { constexpr int P = 64, V = 1; return CALL; }()     \
   : (cols) <= 1024 ? [&] { constexpr int P = 128, V = 1; return CALL; }()    \
   : (cols) <= 2048 ? [&] { constexpr int P = 256, V = 1; return CALL; }()    \
   : (cols) <= 4096 ? [&] { constexpr int P = 512, V = 1; return CALL; }()    \
   : (cols) <= 8192 ? [&] { constexpr int P = 1024, V = 1; return CALL; }()   \
                    : [&] { constexpr int P = 1024, V = 2; return CALL; }())

// Above this many bytes of x bf16 rows are read past the caches, in runs of an XCD: 67
// MB and as much of residual to values took 44 us so and 47 otherwise (54 in runs
// through the caches), to row codes 39 and 44, to both 56 and 61 (without a residual to
// values 26 and 24); MLPBlock's forward pass over 16384 tokens 706 and 724, over 4096,
// where x has 17 MB, 207 and 206.
constexpr int64_t kLargeRows = int64_t(32) << 20;

template <typename T, int TPR, int NV, int OUT>
bfp8_status launch_rows(NormArgs a, const CodesOut& o, hipStream_t stream) {
  a.per_col = 1.0f / static_cast<float>(a.cols);
  a.per_col_low = static_cast<float>(1.0 / a.cols - a.per_col);
  a.large = sizeof(T) == 2 && a.rows * a.cols * 2 > kLargeRows;
  constexpr int kRows = block_threads(TPR) / TPR;
  const int64_t blocks = std::min<int64_t>((a.rows + kRows - 1) / kRows, 1 << 16);
  return launch(norm_rows_kernel<T, TPR, NV, OUT>, dim3(static_cast<unsigned>(blocks)),
                dim3(block_threads(TPR)), stream, a, o);
}
template <typename T, int OUT>
bfp8_status launch_rows_of(const NormArgs& a, const CodesOut& o, hipStream_t stream) {
  return BFP8_WITH_ROW(a.cols, (launch_rows<T, P, V, OUT>(a, o, stream)));
}

// The transposed codes of a tile from r and the rows' statistics.  Statistics need
// the whole row and a token group needs 128 rows, which no workgroup holds at once:
// so r is read a second time, from the last-level cache where it fits.  (The row
// codes leave with the statistics, in whole rows: 16384 x 2048 55 us, and 57 with
// them in these tiles.)
template <typename T, int FORMAT>
__global__ __launch_bounds__(kTileThreads) void norm_tile_kernel(const void* r, int64_t ldr,
                                                                 const float* rstd, const void* w,
                                                                 bool w_f32, unsigned col_tiles,
                                                                 CodesOut o) {
  __shared__ __attribute__((aligned(16))) TileShared sh;
  const unsigned tile = xcd_run(blockIdx.x, gridDim.x);
  const unsigned tm = tile / col_tiles, tc = tile - tm * col_tiles;
  const int64_t m0 = static_cast<int64_t>(tm) * 128, c0 = static_cast<int64_t>(tc) * 128;
  const int lane16 = threadIdx.x & 15, rsub = threadIdx.x >> 4;
  Raw8<T> raw[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) raw[u].load(r, (m0 + 4 * rsub + u) * ldr + c0 + lane16 * 8, 8);
  float wv[8], v[4][8];
  if (w_f32) Load8<float>::run(static_cast<const float*>(w) + c0 + lane16 * 8, wv, 8);
  else Load8<uint16_t>::run(static_cast<const uint16_t*>(w) + c0 + lane16 * 8, wv, 8);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float rs = rstd[m0 + 4 * rsub + u];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] = raw[u].get(k) * rs * wv[k];
  }
  emit_tile<FORMAT, false>(o, m0, c0, v, sh);
}

template <typename T>
bfp8_status quantize_typed(const NormArgs& a, bfp8_code_format format, const CodesOut& o,
                           hipStream_t stream) {
  const bfp8_status st = BFP8_WITH_FORMAT(format, (launch_rows_of<T, F>(a, o, stream)));
  if (st != BFP8_OK || o.qt == nullptr) return st;
  const bool added = a.residual != nullptr;
  const int64_t col_tiles = a.cols / 128, tiles = a.rows / 128 * col_tiles;
  return BFP8_WITH_FORMAT(
      format, (launch(norm_tile_kernel<T, F>, dim3(static_cast<unsigned>(tiles)),
                      dim3(kTileThreads), stream, added ? a.sum : a.x, added ? a.ldsum : a.ldx,
                      a.rstd, a.w, a.w_f32, static_cast<unsigned>(col_tiles), o)));
}

// ---- gradient ------------------------------------------------------------------

// Rows in turn, the weight and this workgroup's share of dw in registers; the
// waves' shares meet in LDS at the end and leave as one row of `partial`.  The
// rows are read past the caches (16384 x 2048 51 us, and 55 through them).
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(block_threads(TPR)) void norm_grad_kernel(NormGradArgs a) {
  constexpr int kThreads = block_threads(TPR), kRows = kThreads / TPR;
  __shared__ float parts[2][TPR <= 64 ? 1 : TPR / 64];
  __shared__ __attribute__((aligned(16))) float joined[kRows > 1 ? kRows / 2 * TPR * NV * 8 : 4];
  const int lane = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  float w[NV][8], dw[NV][8];
  load_weight<TPR, NV>(a.w, a.w_f32, lane, a.cols, w);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + slot; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1) {
    Raw8<T> dy[NV], r[NV], ds[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * 8, n = valid8(c, a.cols);
      if (n == 8) {
        dy[j].load_once(a.dy, row * a.lddy + c);
        r[j].load_once(a.r, row * a.ldr + c);
        if (a.dsum != nullptr) ds[j].load_once(a.dsum, row * a.lddsum + c);
      } else {
        dy[j].load(a.dy, row * a.lddy + c, n);
        r[j].load(a.r, row * a.ldr + c, n);
        if (a.dsum != nullptr) ds[j].load(a.dsum, row * a.lddsum + c, n);
      }
    }
    const float rstd = a.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = dy[j].get(i) * (r[j].get(i) * rstd);
        dw[j][i] += p;
        dot = fmaf(p, w[j][i], dot);
      }
    const float mean = row_sum<TPR>(dot, parts[turn]) / static_cast<float>(a.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * 8, n = valid8(c, a.cols);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = r[j].get(i) * rstd;
        v[i] = rstd * (dy[j].get(i) * w[j][i] - t * mean);
        if (a.dsum != nullptr) v[i] += ds[j].get(i);
      }
      store8(static_cast<T*>(a.dx) + row * a.lddx + c, v, n);
    }
  }
  // the upper half of the slots gives its sums to the lower half, until one is left
#pragma unroll
  for (int half = kRows / 2; half > 0; half /= 2) {
    if (slot >= half && slot < 2 * half) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          joined[(((slot - half) * NV + j) * 8 + i) * TPR + lane] = dw[j][i];
    }
    __syncthreads();
    if (slot < half) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] += joined[((slot * NV + j) * 8 + i) * TPR + lane];
    }
    __syncthreads();
  }
  if (slot == 0) {
    float* p = a.partial + static_cast<int64_t>(blockIdx.x) * norm_grad_ld(a.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + lane) * 8;
      if (c < a.cols) store8(p + c, dw[j], 8);
    }
  }
}

// dw [cols] as the sum of `groups` rows of partial sums: 32 columns a
// workgroup, four a lane, so that 128 rows are under way at once; their sums
// meet in LDS.
constexpr int kSumSlots = 128;
__global__ __launch_bounds__(8 * kSumSlots) void norm_grad_sum_kernel(const float* partial, int groups,
                                                                      int cols, float* dw) {
  __shared__ __attribute__((aligned(16))) float sums[kSumSlots][36];  // 32, and 4 to spread a column
  const int lane = threadIdx.x & 7, slot = threadIdx.x >> 3;
  const int64_t ld = norm_grad_ld(cols);
  const int c = blockIdx.x * 32 + lane * 4;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < ld) {
#pragma unroll 4
    for (int g = slot; g < groups; g += kSumSlots) {
      const float4 p = *reinterpret_cast<const float4*>(partial + g * ld + c);
      s[0] += p.x, s[1] += p.y, s[2] += p.z, s[3] += p.w;
    }
  }
  *reinterpret_cast<float4*>(&sums[slot][lane * 4]) = make_float4(s[0], s[1], s[2], s[3]);
  __syncthreads();
  // 32 columns by 32 threads, four slots each; then a row of 32 lanes' tree
  const int col = threadIdx.x >> 5, part = threadIdx.x & 31;
  float sum = (sums[part][col] + sums[part + 32][col]) + (sums[part + 64][col] + sums[part + 96][col]);
#pragma unroll
  for (int m = 1; m < 32; m *= 2) sum += __shfl_xor(sum, m);
  if (part == 0 && blockIdx.x * 32 + col < cols) dw[blockIdx.x * 32 + col] = sum;
}

template <typename T, int TPR, int NV>
bfp8_status launch_grad(const NormGradArgs& a, hipStream_t stream) {
  constexpr int kRows = block_threads(TPR) / TPR;
  const int64_t groups = std::min((a.rows + kRows - 1) / kRows, norm_grad_groups(a.rows, a.cols));
  if (groups > 0) {
    const bfp8_status st = launch(norm_grad_kernel<T, TPR, NV>, dim3(static_cast<unsigned>(groups)),
                                  dim3(block_threads(TPR)), stream, a);
    if (st != BFP8_OK) return st;
  }
  return launch(norm_grad_sum_kernel, dim3((a.cols + 31) / 32), dim3(8 * kSumSlots), stream,
                a.partial, static_cast<int>(groups), a.cols, a.dw);
}
// Two vectors a thread, whose sums of dw stay in registers (32768 x 1024 with dsum 50 us, 80
// with one in twice the threads).  bf16 rows of up to 2048 a wave each, so that none waits
// for another wave (16384 x 2048 with dsum 52 us, 76 with two waves a row); fp32 rows need
// too many registers for that (8192 x 2048 61 us, 54 with two waves).  Few channels as in
// the forward pass (262144 x 128 with dsum 48 us, 184 with a wave a row; 65536 x 512 48,
// 147 with two waves).
template <typename T>
bfp8_status launch_grad_of(const NormGradArgs& a, hipStream_t stream) {
  constexpr bool kBf16 = sizeof(T) == 2;
  return a.cols <= 128    ? launch_grad<T, 16, 1>(a, stream)
         : a.cols <= 512  ? launch_grad<T, 64, 1>(a, stream)
         : a.cols <= 1024 ? launch_grad<T, 64, 2>(a, stream)
         : a.cols <= 2048 ? launch_grad<T, kBf16 ? 64 : 128, kBf16 ? 4 : 2>(a, stream)
         : a.cols <= 4096 ? launch_grad<T, 256, 2>(a, stream)
         : a.cols <= 8192 ? launch_grad<T, 512, 2>(a, stream)
                          : launch_grad<T, 1024, 2>(a, stream);
}

}  // namespace

bfp8_status launch_rmsnorm(const NormArgs& a, bfp8_in_dtype dt, hipStream_t stream) {
  return dt == BFP8_IN_F32 ? launch_rows_of<float, kValues>(a, CodesOut{}, stream)
                           : launch_rows_of<uint16_t, kValues>(a, CodesOut{}, stream);
}

bfp8_status launch_rmsnorm_quantize(const NormArgs& a, bfp8_in_dtype dt, bfp8_code_format format,
                                    const CodesOut& o, hipStream_t stream) {
  return dt == BFP8_IN_F32 ? quantize_typed<float>(a, format, o, stream)
                           : quantize_typed<uint16_t>(a, format, o, stream);
}

// Workgroups of the gradient at most.  Each has partial sums of dw to write and to
// be read: as many as run at once, two a CU by their registers, or one of 1024
// threads.  (The whole call at 16384 x 2048 with 256, 512 and 1024: 57, 52, 55 us.)
int64_t norm_grad_groups(int64_t rows, int64_t cols) {
  return std::min<int64_t>(rows, cols <= 8192 ? 512 : 256);
}

bfp8_status launch_rmsnorm_backward(const NormGradArgs& a, bfp8_in_dtype dt, hipStream_t stream) {
  return dt == BFP8_IN_F32 ? launch_grad_of<float>(a, stream) : launch_grad_of<uint16_t>(a, stream);
}

}  // namespace bfp8
