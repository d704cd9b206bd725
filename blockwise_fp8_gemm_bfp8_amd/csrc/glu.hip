// The gated activation, its gradient, and the codes of either (bfp8_layer.h).
// Element by element and memory-bound: every input is read once and only
// results are written; in the tiles of codes the values stay in registers
// between the row groups and the token groups.

#include "layer.h"

namespace bfp8 {
namespace {

// 1 / (1 + exp(-g)) with exp(-g) = 2^y e^rho: y = -g H rounded, H the 16 leading bits of
// log2(e); rho, what H leaves of log2(e) and the rounding leaves of y, is under 5e-4 and
// goes in as 1 + rho.  A rounded -g log2(e) alone was off by |g| 2^-24, 65 U at g = -87 (U
// = 2^-24); silu is within 6 U now (9 from -87.3 to -88.7, where sigma is subnormal), and
// 3.5 U for bf16 gates, whose product with H is exact: there rho takes one instruction, and
// the bits are the same.  (16384 x 6144 with row codes 89 us, and 87 without rho; no call,
// float32 ones too, lost more than 2 %.)
//   All of it at 2^-24 of its size, so that the reciprocal stays a normal number until
// exp(-g) overflows (g = -88.72); from there on the result is 0.
template <bool F32>
__device__ __forceinline__ float sigma(float g) {
  constexpr double kLog2e = 1.44269504088896340736, kLn2 = 0.69314718055994530942;
  constexpr float kUnit = 0x1p-24f, kHead = 47274.0f / 32768.0f;
  constexpr float kTail = static_cast<float>((kHead - kLog2e) * kLn2 * 0x1p-24);
  if (F32) g = __builtin_amdgcn_fmed3f(g, -1e30f, 1e30f);  // y finite: no inf - inf in rho
  const float y = g * -kHead;
  float scale = kUnit;  // 2^-24 (1 + rho)
  if (F32) scale = fmaf(fmaf(g, -kHead, -y), static_cast<float>(kLn2 * 0x1p-24), scale);
  scale = fmaf(g, kTail, scale);
  return __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(y), scale, kUnit)) * kUnit;
}

template <bool F32>
__device__ __forceinline__ float silu_gate(float g, float u) {
  return g * sigma<F32>(g) * u;
}

// dgate = dh u sigma (1 + g (1 - sigma)).  1 - sigma is within 3.5 U for g > 0 (the sum's
// and the reciprocal's roundings), which g raises to 2^-18 at most: from 17.4 on it is
// exactly 0 (measured: 2^-20, the same as with correctly rounded operations).
template <bool F32>
__device__ __forceinline__ void silu_gate_grad(float dh, float g, float u, float& dg, float& du) {
  const float s = sigma<F32>(g);
  dg = dh * u * (s * fmaf(g, 1.0f - s, 1.0f));
  du = dh * (g * s);
}

// Vectors of 8 values, one a thread.  ONCE: loads past the caches.
template <typename T, bool GRAD, bool ONCE>
__global__ __launch_bounds__(256) void glu_values_kernel(GluArgs a, unsigned per_row, unsigned count) {
  const unsigned item = blockIdx.x * 256u + threadIdx.x;
  if (item >= count) return;
  const unsigned row = item / per_row;
  const int64_t c = static_cast<int64_t>(item - row * per_row) * 8;
  const int n = valid8(c, a.cols);
  Raw8<T> g, u, dh;
  if (ONCE && n == 8) {
    g.load_once(a.gate, row * a.ldg + c);
    u.load_once(a.up, row * a.ldu + c);
    if (GRAD) dh.load_once(a.dh, row * a.lddh + c);
  } else {
    g.load(a.gate, row * a.ldg + c, n);
    u.load(a.up, row * a.ldu + c, n);
    if (GRAD) dh.load(a.dh, row * a.lddh + c, n);
  }
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (GRAD) silu_gate_grad<sizeof(T) == 4>(dh.get(i), g.get(i), u.get(i), x[i], y[i]);
    else x[i] = silu_gate<sizeof(T) == 4>(g.get(i), u.get(i));
  }
  store8(static_cast<T*>(a.a) + row * a.lda + c, x, n);
  if (GRAD) store8(static_cast<T*>(a.b) + row * a.ldb + c, y, n);
}

// Row groups: 16 lanes a chunk of 128 columns, 16 rows a workgroup, whose
// K-block-major scales lie side by side; workgroups along the rows, in runs of
// an XCD.  (The 16384 x 6144 activation 89 us and its gradient 145; down the columns with
// loads through the caches 119 and 178, along the rows with such loads 94 and 144.)
template <typename T, int FORMAT, bool GRAD>
__global__ __launch_bounds__(256) void glu_rows_kernel(GluArgs a, unsigned per_row, CodesOut o) {
  const unsigned chunk = xcd_run(blockIdx.x, gridDim.x);
  const unsigned block = chunk / per_row;
  const int64_t row = static_cast<int64_t>(block) * 16 + (threadIdx.x >> 4);
  if (row >= a.rows) return;
  const int lane16 = threadIdx.x & 15;
  const int64_t c0 = static_cast<int64_t>(chunk - block * per_row) * 128, c = c0 + lane16 * 8;
  Raw8<T> g, u, dh;
  g.load_once(a.gate, row * a.ldg + c);
  u.load_once(a.up, row * a.ldu + c);
  if (GRAD) dh.load_once(a.dh, row * a.lddh + c);
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (GRAD) silu_gate_grad<sizeof(T) == 4>(dh.get(i), g.get(i), u.get(i), x[i], y[i]);
    else x[i] = silu_gate<sizeof(T) == 4>(g.get(i), u.get(i));
  }
  emit_row_chunk<FORMAT>(o, row, c0, lane16, x);
  if (GRAD) emit_row_chunk<FORMAT>(o, row, a.cols + c0, lane16, y);
}

template <typename T, int FORMAT, bool GRAD>
__global__ __launch_bounds__(kTileThreads) void glu_tile_kernel(GluArgs a, unsigned col_tiles,
                                                                CodesOut o) {
  __shared__ __attribute__((aligned(16))) TileShared sh;
  const unsigned tile = xcd_run(blockIdx.x, gridDim.x);
  const unsigned tm = tile / col_tiles, tc = tile - tm * col_tiles;
  const int64_t m0 = static_cast<int64_t>(tm) * 128, c0 = static_cast<int64_t>(tc) * 128;
  const int64_t c = c0 + (threadIdx.x & 15) * 8, m = m0 + (threadIdx.x >> 4) * 4;
  Raw8<T> g[4], u[4], dh[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    g[i].load_once(a.gate, (m + i) * a.ldg + c);
    u[i].load_once(a.up, (m + i) * a.ldu + c);
    if (GRAD) dh[i].load_once(a.dh, (m + i) * a.lddh + c);
  }
  // Row by row, each one's results pinned before the next: left to itself the
  // compiler unpacks everything first, 156 registers, and one workgroup fits a
  // CU (93, two: 238 -> 199 us for the gradient of 16384 x 6144, 60 -> 47 for 4096 x 6144).
  float x[4][8], y[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (GRAD) silu_gate_grad<sizeof(T) == 4>(dh[i].get(k), g[i].get(k), u[i].get(k), x[i][k], y[i][k]);
      else x[i][k] = silu_gate<sizeof(T) == 4>(g[i].get(k), u[i].get(k));
    }
    if (GRAD) {
#pragma unroll
      for (int k = 0; k < 8; ++k) asm volatile("" : "+v"(x[i][k]), "+v"(y[i][k]));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  emit_tile<FORMAT, true>(o, m0, c0, x, sh);
  if (GRAD) emit_tile<FORMAT, true>(o, m0, a.cols + c0, y, sh);
}

// Above this many bytes of gate the loads of bf16 values go past the caches: 201 MB
// with as much of up took 99 us so and 107 otherwise (the gradient 174 and 179), where 17
// MB with up and dh took 15.5 and 14.6.
constexpr int64_t kLargeGate = int64_t(64) << 20;

template <typename T, bool GRAD>
bfp8_status values_typed(const GluArgs& a, hipStream_t stream) {
  const int64_t per_row = (a.cols + 7) / 8, count = a.rows * per_row, blocks = (count + 255) / 256;
  if (!threads_fit(blocks, 256)) return BFP8_ERR_SHAPE;
  const bool once = sizeof(T) == 2 && a.rows * a.cols * 2 > kLargeGate;
  return launch(once ? glu_values_kernel<T, GRAD, sizeof(T) == 2> : glu_values_kernel<T, GRAD, false>,
                dim3(static_cast<unsigned>(blocks)), dim3(256), stream, a,
                static_cast<unsigned>(per_row), static_cast<unsigned>(count));
}

template <typename T, bool GRAD>
bfp8_status codes_typed(const GluArgs& a, bfp8_code_format format, const CodesOut& o,
                        hipStream_t stream) {
  const int64_t per_row = a.cols / 128;
  if (o.qt == nullptr) {
    const int64_t blocks = (a.rows + 15) / 16 * per_row;
    if (!threads_fit(blocks, 256)) return BFP8_ERR_SHAPE;
    return BFP8_WITH_FORMAT(
        format, (launch(glu_rows_kernel<T, F, GRAD>, dim3(static_cast<unsigned>(blocks)), dim3(256),
                        stream, a, static_cast<unsigned>(per_row), o)));
  }
  const int64_t tiles = a.rows / 128 * per_row;
  return BFP8_WITH_FORMAT(
      format, (launch(glu_tile_kernel<T, F, GRAD>, dim3(static_cast<unsigned>(tiles)),
                      dim3(kTileThreads), stream, a, static_cast<unsigned>(per_row), o)));
}

}  // namespace

bfp8_status launch_swiglu(const GluArgs& a, bfp8_in_dtype dt, hipStream_t stream) {
  if (a.dh == nullptr)
    return dt == BFP8_IN_F32 ? values_typed<float, false>(a, stream)
                             : values_typed<uint16_t, false>(a, stream);
  return dt == BFP8_IN_F32 ? values_typed<float, true>(a, stream)
                           : values_typed<uint16_t, true>(a, stream);
}

bfp8_status launch_swiglu_quantize(const GluArgs& a, bfp8_in_dtype dt, bfp8_code_format format,
                                   const CodesOut& o, hipStream_t stream) {
  if (a.dh == nullptr)
    return dt == BFP8_IN_F32 ? codes_typed<float, false>(a, format, o, stream)
                             : codes_typed<uint16_t, false>(a, format, o, stream);
  return dt == BFP8_IN_F32 ? codes_typed<float, true>(a, format, o, stream)
                           : codes_typed<uint16_t, true>(a, format, o, stream);
}

}  // namespace bfp8
