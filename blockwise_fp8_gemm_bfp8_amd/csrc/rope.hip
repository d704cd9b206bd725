// Rotary positions for gfx950: the table of cosines and sines, and the turn of
// every head's pairs.  Memory-bound: x is read and y written once, the table's
// rows stay in the L1 across the heads of a token.  16384 tokens of 24 heads of
// 128 (bf16, in rows of 32 heads) take 33 us, 6.4 TB/s; 16 tokens 2.9 us, a
// launch's own time; 5003 tokens of 12 heads of 96, 64 of them turned in
// interleaved pairs (float32), 9.4 us, 4.9 TB/s.
#include "attention.h"

namespace bfp8 {
namespace {

// One (cos, sin) pair per thread, its angle in float64: a float32 product of
// a position p and a frequency is off by p * 2^-24 rad.  It runs once per
// model, so its time does not matter.
__global__ __launch_bounds__(256) void rope_table_kernel(float2* table, int64_t count, int half,
                                                         int rot_dim, double base, double factor,
                                                         double original, int scaling) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= count) return;
  const int64_t p = at / half;
  const int i = static_cast<int>(at - p * half);
  if (scaling == BFP8_ROPE_NTK && rot_dim > 2)
    base *= pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  double f = pow(base, -2.0 * i / rot_dim), m = 1.0;
  if (scaling == BFP8_ROPE_LINEAR) f /= factor;
  if (scaling == BFP8_ROPE_YARN) {
    const double turns = original * f / 6.283185307179586476925;
    const double keep = fmin(fmax((turns - 1.0) / 31.0, 0.0), 1.0);
    f = keep * f + (1.0 - keep) * f / factor;
    m = 0.1 * log(factor) + 1.0;
  }
  double sn, cs;
  sincos(static_cast<double>(p) * f, &sn, &cs);
  table[at] = make_float2(static_cast<float>(m * cs), static_cast<float>(m * sn));
}

// N consecutive values, aligned to N of them, to and from float32.
template <typename T, int N>
struct Values {
  typedef T V __attribute__((ext_vector_type(N)));
};
template <typename T>
struct Values<T, 1> {
  typedef T V;
};
__device__ __forceinline__ float widen(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void narrow_to(float v, uint16_t& r) {
  r = static_cast<uint16_t>(pack_bf16x2(v, v));
}
__device__ __forceinline__ void narrow_to(float v, float& r) { r = v; }

template <typename T, int N>
__device__ __forceinline__ void load_values(const T* p, float (&x)[N]) {
  const typename Values<T, N>::V w = *reinterpret_cast<const typename Values<T, N>::V*>(p);
  T e[N];
  __builtin_memcpy(e, &w, sizeof(e));
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = widen(e[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_values(T* p, const float (&x)[N]) {
  T e[N];
#pragma unroll
  for (int i = 0; i < N; ++i) narrow_to(x[i], e[i]);
  typename Values<T, N>::V w;
  __builtin_memcpy(&w, e, sizeof(e));
  *reinterpret_cast<typename Values<T, N>::V*>(p) = w;
}

// A pair (a, b) turned by an angle that is not known: NaN, but a zero stays one.
__device__ __forceinline__ void turn_unknown(float a, float b, float& ya, float& yb) {
  ya = yb = a == 0.0f && b == 0.0f ? 0.0f : NAN;
}

// A unit is V pairs of one head (2 V values), or 2 V of its values past
// rot_dim, which are copied.  A workgroup's threads are `slots` heads of
// `units` units each; consecutive slots are consecutive heads, then tokens.
template <typename T, int V, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int units, int slots, int turned) {
  const int slot = threadIdx.x / units;
  const int u = threadIdx.x - slot * units;
  const unsigned item = blockIdx.x * static_cast<unsigned>(slots) + slot;
  const unsigned heads = static_cast<unsigned>(a.heads);
  const int64_t t = item / heads;
  const int h = item - static_cast<unsigned>(t) * heads;
  if (slot >= slots || t >= a.tokens) return;
  const T* x = static_cast<const T*>(a.x) + t * a.x_row + h * a.x_head;
  T* y = static_cast<T*>(a.y) + t * a.y_row + h * a.y_head;
  if (u >= turned) {
    const int d = a.rot_dim + (u - turned) * 2 * V;
    float w[2 * V];
    load_values<T, 2 * V>(x + d, w);
    store_values<T, 2 * V>(y + d, w);
    return;
  }
  const int64_t p = a.positions == nullptr ? t : a.positions[t];
  const bool inside = p >= 0 && p < a.table_rows;
  const int half = a.rot_dim / 2;
  float cs[2 * V], c[V], s[V];
  load_values<float, 2 * V>(a.table + ((inside ? p : 0) * half + u * V) * 2, cs);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    c[e] = cs[2 * e];
    s[e] = a.inverse ? -cs[2 * e + 1] : cs[2 * e + 1];
  }
  if (INTERLEAVED) {
    float w[2 * V], r[2 * V];
    load_values<T, 2 * V>(x + u * 2 * V, w);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      r[2 * e] = w[2 * e] * c[e] - w[2 * e + 1] * s[e];
      r[2 * e + 1] = w[2 * e] * s[e] + w[2 * e + 1] * c[e];
      if (!inside) turn_unknown(w[2 * e], w[2 * e + 1], r[2 * e], r[2 * e + 1]);
    }
    store_values<T, 2 * V>(y + u * 2 * V, r);
  } else {
    float w0[V], w1[V], r0[V], r1[V];
    load_values<T, V>(x + u * V, w0);
    load_values<T, V>(x + half + u * V, w1);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      r0[e] = w0[e] * c[e] - w1[e] * s[e];
      r1[e] = w0[e] * s[e] + w1[e] * c[e];
      if (!inside) turn_unknown(w0[e], w1[e], r0[e], r1[e]);
    }
    store_values<T, V>(y + u * V, r0);
    store_values<T, V>(y + half + u * V, r1);
  }
}

template <typename T, int V, bool INTERLEAVED>
bfp8_status launch_units(const RopeArgs& a, hipStream_t stream) {
  const int turned = a.rot_dim / 2 / V;
  const int copied = a.x == a.y ? 0 : (a.head_dim - a.rot_dim) / (2 * V);
  const int units = turned + copied;  // at most head_dim / 2
  const int slots = 256 / units;
  const int64_t blocks = (a.tokens * a.heads + slots - 1) / slots;
  if (!grid_fits(blocks, 256)) return BFP8_ERR_SHAPE;
  return launch(rope_kernel<T, V, INTERLEAVED>, dim3(static_cast<unsigned>(blocks)), dim3(256),
                stream, a, units, slots, turned);
}

// The widest unit that the sizes allow: 16 bytes a load (interleaved pairs are
// one run of 2 V values, pairs of halves two runs of V), or 8, or one value.
template <typename T>
bfp8_status launch_rope_typed(const RopeArgs& a, bool interleaved, hipStream_t stream) {
  constexpr int kWide = 16 / sizeof(T);
  const int half = a.rot_dim / 2, rest = a.head_dim - a.rot_dim;
  auto fits = [&](int v) { return half % v == 0 && rest % (2 * v) == 0; };
  if (interleaved)
    return fits(kWide / 2) ? launch_units<T, kWide / 2, true>(a, stream)
                           : launch_units<T, 1, true>(a, stream);
  if (fits(kWide)) return launch_units<T, kWide, false>(a, stream);
  if (fits(kWide / 2)) return launch_units<T, kWide / 2, false>(a, stream);
  return launch_units<T, 1, false>(a, stream);
}

}  // namespace

bfp8_status launch_rope_table(float* table, int64_t positions, int rot_dim, double base,
                              double factor, double original_length, int scaling,
                              hipStream_t stream) {
  const int64_t count = positions * (rot_dim / 2), blocks = (count + 255) / 256;
  if (!grid_fits(blocks, 256)) return BFP8_ERR_SHAPE;
  return launch(rope_table_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), stream,
                reinterpret_cast<float2*>(table), count, rot_dim / 2, rot_dim, base, factor,
                original_length, scaling);
}

bfp8_status launch_rope(const RopeArgs& a, bfp8_in_dtype dt, bool interleaved, hipStream_t stream) {
  return dt == BFP8_IN_F32 ? launch_rope_typed<float>(a, interleaved, stream)
                           : launch_rope_typed<uint16_t>(a, interleaved, stream);
}

}  // namespace bfp8
