// E4M3 codes of float32 values in registers: what the quantisers and the
// kernels that write their results as codes share (not part of the ABI).
#pragma once

#include "bfp8_layer.h"
#include "common.h"

namespace bfp8 {

// Eight consecutive input elements as float32.  bf16 elements are widened
// exactly; `nvalid` (0..8) masks a ragged tail to +0.
template <typename T>
struct Load8;

template <>
struct Load8<uint16_t> {
  static __device__ __forceinline__ void run(const uint16_t* p, float (&v)[8], int nvalid) {
    if (nvalid >= 8) {
      uint4 u = *reinterpret_cast<const uint4*>(p);
      uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < nvalid ? bf16_bits_to_f32(p[i]) : 0.0f;
    }
  }
};

template <>
struct Load8<float> {
  static __device__ __forceinline__ void run(const float* p, float (&v)[8], int nvalid) {
    if (nvalid >= 8) {
      float4 a = reinterpret_cast<const float4*>(p)[0];
      float4 b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < nvalid ? p[i] : 0.0f;
    }
  }
};

__device__ __forceinline__ float absmax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  uint2 r;
  r.x = encode4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  r.y = encode4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
  return r;
}

// Max over the lanes of one group: 16 lanes per 128-group, 4 per 32-group.
template <int GROUP>
__device__ __forceinline__ float group_lanes_max(float v) {
  return GROUP == 128 ? row16_max(v) : quad_max(v);
}

// Loads and stores of what is read or written once and by nobody else soon:
// they leave the caches to data in between.
typedef uint32_t Words4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Words4 load_once(const void* p) {
  return __builtin_nontemporal_load(static_cast<const Words4*>(p));
}
__device__ __forceinline__ void store_once(void* p, uint4 v) {
  __builtin_nontemporal_store(Words4{v.x, v.y, v.z, v.w}, static_cast<Words4*>(p));
}

// Eight elements as loaded, `n` (0..8) of them valid, the others zero: loads
// of several vectors are issued together and widened afterwards.
template <typename T>
struct Raw8;

template <>
struct Raw8<uint16_t> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* base, int64_t at, int n) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (n >= 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = 2 * i < n ? p[2 * i] : 0u;
        if (2 * i + 1 < n) w[i] |= static_cast<uint32_t>(p[2 * i + 1]) << 16;
      }
    }
  }
  __device__ __forceinline__ void load_once(const void* base, int64_t at) {
    const Words4 u = bfp8::load_once(static_cast<const uint16_t*>(base) + at);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
  __device__ __forceinline__ float get(int i) const {
    return i & 1 ? __uint_as_float(w[i >> 1] & 0xFFFF0000u) : __uint_as_float(w[i >> 1] << 16);
  }
};

template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ void load(const void* base, int64_t at, int n) {
    Load8<float>::run(static_cast<const float*>(base) + at, v, n);
  }
  // a lane's two halves share lines with its neighbours' and are loaded apart:
  // through the caches after all
  __device__ __forceinline__ void load_once(const void* base, int64_t at) { load(base, at, 8); }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
};

// The first `n` (0..8) of eight values, rounded to T.
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  if (n >= 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int n) {
  if (n >= 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// How many of the eight elements from column c on lie in a row of `cols`.
__device__ __forceinline__ int valid8(int64_t c, int64_t cols) {
  const int64_t left = cols - c;
  return left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0);
}

// ---- codes of computed results ------------------------------------------------

// ScaleRule for results, whose size is not the caller's to choose: a float32
// group under 2^-117, where 448 / amax would pass float32's range, counts as
// zeros.
constexpr float kTinyGroup = 0x1p-117f;
template <int RULE>
__device__ __forceinline__ typename ScaleRule<RULE>::type result_scale(float amax, float& inv) {
  return ScaleRule<RULE>::make(RULE == 0 && amax < kTinyGroup ? 0.0f : amax, inv);
}

// encode4 without its clamp: |v| <= amax gives |v * inv| <= 448 (1 + 2^-23),
// which rounds to 448.  (The first conversion leaves the upper half of the
// register as it was, for the second; any dead one will do.)
__device__ __forceinline__ uint32_t encode4_within(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, __float_as_int(a), false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}
__device__ __forceinline__ uint2 encode8_within(const float (&v)[8], float inv) {
  return make_uint2(encode4_within(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    encode4_within(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// The formats of bfp8_layer.h: the scales' rule, the groups' length, and
// whether the scale tensors are K-block major.
template <int FORMAT>
struct Codes {
  static constexpr int kRule = FORMAT == BFP8_CODES_F32 ? 0 : 1;
  static constexpr int kGroupLen = FORMAT == BFP8_CODES_E8M0_32 ? 32 : 128;
  static constexpr bool kMajor = FORMAT != BFP8_CODES_E8M0_32;
  typedef typename ScaleRule<kRule>::type S;
};

// Where a call's codes go.  `rows` and `cols` are the result's.
struct CodesOut {
  uint8_t* q;
  int64_t ldq;
  void* s;
  uint8_t* qt;  // null: row groups only
  int64_t ldqt;
  void* st;
  int64_t rows, cols;
};

// Largest sizes.  Sizes are not negative, so that their bits order as they do
// and meet as integers: a maximum with another lane's is one instruction then.
__device__ __forceinline__ uint32_t size8(const float (&v)[8]) {
  return __float_as_uint(absmax8(v));
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_with_lane(uint32_t v) {
  const uint32_t w = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true);
  return v > w ? v : w;
}
// Of every row's sizes the largest in its group's lanes (16, or 4 for groups of 32).
template <int GROUP, int N>
__device__ __forceinline__ void group_max(uint32_t (&m)[N]) {
  // quad_perm [1,0,3,2] and [2,3,0,1], row_half_mirror, row_mirror
#pragma unroll
  for (int u = 0; u < N; ++u) m[u] = max_with_lane<0xB1>(m[u]);
#pragma unroll
  for (int u = 0; u < N; ++u) m[u] = max_with_lane<0x4E>(m[u]);
  if (GROUP == 32) return;
#pragma unroll
  for (int u = 0; u < N; ++u) m[u] = max_with_lane<0x141>(m[u]);
#pragma unroll
  for (int u = 0; u < N; ++u) m[u] = max_with_lane<0x140>(m[u]);
}

// Row groups from a row of 16 lanes that hold columns c0 + 8 lane .. + 7 of a
// row (c0 a multiple of 128): codes and scales.
template <int FORMAT>
__device__ __forceinline__ void emit_row_chunk(const CodesOut& o, int64_t row, int64_t c0,
                                               int lane16, const float (&v)[8]) {
  typedef Codes<FORMAT> F;
  uint32_t m[1] = {size8(v)};
  group_max<F::kGroupLen>(m);
  float inv;
  const typename F::S sc = result_scale<F::kRule>(__uint_as_float(m[0]), inv);
  *reinterpret_cast<uint2*>(o.q + row * o.ldq + c0 + lane16 * 8) = encode8_within(v, inv);
  typename F::S* s = static_cast<typename F::S*>(o.s);
  if (F::kMajor) {
    if (lane16 == 0) s[c0 / 128 * o.rows + row] = sc;
  } else if (lane16 % 4 == 0) {
    s[row * (o.cols / 32) + c0 / 32 + lane16 / 4] = sc;
  }
}

// max over the two halves (rows of 16) of a wave for two sizes at once:
// lanes of the lower half (of even rows) get a's, the others b's.
__device__ __forceinline__ uint32_t halves_max(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return r[0] > r[1] ? r[0] : r[1];
}
__device__ __forceinline__ uint32_t rows_max(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  return r[0] > r[1] ? r[0] : r[1];
}
template <int U>
__device__ __forceinline__ float quad_broadcast(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), U * 0x55, 0xF, 0xF, true));
}

// The place of workgroup b of n in an order that gives each XCD (b mod 8) one
// run of neighbours: what neighbouring tiles write of a row meets in one L2.
__device__ __forceinline__ unsigned xcd_run(unsigned b, unsigned n) {
  const unsigned x = b & 7, each = n >> 3, more = n & 7;
  return x * each + (x < more ? x : more) + (b >> 3);
}

// A 128 x 128 tile's codes in both layouts, from 512 threads: thread
// (rsub = tid / 16, lane16 = tid % 16) holds tokens m0 + 4 rsub .. + 3 of
// channels c0 + 8 lane16 .. + 7.
//   Row groups lie in 16 lanes of a row (quads for groups of 32); lane l makes
// the scale of the thread's row l % 4 and the quad passes the four factors
// round, so that a thread divides once for its four rows.  Column maxima meet
// within the wave by lane swaps that halve the values they reduce, then over
// the waves in LDS, where one thread a group makes the scale.  The codes of a
// channel's four tokens are one dword of the LDS tile [channel][token], whose
// 16-byte chunks are permuted by channel / 8 to spread the writes over the
// banks; its rows leave as 128-byte runs, past the caches, which are left to the
// row codes: those are the next GEMM's operand, the transposed ones wait for the
// backward pass.  (MLPBlock's forward pass over 16384 tokens 719 us so, 740 the
// other way round; alone the activation's tiles take 97 us either way and 120
// with both kept, their gradient's 198 and 202.)
//   The last barrier's reads are of the code tile alone, which the next call
// writes after its own first barrier: tiles can follow each other.
struct TileShared {
  uint8_t ct[128 * 128];
  uint32_t colmax[8][128];
  float colinv[4][128];
  float rowscale[128];
};
constexpr int kTileThreads = 512;

// ROWS false: the transposed codes alone.
template <int FORMAT, bool ROWS>
__device__ __forceinline__ void emit_tile(const CodesOut& o, int64_t m0, int64_t c0,
                                          const float (&v)[4][8], TileShared& sh) {
  typedef Codes<FORMAT> F;
  typedef typename F::S S;
  const int tid = threadIdx.x, lane16 = tid & 15, rsub = tid >> 4, wave = tid >> 6;
  S* s = static_cast<S*>(o.s);
  S* st = static_cast<S*>(o.st);

  S* rowscale = reinterpret_cast<S*>(sh.rowscale);
  if constexpr (ROWS) {
    uint32_t am[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) am[u] = size8(v[u]);
    group_max<F::kGroupLen>(am);
    const int mine = tid & 3;
    const uint32_t m01 = mine & 1 ? am[1] : am[0], m23 = mine & 1 ? am[3] : am[2];
    float inv;
    const S sc = result_scale<F::kRule>(__uint_as_float(mine & 2 ? m23 : m01), inv);
    const float invs[4] = {quad_broadcast<0>(inv), quad_broadcast<1>(inv), quad_broadcast<2>(inv),
                           quad_broadcast<3>(inv)};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<uint2*>(o.q + (m0 + 4 * rsub + u) * o.ldq + c0 + lane16 * 8) =
          encode8_within(v[u], invs[u]);
    if (F::kMajor) {
      if (lane16 < 4) rowscale[4 * rsub + lane16] = sc;
    } else {
      s[(m0 + 4 * rsub + mine) * (o.cols / 32) + c0 / 32 + lane16 / 4] = sc;
    }
  }

  // column maxima of the wave's 16 tokens
  uint32_t cm[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    cm[k] = __float_as_uint(
        fmaxf(fmaxf(fmaxf(fabsf(v[0][k]), fabsf(v[1][k])), fabsf(v[2][k])), fabsf(v[3][k])));
  const uint32_t low = rows_max(halves_max(cm[0], cm[1]), halves_max(cm[2], cm[3]));
  const uint32_t high = rows_max(halves_max(cm[4], cm[5]), halves_max(cm[6], cm[7]));
  const int kk = ((rsub & 1) << 1) | ((rsub >> 1) & 1);  // the channel this lane's row is left with
  sh.colmax[wave][lane16 * 8 + kk] = low;
  sh.colmax[wave][lane16 * 8 + kk + 4] = high;
  __syncthreads();

  if (ROWS && F::kMajor && tid >= 128 && tid < 256)
    s[c0 / 128 * o.rows + m0 + tid - 128] = rowscale[tid - 128];
  if (F::kGroupLen == 32 || tid < 128) {
    const int c = tid & 127, p = tid >> 7;
    uint32_t m = max(sh.colmax[2 * p][c], sh.colmax[2 * p + 1][c]);
    if (F::kGroupLen == 128) {
#pragma unroll
      for (int w = 2; w < 8; ++w) m = max(m, sh.colmax[w][c]);
    }
    float cinv;
    const S tsc = result_scale<F::kRule>(__uint_as_float(m), cinv);
    sh.colinv[p][c] = cinv;
    if (F::kMajor) st[m0 / 128 * o.cols + c0 + c] = tsc;
    else st[(c0 + c) * (o.rows / 32) + m0 / 32 + p] = tsc;
  }
  __syncthreads();

  const float* ci = &sh.colinv[F::kGroupLen == 32 ? wave >> 1 : 0][lane16 * 8];
  float ck[8];
  *reinterpret_cast<float4*>(&ck[0]) = *reinterpret_cast<const float4*>(ci);
  *reinterpret_cast<float4*>(&ck[4]) = *reinterpret_cast<const float4*>(ci + 4);
  const int chunk = (wave ^ (lane16 & 7)) * 16 + (rsub & 3) * 4;  // tokens 4 rsub .. + 3
#pragma unroll
  for (int k = 0; k < 8; ++k)
    *reinterpret_cast<uint32_t*>(&sh.ct[(lane16 * 8 + k) * 128 + chunk]) = encode4_within(
        v[0][k] * ck[k], v[1][k] * ck[k], v[2][k] * ck[k], v[3][k] * ck[k]);
  __syncthreads();

#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    const int c = pass * 64 + (tid >> 3), ch = tid & 7;
    const uint4 w = *reinterpret_cast<const uint4*>(&sh.ct[c * 128 + (ch ^ ((c >> 3) & 7)) * 16]);
    store_once(o.qt + (c0 + c) * o.ldqt + m0 + ch * 16, w);
  }
}

}  // namespace bfp8
