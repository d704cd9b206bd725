// Attention forward for gfx950: O = softmax(scale Q K^T) V and its
// log-sum-exp, one pass over the keys with a running maximum and sum.
//
// All products are turned so that a lane owns its query rows throughout:
//   S^T [key][query] = K Q^T   (K rows from LDS, Q rows in registers)
//   O^T [dim][query] = V^T P^T (V columns by transposing LDS reads, P^T the
//                               accumulator of S^T rounded to bf16 in place)
// With v_mfma_f32_16x16x32_bf16 lane l holds query l % 16 of both results, so
// the row maximum and sum are taken over registers and then over the lanes l,
// l ^ 16, l ^ 32, l ^ 48, the rescaling factor is one register, and P never
// moves between lanes.  P is rounded to bf16 for its product only (an error
// like the output's own rounding); its sum is of the float32 values.
//
// A workgroup of 8 waves takes 256 rows of one kv head, a row being one
// (query, head of the group) pair: the heads that share keys share their
// tiles, and few queries fill more of a tile.  Each wave owns 32 rows, two
// sets of 16; tiles of 64 keys pass through three LDS stages, filled by
// LDS-DMA two tiles ahead with one barrier a tile.
//
// What bounds it: the matrix cores and, above that, the card's power.  16 query
// and 8 key/value heads of 128, causal: 4 sequences of 4096 take 250 to 262 us
// (1068 TFLOP/s and more: cards differ), one of 16384 takes 897 to 954 us
// (1157), 13 sequences of 1 to 2417 tokens, 8274 in all, 67 us (the longest
// workgroup: 38 tiles of keys one after another where an even share is 29 a CU;
// and the starts and ends of 2.4 workgroups a CU, one at a time).
// The same long sequence of zeros, which draws less power, takes 726 us.  Of 967
// us, before its last steps, it took 13 % less without the softmax's arithmetic,
// 12 % without LDS reads, 4 % without copies and barriers: none of them alone
// bounds it.  Workgroups of 4 waves, two to a CU, and half of the waves starting
// half a tile late were within 1 % or slower; 64 rows a wave does not fit the
// registers.
#include "attention.h"

namespace bfp8 {
namespace {

using namespace attn;

constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;  // rows of a workgroup
constexpr int kKeys = 64;           // keys of a tile
constexpr int kStages = 3;          // tiles in LDS: one being read, two under way

// The rows are scaled back to the running maximum only when it has grown by
// more than this many powers of two: probabilities stay below 2^8 (float32
// sums and bf16 products hold that without loss), and most tiles skip the
// multiplication of the accumulators.
constexpr float kSlack = 8.0f;

// What a row's sum over its maximum (in powers of two) makes of its output and
// its log-sum-exp: a sum of zero is a row that sees no key, one that is NaN stays
// NaN in both.
__device__ __forceinline__ float row_factor(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
__device__ __forceinline__ float row_lse(float top, float sum) {
  return sum == 0.0f ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// The running maxima of two sets of rows take in `either` (column_max of both),
// and their sums and accumulators are scaled to them.
template <int DP>
__device__ __forceinline__ void raise_maxima(float either, float (&m)[2], float (&l)[2],
                                             f32x4 (&o)[2][DP / 16]) {
  float top[2];
  both_columns(either, top);
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float next = fmaxf(m[n], top[n]);
    const float alpha = __builtin_amdgcn_exp2f(m[n] - (next == -INFINITY ? 0.0f : next));
    m[n] = next;
    l[n] *= alpha;
#pragma unroll
    for (int ct = 0; ct < DP / 16; ++ct) o[n][ct] *= alpha;
  }
}

template <int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_forward_kernel(AttentionArgs a,
                                                                          int places) {
  typedef Tile<DP, kKeys, kWaves> KTile;
  constexpr int kDims = DP / 16;   // 16-column results
  constexpr int kSteps = DP / 32;  // products of one 16x16 square
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStages][2][KTile::kBytes];
  if (blockIdx.x >= a.clear_from) return clear_forward(a);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int g = blockIdx.x % a.kv_heads;
  Sequence s;
  int rank, tiles;
  const int place = blockIdx.x / a.kv_heads;
  const int split = place / places;  // first every tile's first part
  if (!find_tile<false>(a, a.group, kRows, place - split * places, s, rank, tiles)) return;
  const int row0 = rank * kRows;  // the last rows see the most keys
  const int rows = s.qn * a.group;
  const int all = key_tiles(a, s, row0, kRows);
  const int parts = a.split_q.parts(all);
  if (split >= parts) return;
  const int j0 = static_cast<int>(static_cast<int64_t>(all) * split / parts);
  const int nj = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / parts);
  // last key that the wave's last row sees, and its first
  const int wave_first = row0 + wave * 32;
  const int wave_lim = wave_first < rows ? last_key(a, s, min(wave_first + 32, rows) - 1) : -1;
  const int wave_free = last_key(a, s, wave_first);  // seen by every row

  KTile kt, vt;
  kt.init(wave, lane, a.k.row, a.head_dim);
  vt.init(wave, lane, a.v.row, a.head_dim);
  Walk kw(a.k, (int64_t)s.k0 + j0 * kKeys, g, a.head_dim);
  Walk vw(a.v, (int64_t)s.k0 + j0 * kKeys, g, a.head_dim);
  int left = s.kn - j0 * kKeys, ahead = 0;  // keys from there on; stage of the next copies
  auto copy_tile = [&]() {     // tiles in their order; past the end zeros, counted as the others
    const int n = min(left, kKeys);
    kt.copy(lds[ahead][0], wave, kw.rows(n));
    vt.copy(lds[ahead][1], wave, vw.rows(n));
    kw.step(kKeys);
    vw.step(kKeys);
    left -= kKeys;
    ahead = ahead == kStages - 1 ? 0 : ahead + 1;
  };
  if (nj > j0) {
#pragma unroll
    for (int n = 0; n < kStages - 1; ++n) copy_tile();
  }
  // two sets of 16 rows: a lane's row, its query, head and last visible key
  int64_t t[2];
  int h[2], lim[2];
  bool valid[2];
  bf16x8 q[2][kSteps];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int r = wave_first + 16 * n + (lane & 15);
    valid[n] = r < rows;
    h[n] = g * a.group + r % a.group;
    lim[n] = last_key(a, s, min(r, rows - 1));
    t[n] = s.q0 + min(r, rows - 1) / a.group;
    const uint16_t* qrow = a.q.p + t[n] * a.q.row + h[n] * a.q.head;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
      q[n][ks] = load8(qrow, ks * 32 + 8 * (lane >> 4), a.head_dim, valid[n]);
  }
  wait_copies<0>();  // and the loads of q

  f32x4 o[2][kDims] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {};
  float bound = -INFINITY;  // of the set whose maximum column_max leaves in this lane
  int stage = 0;
  for (int j = j0; j < nj; ++j) {
    wait_copies<2 * (kStages - 2) * KTile::kCopies>();  // later tiles' may still be under way
    __syncthreads();
    copy_tile();
    const uint8_t* K = lds[stage][0];
    const uint8_t* V = lds[stage][1];
    stage = stage == kStages - 1 ? 0 : stage + 1;
    if (j * kKeys > wave_lim) continue;
    // S^T: the K rows of 8 reads are in flight ahead of the products, and the
    // V columns of the first P V products follow them
    f32x4 p[4][2] = {};
    bf16x8 kf[kSteps][4], vf[2][kDims];
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int k = 0; k < 4; ++k) kf[ks][k] = KTile::rows(K, 16 * k, ks, lane);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int n = 0; n < 2; ++n) p[k][n] = mma(kf[ks][k], q[n][ks], p[k][n]);
#pragma unroll
    for (int ct = 0; ct < kDims; ++ct) vf[0][ct] = KTile::columns(V, 0, ct, lane);
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 8, 0);
#pragma unroll
    for (int i = 0; i < 4 * kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
    }
    if (j * kKeys + kKeys - 1 > wave_free) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j * kKeys + 16 * k + acc_row(e, lane) > lim[n]) p[k][n][e] = -INFINITY;
    }
    float top[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      top[n] = p[0][n][0];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) top[n] = fmaxf(top[n], p[k][n][e]);
    }
    const float either = column_max(top[0], top[1]) * a.scale_log2;
    if (__any(either > bound)) {
      raise_maxima<DP>(either, m, l, o);
      bound = ((lane & 16) ? m[1] : m[0]) + kSlack;
    }
    // P and O^T, 32 keys of 16 rows at a time: the exponentials of the next go
    // between the products of one
    const float base[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u == 0) {
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct) vf[1][ct] = KTile::columns(V, 32, ct, lane);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int k = 2 * u; k < 2 * u + 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[k][n][e] = __builtin_amdgcn_exp2f(fmaf(p[k][n][e], a.scale_log2, -base[n]));
            l[n] += p[k][n][e];
          }
        const bf16x8 pu = narrow(p[2 * u][n], p[2 * u + 1][n]);
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct) o[n][ct] = mma(vf[u][ct], pu, o[n][ct]);
      }
    }
    __builtin_amdgcn_sched_group_barrier(kSchedValu, 28, 1);
#pragma unroll
    for (int i = 0; i < 4 * kDims; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 28 / kDims + 1, 1);
    }
  }
  wait_copies<0>();  // no copy may land after the workgroup has given up its LDS
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const float sum = column_sum(l[n]);
    if (!valid[n]) continue;
    if (parts > 1) {
      const int64_t part = ((int64_t)split * a.heads + h[n]) * a.total_q + t[n];
#pragma unroll
      for (int ct = 0; ct < kDims; ++ct) {
        const int d = ct * 16 + 4 * (lane >> 4);
        if (d < a.head_dim)
          *reinterpret_cast<f32x4*>(a.part_o + part * a.head_dim + d) = o[n][ct];
      }
      if (lane < 16) a.part_ml[part] = make_float2(m[n], sum);
      continue;
    }
    uint16_t* orow = a.o.p + t[n] * a.o.row + h[n] * a.o.head;
    store_row<DP>(orow, o[n], row_factor(sum), a.head_dim, lane);
    if (lane < 16)
      a.lse[(int64_t)h[n] * a.total_q + t[n]] = row_lse(m[n], sum);
  }
}

// Joins the parts of each row that has several, in their order (memory-bound:
// the parts once, the output once): one thread per 4
// values of one row of sequence blockIdx.y, whole rows to a workgroup.
__global__ __launch_bounds__(256) void attention_join_splits_kernel(AttentionArgs a) {
  const Sequence s = load_sequence(a, blockIdx.y);
  const unsigned per_row = a.head_dim / 4, slots = 256 / per_row;
  const unsigned slot = threadIdx.x / per_row;
  const int d = (threadIdx.x - slot * per_row) * 4;
  if (slot >= slots) return;
  const int64_t rows = (int64_t)a.heads * a.total_q;
  const unsigned heads = a.heads;
  for (unsigned r = blockIdx.x * slots + slot; r < s.qn * heads; r += gridDim.x * slots) {
    const unsigned i = r / heads, h = r - i * heads;
    const int tile = static_cast<int>(i * a.group + h % a.group) / kRows;
    const int parts = a.split_q.parts(key_tiles(a, s, tile * kRows, kRows));
    if (parts == 1) continue;
    const int64_t t = s.q0 + i;
    const int64_t row = (int64_t)h * a.total_q + t;
    float top = -INFINITY, sum = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int n = 0; n < parts; ++n) {
      const float2 x = a.part_ml[n * rows + row];
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.part_o + (n * rows + row) * a.head_dim + d);
      const float next = fmaxf(top, x.x);
      const float base = next == -INFINITY ? 0.0f : next;
      const float keep = __builtin_amdgcn_exp2f(top - base);
      const float mul = __builtin_amdgcn_exp2f(x.x - base);
      top = next;
      sum = sum * keep + x.y * mul;
      o = o * keep + v * mul;
    }
    const float inv = row_factor(sum);
    u32x2 w;
    w.x = pack_bf16x2(o[0] * inv, o[1] * inv);
    w.y = pack_bf16x2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<u32x2*>(a.o.p + t * a.o.row + h * a.o.head + d) = w;
    if (d == 0) a.lse[row] = row_lse(top, sum);
  }
}

// ---- few query rows ---------------------------------------------------------
//
// Generation: one or a few queries of each sequence over its cached keys.  The
// work is reading K and V once, so what counts is that every CU streams, all
// the time and equally long.  The work is a line of tiles of 32 keys: sequence
// after sequence, kv head after kv head (and 32 rows after 32 rows, should a
// head have more), key tile after key tile.  Each wave, a workgroup of its own,
// takes an equal stretch of the line through two LDS stages, without barriers.
// Where a stretch ends inside a segment (one kv head's 32 rows), its float32
// results go to the workspace, and a second kernel joins a segment's parts in
// their order.
//
// What bounds it: latency and the reading of K and V.  16 sequences of 1 query
// over 1 to 4096 cached keys, 16/8 heads of 128 (103 MB of K and V): 22 us, 4.7
// TB/s, and 8 us to join; a copy's rate would take 20.  A workgroup of 4 waves
// per (sequence, head, stretch) took 65 us for both, one persistent workgroup
// of joined waves per CU 88.
// One on each SIMD.  With heads of 128 its registers (244) would leave room for
// two, the LDS of a CU for five in all; 1280 and 2048 of them took 36 us for both
// kernels where 1024 take 30.
constexpr int kStreams = 1024;
constexpr int kMinShare = 3;    // line units of a stretch at least
// A segment counts for so many tiles more than it has, for the latency of its
// first loads; they come first.
constexpr int kSegmentCost = 1;

// The results of a stretch that covers a part of a segment: part 2 w is of the
// segment that stretch w began in, part 2 w + 1 of the one it ended in.
struct Parts {
  float* o;    // [2 kStreams][32][head_dim], each over its own maximum
  float2* ml;  // [2 kStreams][32]: maximum (in powers of two) and sum
};

// A place on the line of tiles.
struct Place {
  Sequence s;
  int b;                // its index
  int segment;          // in it: kv head, then 32 rows
  int unit;             // in the segment: kSegmentCost, then its key tiles
  int units, segments;  // of the sequence's segments
};

__device__ __forceinline__ void line_units(const AttentionArgs& a, const Sequence& s, int& units,
                                           int& segments) {
  units = kSegmentCost + max((s.kn + 31) / 32, 1);  // rows without keys have a result, too
  segments = (s.qn * a.group + 31) / 32 * a.kv_heads;
}

// Length of the line and the place of unit number `share(length)` * n; false
// past its end.  Each wave by itself, 64 sequences at a time.
template <typename Share>
__device__ __forceinline__ bool find_place(const AttentionArgs& a, int n, Share share, int& length,
                                           int& at, Place& p) {
  const int lane = threadIdx.x & 63;
  length = 0;
  Sequence mine;
  int units = 0, segments = 0;
  auto load = [&](int b0) {
    mine = lane_sequence(a, min(b0 + lane, a.batch - 1));
    line_units(a, mine, units, segments);
    if (b0 + lane >= a.batch) segments = 0;
  };
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    load(b0);
    length += wave_sum(units * segments);
  }
  at = n * share(length);
  if (at >= length) return false;
  int base = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    if (a.batch > 64) load(b0);
    int sum = units * segments;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const uint64_t past = __ballot(at < base + sum);
    if (past != 0) {
      const int l = uniform(__ffsll(static_cast<unsigned long long>(past)) - 1);
      p.s = from_lane(mine, l);
      p.b = b0 + l;
      p.units = __builtin_amdgcn_readlane(units, l);
      p.segments = __builtin_amdgcn_readlane(segments, l);
      const int in = at - base - (__builtin_amdgcn_readlane(sum, l) - p.units * p.segments);
      p.segment = in / p.units;
      p.unit = in - p.segment * p.units;
      return true;
    }
    base += __builtin_amdgcn_readlane(sum, 63);
  }
  return false;
}

__device__ __forceinline__ int stream_share(int length) {
  return max((length + kStreams - 1) / kStreams, kMinShare);
}

template <int DP>
__global__ __launch_bounds__(64, 1) void attention_stream_kernel(AttentionArgs a, Parts parts) {
  typedef Tile<DP, 32, 1> KTile;
  constexpr int kDims = DP / 16, kSteps = DP / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][KTile::kBytes];
  const int lane = threadIdx.x;
  int length, at;
  Place p;
  if (!find_place(a, blockIdx.x, stream_share, length, at, p)) return;
  int remaining = min(stream_share(length), length - at);

  KTile kt, vt;
  kt.init(0, lane, a.k.row, a.head_dim);
  vt.init(0, lane, a.v.row, a.head_dim);
  while (true) {
    const Sequence s = p.s;
    const int end = min(p.unit + remaining, p.units);
    remaining -= end - p.unit;
    const int t0 = max(p.unit - kSegmentCost, 0), t1 = max(end - kSegmentCost, 0);
    if (t0 < t1) {  // this stretch has tiles of the segment
      const int row_tiles = p.segments / a.kv_heads;
      const int g = p.segment / row_tiles;
      const int row0 = (p.segment - g * row_tiles) * 32;
      const int rows = s.qn * a.group;
      const int shift = a.causal ? s.kn - s.qn : s.kn;
      const int free = min(row0 / a.group + shift, s.kn - 1);  // seen by every row
      Walk kw(a.k, (int64_t)s.k0 + t0 * 32, g, a.head_dim);
      Walk vw(a.v, (int64_t)s.k0 + t0 * 32, g, a.head_dim);
      int left = min(t1 * 32, s.kn) - t0 * 32;  // keys from the walks' place on
      auto copy_tile = [&](int stage) {         // past the end: zeros, counted as the others
        kt.copy(lds[stage][0], 0, kw.rows(min(left, 32)));
        vt.copy(lds[stage][1], 0, vw.rows(min(left, 32)));
        kw.step(32);
        vw.step(32);
        left -= 32;
      };
      int64_t at[2];  // two sets of 16 rows
      int h[2], lim[2];
      bool valid[2];
      bf16x8 q[2][kSteps];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int r = row0 + 16 * n + (lane & 15);
        valid[n] = r < rows;
        const int i = min(r, rows - 1) / a.group;
        h[n] = g * a.group + r % a.group;
        lim[n] = min(i + shift, s.kn - 1);
        at[n] = s.q0 + i;
        const uint16_t* qrow = a.q.p + at[n] * a.q.row + h[n] * a.q.head;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
          q[n][ks] = load8(qrow, ks * 32 + 8 * (lane >> 4), a.head_dim, valid[n]);
      }
      copy_tile(0);
      copy_tile(1);
      f32x4 o[2][kDims] = {};
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {};
      float bound = -INFINITY;
      int stage = 0;
      for (int t = t0; t < t1; ++t) {
        wait_copies<2 * KTile::kCopies>();
        const uint8_t* K = lds[stage][0];
        const uint8_t* V = lds[stage][1];
        f32x4 x[2][2] = {};
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bf16x8 kf = KTile::rows(K, 16 * k, ks, lane);
#pragma unroll
            for (int n = 0; n < 2; ++n) x[k][n] = mma(kf, q[n][ks], x[k][n]);
          }
        if (t * 32 + 31 > free) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (t * 32 + 16 * k + acc_row(e, lane) > lim[n]) x[k][n][e] = -INFINITY;
        }
        float top[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          top[n] = x[0][n][0];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[n] = fmaxf(top[n], x[k][n][e]);
        }
        const float either = column_max(top[0], top[1]) * a.scale_log2;
        if (__any(either > bound)) {
          raise_maxima<DP>(either, m, l, o);
          bound = ((lane & 16) ? m[1] : m[0]) + kSlack;
        }
        bf16x8 xu[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float base = m[n] == -INFINITY ? 0.0f : m[n];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[k][n][e] = __builtin_amdgcn_exp2f(fmaf(x[k][n][e], a.scale_log2, -base));
              l[n] += x[k][n][e];
            }
          xu[n] = narrow(x[0][n], x[1][n]);
        }
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct) {
          const bf16x8 vf = KTile::columns(V, 0, ct, lane);
#pragma unroll
          for (int n = 0; n < 2; ++n) o[n][ct] = mma(vf, xu[n], o[n][ct]);
        }
        wait_lds();  // the stage has been read
        copy_tile(stage);
        stage ^= 1;
      }
      wait_copies<0>();
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float sum = column_sum(l[n]);
        if (!valid[n]) continue;
        if (t0 == 0 && end == p.units) {
          uint16_t* orow = a.o.p + at[n] * a.o.row + h[n] * a.o.head;
          store_row<DP>(orow, o[n], row_factor(sum), a.head_dim, lane);
          if (lane < 16)
            a.lse[(int64_t)h[n] * a.total_q + at[n]] = row_lse(m[n], sum);
        } else {
          const int64_t part = (2 * blockIdx.x + (t0 == 0 ? 1 : 0)) * 32 + 16 * n + (lane & 15);
          float* to = parts.o + part * a.head_dim;
#pragma unroll
          for (int ct = 0; ct < kDims; ++ct) {
            const int d = ct * 16 + 4 * (lane >> 4);
            if (d < a.head_dim) *reinterpret_cast<f32x4*>(to + d) = o[n][ct];
          }
          if (lane < 16) parts.ml[part] = make_float2(m[n], sum);
        }
      }
    }
    if (remaining == 0) return;
    p.unit = 0;
    if (++p.segment == p.segments) {  // on to the next sequence that has rows
      p.segment = 0;
      do {
        p.s = load_sequence(a, ++p.b);  // there is one: units remain
        line_units(a, p.s, p.units, p.segments);
      } while (p.segments == 0);
    }
  }
}

// Joins the parts of one segment in their order.  Workgroup n looks at the
// boundary between stretches n and n + 1: where it lies among the tiles of a
// segment and is the first that does, it joins that segment.  16 rows at a
// time; where there are fewer, several groups of threads share a row's parts.
constexpr int kJoinThreads = 512;
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttentionArgs a,
                                                                      Parts parts) {
  __shared__ f32x4 other_o[kJoinThreads];
  __shared__ float2 other_ml[kJoinThreads];
  if (blockIdx.x >= a.clear_from) return clear_forward(a);
  int length, at;
  Place p;
  const int n = blockIdx.x;
  if (!find_place(a, n + 1, stream_share, length, at, p)) return;
  const int share = stream_share(length);
  // a boundary at or before the first tile leaves the stretch before it no part
  const int first_tile = at - p.unit + kSegmentCost;  // on the line
  if (p.unit <= kSegmentCost || first_tile / share != n) return;
  const int last = (at - p.unit + p.units - 1) / share;  // stretch in which the segment ends
  const Sequence s = p.s;
  const int row_tiles = p.segments / a.kv_heads;
  const int g = p.segment / row_tiles;
  const int row0 = (p.segment - g * row_tiles) * 32;
  const int rows = min(s.qn * a.group - row0, 32);
  const int per_row = a.head_dim / 4;
  const int slots = kJoinThreads / per_row;   // at least 16
  const int shared = max(slots / rows, 1);    // slots of one row
  const int at_once = slots / shared;         // rows
  const int slot = threadIdx.x / per_row;
  const int d = (threadIdx.x - slot * per_row) * 4;
  const int sub = slot / at_once;
  for (int r0 = 0; r0 < rows; r0 += at_once) {
    const int r = r0 + slot - sub * at_once;
    float top = -INFINITY, sum = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    auto add = [&](float2 x, f32x4 v) {
      const float next = fmaxf(top, x.x);
      const float base = next == -INFINITY ? 0.0f : next;
      const float keep = __builtin_amdgcn_exp2f(top - base);
      const float mul = __builtin_amdgcn_exp2f(x.x - base);
      top = next;
      sum = sum * keep + x.y * mul;
      o = o * keep + v * mul;
    };
    if (sub < shared && r < rows) {
#pragma unroll 8
      for (int w = n + sub; w <= last; w += shared) {
        const int64_t part = (2 * w + (w == n ? 1 : 0)) * 32 + r;
        add(parts.ml[part], *reinterpret_cast<const f32x4*>(parts.o + part * a.head_dim + d));
      }
    }
    __syncthreads();
    other_o[threadIdx.x] = o;
    other_ml[threadIdx.x] = make_float2(top, sum);
    __syncthreads();
    if (sub != 0 || r >= rows) continue;
    for (int k = 1; k < shared; ++k) {
      const int from = threadIdx.x + k * at_once * per_row;
      add(other_ml[from], other_o[from]);
    }
    const int i = (row0 + r) / a.group, h = g * a.group + (row0 + r) % a.group;
    const float inv = row_factor(sum);
    u32x2 w;
    w.x = pack_bf16x2(o[0] * inv, o[1] * inv);
    w.y = pack_bf16x2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<u32x2*>(a.o.p + (int64_t)(s.q0 + i) * a.o.row + h * a.o.head + d) = w;
    if (d == 0) a.lse[(int64_t)h * a.total_q + s.q0 + i] = row_lse(top, sum);
  }
}

// Whether the keys are streamed.  The other kernel's time is its longest
// workgroup's, about 1 us for 64 keys whatever its rows, until its workgroups
// fill the CUs; this one's is all 32 x 32 squares over 1024 waves, and the
// join.  So it pays while few rows (R, 32-row tiles over all kv heads) meet
// many keys (K, tiles of an average sequence's room).  Measured with heads of
// 128 in us, the other kernel / this one: R 8: K 16 12 / 15, K 32 19 / 14, K
// 128 62 / 17; R 64: K 64 35 / 34, K 128 92 / 43; R 128: K 32 21 / 26, K 128
// 64 / 55; R 256: K 64 47 / 55, K 128 93 / 97, K 512 350 / 298; R 512: K 128
// 94 / 153.  (Both sides measured up to R 512; the other kernel alone takes 383
// us for 128 requests over 4096 keys each, R 1024, and 760 for 256.)
bool streams_keys(const AttentionArgs& a) {
  if (a.total_q == 0) return false;
  const int64_t row_tiles =
      std::max<int64_t>(a.batch, ((int64_t)a.total_q * a.group + 31) / 32) * a.kv_heads;
  const int64_t key_tiles = (int64_t)a.total_k / a.batch / 32;
  if (key_tiles < 32 || row_tiles > std::min<int64_t>(key_tiles, 256)) return false;
  // The line's units and the starts of its stretches are counted in 32 bits, also
  // where falling starts of sequences give every one of them all rows and keys.
  // (256 row tiles over 2^23 keys in 32 sequences are the smallest refused.)
  const int64_t segments = ((int64_t)a.total_q * a.group + 31) / 32 * a.kv_heads;
  const int64_t units = kSegmentCost + ((int64_t)a.total_k + 31) / 32;
  return segments * units * a.batch < (int64_t(1) << 31) - kStreams;
}

// The split of the row tiles' keys; a tile of 64 keys takes about 1.1 us.
// Measured, without / with the parts: one sequence of 4463, one head of 64,
// causal, 84 / 31 us; 12545 tokens in 9 sequences, 4/2 heads of 64, 47 / 38 us.
Split key_split(const AttentionArgs& a) {
  if (a.total_q == 0 || a.total_k == 0 || a.batch > 65535) return Split{1, 1};
  if ((int64_t)a.total_q * a.heads >= (int64_t(1) << 31)) return Split{1, 1};  // rows in 32 bits
  const Lengths keys(a.cu_k, a.batch, a.total_k);
  const double step = 1.1, tile = step / kKeys, cus = 256;
  const double workgroups = static_cast<double>(
      tile_bound(a.cu_q, a.batch, a.total_q, a.group, kRows) * a.kv_heads);
  const double balanced = workgroups * keys.own * tile * (a.causal ? 0.5 : 1.0) / cus;
  return choose_split(keys.longest * tile, balanced, step,
                      static_cast<double>(a.total_q) * a.heads * (a.head_dim + 2));
}

}  // namespace

size_t attention_forward_workspace(const AttentionArgs& a) {
  const size_t floats = a.head_dim + 2;
  if (streams_keys(a)) return static_cast<size_t>(2 * kStreams) * 32 * floats * sizeof(float);
  const int most = key_split(a).most;
  return most == 1 ? 0 : static_cast<size_t>(most) * a.heads * a.total_q * floats * sizeof(float);
}

bfp8_status launch_attention_forward(const AttentionArgs& given, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  AttentionArgs a = given;
  const unsigned clearing =
      a.clear == 0 ? 0 : clear_workgroups((int64_t)a.total_q * a.heads * a.head_dim);
  const bool room = workspace != nullptr && workspace_bytes >= attention_forward_workspace(a);
  if (room && streams_keys(a)) {
    Parts parts;
    parts.o = static_cast<float*>(workspace);
    parts.ml = reinterpret_cast<float2*>(parts.o + 2 * kStreams * 32 * a.head_dim);
    const bfp8_status st =
        a.head_dim <= 64
            ? launch(attention_stream_kernel<64>, dim3(kStreams), dim3(64), stream, a, parts)
            : launch(attention_stream_kernel<128>, dim3(kStreams), dim3(64), stream, a, parts);
    if (st != BFP8_OK) return st;
    a.clear_from = kStreams - 1;
    return launch(attention_join_kernel, dim3(kStreams - 1 + clearing), dim3(kJoinThreads), stream, a,
                  parts);
  }
  a.split_q = room ? key_split(a) : Split{1, 1};
  const int64_t rows = (int64_t)a.heads * a.total_q;
  if (a.split_q.most > 1) {
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + a.split_q.most * rows * a.head_dim);
  }
  const int64_t places = tile_bound(a.cu_q, a.batch, a.total_q, a.group, kRows);
  const int64_t blocks = places * a.kv_heads * a.split_q.most;
  if (blocks == 0) return BFP8_OK;
  if (!grid_fits(blocks + clearing, 64 * kWaves)) return BFP8_ERR_SHAPE;
  a.clear_from = static_cast<unsigned>(blocks);
  const dim3 grid(a.clear_from + clearing);
  const bfp8_status st =
      a.head_dim <= 64
          ? launch(attention_forward_kernel<64>, grid, dim3(64 * kWaves), stream, a, places)
          : launch(attention_forward_kernel<128>, grid, dim3(64 * kWaves), stream, a, places);
  if (st != BFP8_OK || a.split_q.most == 1) return st;
  const int64_t join = rows / a.batch * (a.head_dim / 4) / 256 + 1;  // of an average sequence
  return launch(attention_join_splits_kernel, dim3(static_cast<unsigned>(join), a.batch), dim3(256),
                stream, a);
}

}  // namespace bfp8
