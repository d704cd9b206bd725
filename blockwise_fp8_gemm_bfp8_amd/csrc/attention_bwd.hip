// Attention backward for gfx950.  The probabilities are recomputed from the
// forward pass's log-sum-exp, P = exp(S - L):
//   stats  L log2(e) and delta = sum_d dO O of every row (memory-bound);
//   dkdv   a workgroup per 128 keys walks the query rows of every head that
//          shares them,  dV = P^T dO,  dK = scale dS^T Q;
//   dq     a workgroup per 256 query rows walks the keys,
//            dS = P (dO V^T - delta),  dQ = scale dS K.
// Seven products instead of five, but no gradient is summed across
// workgroups: no atomics, no float32 copy of dQ for every 128 keys, and one
// fixed order of every sum.  P and dS are rounded to bf16 for their products
// only (an error like the outputs' own rounding); all sums are float32.
//
// As in the forward kernel each product is turned so that a lane owns rows of
// its result (queries in dq, keys in dkdv) and the accumulator of one product
// is the second operand of the next without leaving its registers.
//
// dkdv: a wave's dK and dV of 32 keys take 128 registers, so the V rows stay in
// LDS and the workgroup's 8 waves are two halves that take the squares of 32
// queries in turn, for the same 128 keys; their sums meet at the end.  With 256
// keys to a workgroup (8 waves, all squares) ragged sequences took 1.4 times
// as long (310 us for the 225 us of 13 sequences, 8274 tokens in all).
//
// What bounds it: the matrix cores and the card's power.  16/8 heads of 128,
// causal: 4 sequences of 4096 take 819 to 844 us (stats 30; 1196 TFLOP/s of the
// seven products and more: cards differ), one of 16384 takes 2.9 to 3.1 ms
// (1254), those 13 ragged sequences 208 to 222.  The loops alone do 1386 (dkdv)
// and 1438 TFLOP/s (dq), as a large library product; the rest is the workgroups'
// starts and ends, 8 to 9 us of each, and the XCDs' clocks, which differ.
// Kept from the forward kernel's trials: three stages, 16x16x32 products.
#include "attention.h"

namespace bfp8 {
namespace {

using namespace attn;

constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;
constexpr int kKeys = 64;     // keys of a dq tile
constexpr int kStages = 3;    // tiles in LDS: one being read, two under way
constexpr int kKeyWaves = 4;  // waves over the keys of a dkdv workgroup; two halves of them
constexpr int kKeyRows = 32 * kKeyWaves;
static_assert(kWaves == 2 * kKeyWaves, "two halves");

// lse2 and -delta of every row of every head, for the kernel below: 16 lanes a
// row, 8 values a lane (and zeros in the gradients' rows of no sequence).  Memory-bound: O and dO once (16384 tokens, 16 heads of
// 128: 30 us, 5.4 TB/s).
__global__ __launch_bounds__(256) void attention_stats_kernel(AttentionArgs a) {
  if (blockIdx.x >= a.clear_from) return clear_backward(a);
  const int64_t at = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;  // row, then head
  const int d = threadIdx.x % 16 * 8;
  const int64_t t = at / a.heads;
  const int h = static_cast<int>(at - t * a.heads);
  if (t >= a.total_q) return;
  const bf16x8 o = load8(a.o.p + t * a.o.row + h * a.o.head, d, a.head_dim, true);
  const bf16x8 dout = load8(a.dout.p + t * a.dout.row + h * a.dout.head, d, a.head_dim, true);
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    sum = fmaf(static_cast<float>(dout[e]), static_cast<float>(o[e]), sum);
#pragma unroll
  for (int x = 1; x < 16; x *= 2) sum += __shfl_xor(sum, x);
  if (d == 0) {
    const int64_t row = h * (int64_t)a.total_q + t;
    const float lse = a.lse[row];
    a.lse2[row] = lse == -INFINITY ? 0.0f : lse * kLog2e;
    a.delta[row] = -sum;
  }
}

// The accumulator of one row as float32 part number `row`.
template <int DP>
__device__ __forceinline__ void store_part(float* parts, int64_t row, const f32x4 (&acc)[DP / 16],
                                           int dim, int lane) {
#pragma unroll
  for (int ct = 0; ct < DP / 16; ++ct) {
    const int d = ct * 16 + 4 * (lane >> 4);
    if (d < dim) *reinterpret_cast<f32x4*>(parts + row * dim + d) = acc[ct];
  }
}

template <int DP>
struct DqShared {
  uint8_t tiles[kStages][2][Tile<DP, kKeys, kWaves>::kBytes];  // K and V rows
};

template <int DP>
__device__ __forceinline__ void dq_tile(const AttentionArgs& a, DqShared<DP>& shared, int place,
                                        int places, int g) {
  typedef Tile<DP, kKeys, kWaves> KTile;
  constexpr int kDims = DP / 16;   // 16-column results
  constexpr int kSteps = DP / 32;  // products of one 16x16 square
  auto& lds = shared.tiles;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  Sequence s;
  int rank, tiles;
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
  int64_t at[2];
  int h[2], lim[2];
  bool valid[2];
  float lse2[2], delta[2];
  bf16x8 q[2][kSteps], d[2][kSteps];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int r = wave_first + 16 * n + (lane & 15);
    valid[n] = r < rows;
    h[n] = g * a.group + r % a.group;
    lim[n] = last_key(a, s, min(r, rows - 1));
    at[n] = s.q0 + min(r, rows - 1) / a.group;
    const uint16_t* qrow = a.q.p + at[n] * a.q.row + h[n] * a.q.head;
    const uint16_t* drow = a.dout.p + at[n] * a.dout.row + h[n] * a.dout.head;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      const int c = ks * 32 + 8 * (lane >> 4);
      q[n][ks] = load8(qrow, c, a.head_dim, valid[n]);
      d[n][ks] = load8(drow, c, a.head_dim, valid[n]);
    }
    lse2[n] = delta[n] = 0.0f;
    if (valid[n]) {
      lse2[n] = a.lse2[(int64_t)h[n] * a.total_q + at[n]];
      delta[n] = -a.delta[(int64_t)h[n] * a.total_q + at[n]];
    }
  }
  wait_copies<0>();  // and the loads above

  f32x4 acc[2][kDims] = {};
  int stage = 0;
  for (int j = j0; j < nj; ++j) {
    wait_copies<2 * (kStages - 2) * KTile::kCopies>();  // later tiles' may still be under way
    __syncthreads();
    copy_tile();
    const uint8_t* K = lds[stage][0];
    const uint8_t* V = lds[stage][1];
    stage = stage == kStages - 1 ? 0 : stage + 1;
    if (j * kKeys > wave_lim) continue;
    bf16x8 kf[kSteps][2], vf[kSteps][2], kc[kDims];
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int k = 0; k < 2; ++k) kf[ks][k] = KTile::rows(K, 16 * k, ks, lane);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int key0 = j * kKeys + 32 * half;
      // S^T and dP^T of 32 keys; the V rows are read between the products of
      // S^T, the K columns of dQ^T between those of dP^T
      f32x4 p[2][2] = {}, dp[2][2] = {};
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int k = 0; k < 2; ++k) vf[ks][k] = KTile::rows(V, 32 * half + 16 * k, ks, lane);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < 2; ++n) p[k][n] = mma(kf[ks][k], q[n][ks], p[k][n]);
#pragma unroll
      for (int ct = 0; ct < kDims; ++ct) kc[ct] = KTile::columns(K, 32 * half, ct, lane);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < 2; ++n) dp[k][n] = mma(vf[ks][k], d[n][ks], dp[k][n]);
      if (half == 0) __builtin_amdgcn_sched_group_barrier(kSchedRead, 2 * kSteps, 0);
#pragma unroll
      for (int i = 0; i < 2 * kSteps; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < 2 * kSteps; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
      }
      if (key0 + 31 > wave_free) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + 16 * k + acc_row(e, lane) > lim[n]) p[k][n][e] = -INFINITY;
      }
      // dQ^T; the K rows of the next 32 keys are read meanwhile.  Products begin
      // after the first 24 instructions of dS (36 or 8: 1 % slower).
      bf16x8 ds[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[k][n][e] = __builtin_amdgcn_exp2f(fmaf(p[k][n][e], a.scale_log2, -lse2[n])) *
                         (dp[k][n][e] - delta[n]);
        ds[n] = narrow(p[0][n], p[1][n]);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct) acc[n][ct] = mma(kc[ct], ds[n], acc[n][ct]);
      if (half == 0) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
          for (int k = 0; k < 2; ++k) kf[ks][k] = KTile::rows(K, 32 + 16 * k, ks, lane);
      }
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 24, 1);
#pragma unroll
      for (int i = 0; i < kDims; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedValu, 72 / kDims, 1);
      }
    }
  }
  wait_copies<0>();  // no copy may land after the workgroup has given up its LDS
  const AttentionArgs end = late_args();
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    if (!valid[n]) continue;
    if (parts > 1)
      store_part<DP>(end.part_dq, ((int64_t)split * end.heads + h[n]) * end.total_q + at[n], acc[n],
                     end.head_dim, lane);
    else
      store_row<DP>(end.dq.p + at[n] * end.dq.row + h[n] * end.dq.head, acc[n], end.scale,
                    end.head_dim, lane);
  }
}

template <int DP>
struct DkdvShared {
  typedef Tile<DP, 32, kKeyWaves> QTile;
  typedef Tile<DP, kKeyRows, kWaves> VTile;
  uint8_t tiles[kStages][2][2][QTile::kBytes];  // of each half: Q rows, dO rows
  uint8_t v[VTile::kBytes];                     // the workgroup's V rows
  float stats[kStages][2][2][64];               // of each half: lse2, -delta
};

template <int DP>
__device__ __forceinline__ void dkdv_tile(const AttentionArgs& a, DkdvShared<DP>& shared,
                                          int place, int places, int g) {
  typedef typename DkdvShared<DP>::QTile QTile;
  typedef typename DkdvShared<DP>::VTile VTile;
  constexpr int kDims = DP / 16;   // 16-column results
  constexpr int kSteps = DP / 32;  // products of one 16x16 square
  auto& lds = shared.tiles;
  auto& vlds = shared.v;
  auto& stats = shared.stats;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int half = wave / kKeyWaves, kw = wave % kKeyWaves;
  Sequence s;
  int rank, tiles;
  const int split = place / places;  // first every tile's first part
  if (!find_tile<true>(a, 1, kKeyRows, place - split * places, s, rank, tiles)) return;
  const int row0 = (tiles - 1 - rank) * kKeyRows;  // the first keys are seen by the most queries
  const int key0 = row0 + kw * 32;                 // the wave's first key
  // squares of queries, head after head, of which this part's: n0 .. total - 1
  // (an even n0: the halves take them in turn)
  int per_head;
  const int first = first_square(a, s, row0, per_head);
  const int pairs = (per_head * a.group + 1) / 2;
  const int parts = a.split_k.parts(pairs);
  if (split >= parts) return;
  const int n0 = 2 * static_cast<int>(static_cast<int64_t>(pairs) * split / parts);
  const int total = min(2 * static_cast<int>(static_cast<int64_t>(pairs) * (split + 1) / parts),
                        per_head * a.group);
  // query i sees keys up to i + kn - qn: key j is first seen by query j + back
  const int back = a.causal ? s.qn - s.kn : -s.kn;
  {
    VTile vt;
    vt.init(wave, lane, a.v.row, a.head_dim);
    const Walk vw(a.v, (int64_t)s.k0 + row0, g, a.head_dim);
    vt.copy(vlds, wave, vw.rows(min(s.kn - row0, kKeyRows)));
  }
  const int wave_first = key0 + back;
  // first query of no masking: the one that sees the wave's last key, or none
  // if some of its keys are past the used length and must vanish
  const int wave_free = key0 + 31 < s.kn ? key0 + 31 + back : 0x7FFFFFFF;

  // this half's queries: i0 .. i0 + 31 of the group's hh-th head, n-th of all
  QTile qt, dt;
  qt.init(kw, lane, a.q.row, a.head_dim);
  dt.init(kw, lane, a.dout.row, a.head_dim);
  Walk qw(a.q, (int64_t)s.q0 + first, g * a.group, a.head_dim);
  Walk dw(a.dout, (int64_t)s.q0 + first, g * a.group, a.head_dim);
  const int64_t q_next = a.q.head * 2 - static_cast<int64_t>(per_head) * 32 * qw.row_bytes;
  const int64_t d_next = a.dout.head * 2 - static_cast<int64_t>(per_head) * 32 * dw.row_bytes;
  const int64_t stat_next = (static_cast<int64_t>(a.total_q) - per_head * 32) * 4;
  uint64_t stat_at = reinterpret_cast<uint64_t>(
      (kw == 0 ? a.lse2 : a.delta) + static_cast<int64_t>(g) * a.group * a.total_q + s.q0 + first);
  int left = s.qn - first;  // rows from the walks' place to the end of the sequence
  auto pass = [&](int n) {  // the walks go on by n squares of 32 rows
    qw.step(32 * n);
    dw.step(32 * n);
    stat_at += 32 * 4 * n;
    left -= 32 * n;
#pragma unroll
    for (int twice = 0; twice < 2; ++twice)
      if (left <= 0) {  // into the next head
        qw.at += q_next;
        dw.at += d_next;
        stat_at += stat_next;
        left += per_head * 32;
      }
  };
  if (n0 > 0) {
    const int heads = n0 / per_head, squares = n0 - heads * per_head;
    qw.at += heads * a.q.head * 2;
    dw.at += heads * a.dout.head * 2;
    stat_at += (int64_t)heads * a.total_q * 4;
    pass(squares);
  }
  if (half == 1 && total > n0) pass(1);
  int copied = n0 + half;
  int ahead = 0;  // stage of the next copies
  auto copy_square = [&]() {  // past the last: zeros, counted as the others
    const int rows = copied < total ? min(left, 32) : 0;
    qt.copy(lds[ahead][half][0], kw, qw.rows(rows));
    dt.copy(lds[ahead][half][1], kw, dw.rows(rows));
    if (kw < 2)
      copy4(uniform(lds_offset(&stats[ahead][half][kw][0])), lane * 4, buffer(stat_at, rows * 4));
    ahead = ahead == kStages - 1 ? 0 : ahead + 1;
    copied += 2;  // the halves take squares in turn
    pass(2);
  };
  if (total > n0) {
    copy_square();
    copy_square();
  }
  // two sets of 16 keys: a lane's key, its row, the first query that sees it
  int64_t krow[2];
  int from[2];
  bool mine[2];
  bf16x8 k[2][kSteps];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int key = key0 + 16 * n + (lane & 15);
    const bool used = key < s.kn;
    mine[n] = key < s.ka;
    from[n] = used ? key + back : 0x7FFFFFFF;
    krow[n] = s.k0 + min(key, s.ka - 1);
    const uint16_t* kp = a.k.p + krow[n] * a.k.row + g * a.k.head;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
      k[n][ks] = load8(kp, ks * 32 + 8 * (lane >> 4), a.head_dim, used);
  }
  wait_copies<0>();  // and the loads of k

  f32x4 dk[2][kDims] = {}, dv[2][kDims] = {};
  int at = total > n0 ? (n0 + half) % per_head : 0;  // this half's square of its head
  int next = 0;
  for (int n = n0; n < total; n += 2) {
    // the next square's copies may still be under way
    if (kw < 2) wait_copies<2 * QTile::kCopies + 1>();
    else wait_copies<2 * QTile::kCopies>();
    __syncthreads();
    copy_square();
    const int stage = next;
    next = next == kStages - 1 ? 0 : next + 1;
    const int i0 = first + at * 32;
    at += 2;
    if (at >= per_head) at -= per_head;
    if (at >= per_head) at -= per_head;
    if (n + half >= total || i0 + 31 < wave_first) continue;
    const uint8_t* Q = lds[stage][half][0];
    const uint8_t* D = lds[stage][half][1];
    const float* lses = stats[stage][half][0] + 4 * (lane >> 4);
    const float* deltas = stats[stage][half][1] + 4 * (lane >> 4);
    // S and dP of 32 queries; dP starts from -delta
    f32x4 p[2][2] = {}, dp[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n) dp[i][n] = *reinterpret_cast<const f32x4*>(deltas + 16 * i);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bf16x8 qf = QTile::rows(Q, 16 * i, ks, lane);
#pragma unroll
        for (int n = 0; n < 2; ++n) p[i][n] = mma(qf, k[n][ks], p[i][n]);
      }
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      bf16x8 vf[2], df[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) vf[n] = VTile::rows(vlds, kw * 32 + 16 * n, ks, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) df[i] = QTile::rows(D, 16 * i, ks, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) dp[i][n] = mma(df[i], vf[n], dp[i][n]);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 2 + 4, 0);  // 2 of -delta
#pragma unroll
    for (int i = 0; i < 2 * kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
    }
#pragma unroll
    for (int i = 0; i < 2 * kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 0);
    }
    f32x4 lse2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) lse2[i] = *reinterpret_cast<const f32x4*>(lses + 16 * i);
    if (i0 < wave_free) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i0 + 16 * i + acc_row(e, lane) < from[n]) p[i][n][e] = -INFINITY;
    }
    bf16x8 pu[2], du[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[i][n][e] = __builtin_amdgcn_exp2f(fmaf(p[i][n][e], a.scale_log2, -lse2[i][e]));
          dp[i][n][e] *= p[i][n][e];
        }
      pu[n] = narrow(p[0][n], p[1][n]);
      du[n] = narrow(dp[0][n], dp[1][n]);
    }
#pragma unroll
    for (int ct = 0; ct < kDims; ++ct) {
      const bf16x8 dc = QTile::columns(D, 0, ct, lane);
#pragma unroll
      for (int n = 0; n < 2; ++n) dv[n][ct] = mma(dc, pu[n], dv[n][ct]);
    }
#pragma unroll
    for (int ct = 0; ct < kDims; ++ct) {
      const bf16x8 qc = QTile::columns(Q, 0, ct, lane);
#pragma unroll
      for (int n = 0; n < 2; ++n) dk[n][ct] = mma(qc, du[n], dk[n][ct]);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 8, 1);
#pragma unroll
    for (int i = 0; i < 2 * kDims; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 1);
    }
  }
  // The halves' sums: the first half takes dV, the second dK, a quarter of
  // either at a time through the LDS that the tiles no longer need (nothing is
  // under way)
  wait_copies<0>();
  constexpr int kPieces = 2 * kDims / 4;
  f32x4* mine_lds =
      reinterpret_cast<f32x4*>(&lds[0][0][0][0]) + (half * kKeyWaves + kw) * kPieces * 64 + lane;
  const f32x4* other_lds = reinterpret_cast<f32x4*>(&lds[0][0][0][0]) +
                           ((half ^ 1) * kKeyWaves + kw) * kPieces * 64 + lane;
  static_assert(2 * kKeyWaves * kPieces * 64 * sizeof(f32x4) <= sizeof(shared.tiles), "fits");
#pragma unroll
  for (int part = 0; part < 4; ++part) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int n = (part * kPieces + c) / kDims, ct = (part * kPieces + c) % kDims;
      mine_lds[c * 64] = half == 0 ? dk[n][ct] : dv[n][ct];
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int n = (part * kPieces + c) / kDims, ct = (part * kPieces + c) % kDims;
      const f32x4 add = other_lds[c * 64];
      if (half == 0) dv[n][ct] += add;
      else dk[n][ct] += add;
    }
  }
  const AttentionArgs end = late_args();
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    if (!mine[n]) continue;
    if (parts > 1)
      store_part<DP>(half == 0 ? end.part_dv : end.part_dk,
                     ((int64_t)split * end.kv_heads + g) * end.total_k + krow[n],
                     half == 0 ? dv[n] : dk[n], end.head_dim, lane);
    else if (half == 0)
      store_row<DP>(end.dv.p + krow[n] * end.dv.row + g * end.dv.head, dv[n], 1.0f, end.head_dim,
                    lane);
    else
      store_row<DP>(end.dk.p + krow[n] * end.dk.row + g * end.dk.head, dk[n], end.scale,
                    end.head_dim, lane);
  }
}

// Both kinds of tiles in one launch, so that the second kind's workgroups start
// where the first kind's long ones still run.  Not interleaved: workgroups of
// one kind that run together share the rows they read through their XCD's L2
// (dq and dkdv tiles in turn took 11 % longer at 4 x 4096 and 1 x 16384), and
// dq first took 2 % longer.  The kv head changes fastest, which puts all tiles
// of a head on one XCD where the heads are a multiple of 8.
template <int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_backward_kernel(AttentionArgs a,
                                                                           int k_tiles,
                                                                           int q_tiles) {
  union Shared {
    DqShared<DP> dq;
    DkdvShared<DP> dkdv;
  };
  __shared__ __attribute__((aligned(1024))) Shared shared;
  const int g = blockIdx.x % a.kv_heads;
  const int place = blockIdx.x / a.kv_heads;
  const int k_places = k_tiles * a.split_k.most;
  if (place < k_places)
    dkdv_tile<DP>(a, shared.dkdv, place, k_tiles, g);
  else
    dq_tile<DP>(a, shared.dq, place - k_places, q_tiles, g);
}

// Adds the parts of the gradients' rows that have several, in their order: one
// thread per 4 values of a row of sequence blockIdx.y, whole rows to a workgroup.
__global__ __launch_bounds__(256) void attention_sum_kernel(AttentionArgs a) {
  const unsigned per_row = a.head_dim / 4, slots = 256 / per_row;
  const unsigned slot = threadIdx.x / per_row;
  const int d = (threadIdx.x - slot * per_row) * 4;
  if (slot >= slots) return;
  const Sequence s = load_sequence(a, blockIdx.y);
  auto sum = [&](const float* p, int64_t stride, int parts, const Heads& out, int64_t t, unsigned h,
                 float mul) {
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k = 0; k < parts; ++k) x += *reinterpret_cast<const f32x4*>(p + k * stride);
    u32x2 w;
    w.x = pack_bf16x2(x[0] * mul, x[1] * mul);
    w.y = pack_bf16x2(x[2] * mul, x[3] * mul);
    *reinterpret_cast<u32x2*>(out.p + t * out.row + h * out.head + d) = w;
  };
  if (a.split_q.most > 1) {
    const unsigned heads = a.heads;
    const int64_t stride = (int64_t)a.heads * a.total_q * a.head_dim;
    for (unsigned r = blockIdx.x * slots + slot; r < s.qn * heads; r += gridDim.x * slots) {
      const unsigned i = r / heads, h = r - i * heads;
      const int tile = static_cast<int>(i * a.group + h % a.group) / kRows;
      const int parts = a.split_q.parts(key_tiles(a, s, tile * kRows, kRows));
      if (parts == 1) continue;
      const int64_t t = s.q0 + i;
      sum(a.part_dq + ((int64_t)h * a.total_q + t) * a.head_dim + d, stride, parts, a.dq, t, h,
          a.scale);
    }
  }
  if (a.split_k.most > 1) {
    const unsigned heads = a.kv_heads;
    const int64_t stride = (int64_t)a.kv_heads * a.total_k * a.head_dim;
    for (unsigned r = blockIdx.x * slots + slot; r < s.ka * heads; r += gridDim.x * slots) {
      const unsigned j = r / heads, g = r - j * heads;
      int per_head;
      first_square(a, s, static_cast<int>(j) / kKeyRows * kKeyRows, per_head);
      const int parts = a.split_k.parts((per_head * a.group + 1) / 2);
      if (parts == 1) continue;
      const int64_t t = s.k0 + j, at = ((int64_t)g * a.total_k + t) * a.head_dim + d;
      sum(a.part_dk + at, stride, parts, a.dk, t, g, a.scale);
      sum(a.part_dv + at, stride, parts, a.dv, t, g, 1.0f);
    }
  }
}

struct BackwardPlan {
  int64_t q_tiles, k_tiles;
  Split split_q, split_k;
};

// A dq tile takes about 1.5 us for 64 keys, a dkdv tile 1.5 us for 64 queries
// of one head (a pair of squares).  Measured, causal, without / with the parts:
// 2 sequences of 6553 tokens in all, 8/2 heads of 80, 405 / 215 us; one of 1444,
// 32/8 heads of 128, 157 / 118; one of 3961, 4/4 heads, 62 / 56.
BackwardPlan backward_plan(const AttentionArgs& a) {
  BackwardPlan p{0, 0, Split{1, 1}, Split{1, 1}};
  if (a.batch == 0) return p;
  p.q_tiles = tile_bound(a.cu_q, a.batch, a.total_q, a.group, kRows);
  p.k_tiles = tile_bound(a.cu_k, a.batch, a.total_k, 1, kKeyRows);
  if (a.total_q == 0 || a.total_k == 0 || a.batch > 65535) return p;
  if ((int64_t)a.total_q * a.heads >= (int64_t(1) << 31) ||  // rows counted in 32 bits
      (int64_t)a.total_k * a.kv_heads >= (int64_t(1) << 31))
    return p;
  const Lengths keys(a.cu_k, a.batch, a.total_k), queries(a.cu_q, a.batch, a.total_q);
  const double step = 1.5, cus = 256;
  const double balanced = (p.q_tiles * keys.own + p.k_tiles * queries.own * a.group) * a.kv_heads *
                          step / 64 * (a.causal ? 0.5 : 1.0) / cus;
  p.split_q = choose_split(keys.longest * step / 64, balanced, step,
                           static_cast<double>(a.total_q) * a.heads * a.head_dim);
  p.split_k = choose_split(queries.longest * a.group * step / 64, balanced, step,
                           2.0 * a.total_k * a.kv_heads * a.head_dim);
  return p;
}

}  // namespace

size_t attention_backward_workspace(const AttentionArgs& a) {
  const BackwardPlan p = backward_plan(a);
  const size_t q_rows = static_cast<size_t>(a.heads) * a.total_q;
  const size_t k_rows = static_cast<size_t>(a.kv_heads) * a.total_k;
  size_t floats = 2 * q_rows;
  if (p.split_q.most > 1 || p.split_k.most > 1) floats = (floats + 3) / 4 * 4;  // 16 bytes
  if (p.split_q.most > 1) floats += p.split_q.most * q_rows * a.head_dim;
  if (p.split_k.most > 1) floats += 2 * p.split_k.most * k_rows * a.head_dim;
  return floats * sizeof(float);
}

bfp8_status launch_attention_backward(AttentionArgs a, void* workspace, hipStream_t stream) {
  const BackwardPlan p = backward_plan(a);
  const int64_t q_rows = (int64_t)a.heads * a.total_q, k_rows = (int64_t)a.kv_heads * a.total_k;
  a.split_q = p.split_q;
  a.split_k = p.split_k;
  a.lse2 = static_cast<float*>(workspace);
  a.delta = a.lse2 + q_rows;
  a.part_dq = a.lse2 + (2 * q_rows + 3) / 4 * 4;
  a.part_dk = a.part_dq + (a.split_q.most > 1 ? a.split_q.most * q_rows * a.head_dim : 0);
  a.part_dv = a.part_dk + a.split_k.most * k_rows * a.head_dim;
  const int64_t blocks =
      (p.k_tiles * a.split_k.most + p.q_tiles * a.split_q.most) * a.kv_heads;
  const int64_t stat_blocks = (q_rows + 15) / 16;
  const unsigned clearing =
      a.clear == 0 ? 0 : clear_workgroups((q_rows + 2 * k_rows) * a.head_dim);
  if (!grid_fits(blocks, 64 * kWaves) || !grid_fits(stat_blocks + clearing, 256))
    return BFP8_ERR_SHAPE;
  bfp8_status st = BFP8_OK;
  a.clear_from = static_cast<unsigned>(stat_blocks);
  if (stat_blocks + clearing > 0)
    st = launch(attention_stats_kernel, dim3(a.clear_from + clearing), dim3(256), stream, a);
  if (st != BFP8_OK || blocks == 0) return st;
  const dim3 grid(static_cast<unsigned>(blocks));
  st = a.head_dim <= 64 ? launch(attention_backward_kernel<64>, grid, dim3(64 * kWaves), stream, a,
                                 p.k_tiles, p.q_tiles)
                        : launch(attention_backward_kernel<128>, grid, dim3(64 * kWaves), stream, a,
                                 p.k_tiles, p.q_tiles);
  if (st != BFP8_OK || (a.split_q.most == 1 && a.split_k.most == 1)) return st;
  // workgroups for an average sequence's rows
  const int64_t split_rows =
      std::max(a.split_q.most > 1 ? q_rows : 0, a.split_k.most > 1 ? k_rows : 0);
  const int64_t sum = split_rows / a.batch * (a.head_dim / 4) / 256 + 1;
  return launch(attention_sum_kernel, dim3(static_cast<unsigned>(sum), a.batch), dim3(256), stream,
                a);
}

}  // namespace bfp8
