// Attention backward for gfx950.  The probabilities are recomputed from the
// forward pass's log-sum-exp, P = exp(S - L), in two kernels:
//   dq:    a workgroup per 256 query rows walks the keys,
//            delta = sum_d dO O,  dS = P (dO V^T - delta),  dQ = scale dS K;
//   dkdv:  a workgroup per 256 keys walks the query rows of every head that
//          shares them,  dV = P^T dO,  dK = scale dS^T Q.
// Seven products instead of five, but no gradient is summed across
// workgroups: no atomics, no float32 copy of dQ in memory, and one fixed order
// of every sum.
//
// As in the forward kernel each product is turned so that a lane owns one row
// of its result (a query in dq, a key in dkdv) and the accumulator of one
// product is the second operand of the next without leaving its registers.
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
// row, 8 values a lane.  Memory-bound: O and dO once.
__global__ __launch_bounds__(256) void attention_stats_kernel(AttentionArgs a) {
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

template <int DP>
struct DqShared {
  uint8_t tiles[kStages][2][Tile<DP, kKeys, kWaves>::kBytes];  // K and V rows
};

template <int DP>
__device__ __forceinline__ void dq_tile(const AttentionArgs& a, DqShared<DP>& shared, int n,
                                        int g) {
  typedef Tile<DP, kKeys, kWaves> KTile;
  constexpr int kDims = DP / 16;   // 16-column results
  constexpr int kSteps = DP / 32;  // products of one 16x16 square
  auto& lds = shared.tiles;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  Sequence s;
  int rank, tiles;
  if (!find_tile<false>(a, a.group, kRows, n, s, rank, tiles)) return;
  const int row0 = rank * kRows;  // the last rows see the most keys
  const int rows = s.qn * a.group;
  // last visible key of the workgroup's last row and of the wave's first and last
  const int shift = a.causal ? s.kn - s.qn : s.kn;
  const int block_lim = min((min(row0 + kRows, rows) - 1) / a.group + shift, s.kn - 1);
  const int wave_first = row0 + wave * 32;
  const int wave_lim =
      wave_first < rows ? min((min(wave_first + 32, rows) - 1) / a.group + shift, s.kn - 1) : -1;
  const int wave_free = min(wave_first / a.group + shift, s.kn - 1);  // seen by every row

  KTile kt, vt;
  kt.init(wave, lane, a.k.row, a.head_dim);
  vt.init(wave, lane, a.v.row, a.head_dim);
  Walk kw(a.k, s.k0, g, a.head_dim), vw(a.v, s.k0, g, a.head_dim);
  int left = s.kn, ahead = 0;  // keys from the walks' place on; stage of the next copies
  auto copy_tile = [&]() {     // tiles in their order; past the end zeros, counted as the others
    const int n = min(left, kKeys);
    kt.copy(lds[ahead][0], wave, kw.rows(n));
    vt.copy(lds[ahead][1], wave, vw.rows(n));
    kw.step(kKeys);
    vw.step(kKeys);
    left -= kKeys;
    ahead = ahead == kStages - 1 ? 0 : ahead + 1;
  };
  const int nj = block_lim < 0 ? 0 : block_lim / kKeys + 1;
  if (nj > 0) {
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
    const int i = min(r, rows - 1) / a.group;
    h[n] = g * a.group + r % a.group;
    lim[n] = min(i + shift, s.kn - 1);
    at[n] = s.q0 + i;
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
  for (int j = 0; j < nj; ++j) {
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
      // dQ^T; the K rows of the next 32 keys are read meanwhile
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
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 36, 1);
#pragma unroll
      for (int i = 0; i < kDims; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 2, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedValu, 72 / kDims, 1);
      }
    }
  }
  wait_copies<0>();  // no copy may land after the workgroup has given up its LDS
#pragma unroll
  for (int n = 0; n < 2; ++n)
    if (valid[n])
      store_row<DP>(a.dq.p + at[n] * a.dq.row + h[n] * a.dq.head, acc[n], a.scale, a.head_dim,
                    lane);
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
__device__ __forceinline__ void dkdv_tile(const AttentionArgs& a, DkdvShared<DP>& shared, int n0,
                                          int g) {
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
  if (!find_tile<true>(a, 1, kKeyRows, n0, s, rank, tiles)) return;
  const int row0 = (tiles - 1 - rank) * kKeyRows;  // the first keys are seen by the most queries
  const int key0 = row0 + kw * 32;                 // the wave's first key
  {
    VTile vt;
    vt.init(wave, lane, a.v.row, a.head_dim);
    const Walk vw(a.v, (int64_t)s.k0 + row0, g, a.head_dim);
    vt.copy(vlds, wave, vw.rows(min(s.kn - row0, kKeyRows)));
  }
  // query i sees keys up to i + kn - qn: key j is first seen by query j + back
  const int back = a.causal ? s.qn - s.kn : -s.kn;
  const int first = row0 < s.kn ? max(row0 + back, 0) & ~31 : s.qn;
  const int per_head = first < s.qn ? (s.qn - first + 31) / 32 : 0;
  const int total = per_head * a.group;  // squares of queries, head after head
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
  if (half == 1 && total > 0) pass(1);
  int copied = half;
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
  if (total > 0) {
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
  int at = per_head == 1 ? 0 : half;  // this half's square of its head
  int next = 0;
  for (int n = 0; n < total; n += 2) {
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
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    if (!mine[n]) continue;
    if (half == 0)
      store_row<DP>(a.dv.p + krow[n] * a.dv.row + g * a.dv.head, dv[n], 1.0f, a.head_dim, lane);
    else
      store_row<DP>(a.dk.p + krow[n] * a.dk.row + g * a.dk.head, dk[n], a.scale, a.head_dim, lane);
  }
}

// Both kinds of tiles in one launch, so that neither waits for the other's
// last workgroups: of every total places, q_tiles are dq tiles, evenly spread
// (each kind's come by descending work).  The kv head changes fastest, which
// puts all tiles of a head on one XCD where the heads are a multiple of 8.
template <int DP>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_backward_kernel(AttentionArgs a,
                                                                           unsigned q_tiles,
                                                                           unsigned total) {
  union Shared {
    DqShared<DP> dq;
    DkdvShared<DP> dkdv;
  };
  __shared__ __attribute__((aligned(1024))) Shared shared;
  const int g = blockIdx.x % a.kv_heads;
  const unsigned place = blockIdx.x / a.kv_heads;
  if (place < total - q_tiles)
    dkdv_tile<DP>(a, shared.dkdv, place, g);
  else
    dq_tile<DP>(a, shared.dq, place - (total - q_tiles), g);
}

// An upper bound on the tiles of all sequences, whose lengths are on the device.
int64_t tile_bound(const int32_t* cu, int64_t batch, int64_t total, int64_t mult, int64_t unit) {
  if (cu == nullptr) return batch * ((total / batch * mult + unit - 1) / unit);
  return (total * mult + batch * (unit - 1)) / unit;
}

}  // namespace

bfp8_status launch_attention_backward(const AttentionArgs& a, hipStream_t stream) {
  const int64_t q_tiles = tile_bound(a.cu_q, a.batch, a.total_q, a.group, kRows);
  const int64_t total = q_tiles + tile_bound(a.cu_k, a.batch, a.total_k, 1, kKeyRows);
  const int64_t blocks = total * a.kv_heads;
  const int64_t stat_blocks = ((int64_t)a.total_q * a.heads + 15) / 16;
  if (blocks >= (int64_t(1) << 31) || stat_blocks >= (int64_t(1) << 31)) return BFP8_ERR_SHAPE;
  if (stat_blocks > 0) {
    const bfp8_status st = launch(attention_stats_kernel, dim3(static_cast<unsigned>(stat_blocks)),
                                  dim3(256), stream, a);
    if (st != BFP8_OK) return st;
  }
  if (blocks == 0) return BFP8_OK;
  const dim3 grid(static_cast<unsigned>(blocks));
  return a.head_dim <= 64
             ? launch(attention_backward_kernel<64>, grid, dim3(64 * kWaves), stream, a, q_tiles, total)
             : launch(attention_backward_kernel<128>, grid, dim3(64 * kWaves), stream, a, q_tiles,
                      total);
}

}  // namespace bfp8
