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
  auto& lds = shared.tiles;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  Sequence s;
  int rank, tiles;
  if (!find_tile<false>(a, a.group, kRows, n, s, rank, tiles)) return;
  const int row0 = rank * kRows;
  const int rows = s.qn * a.group;
  const int r = row0 + wave * 32 + (lane & 31);
  const bool valid = r < rows;
  const int i = min(r, rows - 1) / a.group;
  const int h = g * a.group + r % a.group;
  const int shift = a.causal ? s.kn - s.qn : s.kn;
  const int lim = min(i + shift, s.kn - 1);
  const int block_lim = min((min(row0 + kRows, rows) - 1) / a.group + shift, s.kn - 1);
  const int wave_first = row0 + wave * 32;
  const int wave_lim =
      wave_first < rows ? min((min(wave_first + 32, rows) - 1) / a.group + shift, s.kn - 1) : -1;
  const int wave_free = min(wave_first / a.group + shift, s.kn - 1);

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
  const int64_t t = s.q0 + i;
  const uint16_t* qrow = a.q.p + t * a.q.row + h * a.q.head;
  const uint16_t* drow = a.dout.p + t * a.dout.row + h * a.dout.head;
  bf16x8 q[DP / 16], d[DP / 16];
#pragma unroll
  for (int ks = 0; ks < DP / 16; ++ks) {
    const int c = ks * 16 + 8 * (lane >> 5);
    q[ks] = load8(qrow, c, a.head_dim, valid);
    d[ks] = load8(drow, c, a.head_dim, valid);
  }
  float lse2 = 0.0f, delta = 0.0f;
  if (valid) {
    lse2 = a.lse2[(int64_t)h * a.total_q + t];
    delta = -a.delta[(int64_t)h * a.total_q + t];
  }
  wait_copies<0>();  // and the loads above

  f32x16 acc[DP / 32];
#pragma unroll
  for (int ct = 0; ct < DP / 32; ++ct) acc[ct] = f32x16{};
  int stage = 0;
  for (int j = 0; j < nj; ++j) {
    wait_copies<2 * (kStages - 2) * KTile::kCopies>();  // later tiles' may still be under way
    __syncthreads();
    copy_tile();
    const uint8_t* K = lds[stage][0];
    const uint8_t* V = lds[stage][1];
    stage = stage == kStages - 1 ? 0 : stage + 1;
    if (j * kKeys > wave_lim) continue;
    constexpr int kDims = DP / 32;   // 32-column panels
    constexpr int kSteps = DP / 16;  // products of one 32x32 square
    bf16x8 kf[kSteps], vf[kSteps], kc[2][kDims];
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) kf[ks] = KTile::rows(K, 0, ks, lane);
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2) {
      const int key0 = j * kKeys + 32 * t2;
      // S^T and dP^T; the V rows are read between the products of S^T, the K
      // columns of dQ^T between those of dP^T
      f32x16 p = {}, dp = {};
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) vf[ks] = KTile::rows(V, 32 * t2, ks, lane);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) p = mma(kf[ks], q[ks], p);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct)
          kc[u][ct] = KTile::columns(K, 32 * t2 + 16 * u, ct, lane);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) dp = mma(vf[ks], d[ks], dp);
      if (t2 == 0) __builtin_amdgcn_sched_group_barrier(kSchedRead, kSteps, 0);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
      }
      if (key0 + 31 > wave_free) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (key0 + acc_row(e, lane) > lim) p[e] = -INFINITY;
      }
      // dQ^T, 16 keys at a time; the K rows of the next square are read meanwhile
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int e = 8 * u; e < 8 * u + 8; ++e)
          p[e] = __builtin_amdgcn_exp2f(fmaf(p[e], a.scale_log2, -lse2)) * (dp[e] - delta);
        const bf16x8 ds = narrow(p, u);
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct) acc[ct] = mma(kc[u][ct], ds, acc[ct]);
      }
      if (t2 == 0) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) kf[ks] = KTile::rows(K, 32, ks, lane);
      }
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 36, 1);
#pragma unroll
      for (int i = 0; i < 2 * kDims; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedValu, 36 / kDims, 1);
      }
    }
  }
  wait_copies<0>();  // no copy may land after the workgroup has given up its LDS
  if (!valid) return;
  store_row<DP>(a.dq.p + t * a.dq.row + h * a.dq.head, acc, a.scale, a.head_dim, lane);
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
  constexpr int kDims = DP / 32;   // 32-column panels
  constexpr int kSteps = DP / 16;  // products of one 32x32 square
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
  const int key = key0 + (lane & 31);
  const bool used = key < s.kn;
  const int64_t krow = s.k0 + min(key, s.ka - 1);
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
  const int from = used ? key + back : 0x7FFFFFFF;  // first query that sees this lane's key

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
  const uint16_t* kp = a.k.p + krow * a.k.row + g * a.k.head;
  bf16x8 k[kSteps];
#pragma unroll
  for (int ks = 0; ks < kSteps; ++ks)
    k[ks] = load8(kp, ks * 16 + 8 * (lane >> 5), a.head_dim, used);
  wait_copies<0>();  // and the loads of k

  f32x16 dk[kDims], dv[kDims];
#pragma unroll
  for (int ct = 0; ct < kDims; ++ct) dk[ct] = dv[ct] = f32x16{};
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
    const float* lses = stats[stage][half][0] + 4 * (lane >> 5);
    const float* deltas = stats[stage][half][1] + 4 * (lane >> 5);
    // S and dP; dP starts from -delta
    f32x16 p = {}, dp;
#pragma unroll
    for (int e = 0; e < 16; ++e) dp[e] = deltas[8 * (e >> 2) + (e & 3)];
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) p = mma(QTile::rows(Q, 0, ks, lane), k[ks], p);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
      dp = mma(QTile::rows(D, 0, ks, lane), VTile::rows(vlds, kw * 32, ks, lane), dp);
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 4 + 4, 0);  // 4 of -delta
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 0);
    }
    f32x16 lse2;
#pragma unroll
    for (int e = 0; e < 16; ++e) lse2[e] = lses[8 * (e >> 2) + (e & 3)];
    if (i0 < wave_free) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (i0 + acc_row(e, lane) < from) p[e] = -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      p[e] = __builtin_amdgcn_exp2f(fmaf(p[e], a.scale_log2, -lse2[e]));
      dp[e] *= p[e];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bf16x8 pu = narrow(p, u), du = narrow(dp, u);
#pragma unroll
      for (int ct = 0; ct < kDims; ++ct)
        dv[ct] = mma(QTile::columns(D, 16 * u, ct, lane), pu, dv[ct]);
#pragma unroll
      for (int ct = 0; ct < kDims; ++ct)
        dk[ct] = mma(QTile::columns(Q, 16 * u, ct, lane), du, dk[ct]);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 8, 1);
#pragma unroll
    for (int i = 0; i < 4 * kDims; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 1);
    }
  }
  // The halves' sums: the first half takes dV, the second dK, 32 columns at a
  // time through the LDS that the tiles no longer need (nothing is under way)
  wait_copies<0>();
  f32x4* mine = reinterpret_cast<f32x4*>(&lds[0][0][0][0]) + ((half * kKeyWaves + kw) * 4) * 64 + lane;
  const f32x4* other =
      reinterpret_cast<f32x4*>(&lds[0][0][0][0]) + (((half ^ 1) * kKeyWaves + kw) * 4) * 64 + lane;
#pragma unroll
  for (int ct = 0; ct < kDims; ++ct) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const f32x16& give = half == 0 ? dk[ct] : dv[ct];
      mine[c * 64] = f32x4{give[4 * c], give[4 * c + 1], give[4 * c + 2], give[4 * c + 3]};
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const f32x4 add = other[c * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (half == 0) dv[ct][4 * c + e] += add[e];
        else dk[ct][4 * c + e] += add[e];
      }
    }
  }
  if (key >= s.ka) return;
  if (half == 0)
    store_row<DP>(a.dv.p + krow * a.dv.row + g * a.dv.head, dv, 1.0f, a.head_dim, lane);
  else
    store_row<DP>(a.dk.p + krow * a.dk.row + g * a.dk.head, dk, a.scale, a.head_dim, lane);
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
