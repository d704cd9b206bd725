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
constexpr int kKeyWaves = 4;  // waves over the keys of a dkdv workgroup; two halves of them
constexpr int kKeyRows = 32 * kKeyWaves;
static_assert(kWaves == 2 * kKeyWaves, "two halves");

template <int DP>
__global__ __launch_bounds__(512, 2) void attention_dq_kernel(AttentionArgs a) {
  typedef Tile<DP, kKeys, kWaves> KTile;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][KTile::kBytes];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int g = blockIdx.x % a.kv_heads;
  int b, rank, tiles;
  if (!find_tile(a.cu_q, a.batch, a.total_q, a.group, kRows, blockIdx.x / a.kv_heads, b, rank,
                 tiles))
    return;
  const Sequence s = load_sequence(a, b);
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

  const int64_t t = s.q0 + i;
  const uint16_t* qrow = a.q.p + t * a.q.row + h * a.q.head;
  const uint16_t* drow = a.dout.p + t * a.dout.row + h * a.dout.head;
  const uint16_t* orow = a.o.p + t * a.o.row + h * a.o.head;
  bf16x8 q[DP / 16], d[DP / 16];
  float delta = 0.0f;
#pragma unroll
  for (int ks = 0; ks < DP / 16; ++ks) {
    const int c = ks * 16 + 8 * (lane >> 5);
    q[ks] = load8(qrow, c, a.head_dim, valid);
    d[ks] = load8(drow, c, a.head_dim, valid);
    const bf16x8 o = load8(orow, c, a.head_dim, valid);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      delta = fmaf(static_cast<float>(d[ks][e]), static_cast<float>(o[e]), delta);
  }
  delta = pair_sum(delta);
  float lse2 = 0.0f;
  if (valid) {
    const float lse = a.lse[(int64_t)h * a.total_q + t];
    lse2 = lse == -INFINITY ? 0.0f : lse * kLog2e;
    if (lane < 32) {  // for the dkdv kernel
      a.lse2[(int64_t)h * a.total_q + t] = lse2;
      a.delta[(int64_t)h * a.total_q + t] = -delta;
    }
  }

  KTile kt, vt;
  kt.init(wave, lane, a.k.row, a.head_dim);
  vt.init(wave, lane, a.v.row, a.head_dim);
  Walk kw(a.k, s.k0, g, a.head_dim), vw(a.v, s.k0, g, a.head_dim);
  auto copy_tile = [&](int j) {  // tiles in their order
    const int n = min(s.kn - j * kKeys, kKeys);
    kt.copy(lds[j & 1][0], wave, kw.rows(n));
    vt.copy(lds[j & 1][1], wave, vw.rows(n));
    kw.step(kKeys);
    vw.step(kKeys);
  };

  f32x16 acc[DP / 32];
#pragma unroll
  for (int ct = 0; ct < DP / 32; ++ct) acc[ct] = f32x16{};
  const int nj = block_lim < 0 ? 0 : block_lim / kKeys + 1;
  if (nj > 0) copy_tile(0);
  for (int j = 0; j < nj; ++j) {
    wait_copies<0>();
    __syncthreads();
    if (j + 1 < nj) copy_tile(j + 1);
    if (j * kKeys > wave_lim) continue;
    const uint8_t* K = lds[j & 1][0];
    const uint8_t* V = lds[j & 1][1];
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
  if (!valid) return;
  store_row<DP>(a.dq.p + t * a.dq.row + h * a.dq.head, acc, a.scale, a.head_dim, lane);
}

template <int DP>
__global__ __launch_bounds__(512, 2) void attention_dkdv_kernel(AttentionArgs a) {
  typedef Tile<DP, 32, kKeyWaves> QTile;
  typedef Tile<DP, kKeyRows, kWaves> VTile;
  constexpr int kDims = DP / 32;   // 32-column panels
  constexpr int kSteps = DP / 16;  // products of one 32x32 square
  // two stages of each half's Q rows, dO rows and their lse2 and -delta; the V rows
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][2][QTile::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t vlds[VTile::kBytes];
  __shared__ __attribute__((aligned(256))) float stats[2][2][2][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int half = wave / kKeyWaves, kw = wave % kKeyWaves;
  const int g = blockIdx.x % a.kv_heads;
  int b, rank, tiles;
  if (!find_tile(a.cu_k, a.batch, a.total_k, 1, kKeyRows, blockIdx.x / a.kv_heads, b, rank, tiles))
    return;
  const Sequence s = load_sequence(a, b);
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
  auto copy_square = [&](int stage) {
    const int rows = copied < total ? min(left, 32) : 0;
    qt.copy(lds[stage][half][0], kw, qw.rows(rows));
    dt.copy(lds[stage][half][1], kw, dw.rows(rows));
    if (kw < 2)
      copy4(uniform(lds_offset(&stats[stage][half][kw][0])), lane * 4, buffer(stat_at, rows * 4));
    copied += 2;  // the halves take squares in turn
    pass(2);
  };
  if (total > 0) copy_square(0);
  const uint16_t* kp = a.k.p + krow * a.k.row + g * a.k.head;
  bf16x8 k[kSteps];
#pragma unroll
  for (int ks = 0; ks < kSteps; ++ks)
    k[ks] = load8(kp, ks * 16 + 8 * (lane >> 5), a.head_dim, used);

  f32x16 dk[kDims], dv[kDims];
#pragma unroll
  for (int ct = 0; ct < kDims; ++ct) dk[ct] = dv[ct] = f32x16{};
  int at = per_head == 1 ? 0 : half;  // this half's square of its head
  for (int n = 0; n < total; n += 2) {
    const int stage = (n >> 1) & 1;
    wait_copies<0>();
    __syncthreads();
    if (n + 2 < total) copy_square(stage ^ 1);
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

template <int DP>
bfp8_status launch_backward(const AttentionArgs& a, int64_t q_blocks, int64_t k_blocks,
                            hipStream_t stream) {
  bfp8_status st = BFP8_OK;
  if (q_blocks > 0)
    st = launch(attention_dq_kernel<DP>, dim3(static_cast<unsigned>(q_blocks)), dim3(512), stream, a);
  if (st == BFP8_OK && k_blocks > 0)
    st = launch(attention_dkdv_kernel<DP>, dim3(static_cast<unsigned>(k_blocks)), dim3(512), stream,
                a);
  return st;
}

// An upper bound on the tiles of all sequences, whose lengths are on the device.
int64_t tile_bound(const int32_t* cu, int64_t batch, int64_t total, int64_t mult, int64_t unit) {
  if (cu == nullptr) return batch * ((total / batch * mult + unit - 1) / unit);
  return (total * mult + batch * (unit - 1)) / unit;
}

}  // namespace

bfp8_status launch_attention_backward(const AttentionArgs& a, hipStream_t stream) {
  const int64_t q_blocks = tile_bound(a.cu_q, a.batch, a.total_q, a.group, kRows) * a.kv_heads;
  const int64_t k_blocks = tile_bound(a.cu_k, a.batch, a.total_k, 1, kKeyRows) * a.kv_heads;
  if (q_blocks >= (int64_t(1) << 31) || k_blocks >= (int64_t(1) << 31)) return BFP8_ERR_SHAPE;
  return a.head_dim <= 64 ? launch_backward<64>(a, q_blocks, k_blocks, stream)
                          : launch_backward<128>(a, q_blocks, k_blocks, stream);
}

}  // namespace bfp8
