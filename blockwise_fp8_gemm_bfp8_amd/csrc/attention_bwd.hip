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
constexpr int kQueries = 64;  // queries of a dkdv tile

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
  auto copy_tile = [&](int j) {
    const int n = min(s.kn - j * kKeys, kKeys);
    const int64_t row = (int64_t)s.k0 + j * kKeys;
    kt.copy(lds[j & 1][0], wave, head_rows(a.k, row, g, n, a.head_dim));
    vt.copy(lds[j & 1][1], wave, head_rows(a.v, row, g, n, a.head_dim));
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
  typedef Tile<DP, kQueries, kWaves> QTile;
  typedef Tile<DP, kRows, kWaves> VTile;
  // two stages of Q rows, dO rows and their statistics, and the workgroup's V rows
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][QTile::kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t vlds[VTile::kBytes];
  __shared__ __attribute__((aligned(256))) float stats[2][2][kQueries];  // lse2, -delta
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int g = blockIdx.x % a.kv_heads;
  int b, rank, tiles;
  if (!find_tile(a.cu_k, a.batch, a.total_k, 1, kRows, blockIdx.x / a.kv_heads, b, rank, tiles))
    return;
  const Sequence s = load_sequence(a, b);
  const int row0 = (tiles - 1 - rank) * kRows;  // the first keys are seen by the most queries
  const int key = row0 + wave * 32 + (lane & 31);
  const bool used = key < s.kn;
  const int64_t krow = s.k0 + min(key, s.ka - 1);
  const uint16_t* kp = a.k.p + krow * a.k.row + g * a.k.head;
  bf16x8 k[DP / 16];
#pragma unroll
  for (int ks = 0; ks < DP / 16; ++ks)
    k[ks] = load8(kp, ks * 16 + 8 * (lane >> 5), a.head_dim, used);
  {
    VTile vt;
    vt.init(wave, lane, a.v.row, a.head_dim);
    vt.copy(vlds, wave,
            head_rows(a.v, (int64_t)s.k0 + row0, g, min(s.kn - row0, kRows), a.head_dim));
  }
  // query i sees keys up to i + kn - qn
  const int back = a.causal ? s.qn - s.kn : -s.kn;  // first query that sees key: key + back
  const int first = row0 < s.kn ? max(row0 + back, 0) / kQueries * kQueries : s.qn;
  const int wave_first = row0 + wave * 32 + back;  // first query that sees the wave's first key
  // first query of no masking: the one that sees the wave's last key, or none
  // if some of its keys are past the used length and must vanish
  const bool all_used = row0 + wave * 32 + 31 < s.kn;
  const int wave_free = all_used ? row0 + wave * 32 + 31 + back : 0x7FFFFFFF;
  const int from = used ? key + back : 0x7FFFFFFF;  // first query that sees this lane's key

  QTile qt, dt;
  qt.init(wave, lane, a.q.row, a.head_dim);
  dt.init(wave, lane, a.dout.row, a.head_dim);
  // tile of queries i0 .. of the h-th head of the group into stage n
  auto copy_tile = [&](int n, int hh, int i0) {
    const int h = g * a.group + hh;
    const int rows = min(s.qn - i0, kQueries);
    qt.copy(lds[n][0], wave, head_rows(a.q, (int64_t)s.q0 + i0, h, rows, a.head_dim));
    dt.copy(lds[n][1], wave, head_rows(a.dout, (int64_t)s.q0 + i0, h, rows, a.head_dim));
    if (wave < 2) {
      const float* src = wave == 0 ? a.lse2 : a.delta;
      copy4(uniform(lds_offset(&stats[n][wave][0])), lane * 4,
            buffer(src + (int64_t)h * a.total_q + s.q0 + i0, rows * 4));
    }
  };

  f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int ct = 0; ct < DP / 32; ++ct) dk[ct] = dv[ct] = f32x16{};
  int hh = 0, i0 = first, n = 0;
  const bool any = first < s.qn;
  if (any) copy_tile(0, 0, first);
  while (any) {
    int next_h = hh, next_i = i0 + kQueries;
    if (next_i >= s.qn) {
      next_i = first;
      ++next_h;
    }
    wait_copies<0>();
    __syncthreads();
    if (next_h < a.group) copy_tile(n ^ 1, next_h, next_i);
    const uint8_t* Q = lds[n][0];
    const uint8_t* D = lds[n][1];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (i0 + 32 * t + 31 < wave_first) continue;
      constexpr int kDims = DP / 32, kSteps = DP / 16;
      // S and dP; dP starts from -delta
      f32x16 p = {}, dp;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          dp[4 * c + e] = stats[n][1][32 * t + 8 * c + 4 * (lane >> 5) + e];
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) p = mma(QTile::rows(Q, 32 * t, ks, lane), k[ks], p);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
        dp = mma(QTile::rows(D, 32 * t, ks, lane), VTile::rows(vlds, wave * 32, ks, lane), dp);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 4, 0);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 0);
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 0);
      }
      f32x16 lse2;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          lse2[4 * c + e] = stats[n][0][32 * t + 8 * c + 4 * (lane >> 5) + e];
      if (i0 + 32 * t < wave_free) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (i0 + 32 * t + acc_row(e, lane) < from) p[e] = -INFINITY;
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
          dv[ct] = mma(QTile::columns(D, 32 * t + 16 * u, ct, lane), pu, dv[ct]);
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct)
          dk[ct] = mma(QTile::columns(Q, 32 * t + 16 * u, ct, lane), du, dk[ct]);
      }
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 8, 1);
#pragma unroll
      for (int i = 0; i < 4 * kDims; ++i) {
        __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 1);
        __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 1);
      }
    }
    if (next_h == a.group) break;
    hh = next_h;
    i0 = next_i;
    n ^= 1;
  }
  wait_copies<0>();  // no copy may land after the workgroup has given up its LDS
  if (key >= s.ka) return;
  store_row<DP>(a.dv.p + krow * a.dv.row + g * a.dv.head, dv, 1.0f, a.head_dim, lane);
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

int64_t tile_bound(const int32_t* cu, int64_t batch, int64_t total, int64_t mult) {
  if (cu == nullptr) return batch * ((total / batch * mult + kRows - 1) / kRows);
  return (total * mult + batch * (kRows - 1)) / kRows;
}

}  // namespace

bfp8_status launch_attention_backward(const AttentionArgs& a, hipStream_t stream) {
  const int64_t q_blocks = tile_bound(a.cu_q, a.batch, a.total_q, a.group) * a.kv_heads;
  const int64_t k_blocks = tile_bound(a.cu_k, a.batch, a.total_k, 1) * a.kv_heads;
  if (q_blocks >= (int64_t(1) << 31) || k_blocks >= (int64_t(1) << 31)) return BFP8_ERR_SHAPE;
  return a.head_dim <= 64 ? launch_backward<64>(a, q_blocks, k_blocks, stream)
                          : launch_backward<128>(a, q_blocks, k_blocks, stream);
}

}  // namespace bfp8
