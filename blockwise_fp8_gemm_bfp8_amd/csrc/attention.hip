// Attention forward for gfx950: O = softmax(scale Q K^T) V and its
// log-sum-exp, one pass over the keys with a running maximum and sum.
//
// All products are turned so that a lane owns one query row throughout:
//   S^T [key][query] = K Q^T   (K rows from LDS, Q rows in registers)
//   O^T [dim][query] = V^T P^T (V columns by transposing LDS reads, P^T the
//                               accumulator of S^T rounded to bf16 in place)
// With v_mfma_f32_32x32x16_bf16 lane l holds query l % 32 of both results, so
// the row maximum and sum are taken over registers (and one exchange with
// lane l ^ 32), the rescaling factor is one register, and P never moves
// between lanes.
//
// A workgroup of 8 waves takes 256 rows of one kv head, a row being one
// (query, head of the group) pair: the heads that share keys share their
// tiles, and few queries fill more of a tile.  Each wave owns 32 rows; tiles
// of 64 keys pass through two LDS stages, filled by LDS-DMA one tile ahead.
#include "attention.h"

namespace bfp8 {
namespace {

using namespace attn;

constexpr int kWaves = 8;
constexpr int kRows = 32 * kWaves;  // rows of a workgroup
constexpr int kKeys = 64;           // keys of a tile

// The rows are scaled back to the running maximum only when it has grown by
// more than this many powers of two: probabilities stay below 2^8 (float32
// sums and bf16 products hold that without loss), and most tiles skip the
// multiplication of the accumulators.
constexpr float kSlack = 8.0f;

template <int DP>
__global__ __launch_bounds__(512, 2) void attention_forward_kernel(AttentionArgs a) {
  typedef Tile<DP, kKeys, kWaves> KTile;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][2][KTile::kBytes];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int g = blockIdx.x % a.kv_heads;
  int b, rank, tiles;
  if (!find_tile(a.cu_q, a.batch, a.total_q, a.group, kRows, blockIdx.x / a.kv_heads, b, rank,
                 tiles))
    return;
  const Sequence s = load_sequence(a, b);
  const int row0 = rank * kRows;  // the last rows see the most keys
  const int rows = s.qn * a.group;
  const int r = row0 + wave * 32 + (lane & 31);
  const bool valid = r < rows;
  const int i = min(r, rows - 1) / a.group;  // query
  const int h = g * a.group + r % a.group;
  // last visible key of a row, of the workgroup's last and of the wave's first and last
  const int shift = a.causal ? s.kn - s.qn : s.kn;
  const int lim = min(i + shift, s.kn - 1);
  const int block_lim = min((min(row0 + kRows, rows) - 1) / a.group + shift, s.kn - 1);
  const int wave_first = row0 + wave * 32;
  const int wave_lim =
      wave_first < rows ? min((min(wave_first + 32, rows) - 1) / a.group + shift, s.kn - 1) : -1;
  const int wave_free = min(wave_first / a.group + shift, s.kn - 1);  // seen by every row

  const uint16_t* qrow = a.q.p + (int64_t)(s.q0 + i) * a.q.row + h * a.q.head;
  bf16x8 q[DP / 16];
#pragma unroll
  for (int ks = 0; ks < DP / 16; ++ks)
    q[ks] = load8(qrow, ks * 16 + 8 * (lane >> 5), a.head_dim, valid);

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

  f32x16 o[DP / 32];
#pragma unroll
  for (int ct = 0; ct < DP / 32; ++ct) o[ct] = f32x16{};
  float m = -INFINITY, l[2] = {0.0f, 0.0f};  // l: sums of even and odd values
  const int nj = block_lim < 0 ? 0 : block_lim / kKeys + 1;
  if (nj > 0) copy_tile(0);
  for (int j = 0; j < nj; ++j) {
    wait_copies<0>();
    __syncthreads();
    if (j + 1 < nj) copy_tile(j + 1);
    if (j * kKeys > wave_lim) continue;
    const uint8_t* K = lds[j & 1][0];
    const uint8_t* V = lds[j & 1][1];
    constexpr int kDims = DP / 32;    // 32-column panels
    constexpr int kSteps = DP / 16;   // products of one S^T square
    // S^T: the K rows of 8 products are in flight ahead of the products, and
    // the V columns of the first P V products follow them
    f32x16 p[2] = {};
    bf16x8 kf[2][kSteps], vf[2][kDims];
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t) kf[t][ks] = KTile::rows(K, 32 * t, ks, lane);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
      for (int t = 0; t < 2; ++t) p[t] = mma(kf[t][ks], q[ks], p[t]);
#pragma unroll
    for (int ct = 0; ct < kDims; ++ct) vf[0][ct] = KTile::columns(V, 0, ct, lane);
    __builtin_amdgcn_sched_group_barrier(kSchedRead, 8, 0);
#pragma unroll
    for (int i = 0; i < 2 * kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 1, 0);
    }
    if (j * kKeys + kKeys - 1 > wave_free) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (j * kKeys + 32 * t + acc_row(e, lane) > lim) p[t][e] = -INFINITY;
    }
    float top = p[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, p[t][e]);
    top = pair_max(top) * a.scale_log2;
    if (__any(top > m + kSlack)) {
      const float next = fmaxf(m, top);
      const float alpha = __builtin_amdgcn_exp2f(m - (next == -INFINITY ? 0.0f : next));
      m = next;
      l[0] *= alpha;
      l[1] *= alpha;
#pragma unroll
      for (int ct = 0; ct < kDims; ++ct)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[ct][e] *= alpha;
    }
    // P and O^T, 16 keys at a time: the exponentials of the next 16 and the
    // reads of their V columns go between the products of these
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int e = 8 * (u & 1); e < 8 * (u & 1) + 8; ++e) {
        p[u >> 1][e] = __builtin_amdgcn_exp2f(fmaf(p[u >> 1][e], a.scale_log2, -base));
        l[e & 1] += p[u >> 1][e];
      }
      const bf16x8 pu = narrow(p[u >> 1], u & 1);
      if (u < 3) {
#pragma unroll
        for (int ct = 0; ct < kDims; ++ct)
          vf[(u + 1) & 1][ct] = KTile::columns(V, 16 * (u + 1), ct, lane);
      }
#pragma unroll
      for (int ct = 0; ct < kDims; ++ct) o[ct] = mma(vf[u & 1][ct], pu, o[ct]);
    }
    __builtin_amdgcn_sched_group_barrier(kSchedValu, 28, 1);
#pragma unroll
    for (int i = 0; i < 4 * kDims; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedMma, 1, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedRead, 2, 1);
      __builtin_amdgcn_sched_group_barrier(kSchedValu, 28 / kDims, 1);
    }
  }
  const float sum = pair_sum(l[0] + l[1]);
  if (!valid) return;
  uint16_t* orow = a.o.p + (int64_t)(s.q0 + i) * a.o.row + h * a.o.head;
  store_row<DP>(orow, o, sum > 0.0f ? 1.0f / sum : 0.0f, a.head_dim, lane);
  if (lane < 32)
    a.lse[(int64_t)h * a.total_q + s.q0 + i] =
        sum > 0.0f ? (m + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
}

}  // namespace

size_t attention_forward_workspace(const AttentionArgs&) { return 0; }

bfp8_status launch_attention_forward(const AttentionArgs& a, void*, size_t, hipStream_t stream) {
  // an upper bound on the tiles of all sequences: the lengths are on the device
  int64_t tiles;
  if (a.cu_q == nullptr)
    tiles = a.batch * (((int64_t)a.total_q / a.batch * a.group + kRows - 1) / kRows);
  else
    tiles = ((int64_t)a.total_q * a.group + (int64_t)a.batch * (kRows - 1)) / kRows;
  const int64_t blocks = tiles * a.kv_heads;
  if (blocks == 0) return BFP8_OK;
  if (blocks >= (int64_t(1) << 31)) return BFP8_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>(blocks));
  if (a.head_dim <= 64) return launch(attention_forward_kernel<64>, grid, dim3(512), stream, a);
  return launch(attention_forward_kernel<128>, grid, dim3(512), stream, a);
}

}  // namespace bfp8
